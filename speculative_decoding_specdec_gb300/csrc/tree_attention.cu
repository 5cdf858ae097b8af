// Attention of a draft tree over the cache: host entry, and the kernel for fp32 tensors and for
// head sizes that the tensor-core kernels do not take.
//
// attn_fma_kernel.  fp32 has no tensor-core product of full precision, so this is the FMA pipe, R
// query rows at a time.  As in the kernel for few rows, a warp is the unit: it streams its own 16
// columns of each tile into two private stages, one bulk copy per column and lane, without any
// CTA-wide barrier.  For the scores a lane has half of a column's values (one 16-byte read of K
// against R broadcast reads of Q); for O a lane owns 4 (or 8) of the head's values (one read of V
// and R / 4 broadcast reads of the weights for 4 R FMAs).  HBM bounds few rows, the
// operands' shared-memory reads many: 16 rows of up to 4096 columns, 8 K/V heads: 4 query rows 80 us
// (302 MB, 3.8 TB/s); one row of 65536 columns and 8 query rows: 193 us (2.8 TB/s).
// bf16 heads of other sizes than 64 and 128 come here too: chains of 6, 32 heads of 96, 8 rows of up
// to 1024 columns: 55 us.
//
// Columns that batch rows share (specdec_prefix_attention).  A softmax over two sets of columns is that of
// their (m, l, o): m the larger of the maxima, l and o the sums of 2^(m_i - m) (l_i, o_i).  So all query
// rows of a group, which may fill a matrix tile where a row's own do not, attend its prefix in one pass that
// reads the prefix once and leaves (m, l, o) in fp32, and the pass over the rows' own columns takes these
// in where it writes its output.  The second is launched as the first's programmatic dependent: it
// starts where SMs are free, and waits before it reads what the first wrote.  Measured, heads of 128:
//   64 rows of one token, 32 query and 8 K/V heads, one prompt of 65537 columns: 108 us (the shared pass
//     78, 269 MB in 3.4 TB/s; its cut units' merge 12, the own columns 26, partly at once);
//   32 chains of 6 of the same heads, 4 prompts of 6000 to 2400 (264 to 120 query rows): 70 us (38, 10, 27);
//   8 rows of one token of 32 K/V heads, one prompt of 2048: 22 us.
// Rows that fill the tiles by themselves gain nothing from a pass of their group and would pay for (m, l,
// o): they take both parts in one pass, from two tensor maps, the prefix's tiles first (fills_tiles):
//   32 trees of 32 nodes, 32 query and 2 K/V heads, one prompt of 8192 columns: 132 us, 0.97 PFLOP/s.
#include <algorithm>
#include <climits>
#include <cmath>

#include "tree_attention.cuh"

namespace specdec {
namespace {

constexpr int kCols = 16;      // columns of a warp's slice of a tile
constexpr int kStages = 2;
constexpr int kMaxWarps = 8;
constexpr uint32_t kTries = 1u << 17, kNs = 20000;  // a wait gives up after about 2.6 s
constexpr float kGrow = 32.f;  // log2 of the growth of the maximum that is let pass

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bytes of a column in shared memory: 16 more than its values, so that the 16-byte reads of
// eight neighbouring columns fall into different banks.
__host__ __device__ constexpr int pitch_of(int hd, int es) { return hd * es + 16; }

constexpr int kRowsTile = 32;  // columns of a tile of the kernel for more rows
__host__ inline size_t fma_rows_smem(int hd, int es) {
  return static_cast<size_t>(4) * kRowsTile * pitch_of(hd, es) + static_cast<size_t>(32) * hd * 4 + 8 * kRowsTile * 16;
}

// Shared memory of a warp: stages, weights, and its O to be merged; and of the CTA: Q.
__host__ __device__ constexpr int fma_warp_bytes(int R, int hd, int es) {
  return kStages * 2 * kCols * pitch_of(hd, es) + kCols * R * 4 + R * hd * 4;
}

// 4 consecutive values of a column as floats.
template <typename T> __device__ __forceinline__ float4 load4(const char* p);
template <> __device__ __forceinline__ float4 load4<float>(const char* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <> __device__ __forceinline__ float4 load4<uint16_t>(const char* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
}
template <typename T> __device__ __forceinline__ void store4(char* p, float4 v);
template <> __device__ __forceinline__ void store4<float>(char* p, float4 v) {
  *reinterpret_cast<float4*>(p) = v;
}
template <> __device__ __forceinline__ void store4<uint16_t>(char* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pack(v.x, v.y), bf16_pack(v.z, v.w));
}

// Walks the tiles of a share, segment by segment.
struct Cursor {
  AttnSegment seg;
  int tile;   // of the segment
  bool more;  // not behind the last
};

// R: query rows of an M-tile; NB: blocks of 128 head values (1 or 2).
template <typename T, int R, int NB, bool kPrefix>
__global__ void __launch_bounds__(kMaxWarps * 32) attn_fma_kernel(const AttnParams p) {
  extern __shared__ __align__(16) char smem[];
  __shared__ uint64_t s_full[kMaxWarps][kStages];
  __shared__ int s_par[kMaxTree], s_flag, s_bad;
  __shared__ unsigned long long s_anc[kMaxTree];
  __shared__ float2 s_ml[kMaxWarps][R];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
  const int hd = p.hd, es = sizeof(T), pitch = pitch_of(hd, es), col_bytes = hd * es, tile_cols = kCols * warps;
  const int warp_bytes = fma_warp_bytes(R, hd, es);
  float* s_q = reinterpret_cast<float*>(smem);                     // [R][hd], times scale_log2
  char* mem = smem + R * hd * 4 + warp * warp_bytes;               // [stage][K, V][kCols] columns
  float* s_p = reinterpret_cast<float*>(mem + kStages * 2 * kCols * pitch);  // [kCols][R]
  auto merge = [&](int w) {                                        // [R][hd] of warp w
    return reinterpret_cast<float*>(smem + R * hd * 4 + w * warp_bytes + kStages * 2 * kCols * pitch) + kCols * R;
  };
  const AttnPlan plan = attn_plan_at(smem + R * hd * 4 + warps * warp_bytes, kPrefix ? p.P : p.B);
  if (warp == 0) attn_plan<kPrefix ? kPrefixPass : kOwn>(p, tile_cols, plan);
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&s_full[warp][i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (kPrefix) pdl_launch_dependents();  // the pass over own columns may be set up
  const AttnShares sh = attn_shares<kPrefix ? kPrefixPass : kOwn>(p, plan);
  const int g = blockIdx.x / p.MT, mt = blockIdx.x % p.MT;
  if (sh.total == 0 || g >= sh.groups) {
    if (!kPrefix) attn_wait_prior(p);
    return;
  }
  const int x1 = sh.start(g + 1);
  // The warp's columns of the cursor's tile into stage `st`: lanes 0..15 copy K's, the others V's.
  auto fetch = [&](const Cursor& c, int st) {
    const int col = c.tile * tile_cols + warp * kCols, n = max(0, min(kCols, c.seg.cols - col));
    if (lane == 0) mbar_arrive_expect_tx(&s_full[warp][st], 2 * n * col_bytes);
    __syncwarp();
    const int j = lane & 15, kv = lane >> 4;
    if (j < n)
      bulk_g2s(mem + ((st * 2 + kv) * kCols + j) * pitch,
               p.cache.base + kv * p.cache.skv + (p.one_row ? 0 : c.seg.b) * p.cache.srow +
                   c.seg.h * p.cache.shead + static_cast<long long>(c.seg.first + col + j) * col_bytes,
               col_bytes, &s_full[warp][st]);
  };
  auto advance = [&](Cursor& c) {
    if (++c.tile >= c.seg.tile1) {
      c.more = attn_next<kPrefix ? kPrefixPass : kOwn>(p, plan, c.seg.next, x1, c.seg);
      c.tile = c.seg.tile0;
    }
  };
  Cursor ahead;
  ahead.more = attn_next<kPrefix ? kPrefixPass : kOwn>(p, plan, sh.start(g), x1, ahead.seg);
  ahead.tile = ahead.seg.tile0;
  int loaded = 0, used = 0, row_b = -1;  // tiles asked for, tiles done
  for (; loaded < kStages && ahead.more; ++loaded) {
    fetch(ahead, loaded);
    advance(ahead);
  }
  bool ok = true;
  AttnSegment seg;
  for (int x = sh.start(g); attn_next<kPrefix ? kPrefixPass : kOwn>(p, plan, x, x1, seg); x = seg.next) {
    __syncthreads();  // the segment before is done with Q and the tree
    const int nrows = kPrefix ? seg.rows : min(R, p.T * p.G - mt * R);  // query rows of this M-tile: (node, head) pairs
    const bool other = kPrefix ? row_b < 0 : seg.b != row_b;
    row_b = seg.b;
    if (other) {
      if (!kPrefix && p.parents && tid < p.T) s_par[tid] = p.parents[seg.b * p.T + tid];
      if (tid == 0) s_bad = 0;
    }
    for (int i = tid * 4; i < R * hd; i += threads * 4) {
      const int r = i / hd, d = i - r * hd;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nrows) {
        const AttnQuery at = attn_query<kPrefix>(p, seg, mt * R + r);
        v = load4<T>(p.q + at.b * p.qr + at.t * p.qt + (static_cast<long long>(at.h) * hd + d) * es);
      }
      *reinterpret_cast<float4*>(s_q + i) = make_float4(v.x * p.scale_log2, v.y * p.scale_log2,
                                                        v.z * p.scale_log2, v.w * p.scale_log2);
    }
    __syncthreads();
    if (!kPrefix && other) {
      for (int i = tid; i < p.T; i += threads) {
        bool bad = false;
        s_anc[i] = tree_ancestors(p.parents ? s_par : nullptr, i, bad);
        if (bad) {
          s_bad = 1;
          set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
        }
      }
      __syncthreads();
    }
    float m[R], l[R];
    float4 o[R][NB];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int j = 0; j < NB; ++j) o[r][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int tile = seg.tile0; tile < seg.tile1; ++tile, ++used) {
      const int st = used % kStages;
      ok = ok && __all_sync(0xffffffffu, mbar_wait_sleep(&s_full[warp][st], (used / kStages) & 1, kTries, kNs));
      const int col = tile * tile_cols + warp * kCols;
      if (ok && col < seg.cols) {
        const char* sk = mem + (st * 2 * kCols + (lane & 15)) * pitch;
        const char* sv = mem + (st * 2 + 1) * kCols * pitch;
        float z[R];
#pragma unroll
        for (int r = 0; r < R; ++r) z[r] = 0.f;
        const int n4 = hd / 4, mid = (n4 + 1) / 2;  // the two lanes of a column take half each
        for (int i = lane >> 4 ? mid : 0, end = lane >> 4 ? n4 : mid; i < end; ++i) {
          const float4 kk = load4<T>(sk + i * 4 * es);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float4 qq = *reinterpret_cast<const float4*>(s_q + r * hd + i * 4);
            z[r] = fmaf(qq.x, kk.x, z[r]);
            z[r] = fmaf(qq.y, kk.y, z[r]);
            z[r] = fmaf(qq.z, kk.z, z[r]);
            z[r] = fmaf(qq.w, kk.w, z[r]);
          }
        }
        __syncwarp();
        const int node = col + (lane & 15) - seg.old;
        bool up = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          z[r] += __shfl_xor_sync(0xffffffffu, z[r], 16);
          if (node >= 0) {
            const int rr = mt * R + r;
            const bool see = !kPrefix && node < p.T && r < nrows && (s_anc[p.g_shift >= 0 ? rr >> p.g_shift : rr / p.G] >> node & 1);
            if (!see) z[r] = -INFINITY;
          }
          up |= z[r] > m[r] + kGrow || (m[r] == -INFINITY && z[r] > m[r]);
        }
        // the maximum is followed only where it grows much: until then weights, sum and O are that
        // much larger, which fp32 does not mind
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float mx = z[r];
#pragma unroll
            for (int j = 8; j > 0; j >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, j));
            if (mx > m[r]) {
              const float f = ex2(m[r] - mx);
              m[r] = mx;
              l[r] *= f;
#pragma unroll
              for (int j = 0; j < NB; ++j) {
                o[r][j].x *= f;
                o[r][j].y *= f;
                o[r][j].z *= f;
                o[r][j].w *= f;
              }
            }
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          z[r] = ex2(z[r] - (m[r] == -INFINITY ? 0.f : m[r]));
          l[r] += z[r];  // (both lanes of a column: halved at the end)
        }
        if (lane < 16)
#pragma unroll
          for (int r = 0; r < R; r += 4)
            *reinterpret_cast<float4*>(s_p + lane * R + r) = make_float4(z[r], z[r + 1], z[r + 2], z[r + 3]);
        __syncwarp();
        // nodes' columns may hold anything where a row does not see them: weight 0 is skipped there
        const int c_end = min(kCols, seg.cols - col), plain = min(c_end, max(0, seg.old - col));
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const int d = j * 128 + lane * 4;
          if (d < hd) {
            auto column = [&](int c, bool skip) {
              const float4 vv = load4<T>(sv + c * pitch + d * es);
#pragma unroll
              for (int r = 0; r < R; r += 4) {
                const float4 w4 = *reinterpret_cast<const float4*>(s_p + c * R + r);
                const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (!skip || w[k] != 0.f) {
                    o[r + k][j].x = fmaf(w[k], vv.x, o[r + k][j].x);
                    o[r + k][j].y = fmaf(w[k], vv.y, o[r + k][j].y);
                    o[r + k][j].z = fmaf(w[k], vv.z, o[r + k][j].z);
                    o[r + k][j].w = fmaf(w[k], vv.w, o[r + k][j].w);
                  }
              }
            };
            if (plain == kCols) {
#pragma unroll 4
              for (int c = 0; c < kCols; ++c) column(c, false);
            } else {
              for (int c = 0; c < c_end; ++c) column(c, c >= plain);
            }
          }
        }
      }
      __syncwarp();
      if (ok && ahead.more) {
        fetch(ahead, loaded % kStages);
        advance(ahead);
        ++loaded;
      }
    }
    // ------------------------------------------------------------- the warps' parts
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int j = 16; j > 0; j >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], j);
      if (lane == 0) s_ml[warp][r] = make_float2(m[r], 0.5f * l[r]);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int d = j * 128 + lane * 4;
        if (d < hd) *reinterpret_cast<float4*>(merge(warp) + r * hd + d) = o[r][j];
      }
    }
    __syncthreads();
    const bool whole = seg.tile0 == 0 && seg.tile1 == seg.tiles;
    const int g0 = sh.owner(seg.unit0), g1 = sh.owner(seg.unit0 + seg.tiles - 1), n4 = hd / 4;
    // 4 values of row r, merged over `parts` parts that `ml(i)` and `at(i)` give
    auto merged = [&](int parts, auto ml, auto at, float& mm, float& ll) {
      mm = -INFINITY;
#pragma unroll 4
      for (int i = 0; i < parts; ++i) mm = fmaxf(mm, ml(i).x);
      const float off = mm == -INFINITY ? 0.f : mm;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      ll = 0.f;
#pragma unroll 4
      for (int i = 0; i < parts; ++i) {
        const float2 y = ml(i);
        const float4 v = at(i);
        const float f = ex2(y.x - off);
        ll += y.y * f;
        acc.x += v.x * f;
        acc.y += v.y * f;
        acc.z += v.z * f;
        acc.w += v.w * f;
      }
      return acc;
    };
    auto store = [&](int r, int i, float4 acc, float mm, float ll) {
      const AttnQuery row = attn_query<kPrefix>(p, seg, mt * R + r);
      const int t = row.t, qh = row.h;
      if constexpr (kPrefix) {
        const long long at = attn_prior_at(p, row.b, t, qh);
        if (i == 0) p.prior_ml[at] = make_float2(mm, ll);
        *reinterpret_cast<float4*>(p.prior_o + at * hd + i * 4) = acc;
        return;
      }
      const bool live = s_anc[t] != 0;
      if (p.prior) {
        attn_wait_prior(p);
        const int state = p.prior[seg.b];
        if (state < 0) return;
        if (state > 0) {
          const long long at = attn_prior_at(p, seg.b, t, qh);
          float f0, f1;
          const float2 ml = attn_join(mm, ll, __ldcg(p.prior_ml + at), f0, f1);
          const float4 v = __ldcg(reinterpret_cast<const float4*>(p.prior_o + at * hd + i * 4));
          mm = ml.x;
          ll = ml.y;
          acc = make_float4(acc.x * f0 + v.x * f1, acc.y * f0 + v.y * f1, acc.z * f0 + v.z * f1, acc.w * f0 + v.w * f1);
        }
      }
      const float inv = 1.f / ll;
      store4<T>(p.out + seg.b * p.outr + t * p.outt + (static_cast<long long>(qh) * hd + i * 4) * es,
                live ? make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f));
      if (p.lse && i == 0)
        p.lse[(static_cast<long long>(seg.b) * p.T + t) * p.Hq + qh] =
            live ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
    };
    const int slot = whole ? 0 : attn_slot(p, sh, g, mt, seg.unit0);
    if (!s_bad)
      for (int k = tid; k < nrows * n4; k += threads) {
        const int r = k / n4, i = k - r * n4;
        float mm, ll;
        const float4 acc = merged(warps, [&](int w) { return s_ml[w][r]; },
                                  [&](int w) { return *reinterpret_cast<const float4*>(merge(w) + r * hd + i * 4); }, mm, ll);
        if (whole) {
          store(r, i, acc, mm, ll);
        } else {
          const long long at = static_cast<long long>(slot) * R + r;
          if (i == 0) p.part_ml[at] = make_float2(mm, ll);
          *reinterpret_cast<float4*>(p.part_o + at * hd + i * 4) = acc;
        }
      }
    if (whole || s_bad) continue;
    if (!attn_last(p, g0, mt, g1 - g0 + 1, &s_flag)) continue;
    for (int k = tid; k < nrows * n4; k += threads) {
      const int r = k / n4, i = k - r * n4;
      auto at = [&](int j) { return static_cast<long long>(attn_slot(p, sh, g0 + j, mt, seg.unit0)) * R + r; };
      float mm, ll;
      const float4 acc = merged(g1 - g0 + 1, [&](int j) { return __ldcg(p.part_ml + at(j)); },
                                [&](int j) { return __ldcg(reinterpret_cast<const float4*>(p.part_o + at(j) * hd + i * 4)); }, mm, ll);
      store(r, i, acc, mm, ll);
    }
  }
  if (!kPrefix) attn_wait_prior(p);
  if (!ok) {
    set_status(p.status, SPECDEC_ERR_TIMEOUT);
    // no copy outlives the CTA: each stage's last one, which may be the one whose wait gave up, is
    // waited for (a stage is filled again only when its copy before has landed)
    for (int i = max(0, loaded - kStages); i < loaded; ++i)
      (void)mbar_wait_sleep(&s_full[warp][i % kStages], (i / kStages) & 1, kTries, kNs);
  }
}

// More than 32 rows: the FMA pipe bounds it, so 8 warps of 4 rows each share a tile of 32 columns in
// shared memory (cp.async, two stages) in place of streaming their own.  A lane computes the scores
// of one column, the softmax of a row is warp-local, and for O a lane owns 4 (or 8) of the head's
// values.  NB: blocks of 128 head values (1 or 2).
template <typename T, int NB, bool kPrefix>
__global__ void __launch_bounds__(256) attn_fma_rows_kernel(const AttnParams p) {
  constexpr int RG = 8, kThreads = RG * 32, M = RG * 4, kTile = kRowsTile;
  extern __shared__ __align__(16) char smem[];
  __shared__ int s_par[kMaxTree], s_flag, s_bad;
  __shared__ unsigned long long s_anc[kMaxTree];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hd = p.hd, pitch = pitch_of(hd, sizeof(T)), vecs = hd * static_cast<int>(sizeof(T)) / 16;
  char* s_k = smem;                                   // [2][kTile] columns
  char* s_v = s_k + 2 * kTile * pitch;
  float* s_q = reinterpret_cast<float*>(s_v + 2 * kTile * pitch);  // [M][hd], times scale_log2
  float4* s_p = reinterpret_cast<float4*>(s_q + M * hd) + warp * kTile;  // [kTile] x 4 rows
  const AttnPlan plan = attn_plan_at(reinterpret_cast<float4*>(s_q + M * hd) + RG * kTile, kPrefix ? p.P : p.B);
  if (warp == 0) attn_plan<kPrefix ? kPrefixPass : kOwn>(p, kTile, plan);
  __syncthreads();
  if (kPrefix) pdl_launch_dependents();  // the pass over own columns may be set up
  const AttnShares sh = attn_shares<kPrefix ? kPrefixPass : kOwn>(p, plan);
  const int g = blockIdx.x / p.MT, mt = blockIdx.x % p.MT;
  if (sh.total == 0 || g >= sh.groups) {
    if (!kPrefix) attn_wait_prior(p);
    return;
  }
  const int x1 = sh.start(g + 1);
  int row_b = -1;
  AttnSegment seg;
  for (int x = sh.start(g); attn_next<kPrefix ? kPrefixPass : kOwn>(p, plan, x, x1, seg); x = seg.next) {
    const int nrows = kPrefix ? seg.rows : min(M, p.T * p.G - mt * M);  // query rows of this M-tile: (node, head) pairs
    if (kPrefix ? row_b < 0 : seg.b != row_b) {  // a new batch row: its tree
      row_b = seg.b;
      __syncthreads();
      if (!kPrefix && p.parents) {
        for (int i = tid; i < p.T; i += kThreads) s_par[i] = p.parents[seg.b * p.T + i];
        __syncthreads();
      }
      bool bad = false;
      for (int i = tid; !kPrefix && i < p.T; i += kThreads)
        s_anc[i] = tree_ancestors(p.parents ? s_par : nullptr, i, bad);
      if (bad) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
      s_bad = 0;
      __syncthreads();
      if (bad) s_bad = 1;
    }
    __syncthreads();
    if (s_bad) {  // not written; every CTA of the row sees the same
      row_b = -1;
      continue;
    }
    for (int i = tid; i < M * hd; i += kThreads) {
      const int r = i / hd, d = i - r * hd;
      float v = 0.f;
      if (r < nrows) {
        const AttnQuery at = attn_query<kPrefix>(p, seg, mt * M + r);
        v = Vec<T>::scalar(reinterpret_cast<const T*>(p.q + at.b * p.qr + at.t * p.qt) + at.h * hd + d);
      }
      s_q[i] = v * p.scale_log2;
    }
    unsigned long long anc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = warp * 4 + k;
      anc[k] = r < nrows ? (kPrefix ? ~0ull : s_anc[(mt * M + r) / p.G]) : 0ull;
    }
    const long long crow = p.one_row ? 0 : seg.b;
    const char* kbase = p.cache.base + crow * p.cache.srow + seg.h * p.cache.shead +
                        static_cast<long long>(seg.first) * hd * sizeof(T);
    const char* vbase = kbase + p.cache.skv;
    auto fetch = [&](int tile) {
      const int stage = tile & 1;
      for (int i = tid; i < kTile * vecs; i += kThreads) {
        const int c = i / vecs, v = i - c * vecs, col = tile * kTile + c;
        const bool in = col < seg.cols;
        const long long at = (static_cast<long long>(in ? col : 0) * vecs + v) * 16;
        cp_async16(s_k + (stage * kTile + c) * pitch + v * 16, kbase + at, in);
        cp_async16(s_v + (stage * kTile + c) * pitch + v * 16, vbase + at, in);
      }
      cp_async_commit();
    };
    float m[4], l[4];
    float4 o[4][NB];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      m[k] = -INFINITY;
      l[k] = 0.f;
#pragma unroll
      for (int j = 0; j < NB; ++j) o[k][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    fetch(seg.tile0);
    for (int tile = seg.tile0; tile < seg.tile1; ++tile) {
      if (tile + 1 < seg.tile1) {
        fetch(tile + 1);
        cp_async_wait<1>();
      } else {
        cp_async_wait<0>();
      }
      __syncthreads();
      const char* sk = s_k + ((tile & 1) * kTile + lane) * pitch;
      const char* sv = s_v + (tile & 1) * kTile * pitch;
      float z[4] = {0.f, 0.f, 0.f, 0.f};
      const float* qrow = s_q + warp * 4 * hd;
      for (int d = 0; d < hd; d += 4) {
        const float4 kk = load4<T>(sk + d * sizeof(T));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 qq = *reinterpret_cast<const float4*>(qrow + k * hd + d);
          z[k] = fmaf(qq.x, kk.x, z[k]);
          z[k] = fmaf(qq.y, kk.y, z[k]);
          z[k] = fmaf(qq.z, kk.z, z[k]);
          z[k] = fmaf(qq.w, kk.w, z[k]);
        }
      }
      const int col = tile * kTile + lane, node = col - seg.old;
      float4 pr;
      float* pv = reinterpret_cast<float*>(&pr);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool see = node < 0 ? anc[k] != 0 : !kPrefix && node < p.T && (anc[k] >> node & 1);
        float s = see ? z[k] : -INFINITY;
        float mx = s;
#pragma unroll
        for (int j = 16; j > 0; j >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, j));
        const float mn = fmaxf(m[k], mx);
        const float off = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every weight is zero
        const float f = ex2(m[k] - off);
        pv[k] = ex2(s - off);
        float sum = pv[k];
#pragma unroll
        for (int j = 16; j > 0; j >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, j);
        l[k] = l[k] * f + sum;
        m[k] = mn;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          o[k][j].x *= f;
          o[k][j].y *= f;
          o[k][j].z *= f;
          o[k][j].w *= f;
        }
      }
      s_p[lane] = pr;
      __syncwarp();
      // nodes' columns may hold anything where a row does not see them: weight 0 is skipped there
      const int c_end = min(kTile, seg.cols - tile * kTile), plain = min(c_end, max(0, seg.old - tile * kTile));
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int d = j * 128 + lane * 4;
        if (d < hd) {
          for (int c = 0; c < plain; ++c) {
            const float4 w = s_p[c], vv = load4<T>(sv + c * pitch + d * sizeof(T));
            const float* wk = reinterpret_cast<const float*>(&w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              o[k][j].x = fmaf(wk[k], vv.x, o[k][j].x);
              o[k][j].y = fmaf(wk[k], vv.y, o[k][j].y);
              o[k][j].z = fmaf(wk[k], vv.z, o[k][j].z);
              o[k][j].w = fmaf(wk[k], vv.w, o[k][j].w);
            }
          }
          for (int c = plain; c < c_end; ++c) {
            const float4 w = s_p[c], vv = load4<T>(sv + c * pitch + d * sizeof(T));
            const float* wk = reinterpret_cast<const float*>(&w);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (wk[k] != 0.f) {
                o[k][j].x = fmaf(wk[k], vv.x, o[k][j].x);
                o[k][j].y = fmaf(wk[k], vv.y, o[k][j].y);
                o[k][j].z = fmaf(wk[k], vv.z, o[k][j].z);
                o[k][j].w = fmaf(wk[k], vv.w, o[k][j].w);
              }
          }
        }
      }
      __syncthreads();  // the stage may be filled again
    }
    // a row of no used node keeps l = 0; rows the committed columns alone
    if (seg.tile0 > 0 || seg.tile1 < seg.tiles) {
      const int slot = attn_slot(p, sh, g, mt, seg.unit0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = warp * 4 + k;
        if (r >= nrows) continue;
        if (lane == 0) p.part_ml[static_cast<long long>(slot) * M + r] = make_float2(m[k], l[k]);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const int d = j * 128 + lane * 4;
          if (d < hd)
            *reinterpret_cast<float4*>(p.part_o + (static_cast<long long>(slot) * M + r) * hd + d) = o[k][j];
        }
      }
      const int g0 = sh.owner(seg.unit0), g1 = sh.owner(seg.unit0 + seg.tiles - 1);
      const bool last = attn_last(p, g0, mt, g1 - g0 + 1, &s_flag);
      if (!last) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = warp * 4 + k;
        m[k] = -INFINITY;
        l[k] = 0.f;
#pragma unroll
        for (int j = 0; j < NB; ++j) o[k][j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r >= nrows) continue;
        for (int gg = g0; gg <= g1; ++gg) {
          const long long at = static_cast<long long>(attn_slot(p, sh, gg, mt, seg.unit0)) * M + r;
          const float2 ml = __ldcg(p.part_ml + at);
          const float mn = fmaxf(m[k], ml.x), off = mn == -INFINITY ? 0.f : mn;
          const float f = ex2(m[k] - off), f2 = ex2(ml.x - off);
          l[k] = l[k] * f + ml.y * f2;
          m[k] = mn;
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const int d = j * 128 + lane * 4;
            if (d < hd) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * hd + d));
              o[k][j].x = o[k][j].x * f + v.x * f2;
              o[k][j].y = o[k][j].y * f + v.y * f2;
              o[k][j].z = o[k][j].z * f + v.z * f2;
              o[k][j].w = o[k][j].w * f + v.w * f2;
            }
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = warp * 4 + k;
      if (r >= nrows) continue;
      const AttnQuery row = attn_query<kPrefix>(p, seg, mt * M + r);
      const int t = row.t, qh = row.h;
      if constexpr (kPrefix) {
        const long long at = attn_prior_at(p, row.b, t, qh);
        if (lane == 0) p.prior_ml[at] = make_float2(m[k], l[k]);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const int d = j * 128 + lane * 4;
          if (d < hd) *reinterpret_cast<float4*>(p.prior_o + at * hd + d) = o[k][j];
        }
        continue;
      }
      if (p.prior) {
        attn_wait_prior(p);
        const int state = p.prior[seg.b];
        if (state < 0) continue;
        if (state > 0) {
          const long long at = attn_prior_at(p, seg.b, t, qh);
          float f0, f1;
          const float2 ml = attn_join(m[k], l[k], __ldcg(p.prior_ml + at), f0, f1);
          m[k] = ml.x;
          l[k] = ml.y;
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const int d = j * 128 + lane * 4;
            if (d < hd) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(p.prior_o + at * hd + d));
              o[k][j] = make_float4(o[k][j].x * f0 + v.x * f1, o[k][j].y * f0 + v.y * f1, o[k][j].z * f0 + v.z * f1, o[k][j].w * f0 + v.w * f1);
            }
          }
        }
      }
      const float inv = 1.f / l[k];
      char* y = p.out + seg.b * p.outr + t * p.outt + static_cast<long long>(qh) * hd * sizeof(T);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int d = j * 128 + lane * 4;
        if (d < hd)
          store4<T>(y + d * sizeof(T), anc[k] ? make_float4(o[k][j].x * inv, o[k][j].y * inv, o[k][j].z * inv, o[k][j].w * inv)
                                              : make_float4(0.f, 0.f, 0.f, 0.f));
      }
      if (p.lse && lane == 0)
        p.lse[(static_cast<long long>(seg.b) * p.T + t) * p.Hq + qh] =
            anc[k] ? (m[k] + log2f(l[k])) * 0.6931471805599453f : -INFINITY;
    }
  }
  if (!kPrefix) attn_wait_prior(p);
}

// ------------------------------------------------------------------------------------- host

struct AttnShape {
  int M, MT, groups, grid, tile, min_tiles, open, warps;
  size_t smem;
  int kind;
};
enum { kFma = 0, kMma = 1, kTc = 2 };
// (behind a prefix pass the former up to more: 32 rows of 24 query rows, 8 K/V heads, 2400 shared columns:
// 70 us against 91 with up to 512 columns of their own, 101 against 121 with up to 2048; 16 of 4096: 104, 115)
constexpr long long kFewColumns = 128 << 10, kFewBehind = 1024 << 10;

// Rows per M-tile, CTAs and shares of a shape; 0 CTAs if there is no device.
AttnShape fma_shape(int es, int T, int G, int hd) {
  AttnShape s = {};
  const int rows = T * G;
  // (64 rows of 128 values: 122 us against 177 of the other kernel; 32 rows of 64: 51 against 36)
  if (rows > 32) {
    s.M = 32;
    s.MT = (rows + 31) / 32;
    s.warps = 8;
    s.smem = fma_rows_smem(hd, es);
    const int per_sm = std::max(1, static_cast<int>((212 * 1024) / (s.smem + 14 * 1024)));
    s.groups = std::max(1, sm_count() * std::min(per_sm, 2) / s.MT);
    s.grid = sm_count() > 0 ? s.groups * s.MT : 0;
    s.tile = kRowsTile;
    s.min_tiles = 2;
    return s;
  }
  s.M = rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
  s.MT = (rows + s.M - 1) / s.M;
  // one CTA per SM of as many warps as have room (the plan of 1024 rows takes 12 KB)
  const int room = 212 * 1024 - s.M * hd * 4;
  s.warps = std::max(1, std::min(kMaxWarps, room / fma_warp_bytes(s.M, hd, es)));
  s.smem = static_cast<size_t>(s.M) * hd * 4 + static_cast<size_t>(s.warps) * fma_warp_bytes(s.M, hd, es);
  s.groups = std::max(1, sm_count() / s.MT);
  s.grid = sm_count() > 0 ? s.groups * s.MT : 0;
  s.tile = kCols * s.warps;
  s.min_tiles = 1;
  s.open = 2;
  return s;
}

// The kernel and its shape for bf16 heads of 64 and 128 values: tiles of 8 or 16 query rows, or of
// 256.  Up to 16 rows the former, whose tiles the latter would leave nearly empty.  From 17 to 32 rows
// by the columns that the cache has: the former is ahead on few (one row of 6400, 4 K/V heads, 25
// thousand in all: 20 us against 41; 100 thousand: 22 against 27), the latter on many (200 thousand:
// 31.0 against 31.4 and 34.7 against 34.2; 800 thousand: 73 against 67).  So the same tokens in a
// cache of another capacity may take the other kernel, with other roundings.
// `columns`: an upper bound of the columns of all units.
AttnShape attn_shape(int es, int T, int G, int hd, long long columns, bool behind = false) {
  if (es != 2 || (hd != 64 && hd != 128)) return fma_shape(es, T, G, hd);
  AttnShape s = {};
  int per_sm = 1;
  if (T * G <= 16 || (T * G <= 32 && columns <= (behind ? kFewBehind : kFewColumns))) {
    s.kind = kMma;
    attn_mma_shape(T * G, hd, &s.M, &s.MT, &s.tile, &per_sm);
    s.open = 3;
  } else {
    s.kind = kTc;
    attn_tc_shape(T * G, &s.M, &s.MT);
    s.tile = 128;
    s.open = T * G > 128 ? 6 : 4;
  }
  s.groups = std::max(1, sm_count() * per_sm / s.MT);
  s.grid = sm_count() > 0 ? s.groups * s.MT : 0;
  s.min_tiles = 1;
  return s;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// The tickets come first and take the same room whatever the shape, so that no shape's other data
// ever lies where another expects zeros.
constexpr size_t kTicketBytes = 32 << 10;
constexpr int kMaxQueries = 65536;  // query rows per K/V head

struct AttnWorkspace {
  size_t ticket, cuts, ml, o, bytes;  // offsets
};
AttnWorkspace attn_workspace(const AttnShape& s, int hd) {
  AttnWorkspace w;
  w.ticket = 0;
  w.cuts = kTicketBytes;
  w.ml = w.cuts + round256(static_cast<size_t>(s.groups) * 16);
  w.o = w.ml + round256(static_cast<size_t>(s.grid) * 2 * s.M * 8);
  w.bytes = w.o + round256(static_cast<size_t>(s.grid) * 2 * s.M * hd * 4);
  return w;
}

template <typename K>
int launch_fma(K kernel, const AttnParams& p, const AttnShape& s, bool prefix, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(s.smem) + attn_plan_bytes(kAttnMaxRows));
  if (e != cudaSuccess) return map_cuda_error(e);
  return map_cuda_error(attn_launch(kernel, s.grid, s.warps * 32, s.smem + (prefix ? prefix_plan_bytes(p.P) : attn_plan_bytes(p.B)),
                                    !prefix && p.prior, stream, p));
}
template <typename T, int NB, bool kPrefix>
int launch_fma_rows(const AttnParams& p, const AttnShape& s, cudaStream_t stream) {
  switch (s.M) {
    case 4: return launch_fma(attn_fma_kernel<T, 4, NB, kPrefix>, p, s, kPrefix, stream);
    case 8: return launch_fma(attn_fma_kernel<T, 8, NB, kPrefix>, p, s, kPrefix, stream);
    case 16: return launch_fma(attn_fma_kernel<T, 16, NB, kPrefix>, p, s, kPrefix, stream);
    default: return launch_fma(attn_fma_rows_kernel<T, NB, kPrefix>, p, s, kPrefix, stream);
  }
}
// The pass that a shape is for.
template <bool kPrefix>
int launch_attention(const AttnParams& p, const AttnShape& s, int es, int rows, cudaStream_t stream) {
  if (s.kind == kTc) return launch_attn_tc(p, rows, s.grid, kPrefix, stream);
  if (s.kind == kMma) return launch_attn_mma(p, s.M, rows, s.grid, kPrefix, stream);
  if (es == 2)
    return p.hd <= 128 ? launch_fma_rows<uint16_t, 1, kPrefix>(p, s, stream)
                       : launch_fma_rows<uint16_t, 2, kPrefix>(p, s, stream);
  return p.hd <= 128 ? launch_fma_rows<float, 1, kPrefix>(p, s, stream)
                     : launch_fma_rows<float, 2, kPrefix>(p, s, stream);
}

// The shape of a pass over prefixes for at most R query rows per K/V head, in units of up to M.
AttnShape prefix_shape(int es, long long R, int hd, long long columns) {
  AttnShape s = {};
  int per_sm = 1;
  if (es != 2 || (hd != 64 && hd != 128)) {
    s = fma_shape(es, 1, static_cast<int>(std::min<long long>(R, 64)), hd);
    s.groups *= s.MT;  // (units have one M-tile)
  } else {
    if (R <= 16 || (R <= 32 && columns <= kFewColumns)) {
      s.kind = kMma;
      attn_mma_shape(static_cast<int>(R), hd, &s.M, &s.MT, &s.tile, &per_sm);
      s.open = 3;
    } else {
      s.kind = kTc;
      attn_tc_shape(1, &s.M, &s.MT);
      s.tile = 128;
      s.open = R > 128 ? 6 : 4;
    }
    s.groups = std::max(1, sm_count() * per_sm);
    s.min_tiles = 1;
  }
  s.MT = 1;
  s.grid = sm_count() > 0 ? s.groups : 0;
  return s;
}

// A workspace for prefixes too.  The passes may overlap, so each has room of its own for cut units (the
// tickets' first half is for the own columns, its second for the prefixes); what the prefix pass leaves for
// the rows follows.
struct PrefixWorkspace {
  size_t parts, state, ml, o, bytes;  // offsets
};
PrefixWorkspace prefix_workspace(int es, int B, int T, int Hq, int G, int hd) {
  size_t own = 0, prefix = 0;  // of the kernels that the lengths may decide for
  for (const long long columns : {0LL, kFewBehind + 1}) {
    own = std::max(own, attn_workspace(attn_shape(es, T, G, hd, columns), hd).bytes);
    prefix = std::max(prefix, attn_workspace(prefix_shape(es, static_cast<long long>(B) * T * G, hd, columns), hd).bytes);
  }
  const size_t rows = static_cast<size_t>(B) * T * Hq;
  PrefixWorkspace w;
  w.parts = round256(own);
  w.state = w.parts + round256(prefix);
  w.ml = w.state + round256(static_cast<size_t>(B) * 4);
  w.o = w.ml + round256(rows * 8);
  w.bytes = w.o + round256(rows * hd * 4);
  return w;
}

bool attn_sizes_ok(int dtype, int B, int T, int heads_q, int heads_kv, int head_dim) {
  const int es = elem_size(dtype);
  return es != 0 && B >= 1 && B <= kAttnMaxRows && T >= 1 && T <= SPECDEC_MAX_TREE &&
         heads_kv >= 1 && heads_q >= heads_kv && heads_q % heads_kv == 0 && head_dim >= 1 &&
         head_dim <= 256 && head_dim * es % 16 == 0 && heads_q / heads_kv <= kMaxQueries / T;
}

// Host checks of a call (SPECDEC_OK with B == 0: nothing to do).
int check_attention(const specdec_tree_attention_args* a) {
  if (a->B < 0 || a->T < 1 || a->heads_q < 1 || a->layer < 0 || !std::isfinite(a->scale))
    return SPECDEC_ERR_INVALID_ARG;
  if (a->B > kAttnMaxRows || a->T > SPECDEC_MAX_TREE) return SPECDEC_ERR_UNSUPPORTED;
  if (a->B == 0) return SPECDEC_OK;
  const int st = check_view(a->cache, 0);
  if (st) return st;
  const specdec_kv_view& c = a->cache;
  const long long es = elem_size(c.dtype);
  if (a->layer >= c.layers || !(c.rows >= a->B || c.rows == 1) || a->heads_q % c.heads)
    return SPECDEC_ERR_INVALID_ARG;
  if (!attn_sizes_ok(c.dtype, a->B, a->T, a->heads_q, c.heads, c.head_dim))
    return SPECDEC_ERR_UNSUPPORTED;
  if (!a->q || !a->out || !a->n_committed || !a->dev_status || !a->workspace)
    return SPECDEC_ERR_INVALID_ARG;
  if (!a->first_col && (!a->width || a->rows || (c.rows == 1 && a->B > 1)))
    return SPECDEC_ERR_INVALID_ARG;
  const long long strides = a->q_stride_row | a->q_stride_token | a->out_stride_row |
                            a->out_stride_token;
  if (a->q_stride_row < 0 || a->q_stride_token < 0 || a->out_stride_row < 0 ||
      a->out_stride_token < 0)
    return SPECDEC_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(a->q) % 16 || reinterpret_cast<uintptr_t>(a->out) % 16 ||
      (strides * es) % 16 || reinterpret_cast<uintptr_t>(a->lse) % 4)
    return SPECDEC_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(a->workspace) % 256) return SPECDEC_ERR_INVALID_ARG;
  return SPECDEC_OK;
}

// What both passes take from the arguments.
AttnParams attention_params(const specdec_tree_attention_args* a) {
  const specdec_kv_view& c = a->cache;
  const long long es = elem_size(c.dtype);
  const int G = a->heads_q / c.heads;
  AttnParams p = {};
  p.cache = to_bytes(c);
  p.cache.base += a->layer * p.cache.sl;
  p.q = static_cast<const char*>(a->q);
  p.out = static_cast<char*>(a->out);
  p.lse = a->lse;
  p.qr = a->q_stride_row * es;
  p.qt = a->q_stride_token * es;
  p.outr = a->out_stride_row * es;
  p.outt = a->out_stride_token * es;
  p.n_committed = a->n_committed;
  p.width = a->width;
  p.parents = a->parents;
  p.rows = a->rows;
  p.first_col = a->first_col;
  p.status = a->dev_status;
  p.scale_log2 = a->scale * kLog2e;
  p.B = a->B;
  p.T = a->T;
  p.Hq = a->heads_q;
  p.H = c.heads;
  p.G = G;
  p.hd = c.head_dim;
  p.cap = c.cap_cols;
  p.one_row = c.rows == 1 ? 1 : 0;
  p.g_shift = (G & (G - 1)) == 0 ? __builtin_ctz(G) : -1;
  return p;
}

// How a shape's work is shared out, and where in the workspace its cut units go.
void set_shape(AttnParams& p, const AttnShape& s, void* workspace) {
  const AttnWorkspace w = attn_workspace(s, p.hd);
  char* ws = static_cast<char*>(workspace);
  p.ticket = reinterpret_cast<unsigned*>(ws + w.ticket);
  p.cuts = reinterpret_cast<int4*>(ws + w.cuts);
  p.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  p.part_o = reinterpret_cast<float*>(ws + w.o);
  p.MT = s.MT;
  p.M = s.M;
  p.groups = s.groups;
  p.min_tiles = s.min_tiles;
  p.open = s.open;
}

// Whether a batch row's own query rows fill the tensor cores' tiles to three quarters and more, so that
// its prefix is attended with its own columns in one pass.
// (16384 rows in all per K/V head over 8192 columns and 512 a row over up to 1056 of its own, 32 rows
// and 2 K/V heads: 132 us against 201 in two passes.  32 rows of up to 512 columns, 8 K/V heads, behind one
// prefix of 8192 and of 1024, one pass and two: 96 query rows a row 134, 170 and 51, 103 us; 128: 137, 203 and
// 54, 116; 192: 237, 278 and 77, 150; 256: 243, 335 and 81, 172.  Below the border one pass is ahead too,
// 64 rows 133, 137 and 50, 88, 160 rows 220, 243 and 70, 138, down to 32 rows: 117, 82 and 46, 53.)
bool fills_tiles(const AttnShape& s, long long R) {
  const long long room = R <= 128 ? 128 : (R + 255) / 256 * 256;
  return s.kind == kTc && R * 4 >= room * 3;
}

// The shape of the pass over the rows' own columns, and whether it can run; p from attention_params, behind
// a prefix pass with where that leaves its parts.  both: over their prefixes' columns too.
int own_shape(const AttnParams& p, const specdec_tree_attention_args* a, const specdec_kv_view* both, AttnShape& s) {
  if (sm_count() <= 0) return SPECDEC_ERR_CUDA;
  const specdec_kv_view& c = a->cache;
  s = attn_shape(elem_size(c.dtype), a->T, p.G, c.head_dim, static_cast<long long>(a->B) * c.heads * c.cap_cols, p.prior != nullptr);
  // no more groups than the longest rows could give work to
  const long long columns = static_cast<long long>(c.cap_cols) + (both ? both->cap_cols + s.tile : 0);
  const long long tiles = static_cast<long long>(a->B) * c.heads * ((columns - 1) / s.tile + 1 + s.open);
  s.groups = static_cast<int>(std::min<long long>(s.groups, std::max<long long>(1, tiles / s.min_tiles)));
  s.grid = s.groups * s.MT;
  if (a->workspace_bytes < attn_workspace(s, c.head_dim).bytes) return SPECDEC_ERR_INVALID_ARG;
  if (s.grid > static_cast<int>(kTicketBytes / (p.prior ? 8 : 4))) return SPECDEC_ERR_UNSUPPORTED;
  if (static_cast<long long>(a->B) * c.heads * (columns / kCols + 16) >= (1LL << 31))
    return SPECDEC_ERR_UNSUPPORTED;  // the sequence of tiles is numbered in 32 bits
  return SPECDEC_OK;
}

int launch_own(AttnParams p, const specdec_tree_attention_args* a, const specdec_kv_view* both, const AttnShape& s, cudaStream_t stream) {
  const specdec_kv_view& c = a->cache;
  set_shape(p, s, a->workspace);
  if (both) {
    ByteView prefix = to_bytes(*both);
    prefix.base += a->layer * prefix.sl;
    return launch_attn_tc_both(p, c.rows, prefix, both->rows, s.grid, stream);
  }
  return launch_attention<false>(p, s, elem_size(c.dtype), c.rows, stream);
}

int own_pass(const AttnParams& p, const specdec_tree_attention_args* a, cudaStream_t stream, const specdec_kv_view* both = nullptr) {
  AttnShape s;
  const int rc = own_shape(p, a, both, s);
  return rc ? rc : launch_own(p, a, both, s, stream);
}

}  // namespace
}  // namespace specdec

extern "C" size_t specdec_tree_attention_workspace(int dtype, int B, int T, int heads_q,
                                                   int heads_kv, int head_dim) {
  using namespace specdec;
  if (!attn_sizes_ok(dtype, B, T, heads_q, heads_kv, head_dim)) return 0;
  size_t most = 0;  // of the kernels that the lengths may decide for
  for (const long long columns : {0LL, kFewColumns + 1}) {
    const AttnShape s = attn_shape(elem_size(dtype), T, heads_q / heads_kv, head_dim, columns);
    most = std::max(most, attn_workspace(s, head_dim).bytes);
  }
  return most;
}

extern "C" int specdec_tree_attention(const specdec_tree_attention_args* a, void* stream) {
  using namespace specdec;
  if (!a) return SPECDEC_ERR_INVALID_ARG;
  const int rc = check_attention(a);
  if (rc || a->B == 0) return rc;
  return own_pass(attention_params(a), a, static_cast<cudaStream_t>(stream));
}

extern "C" size_t specdec_prefix_attention_workspace(int dtype, int B, int T, int heads_q, int heads_kv,
                                                     int head_dim, int P) {
  using namespace specdec;
  if (!attn_sizes_ok(dtype, B, T, heads_q, heads_kv, head_dim) || P < 0 || P > kAttnMaxPrefixes) return 0;
  return prefix_workspace(elem_size(dtype), B, T, heads_q, heads_q / heads_kv, head_dim).bytes;
}

extern "C" int specdec_prefix_attention(const specdec_prefix_attention_args* args, void* stream) {
  using namespace specdec;
  if (!args || args->P < 0) return SPECDEC_ERR_INVALID_ARG;
  if (args->P > kAttnMaxPrefixes) return SPECDEC_ERR_UNSUPPORTED;
  const specdec_tree_attention_args* a = &args->own;
  const int rc = check_attention(a);
  if (rc || a->B == 0) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  AttnParams own = attention_params(a);
  if (args->P == 0) return own_pass(own, a, s);
  const specdec_kv_view &c = a->cache, &f = args->prefix;
  const int st = check_view(f, elem_size(c.dtype));
  if (st) return st;
  if (f.dtype != c.dtype || f.heads != c.heads || f.head_dim != c.head_dim || a->layer >= f.layers ||
      !(f.rows >= args->P || (f.rows == 1 && args->prefix_first)))
    return SPECDEC_ERR_INVALID_ARG;
  auto off = [](const void* x) { return reinterpret_cast<uintptr_t>(x) % 4 != 0; };
  if (!args->prefix_len || !args->group_start || off(args->prefix_len) || off(args->group_start) || off(args->prefix_first))
    return SPECDEC_ERR_INVALID_ARG;
  if (sm_count() <= 0) return SPECDEC_ERR_CUDA;
  const int es = elem_size(c.dtype);
  const PrefixWorkspace w = prefix_workspace(es, a->B, a->T, a->heads_q, own.G, c.head_dim);
  if (a->workspace_bytes < w.bytes) return SPECDEC_ERR_INVALID_ARG;
  own.prefix_len = args->prefix_len;
  own.prefix_first = args->prefix_first;
  own.group_start = args->group_start;
  own.P = args->P;
  own.prefix_cap = f.cap_cols;
  own.prefix_one_row = f.rows == 1 ? 1 : 0;
  const AttnShape alone = attn_shape(es, a->T, own.G, c.head_dim, static_cast<long long>(a->B) * c.heads * c.cap_cols);
  if (fills_tiles(alone, static_cast<long long>(a->T) * own.G)) return own_pass(own, a, s, &f);
  char* ws = static_cast<char*>(a->workspace);
  own.prior = reinterpret_cast<int32_t*>(ws + w.state);
  own.prior_ml = reinterpret_cast<float2*>(ws + w.ml);
  own.prior_o = reinterpret_cast<float*>(ws + w.o);
  AttnShape behind;  // (refused before anything is launched)
  const int rc_own = own_shape(own, a, nullptr, behind);
  if (rc_own) return rc_own;
  AttnParams p = own;
  p.cache = to_bytes(f);
  p.cache.base += a->layer * p.cache.sl;
  p.cap = f.cap_cols;
  p.one_row = f.rows == 1 ? 1 : 0;
  const long long R = static_cast<long long>(a->B) * a->T * own.G;
  p.two = R > 128 ? 1 : 0;
  AttnShape shape = prefix_shape(es, R, c.head_dim, static_cast<long long>(args->P) * c.heads * f.cap_cols);
  // (a group's last unit may be nearly empty, so there are at most P more than full ones)
  const long long units = ((R - 1) / shape.M + 1 + args->P) * c.heads;
  if (units * (f.cap_cols / kCols + 16) >= (1LL << 31)) return SPECDEC_ERR_UNSUPPORTED;
  const long long tiles = units * ((f.cap_cols - 1) / shape.tile + 1 + shape.open);
  shape.groups = static_cast<int>(std::min<long long>(shape.groups, std::max<long long>(1, tiles / shape.min_tiles)));
  shape.grid = shape.groups;
  if (shape.grid > static_cast<int>(kTicketBytes / 8)) return SPECDEC_ERR_UNSUPPORTED;
  set_shape(p, shape, ws + w.parts);
  p.ticket = reinterpret_cast<unsigned*>(ws) + kTicketBytes / 8;
  const int rp = launch_attention<true>(p, shape, es, f.rows, s);
  if (rp) return rp;
  return launch_own(own, a, nullptr, behind, s);
}
