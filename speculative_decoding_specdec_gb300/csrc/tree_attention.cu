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
template <typename T, int R, int NB>
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
  const AttnPlan plan = attn_plan_at(smem + R * hd * 4 + warps * warp_bytes, p.B);
  if (warp == 0) attn_plan(p, tile_cols, plan);
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&s_full[warp][i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  const AttnShares sh = attn_shares(p, plan);
  const int g = blockIdx.x / p.MT, mt = blockIdx.x % p.MT;
  if (sh.total == 0 || g >= sh.groups) return;
  const int x1 = sh.start(g + 1);
  const int nrows = min(R, p.T * p.G - mt * R);  // query rows of this M-tile: (node, head) pairs
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
      c.more = attn_next(p, plan, c.seg.next, x1, c.seg);
      c.tile = c.seg.tile0;
    }
  };
  Cursor ahead;
  ahead.more = attn_next(p, plan, sh.start(g), x1, ahead.seg);
  ahead.tile = ahead.seg.tile0;
  int loaded = 0, used = 0, row_b = -1;  // tiles asked for, tiles done
  for (; loaded < kStages && ahead.more; ++loaded) {
    fetch(ahead, loaded);
    advance(ahead);
  }
  bool ok = true;
  AttnSegment seg;
  for (int x = sh.start(g); attn_next(p, plan, x, x1, seg); x = seg.next) {
    __syncthreads();  // the segment before is done with Q and the tree
    const bool other = seg.b != row_b;
    row_b = seg.b;
    if (other) {
      if (p.parents && tid < p.T) s_par[tid] = p.parents[seg.b * p.T + tid];
      if (tid == 0) s_bad = 0;
    }
    for (int i = tid * 4; i < R * hd; i += threads * 4) {
      const int r = i / hd, d = i - r * hd, rr = mt * R + r;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nrows) {
        const int t = rr / p.G, qh = seg.h * p.G + rr - t * p.G;
        v = load4<T>(p.q + seg.b * p.qr + t * p.qt + (static_cast<long long>(qh) * hd + d) * es);
      }
      *reinterpret_cast<float4*>(s_q + i) = make_float4(v.x * p.scale_log2, v.y * p.scale_log2,
                                                        v.z * p.scale_log2, v.w * p.scale_log2);
    }
    __syncthreads();
    if (other) {
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
            const bool see = node < p.T && r < nrows && (s_anc[p.g_shift >= 0 ? rr >> p.g_shift : rr / p.G] >> node & 1);
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
      const int rr = mt * R + r, t = rr / p.G, qh = seg.h * p.G + rr - t * p.G;
      const bool live = s_anc[t] != 0;
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
template <typename T, int NB>
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
  const AttnPlan plan = attn_plan_at(reinterpret_cast<float4*>(s_q + M * hd) + RG * kTile, p.B);
  if (warp == 0) attn_plan(p, kTile, plan);
  __syncthreads();
  const AttnShares sh = attn_shares(p, plan);
  const int g = blockIdx.x / p.MT, mt = blockIdx.x % p.MT;
  if (sh.total == 0 || g >= sh.groups) return;
  const int x1 = sh.start(g + 1);
  const int nrows = min(M, p.T * p.G - mt * M);  // query rows of this M-tile: (node, head) pairs
  int row_b = -1;
  AttnSegment seg;
  for (int x = sh.start(g); attn_next(p, plan, x, x1, seg); x = seg.next) {
    if (seg.b != row_b) {  // a new batch row: its tree
      row_b = seg.b;
      __syncthreads();
      if (p.parents) {
        for (int i = tid; i < p.T; i += kThreads) s_par[i] = p.parents[seg.b * p.T + i];
        __syncthreads();
      }
      bool bad = false;
      for (int i = tid; i < p.T; i += kThreads)
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
      const int r = i / hd, d = i - r * hd, rr = mt * M + r;
      float v = 0.f;
      if (r < nrows) {
        const int t = rr / p.G, qh = seg.h * p.G + rr % p.G;
        v = Vec<T>::scalar(reinterpret_cast<const T*>(p.q + seg.b * p.qr + t * p.qt) + qh * hd + d);
      }
      s_q[i] = v * p.scale_log2;
    }
    unsigned long long anc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = warp * 4 + k;
      anc[k] = r < nrows ? s_anc[(mt * M + r) / p.G] : 0ull;
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
        const bool see = node < 0 ? anc[k] != 0 : node < p.T && (anc[k] >> node & 1);
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
      const int r = warp * 4 + k, rr = mt * M + r;
      if (r >= nrows) continue;
      const int t = rr / p.G, qh = seg.h * p.G + rr % p.G;
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
}

// ------------------------------------------------------------------------------------- host

struct AttnShape {
  int M, MT, groups, grid, tile, min_tiles, open, warps;
  size_t smem;
  int kind;
};
enum { kFma = 0, kMma = 1, kTc = 2 };
constexpr long long kFewColumns = 128 << 10;

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
AttnShape attn_shape(int es, int T, int G, int hd, long long columns) {
  if (es != 2 || (hd != 64 && hd != 128)) return fma_shape(es, T, G, hd);
  AttnShape s = {};
  int per_sm = 1;
  if (T * G <= 16 || (T * G <= 32 && columns <= kFewColumns)) {
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

template <typename T, typename K>
int launch_fma(K kernel, const AttnParams& p, const AttnShape& s, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(s.smem) + attn_plan_bytes(kAttnMaxRows));
  if (e != cudaSuccess) return map_cuda_error(e);
  kernel<<<s.grid, s.warps * 32, s.smem + attn_plan_bytes(p.B), stream>>>(p);
  return map_cuda_error(cudaGetLastError());
}
template <typename T, int NB>
int launch_fma_rows(const AttnParams& p, const AttnShape& s, cudaStream_t stream) {
  switch (s.M) {
    case 4: return launch_fma<T>(attn_fma_kernel<T, 4, NB>, p, s, stream);
    case 8: return launch_fma<T>(attn_fma_kernel<T, 8, NB>, p, s, stream);
    case 16: return launch_fma<T>(attn_fma_kernel<T, 16, NB>, p, s, stream);
    default: return launch_fma<T>(attn_fma_rows_kernel<T, NB>, p, s, stream);
  }
}

bool attn_sizes_ok(int dtype, int B, int T, int heads_q, int heads_kv, int head_dim) {
  const int es = elem_size(dtype);
  return es != 0 && B >= 1 && B <= kAttnMaxRows && T >= 1 && T <= SPECDEC_MAX_TREE &&
         heads_kv >= 1 && heads_q >= heads_kv && heads_q % heads_kv == 0 && head_dim >= 1 &&
         head_dim <= 256 && head_dim * es % 16 == 0 && heads_q / heads_kv <= kMaxQueries / T;
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
  if (sm_count() <= 0) return SPECDEC_ERR_CUDA;
  const int G = a->heads_q / c.heads;
  AttnShape s = attn_shape(static_cast<int>(es), a->T, G, c.head_dim,
                           static_cast<long long>(a->B) * c.heads * c.cap_cols);
  // no more groups than the longest rows could give work to
  const long long tiles = static_cast<long long>(a->B) * c.heads * ((c.cap_cols - 1) / s.tile + 1 + s.open);
  s.groups = static_cast<int>(std::min<long long>(s.groups, std::max<long long>(1, tiles / s.min_tiles)));
  s.grid = s.groups * s.MT;
  const AttnWorkspace w = attn_workspace(s, c.head_dim);
  if (a->workspace_bytes < w.bytes) return SPECDEC_ERR_INVALID_ARG;
  if (s.grid > static_cast<int>(kTicketBytes / 4)) return SPECDEC_ERR_UNSUPPORTED;
  if (static_cast<long long>(a->B) * c.heads * (c.cap_cols / kCols + 16) >= (1LL << 31))
    return SPECDEC_ERR_UNSUPPORTED;  // the sequence of tiles is numbered in 32 bits
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
  char* ws = static_cast<char*>(a->workspace);
  p.ticket = reinterpret_cast<unsigned*>(ws + w.ticket);
  p.cuts = reinterpret_cast<int4*>(ws + w.cuts);
  p.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  p.part_o = reinterpret_cast<float*>(ws + w.o);
  p.scale_log2 = a->scale * kLog2e;
  p.B = a->B;
  p.T = a->T;
  p.Hq = a->heads_q;
  p.H = c.heads;
  p.G = G;
  p.hd = c.head_dim;
  p.cap = c.cap_cols;
  p.one_row = c.rows == 1 ? 1 : 0;
  p.MT = s.MT;
  p.groups = s.groups;
  p.min_tiles = s.min_tiles;
  p.open = s.open;
  p.g_shift = (G & (G - 1)) == 0 ? __builtin_ctz(G) : -1;
  cudaStream_t stream_ = static_cast<cudaStream_t>(stream);
  if (s.kind == kTc) return launch_attn_tc(p, c.rows, s.grid, stream_);
  if (s.kind == kMma) return launch_attn_mma(p, s.M, c.rows, s.grid, stream_);
  if (es == 2)
    return c.head_dim <= 128 ? launch_fma_rows<uint16_t, 1>(p, s, stream_)
                             : launch_fma_rows<uint16_t, 2>(p, s, stream_);
  return c.head_dim <= 128 ? launch_fma_rows<float, 1>(p, s, stream_)
                           : launch_fma_rows<float, 2>(p, s, stream_);
}
