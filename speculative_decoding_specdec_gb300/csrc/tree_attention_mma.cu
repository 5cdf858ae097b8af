// Attention of a draft tree over the cache for few query rows per K/V head: bf16, head sizes 64
// and 128, M-tiles of 8 or 16 rows.
//
// With at most 16 rows (a token or a short chain with one or a few query heads per K/V head) a
// K/V column of 512 bytes meets 16 * 512 flops: HBM bounds it, and tensor memory's 128-row tiles
// would be nearly empty.  So a warp is the unit: it streams its own 16 columns of each 64-column
// tile by TMA (128-byte swizzle) into two private stages, without any CTA-wide barrier, and runs
// both products with m16n8k16, transposed so that the columns (or the head's values) fill the 16
// and the query rows the 8: S^T = K Q^T (Q in registers for the whole segment) and O^T += V^T P^T,
// the weights turned by one movmatrix per 8 x 8.  (Query rows as the 16 took twice the
// instructions for 8 rows.)  Each warp keeps
// maximum, sum and O of its columns; the CTA's are merged in shared memory when the segment ends,
// while the next segment's tiles are already on their way.
// Measured: 8 rows of 128 to 1024 columns, 32 K/V heads, chains of 6: 24 us (3.2 TB/s, in
// 256 units); one row of 131071 columns, 8 K/V heads of 4 query heads: 89 us (6.0 TB/s).
#include <cmath>

#include "tcgen05.cuh"
#include "tree_attention.cuh"

namespace specdec {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kCols = 16;                // columns of a warp's slice of a tile
constexpr int kTileCols = kCols * kWarps;
constexpr int kStages = 2;
constexpr uint32_t kTries = 1u << 17, kNs = 20000;  // a wait gives up after about 2.6 s
constexpr float kGrow = 32.f;  // log2 of the growth of the maximum that is let pass

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ldmatrix4(uint32_t a, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                          uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t a, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                           uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit values held as a product's result is.
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

template <int HD, int NT> struct Smem {
  static constexpr int kSlice = kCols * HD * 2;               // K or V of a warp's slice
  static constexpr int kWarp = kStages * 2 * kSlice;          // [stage][K, V]
  static constexpr int kRows = 8 * NT;
  static constexpr int kPitch = HD + 4;                       // floats of a row to merge
  static constexpr int merge = kWarps * kWarp;                // [warp][kRows][kPitch]
  static constexpr int bytes = merge + kWarps * kRows * kPitch * 4 + 1024;
};

// Walks the tiles of a share, segment by segment.
struct Cursor {
  AttnSegment seg;
  int tile;   // of the segment
  bool more;  // not behind the last
};

// NT: groups of 8 query rows.
template <int HD, int NT>
__global__ void __launch_bounds__(kThreads)
attn_mma_kernel(const AttnParams p, const __grid_constant__ CUtensorMap map) {
  using S = Smem<HD, NT>;
  constexpr int kSteps = HD / 16, kPanels = HD / 64, kRows = S::kRows;
  extern __shared__ char raw[];
  __shared__ uint64_t s_full[kWarps][kStages];
  __shared__ int s_par[kMaxTree], s_flag, s_bad;
  __shared__ unsigned long long s_anc[kMaxTree], s_poison[kWarps];
  __shared__ float2 s_ml[kWarps][kRows];
  char* smem = raw + (1024 - smem_addr(raw) % 1024) % 1024;
  const AttnPlan plan = attn_plan_at(smem + S::bytes - 1024, p.B);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gr = lane >> 2, qd = lane & 3;
  if (warp == 0) attn_plan(p, kTileCols, plan);
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&s_full[warp][i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  const AttnShares sh = attn_shares(p, plan);
  const int g = blockIdx.x / p.MT, mt = blockIdx.x % p.MT;
  if (sh.total == 0 || g >= sh.groups) return;
  const int x1 = sh.start(g + 1);
  const int nrows = min(kRows, p.T * p.G - mt * kRows);
  const float scale = fmaxf(fabsf(p.scale_log2), 1.2e-38f);  // hidden scores stay -infinity
  const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
  char* mem = smem + warp * S::kWarp;
  float* merge = reinterpret_cast<float*>(smem + S::merge);

  // The warp's slice of the cursor's tile into stage `st` (nothing if the row ends before it).
  auto fetch = [&](const Cursor& c, int st) {
    const int col = c.tile * kTileCols + warp * kCols;
    if (lane == 0) {
      if (col < c.seg.cols) {
        mbar_arrive_expect_tx(&s_full[warp][st], 2 * S::kSlice);
        const int crow = p.one_row ? 0 : c.seg.b;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
          for (int j = 0; j < kPanels; ++j)
            tma_load_5d(mem + (st * 2 + kv) * S::kSlice + j * kCols * 128, &map, j * 64,
                        c.seg.first + col, c.seg.h, crow, kv, &s_full[warp][st]);
      } else {
        mbar_arrive_expect_tx(&s_full[warp][st], 0);
      }
    }
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
  int loaded = 0;  // tiles asked for so far
  for (; loaded < kStages && ahead.more; ++loaded) {
    fetch(ahead, loaded);
    advance(ahead);
  }
  int used = 0, row_b = -1;
  bool ok = true;
  AttnSegment seg;
  for (int x = sh.start(g); attn_next(p, plan, x, x1, seg); x = seg.next) {
    if (seg.b != row_b) {
      row_b = seg.b;
      __syncthreads();
      if (p.parents && tid < p.T) s_par[tid] = p.parents[seg.b * p.T + tid];
      if (tid == 0) s_bad = 0;
      __syncthreads();
      if (tid < p.T) {
        bool bad = false;
        s_anc[tid] = tree_ancestors(p.parents ? s_par : nullptr, tid, bad);
        if (bad) {
          s_bad = 1;
          set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
        }
      }
      __syncthreads();
    }
    // Q as B operand (this thread's rows 8n + gr), and the ancestors of its results' rows
    // 8n + 2 qd and one more
    uint32_t q[NT][kSteps][2];
    unsigned long long anc[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + gr, rr = mt * kRows + r;
      const int t = r < nrows ? rr / p.G : 0, h = seg.h * p.G + (r < nrows ? rr % p.G : 0);
      const char* src = p.q + seg.b * p.qr + t * p.qt + static_cast<long long>(h) * HD * 2 + qd * 4;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          q[n][s][i] = r < nrows ? __ldg(reinterpret_cast<const uint32_t*>(src + s * 32 + i * 16)) ^ flip : 0u;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ro = 8 * n + 2 * qd + i;
        anc[n][i] = ro < nrows ? s_anc[(mt * kRows + ro) / p.G] : 0ull;
      }
    }
    float o[NT][kSteps][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[n][j][k] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }
    unsigned long long poison = 0;  // nodes whose V is not finite somewhere
    for (int tile = seg.tile0; tile < seg.tile1; ++tile, ++used) {
      const int st = used % kStages;
      ok = ok && __all_sync(0xffffffffu, mbar_wait_sleep(&s_full[warp][st], (used / kStages) & 1,
                                                         kTries, kNs));
      const int col = tile * kTileCols + warp * kCols, base = col - seg.old;
      if (ok && col < seg.cols) {
        char* vm = mem + (st * 2 + 1) * S::kSlice;
        const uint32_t ka = smem_addr(mem + st * 2 * S::kSlice), va = smem_addr(vm);
        const int mi = lane >> 3, mr = lane & 7;  // matrix and row this lane addresses
        float s[NT][2][4];  // (two sums of every other step: shorter chains)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[n][0][k] = s[n][1][k] = 0.f;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const int c = (mi & 1) * 8 + mr, ch = k * 2 + (mi >> 1);
          uint32_t f[4];
          ldmatrix4(ka + (ch >> 3) * kCols * 128 + c * 128 + (((ch & 7) ^ mr) << 4), f[0], f[1], f[2], f[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(s[n][k & 1], f, q[n][k][0], q[n][k][1]);
        }
        float z[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) z[n][k] = (s[n][0][k] + s[n][1][k]) * scale;
        if (base + kCols > 0) {
          // columns behind the committed ones: what each row sees, and V where it may hold anything
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int node = base + gr + (k >> 1) * 8;
              if (node >= 0 && !(node < p.T && (anc[n][k & 1] >> node & 1))) z[n][k] = -INFINITY;
            }
          const int c = lane & 15, node = base + c;  // two lanes look after a column
          bool bad = false, drop = false;
          const int ch0 = (lane >> 4) * (HD / 16), ch1 = ch0 + HD / 16;
          auto at = [&](int ch) {
            return reinterpret_cast<uint4*>(vm + (ch >> 3) * kCols * 128 + c * 128 + (((ch & 7) ^ (c & 7)) << 4));
          };
          if (node >= 0) {
            drop = node >= p.T || s_anc[node] == 0;
            if (!drop)
              for (int ch = ch0; ch < ch1; ++ch) bad |= inf_or_nan(*at(ch));
          }
          if (drop)
            for (int ch = ch0; ch < ch1; ++ch) *at(ch) = make_uint4(0, 0, 0, 0);
          if (bad) attn_make_finite(vm, c, kCols, ch0, ch1);
          unsigned long long which = __ballot_sync(0xffffffffu, bad);
          which = (which | which >> 16) & 0xffffu;
          poison |= base >= 0 ? which << base : which >> -base;
          fence_async_smem();
          __syncwarp();
        }
        // the maximum is followed only where it grows much: until then weights, sum and O are that
        // much larger, which neither fp32 nor bf16 minds
        bool up = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mx = fmaxf(z[n][i], z[n][i + 2]);
            up |= mx > m[n][i] + kGrow || (m[n][i] == -INFINITY && mx > m[n][i]);
          }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float mx = fmaxf(z[n][i], z[n][i + 2]);
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              if (mx > m[n][i]) {
                const float f = ex2(m[n][i] - mx);
                m[n][i] = mx;
                l[n][i] *= f;
#pragma unroll
                for (int j = 0; j < kSteps; ++j) {
                  o[n][j][i] *= f;
                  o[n][j][i + 2] *= f;
                }
              }
            }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) e[k] = ex2(z[n][k] - (m[n][k & 1] == -INFINITY ? 0.f : m[n][k & 1]));
          l[n][0] += e[0] + e[2];
          l[n][1] += e[1] + e[3];
          // the weights, rounded to bf16: with V in bf16 the product takes nothing wider
          pb[n][0] = transposed(bf16_pack(e[0], e[1]));
          pb[n][1] = transposed(bf16_pack(e[2], e[3]));
        }
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          const int c = (mi >> 1) * 8 + mr, ch = j * 2 + (mi & 1);
          uint32_t f[4];
          ldmatrix4t(va + (ch >> 3) * kCols * 128 + c * 128 + (((ch & 7) ^ mr) << 4), f[0], f[1], f[2], f[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(o[n][j], f, pb[n][0], pb[n][1]);
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
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], 4);
        l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], 8);
        l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], 16);
      }
    __syncthreads();  // the segment before has been merged
    if (lane == 0) s_poison[warp] = poison;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (gr == 0) {
        s_ml[warp][8 * n + 2 * qd] = make_float2(m[n][0], l[n][0]);
        s_ml[warp][8 * n + 2 * qd + 1] = make_float2(m[n][1], l[n][1]);
      }
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          merge[(warp * kRows + 8 * n + 2 * qd + (k & 1)) * S::kPitch + j * 16 + gr + (k >> 1) * 8] = o[n][j][k];
    }
    const bool poisoned = __syncthreads_or(poison != 0);
    // kPer threads per row: every kPer-th group of 4 values from d0
    constexpr int kPer = kThreads / kRows, kVecs = HD / 4 / kPer;
    const int r = tid / kPer, d0 = tid % kPer * 4;
    const int rr = mt * kRows + r;
    const bool mine = r < nrows && !s_bad;
    const int t = mine ? rr / p.G : 0, h = seg.h * p.G + (mine ? rr % p.G : 0);
    const bool live = mine && s_anc[t] != 0;
    float mm = -INFINITY, ll = 0.f;
    float4 acc[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float2 ml, auto at) {  // one more part of the row
      const float mn = fmaxf(mm, ml.x), off = mn == -INFINITY ? 0.f : mn;
      const float fa = ex2(mm - off), fb = ex2(ml.x - off);
      ll = ll * fa + ml.y * fb;
      mm = mn;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        const float4 v = at(j);
        acc[j].x = acc[j].x * fa + v.x * fb;
        acc[j].y = acc[j].y * fa + v.y * fb;
        acc[j].z = acc[j].z * fa + v.z * fb;
        acc[j].w = acc[j].w * fa + v.w * fb;
      }
    };
    if (mine)
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        add(s_ml[w][r], [&](int j) {
          return *reinterpret_cast<const float4*>(merge + (w * kRows + r) * S::kPitch + d0 + j * kPer * 4);
        });
    unsigned long long hit = 0;
    if (poisoned && mine) hit = (s_poison[0] | s_poison[1] | s_poison[2] | s_poison[3]) & s_anc[t];
    if (seg.tile0 > 0 || seg.tile1 < seg.tiles) {
      const long long at = static_cast<long long>(attn_slot(p, sh, g, mt, seg.unit0)) * kRows + r;
      if (mine) {
        if (d0 == 0) p.part_ml[at] = make_float2(mm, ll);
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
          *reinterpret_cast<float4*>(p.part_o + at * HD + d0 + j * kPer * 4) = acc[j];
        if (hit) attn_add_not_finite(hit, attn_node_v(p, seg), HD, d0, kPer * 4, nullptr, reinterpret_cast<float4*>(p.part_o + at * HD), 1);
        hit = 0;
      }
      if (s_bad) continue;
      const int g0 = sh.owner(seg.unit0), g1 = sh.owner(seg.unit0 + seg.tiles - 1);
      if (!attn_last(p, g0, mt, g1 - g0 + 1, &s_flag)) continue;
      mm = -INFINITY;
      ll = 0.f;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (mine) {
        // the maximum first, so that the parts' loads depend on nothing and wait together
        const auto at = [&](int gg) { return static_cast<long long>(attn_slot(p, sh, gg, mt, seg.unit0)) * kRows + r; };
#pragma unroll 8
        for (int gg = g0; gg <= g1; ++gg) mm = fmaxf(mm, __ldcg(&p.part_ml[at(gg)].x));
        const float off = mm == -INFINITY ? 0.f : mm;
#pragma unroll 4
        for (int gg = g0; gg <= g1; ++gg) {
          const float2 ml = __ldcg(p.part_ml + at(gg));
          const float f = ex2(ml.x - off);
          ll += ml.y * f;
#pragma unroll
          for (int j = 0; j < kVecs; ++j) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part_o + at(gg) * HD + d0 + j * kPer * 4));
            acc[j].x += v.x * f;
            acc[j].y += v.y * f;
            acc[j].z += v.z * f;
            acc[j].w += v.w * f;
          }
        }
      }
    }
    if (!mine) continue;
    const float inv = 1.f / ll;
    char* y = p.out + seg.b * p.outr + t * p.outt + static_cast<long long>(h) * HD * 2;
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      *reinterpret_cast<uint2*>(y + (d0 + j * kPer * 4) * 2) =
          live ? make_uint2(bf16_pack(acc[j].x * inv, acc[j].y * inv), bf16_pack(acc[j].z * inv, acc[j].w * inv)) : make_uint2(0, 0);
    if (hit) attn_add_not_finite(hit, attn_node_v(p, seg), HD, d0, kPer * 4, y, nullptr, 0);
    if (p.lse && d0 == 0)
      p.lse[(static_cast<long long>(seg.b) * p.T + t) * p.Hq + h] =
          live ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
  }
  if (!ok) {
    set_status(p.status, SPECDEC_ERR_TIMEOUT);
    // no copy outlives the CTA: each stage's last one, which may be the one whose wait gave up, is
    // waited for (a stage is filled again only when its copy before has landed)
    for (int i = max(0, loaded - kStages); i < loaded; ++i)
      (void)mbar_wait_sleep(&s_full[warp][i % kStages], (i / kStages) & 1, kTries, kNs);
  }
}

template <int HD, int NT>
int launch_mma(const AttnParams& p, const CUtensorMap& map, int grid, cudaStream_t stream) {
  auto kernel = attn_mma_kernel<HD, NT>;
  constexpr int smem = Smem<HD, NT>::bytes;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             smem + attn_plan_bytes(kAttnMaxRows));
  if (e != cudaSuccess) return map_cuda_error(e);
  kernel<<<grid, kThreads, smem + attn_plan_bytes(p.B), stream>>>(p, map);
  return map_cuda_error(cudaGetLastError());
}

}  // namespace

void attn_mma_shape(int R, int hd, int* M, int* MT, int* tile, int* per_sm) {
  *M = R <= 8 ? 8 : 16;
  *MT = (R + *M - 1) / *M;
  *tile = kTileCols;
  *per_sm = hd == 64 ? 4 : 2;  // by shared memory: one CTA opens or merges while another streams
}

int launch_attn_mma(const AttnParams& p, int M, int rows, int grid, cudaStream_t stream) {
  CUtensorMap map;
  if (!kv_tensor_map(&map, p.cache, p.hd, p.cap, p.H, rows, kCols)) return SPECDEC_ERR_UNSUPPORTED;
  if (M == 8)
    return p.hd == 64 ? launch_mma<64, 1>(p, map, grid, stream) : launch_mma<128, 1>(p, map, grid, stream);
  return p.hd == 64 ? launch_mma<64, 2>(p, map, grid, stream) : launch_mma<128, 2>(p, map, grid, stream);
}

}  // namespace specdec
