// Attention of a draft tree over the cache for few query rows per K/V head: bf16, head sizes 64
// and 128, M-tiles of 16 rows.
//
// With at most 16 rows (a token or a short chain with one or a few query heads per K/V head) a
// K/V column of 512 bytes meets 16 * 512 flops: HBM bounds it, and tensor memory's 128-row tiles
// would be nearly empty.  So a warp is the unit: it streams its own 32 columns of each 128-column
// tile by TMA (128-byte swizzle) into two private stages, without any CTA-wide barrier, and runs
// both products with m16n8k16: S = Q K^T (Q in registers for the whole segment), the softmax
// weights' accumulator layout is the next product's A operand as it stands, O += P V.  Each warp
// keeps maximum, sum and O of its columns; the four are merged in shared memory when the
// segment ends, while the next segment's tiles are already on their way.
#include <cmath>

#include "tcgen05.cuh"
#include "tree_attention.cuh"

namespace specdec {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kRows = 16;
constexpr int kCols = 32;                // columns of a warp's slice of a tile
constexpr int kTileCols = kCols * kWarps;
constexpr int kStages = 2;
constexpr uint32_t kTries = 1u << 17, kNs = 20000;  // a wait gives up after about 2.6 s

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
__device__ __forceinline__ bool inf_or_nan(uint32_t w) {  // either of two bf16 values
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

template <int HD> struct Smem {
  static constexpr int kSlice = kCols * HD * 2;               // K or V of a warp's slice
  static constexpr int kWarp = kStages * 2 * kSlice;          // [stage][K, V]
  static constexpr int kPitch = HD + 4;                       // floats of a row to merge
  static constexpr int merge = kWarps * kWarp;                // [warp][16][kPitch]
  static constexpr int bytes = merge + kWarps * kRows * kPitch * 4 + 1024;
};

// Walks the tiles of a share, segment by segment.
struct Cursor {
  AttnSegment seg;
  int tile;   // of the segment
  bool more;  // not behind the last
};

template <int HD>
__global__ void __launch_bounds__(kThreads)
attn_mma_kernel(const AttnParams p, const __grid_constant__ CUtensorMap map) {
  using S = Smem<HD>;
  constexpr int kSteps = HD / 16, kPanels = HD / 64;
  extern __shared__ char raw[];
  __shared__ AttnPlan plan;
  __shared__ uint64_t s_full[kWarps][kStages];
  __shared__ int s_par[kMaxTree], s_flag, s_bad;
  __shared__ unsigned long long s_anc[kMaxTree];
  __shared__ float2 s_ml[kWarps][kRows];
  char* smem = raw + (1024 - smem_addr(raw) % 1024) % 1024;
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
    // this thread's rows gr and gr + 8: Q as A operand, ancestors
    uint32_t q[kSteps][4];
    unsigned long long anc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = gr + 8 * i, rr = mt * kRows + r;
      const bool in = r < nrows;
      const int t = in ? rr / p.G : 0, h = seg.h * p.G + (in ? rr % p.G : 0);
      anc[i] = in ? s_anc[t] : 0ull;
      const char* src = p.q + seg.b * p.qr + t * p.qt + static_cast<long long>(h) * HD * 2 + qd * 4;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        q[s][i] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + s * 32)) ^ flip : 0u;
        q[s][i + 2] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + s * 32 + 16)) ^ flip : 0u;
      }
    }
    float o[HD / 8][4];
#pragma unroll
    for (int j = 0; j < HD / 8; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[j][k] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    unsigned long long poison = 0;
    for (int tile = seg.tile0; tile < seg.tile1; ++tile, ++used) {
      const int st = used % kStages;
      ok = ok && __all_sync(0xffffffffu, mbar_wait_sleep(&s_full[warp][st], (used / kStages) & 1,
                                                         kTries, kNs));
      const int col = tile * kTileCols + warp * kCols, base = col - seg.old;
      if (ok && col < seg.cols) {
        const char* km = mem + st * 2 * S::kSlice;
        char* vm = mem + (st * 2 + 1) * S::kSlice;
        const uint32_t ka = smem_addr(km), va = smem_addr(vm);
        float s[kCols / 8][4];
#pragma unroll
        for (int j = 0; j < kCols / 8; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[j][k] = 0.f;
        const int mi = lane >> 3, mr = lane & 7;  // matrix and row this lane addresses
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
#pragma unroll
          for (int j = 0; j < kCols / 16; ++j) {
            const int c = j * 16 + (mi >> 1) * 8 + mr, ch = k * 2 + (mi & 1);
            uint32_t b0, b1, b2, b3;
            ldmatrix4(ka + (ch >> 3) * kCols * 128 + c * 128 + (((ch & 7) ^ mr) << 4), b0, b1, b2, b3);
            mma16816(s[2 * j], q[k], b0, b1);
            mma16816(s[2 * j + 1], q[k], b2, b3);
          }
        }
        if (base + kCols > 0) {
          // columns behind the committed ones: what each row sees, and V where it may hold anything
#pragma unroll
          for (int j = 0; j < kCols / 8; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int node = base + j * 8 + qd * 2 + (k & 1);
              if (node >= 0 && !(node < p.T && (anc[k >> 1] >> node & 1))) s[j][k] = -INFINITY;
            }
          const int node = base + lane;  // a lane looks after one column
          bool bad = false;
          if (node >= 0) {
            const bool live = node < p.T && s_anc[node] != 0;
            if (live)
              for (int ch = 0; ch < HD / 8; ++ch) {
                const uint4 v = *reinterpret_cast<const uint4*>(vm + (ch >> 3) * kCols * 128 + lane * 128 + (((ch & 7) ^ (lane & 7)) << 4));
                bad |= inf_or_nan(v.x) || inf_or_nan(v.y) || inf_or_nan(v.z) || inf_or_nan(v.w);
              }
            if (!live || bad)
              for (int ch = 0; ch < HD / 8; ++ch)
                *reinterpret_cast<uint4*>(vm + (ch >> 3) * kCols * 128 + lane * 128 + (((ch & 7) ^ (lane & 7)) << 4)) = make_uint4(0, 0, 0, 0);
          }
          const unsigned long long which = __ballot_sync(0xffffffffu, bad);
          if (which) poison |= base >= 0 ? which << base : which >> -base;
          fence_async_smem();
          __syncwarp();
        }
        float f[2];
        bool up = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = s[0][2 * i];
#pragma unroll
          for (int j = 0; j < kCols / 8; ++j) mx = fmaxf(mx, fmaxf(s[j][2 * i], s[j][2 * i + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * scale;
          const float mn = fmaxf(m[i], mx);
          up |= mn > m[i];
          f[i] = mn > m[i] ? ex2(m[i] - mn) : 1.f;
          m[i] = mn;
          const float off = mn == -INFINITY ? 0.f : mn;
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < kCols / 8; ++j) {
            s[j][2 * i] = ex2(fmaf(s[j][2 * i], scale, -off));
            s[j][2 * i + 1] = ex2(fmaf(s[j][2 * i + 1], scale, -off));
            sum += s[j][2 * i] + s[j][2 * i + 1];
          }
          l[i] = l[i] * f[i] + sum;
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int j = 0; j < HD / 8; ++j) {
            o[j][0] *= f[0];
            o[j][1] *= f[0];
            o[j][2] *= f[1];
            o[j][3] *= f[1];
          }
        }
#pragma unroll
        for (int kb = 0; kb < kCols / 16; ++kb) {
          // the weights, rounded to bf16: with V in bf16 the product takes nothing wider
          const uint32_t pa[4] = {bf16_pack(s[2 * kb][0], s[2 * kb][1]), bf16_pack(s[2 * kb][2], s[2 * kb][3]),
                                  bf16_pack(s[2 * kb + 1][0], s[2 * kb + 1][1]), bf16_pack(s[2 * kb + 1][2], s[2 * kb + 1][3])};
#pragma unroll
          for (int n = 0; n < HD / 16; ++n) {
            const int c = kb * 16 + (mi & 1) * 8 + mr, ch = n * 2 + (mi >> 1);
            uint32_t b0, b1, b2, b3;
            ldmatrix4t(va + (ch >> 3) * kCols * 128 + c * 128 + (((ch & 7) ^ mr) << 4), b0, b1, b2, b3);
            mma16816(o[2 * n], pa, b0, b1);
            mma16816(o[2 * n + 1], pa, b2, b3);
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
    // ------------------------------------------------------------- the four warps' parts
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (anc[i] & poison) l[i] = __int_as_float(0x7FC00000);  // the row sees a column that is not finite
    }
    __syncthreads();  // the segment before has been merged
    if (qd == 0) {
      s_ml[warp][gr] = make_float2(m[0], l[0]);
      s_ml[warp][gr + 8] = make_float2(m[1], l[1]);
    }
#pragma unroll
    for (int j = 0; j < HD / 8; ++j) {
      float* w = merge + (warp * kRows + gr) * S::kPitch + j * 8 + qd * 2;
      *reinterpret_cast<float2*>(w) = make_float2(o[j][0], o[j][1]);
      *reinterpret_cast<float2*>(w + 8 * S::kPitch) = make_float2(o[j][2], o[j][3]);
    }
    __syncthreads();
    const int r = tid >> 3, d0 = (tid & 7) * 4;  // row, and every 32nd group of 4 values from d0
    const int rr = mt * kRows + r;
    const bool mine = r < nrows && !s_bad;
    const int t = mine ? rr / p.G : 0, h = seg.h * p.G + (mine ? rr % p.G : 0);
    const bool live = mine && s_anc[t] != 0;
    float mm = -INFINITY, ll = 0.f;
    float4 acc[HD / 32];
#pragma unroll
    for (int j = 0; j < HD / 32; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float2 ml, auto at) {  // one more part of the row
      const float mn = fmaxf(mm, ml.x), off = mn == -INFINITY ? 0.f : mn;
      const float fa = ex2(mm - off), fb = ex2(ml.x - off);
      ll = ll * fa + ml.y * fb;
      mm = mn;
#pragma unroll
      for (int j = 0; j < HD / 32; ++j) {
        const float4 v = at(j);
        acc[j].x = acc[j].x * fa + v.x * fb;
        acc[j].y = acc[j].y * fa + v.y * fb;
        acc[j].z = acc[j].z * fa + v.z * fb;
        acc[j].w = acc[j].w * fa + v.w * fb;
      }
    };
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      add(s_ml[w][r], [&](int j) {
        return *reinterpret_cast<const float4*>(merge + (w * kRows + r) * S::kPitch + d0 + j * 32);
      });
    if (seg.tile0 > 0 || seg.tile1 < seg.tiles) {
      const long long at = static_cast<long long>(attn_slot(p, sh, g, mt, seg.unit0)) * kRows + r;
      if (mine) {
        if (d0 == 0) p.part_ml[at] = make_float2(mm, ll);
#pragma unroll
        for (int j = 0; j < HD / 32; ++j)
          *reinterpret_cast<float4*>(p.part_o + at * HD + d0 + j * 32) = acc[j];
      }
      if (s_bad) continue;
      const int g0 = sh.owner(seg.unit0), g1 = sh.owner(seg.unit0 + seg.tiles - 1);
      if (!attn_last(p, seg.b, seg.h, mt, g1 - g0 + 1, &s_flag)) continue;
      mm = -INFINITY;
      ll = 0.f;
#pragma unroll
      for (int j = 0; j < HD / 32; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (mine)
        for (int gg = g0; gg <= g1; ++gg) {
          const long long a2 = static_cast<long long>(attn_slot(p, sh, gg, mt, seg.unit0)) * kRows + r;
          add(__ldcg(p.part_ml + a2), [&](int j) {
            return __ldcg(reinterpret_cast<const float4*>(p.part_o + a2 * HD + d0 + j * 32));
          });
        }
    }
    if (!mine) continue;
    const float inv = live ? 1.f / ll : 0.f;
    char* y = p.out + seg.b * p.outr + t * p.outt + static_cast<long long>(h) * HD * 2;
#pragma unroll
    for (int j = 0; j < HD / 32; ++j)
      *reinterpret_cast<uint2*>(y + (d0 + j * 32) * 2) =
          make_uint2(bf16_pack(acc[j].x * inv, acc[j].y * inv), bf16_pack(acc[j].z * inv, acc[j].w * inv));
    if (p.lse && d0 == 0)
      p.lse[(static_cast<long long>(seg.b) * p.T + t) * p.Hq + h] =
          live ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
  }
  if (!ok) {
    set_status(p.status, SPECDEC_ERR_TIMEOUT);
    // no copy outlives the CTA: those asked for and not waited for have landed
    for (int i = used; i < loaded; ++i)
      (void)mbar_wait_sleep(&s_full[warp][i % kStages], (i / kStages) & 1, kTries, kNs);
  }
}

template <int HD>
int launch_mma(const AttnParams& p, const CUtensorMap& map, int grid, cudaStream_t stream) {
  auto kernel = attn_mma_kernel<HD>;
  constexpr int smem = Smem<HD>::bytes;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return map_cuda_error(e);
  kernel<<<grid, kThreads, smem, stream>>>(p, map);
  return map_cuda_error(cudaGetLastError());
}

}  // namespace

void attn_mma_shape(int R, int hd, int* M, int* MT, int* per_sm) {
  *M = kRows;
  *MT = (R + kRows - 1) / kRows;
  *per_sm = hd == 64 ? 2 : 1;  // by shared memory
}

int launch_attn_mma(const AttnParams& p, int rows, int grid, cudaStream_t stream) {
  CUtensorMap map;
  if (!kv_tensor_map(&map, p.cache, p.hd, p.cap, p.H, rows, kCols)) return SPECDEC_ERR_UNSUPPORTED;
  return p.hd == 64 ? launch_mma<64>(p, map, grid, stream) : launch_mma<128>(p, map, grid, stream);
}

}  // namespace specdec
