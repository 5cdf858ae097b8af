// Attention of a draft tree over the cache on the tensor cores: bf16, head sizes 64 and 128.
//
// One CTA per SM, two accumulators of 128 query rows each, A and B.  With more than 128 rows in an
// M-tile pair, A and B are different rows over the same columns; with at most 128, they are the
// same rows over alternate column tiles and are merged at the end.  Either way one accumulator's
// softmax runs while the tensor cores work for the other.
//   warps 0-3, 4-7  softmax of A, B: one thread per row reads its 128 scores from tensor memory,
//                   keeps maximum and sum, writes the weights back as bf16 over the scores;
//   warp 8          TMA: K and V tiles of 128 columns into two stages each (128-byte swizzle);
//   warp 9          one thread issues S = Q K^T (both operands in shared memory) and
//                   O += P V (P from tensor memory, V as it lies: MN-major).
// Tensor memory (512 columns): S/P of A and B, O of A and B, 128 columns each.
// The running maximum is only followed when it grows by more than 2^8 in weight: O is then rescaled
// by the row's thread between its scores' arrival and its weights' release, when no MMA of that
// accumulator is in flight.  Weights below 2^8 lose nothing: bf16 and fp32 have the range.
//
// A tile that holds nodes' columns or the end of a row needs care: its V columns behind the nodes
// and of unused nodes are zeroed in shared memory (0 * NaN is NaN in a matrix product), and so are
// those of used nodes that hold something that is not finite; rows that see such a node get NaN.
#include <cmath>

#include "tcgen05.cuh"
#include "tree_attention.cuh"

namespace specdec {

namespace {

constexpr int kThreads = 384;  // the last two warps only make whole warpgroups of registers
// Registers per thread: 384 x 168 at launch; 2 x 128 x 216 + 128 x 64 = 63488 of those 64512.
constexpr int kRegsSoftmax = 216, kRegsOther = 64;
constexpr int kCols = 128;     // columns of a K/V tile
constexpr int kRows = 128;     // rows of an accumulator
constexpr int kStages = 2;
constexpr uint32_t kTries = 1u << 17, kNs = 20000;  // a wait gives up after about 2.6 s
constexpr float kGrow = 8.f;   // log2 of the growth of the maximum that is let pass

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
  return mbar_wait_sleep(bar, parity, kTries, kNs);
}
// The wait of a whole warp: one answer, so that its lanes stay together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(bar, parity));
}
// named_bar_sync that tells whether `ok` held in all n threads.
__device__ __forceinline__ bool named_bar_all(int id, int n, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(id), "r"(n), "r"(ok ? 1 : 0) : "memory");
  return r != 0;
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

struct Bars {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t q_full, v_clean, s_full[2], p_ready[2], o_done[2];
};

__device__ __forceinline__ bool inf_or_nan(uint32_t w) {  // either of two bf16 values
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

template <int HD> struct Smem {
  static constexpr int kQ = kRows * HD * 2, kTile = kCols * HD * 2;
  static constexpr int q = 0;                          // A's rows, then B's
  static constexpr int k = 2 * kQ, v = k + kStages * kTile;
  static constexpr int bytes = v + kStages * kTile + 1024;  // and alignment to 1024
};

// Byte offset of 16-byte chunk `c` of row `r` in a [rows][HD] bf16 tile: panels of 64 values,
// rows of 128 bytes, chunks xor-ed with the row (the 128-byte swizzle).
__device__ __forceinline__ int swizzled(int r, int c, int rows) {
  return (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Visibility of 32 columns that start `base` columns behind the committed ones.
__device__ __forceinline__ uint32_t visible32(unsigned long long anc, int base) {
  if (base >= 0) return base < 64 ? static_cast<uint32_t>(anc >> base) : 0u;
  if (base <= -32) return 0xffffffffu;
  return static_cast<uint32_t>(anc << -base) | ((1u << -base) - 1u);
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const AttnParams p, const __grid_constant__ CUtensorMap map) {
  using S = Smem<HD>;
  constexpr int kSteps = HD / 16, kPanels = HD / 64;
  extern __shared__ char raw[];
  __shared__ AttnPlan plan;
  __shared__ Bars bar;
  __shared__ uint32_t s_tmem;
  __shared__ int s_par[kMaxTree], s_flag, s_bad;
  __shared__ unsigned long long s_anc[kMaxTree], s_poison;
  __shared__ float2 s_ml[kRows];
  char* smem = raw + (1024 - smem_addr(raw) % 1024) % 1024;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == 0) attn_plan(p, kCols, plan);
  if (warp == 9) tmem_alloc(&s_tmem, 512);
  if (tid == 32) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_full[i], 1);
      mbar_init(&bar.v_empty[i], 1);
    }
    mbar_init(&bar.q_full, 256);
    mbar_init(&bar.v_clean, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_ready[i], 128);
      mbar_init(&bar.o_done[i], 1);
    }
    fence_mbar_init();
    s_poison = 0;
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = s_tmem;
  const AttnShares sh = attn_shares(p, plan);
  const int g = blockIdx.x / p.MT, mt = blockIdx.x % p.MT;
  const bool work = sh.total > 0 && g < sh.groups;
  const int x0 = work ? sh.start(g) : 0, x1 = work ? sh.start(g + 1) : 0;
  const int nrows = min(2 * kRows, p.T * p.G - mt * 2 * kRows);  // query rows of this pair
  const bool two = nrows > kRows;  // A and B are different rows, else alternate tiles
  bool ok = true;

  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
  if (warp == 8) {
    // ------------------------------------------------------------------------------- TMA
    if (lane == 0) {
      int kv = 0;  // tiles so far
      for (int x = x0; x < x1 && ok;) {
        const AttnSegment seg = attn_segment(p, plan, x, x1);
        x += seg.tile1 - seg.tile0;
        int err;
        const AttnRow row = attn_row(p, seg.b, &err);
        const int crow = p.one_row ? 0 : seg.b;
        for (int tile = seg.tile0; tile < seg.tile1; ++tile, ++kv) {
          const int st = kv % kStages, col = row.first + tile * kCols;
          const uint32_t ph = (kv / kStages) & 1;
          if (!(ok = wait(&bar.k_empty[st], ph ^ 1))) break;
          mbar_arrive_expect_tx(&bar.k_full[st], S::kTile);
          for (int j = 0; j < kPanels; ++j)
            tma_load_5d(smem + S::k + st * S::kTile + j * kCols * 128, &map, j * 64, col, seg.h,
                        crow, 0, &bar.k_full[st]);
          if (!(ok = wait(&bar.v_empty[st], ph ^ 1))) break;
          mbar_arrive_expect_tx(&bar.v_full[st], S::kTile);
          for (int j = 0; j < kPanels; ++j)
            tma_load_5d(smem + S::v + st * S::kTile + j * kCols * 128, &map, j * 64, col, seg.h,
                        crow, 1, &bar.v_full[st]);
        }
      }
      // no copy outlives the CTA: the last ones issued have landed (their tiles were used) unless
      // a wait gave up
      if (!ok)
        for (int i = max(0, kv - kStages); i <= kv; ++i) {
          (void)wait(&bar.k_full[i % kStages], (i / kStages) & 1);
          (void)wait(&bar.v_full[i % kStages], (i / kStages) & 1);
        }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------------------- MMA
    constexpr uint32_t id_s = mma_idesc(kRows, kCols, false), id_o = mma_idesc(kRows, HD, true);
    int kv = 0, seg_no = 0, done[2] = {0, 0};  // tiles, segments, jobs of A and B so far
    for (int x = x0; x < x1 && ok; ++seg_no) {
      const AttnSegment seg = attn_segment(p, plan, x, x1);
      const int n = seg.tile1 - seg.tile0, jobs = two ? 2 * n : n;
      x += n;
      int err;
      const AttnRow row = attn_row(p, seg.b, &err);
      // S = Q K^T of job i: tile i / 2 for A or B (two), or tile i
      auto scores = [&](int i) {
        const int a = i & 1, t = kv + (two ? i >> 1 : i), st = t % kStages;
        if (!two || a == 0) ok = ok && warp_wait(&bar.k_full[st], (t / kStages) & 1);
        if (!ok) return;
        if (lane == 0) {
          const uint32_t qa = smem_addr(smem + S::q + (two ? a : 0) * S::kQ);
          const uint32_t ka = smem_addr(smem + S::k + st * S::kTile);
          for (int s = 0; s < kSteps; ++s)
            mma_ss(tmem + a * kCols,
                   mma_desc(qa + (s >> 2) * kRows * 128 + (s & 3) * 32, 16, 1024),
                   mma_desc(ka + (s >> 2) * kCols * 128 + (s & 3) * 32, 16, 1024), id_s, s > 0);
          mma_commit(&bar.s_full[a]);
          if (!two || a == 1) mma_commit(&bar.k_empty[st]);
        }
        __syncwarp();
      };
      ok = warp_wait(&bar.q_full, seg_no & 1);
      tmem_fence_after();
      for (int i = 0; i < 2 && i < jobs && ok; ++i) scores(i);
      for (int i = 0; i < jobs && ok; ++i) {
        const int a = i & 1, tile = two ? i >> 1 : i, t = kv + tile, st = t % kStages;
        char* vt = smem + S::v + st * S::kTile;
        if (!two || a == 0) {
          if (!(ok = warp_wait(&bar.v_full[st], (t / kStages) & 1))) break;
          const int col0 = (seg.tile0 + tile) * kCols;
          if (col0 + kCols > row.old) {  // clean V where it may hold anything
            for (int c = max(0, row.old - col0); c < kCols; ++c) {
              const int node = col0 + c - row.old;
              const bool used = node < p.T && s_anc[node] != 0;
              uint4* v = reinterpret_cast<uint4*>(vt + swizzled(c, lane, kCols));
              bool bad = false;
              if (used) {
                if (lane < HD / 8) {
                  const uint4 w = *v;
                  bad = inf_or_nan(w.x) || inf_or_nan(w.y) || inf_or_nan(w.z) || inf_or_nan(w.w);
                }
                bad = __any_sync(0xffffffffu, bad);
                if (bad && lane == 0) s_poison |= 1ull << node;
              }
              if ((!used || bad) && lane < HD / 8) *v = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            __syncwarp();
          }
        }
        if (i == jobs - 1 && lane == 0) arrive(&bar.v_clean);  // the segment's V has been seen
        if (!(ok = warp_wait(&bar.p_ready[a], done[a] & 1))) break;
        ++done[a];
        tmem_fence_after();
        if (lane == 0) {
          const uint32_t va = smem_addr(vt);
          for (int s = 0; s < kCols / 16; ++s)
            mma_ts(tmem + (2 + a) * kCols, tmem + a * kCols + s * 8,
                   mma_desc(va + s * 2048, kCols * 128, 1024), id_o, i >= 2 || s > 0);
          if (!two || a == 1) mma_commit(&bar.v_empty[st]);
          if (i + 2 >= jobs) mma_commit(&bar.o_done[a]);
        }
        __syncwarp();
        if (i + 2 < jobs) scores(i + 2);
      }
      kv += n;
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------------------------- softmax
    const int a = warp >> 2, r = tid & (kRows - 1);       // accumulator, row of it
    const int pr = two ? a * kRows + r : r;               // row of the pair
    const int rr = mt * 2 * kRows + pr;                   // query row of the unit
    const bool mine = pr < nrows;
    const bool idle = (two ? a * kRows : 0) + (warp & 3) * 32 >= nrows;  // a warp without rows
    const int t_of = mine ? rr / p.G : 0;
    const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // lane 32 * (warp % 4)
    const uint32_t t_s = tmem + lane_base + a * kCols, t_o = tmem + lane_base + (2 + a) * kCols;
    // a scale of zero as the smallest one: hidden scores are -infinity and have to stay so
    const float scale = fmaxf(fabsf(p.scale_log2), 1.2e-38f);
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale turns Q
    int seg_no = 0, seen = 0, ends = 0, row_b = -1;  // segments, jobs, accumulations so far
    for (int x = x0; x < x1 && ok; ++seg_no) {
      const AttnSegment seg = attn_segment(p, plan, x, x1);
      const int n = seg.tile1 - seg.tile0;
      x += n;
      int err;
      const AttnRow row = attn_row(p, seg.b, &err);
      // the segment before is done with what is written now; all agree to go on
      if (!(ok = named_bar_all(1, 256, ok))) break;
      if (seg.b != row_b) {
        row_b = seg.b;
        if (p.parents && tid < p.T) s_par[tid] = p.parents[seg.b * p.T + tid];
        if (tid == 0) s_bad = 0;
        named_bar_sync(1, 256);
        if (tid < p.T) {
          bool bad = false;
          s_anc[tid] = tree_ancestors(p.parents ? s_par : nullptr, tid, bad);
          if (bad) {
            s_bad = 1;
            set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
          }
        }
      }
      if (tid == 0) s_poison = 0;
      {  // Q rows, swizzled; rows that do not exist are zero
        constexpr int kChunks = HD / 8;
        for (int i = tid; i < (two ? 2 : 1) * kRows * kChunks; i += 256) {
          const int q = i / kChunks, c = i % kChunks, qq = mt * 2 * kRows + q;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (q < nrows) {
            const int t = qq / p.G, h = seg.h * p.G + qq % p.G;
            v = __ldg(reinterpret_cast<const uint4*>(p.q + seg.b * p.qr + t * p.qt +
                                                     static_cast<long long>(h) * HD * 2) + c);
            v.x ^= flip;
            v.y ^= flip;
            v.z ^= flip;
            v.w ^= flip;
          }
          *reinterpret_cast<uint4*>(smem + S::q + (q / kRows) * S::kQ +
                                    swizzled(q % kRows, c, kRows)) = v;
        }
        fence_async_smem();
        arrive(&bar.q_full);
      }
      named_bar_sync(1, 256);
      const unsigned long long anc = mine ? s_anc[t_of] : 0ull;
      const int jobs = two ? n : (n - a + 1) >> 1;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < jobs; ++j, ++seen) {
        if (!(ok = warp_wait(&bar.s_full[a], seen & 1))) break;
        if (!idle) {
          tmem_fence_after();
          const int base = (seg.tile0 + (two ? j : 2 * j + a)) * kCols - row.old;
          // Two passes over the scores in tensor memory, 32 columns at a time: all 128 in registers
          // would leave too few for the rest.
          const auto load = [&](int c, uint32_t (&s)[32]) {
            tmem_ld32(t_s + c * 32, s);
            tmem_wait_ld();
            if (base + kCols > 0) {
              const uint32_t vis = visible32(anc, base + c * 32);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(vis >> k & 1)) s[k] = __float_as_uint(-INFINITY);
            }
          };
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t s[32];
            load(c, s);
            float q[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 32; ++k) q[k & 3] = fmaxf(q[k & 3], __uint_as_float(s[k]));
            mx = fmaxf(fmaxf(q[0], q[1]), fmaxf(q[2], q[3]));
          }
          mx *= scale;
          const bool up = mx > m + kGrow || (m == -INFINITY && mx > m);
          if (__any_sync(0xffffffffu, up)) {
            const float mn = up ? mx : m;
            const float f = up ? ex2(m - mn) : 1.f;
            l *= f;
            m = mn;
            if (j > 0) {
#pragma unroll 1
              for (int c = 0; c < HD / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(t_o + c * 16, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st16(t_o + c * 16, o);
              }
            }
          }
          const float off = m == -INFINITY ? 0.f : m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {  // the weights go over scores that have been read
            uint32_t s[32], w[16];
            load(c, s);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float e0 = ex2(fmaf(__uint_as_float(s[2 * k]), scale, -off));
              const float e1 = ex2(fmaf(__uint_as_float(s[2 * k + 1]), scale, -off));
              sum[k & 3] += e0 + e1;
              w[k] = bf16_pack(e0, e1);
            }
            tmem_st16(t_s + c * 16, w);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
          tmem_fence_before();
        }
        arrive(&bar.p_ready[a]);
      }
      // ----------------------------------------------------------------------------- output
      if (jobs > 0) ok = ok && warp_wait(&bar.o_done[a], ends++ & 1);
      ok = ok && warp_wait(&bar.v_clean, seg_no & 1);
      tmem_fence_after();
      if (anc & s_poison) l = __int_as_float(0x7FC00000);
      // this row's sums, B's merged into A's where both hold parts of one row
      float fa = 1.f, fb = 0.f;
      float* swap = reinterpret_cast<float*>(smem + S::q + S::kQ);  // [HD / 2][128], Q of B's rows
      auto part = [&](int c, float (&o)[32]) {  // columns 32c .. of this accumulator's O
        uint32_t u[32];
        if (jobs > 0 && !idle) {
          tmem_ld32(t_o + c * 32, u);
          tmem_wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = jobs > 0 && !idle ? __uint_as_float(u[k]) : 0.f;
      };
      const bool whole = seg.tile0 == 0 && seg.tile1 == seg.tiles;
      const int slot = whole ? 0 : attn_slot(p, sh, g, mt, seg.unit0);
      char* y = p.out + seg.b * p.outr + t_of * p.outt +
                static_cast<long long>(seg.h * p.G + (mine ? rr % p.G : 0)) * HD * 2;
      auto store_out = [&](int c, const float (&o)[32], float inv) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(y + c * 64 + k * 16) =
              make_uint4(bf16_pack(o[8 * k] * inv, o[8 * k + 1] * inv),
                         bf16_pack(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                         bf16_pack(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                         bf16_pack(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
      };
      auto store_lse = [&](float mm, float ll) {
        if (p.lse)
          p.lse[(static_cast<long long>(seg.b) * p.T + t_of) * p.Hq + seg.h * p.G + rr % p.G] =
              anc ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
      };
      const bool write = mine && !s_bad && ok;
      // one chunk of the row's merged sums goes to the output, or to the partial results
      auto emit = [&](int c, const float (&o)[32]) {
        if (!write) return;
        if (whole) {
          store_out(c, o, anc ? 1.f / l : 0.f);
        } else {
          float4* w = reinterpret_cast<float4*>(p.part_o) +
                      (static_cast<long long>(slot) * (HD / 4) + c * 8) * 2 * kRows + pr;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            w[k * 2 * kRows] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      };
      if (two) {
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          float o[32];
          part(c, o);
          emit(c, o);
        }
      } else {
        if (a == 1) s_ml[r] = make_float2(m, l);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (half) named_bar_sync(3, 256);  // A has read the first half
          if (a == 1) {
#pragma unroll 1
            for (int c = 0; c < HD / 64; ++c) {
              float o[32];
              part(half * (HD / 64) + c, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) swap[(c * 32 + k) * kRows + r] = o[k];
            }
          }
          named_bar_sync(2, 256);
          if (a == 0) {
            if (half == 0) {
              const float2 b = s_ml[r];
              const float mn = fmaxf(m, b.x), off = mn == -INFINITY ? 0.f : mn;
              fa = ex2(m - off);
              fb = ex2(b.x - off);
              l = l * fa + b.y * fb;
              m = mn;
            }
#pragma unroll 1
            for (int c = 0; c < HD / 64; ++c) {
              float o[32];
              part(half * (HD / 64) + c, o);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                o[k] = o[k] * fa + swap[(c * 32 + k) * kRows + r] * fb;
              emit(half * (HD / 64) + c, o);
            }
          }
        }
      }
      const bool owner = write && (two || a == 0);
      if (whole) {
        if (owner) store_lse(m, l);
        continue;
      }
      if (owner) p.part_ml[static_cast<long long>(slot) * 2 * kRows + pr] = make_float2(m, l);
      if (s_bad) continue;
      // the unit's last CTA merges the parts in share order
      const int g0 = sh.owner(seg.unit0), g1 = sh.owner(seg.unit0 + seg.tiles - 1);
      __threadfence();
      named_bar_sync(1, 256);
      if (tid == 0) {
        unsigned* t = &p.ticket[(static_cast<long long>(seg.b) * p.H + seg.h) * p.MT + mt];
        const unsigned old = atomicAdd(t, 1u);
        s_flag = old + 1 == static_cast<unsigned>(g1 - g0 + 1);
        if (s_flag) *t = 0;
        __threadfence();
      }
      named_bar_sync(1, 256);
      if (!s_flag || !mine) continue;
      float mm = -INFINITY, ll = 0.f;
      for (int gg = g0; gg <= g1; ++gg) {
        const float2 w = __ldcg(p.part_ml + static_cast<long long>(attn_slot(p, sh, gg, mt, seg.unit0)) * 2 * kRows + pr);
        const float mn = fmaxf(mm, w.x), of = mn == -INFINITY ? 0.f : mn;
        ll = ll * ex2(mm - of) + w.y * ex2(w.x - of);
        mm = mn;
      }
      const float of = mm == -INFINITY ? 0.f : mm, inv = anc ? 1.f / ll : 0.f;
      // one row per thread, or (with A and B on the same rows) half of a row's values each
      const int c0 = two ? 0 : a * (HD / 64), c1 = two ? HD / 32 : c0 + HD / 64;
#pragma unroll 1
      for (int c = c0; c < c1; ++c) {
        float o[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0.f;
        for (int gg = g0; gg <= g1; ++gg) {
          const long long sl = attn_slot(p, sh, gg, mt, seg.unit0);
          const float f = ex2(__ldcg(p.part_ml + sl * 2 * kRows + pr).x - of);
          const float4* w = reinterpret_cast<const float4*>(p.part_o) + (sl * (HD / 4) + c * 8) * 2 * kRows + pr;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 v = __ldcg(w + k * 2 * kRows);
            o[4 * k] += v.x * f;
            o[4 * k + 1] += v.y * f;
            o[4 * k + 2] += v.z * f;
            o[4 * k + 3] += v.w * f;
          }
        }
        store_out(c, o, inv);
      }
      if (two || a == 0) store_lse(mm, ll);
    }
  }
  if (!ok) set_status(p.status, SPECDEC_ERR_TIMEOUT);
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == 9) {
    tmem_fence_after();
    tmem_free(tmem, 512);
  }
}

template <int HD>
int launch_tc(const AttnParams& p, const CUtensorMap& map, int grid, cudaStream_t stream) {
  auto kernel = attn_tc_kernel<HD>;
  constexpr int smem = Smem<HD>::bytes;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return map_cuda_error(e);
  kernel<<<grid, kThreads, smem, stream>>>(p, map);
  return map_cuda_error(cudaGetLastError());
}

}  // namespace

bool kv_tensor_map(CUtensorMap* map, const ByteView& v, int head_dim, int cap, int heads, int rows,
                   int box_cols) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess || q != cudaDriverEntryPointSuccess)
      f = nullptr;
    (void)cudaGetLastError();
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return false;
  // a dimension of one entry has no stride that matters, but the driver wants a valid one
  const cuuint64_t col = static_cast<cuuint64_t>(head_dim) * 2;
  const cuuint64_t dims[5] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(cap),
                              static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows), 2};
  const cuuint64_t strides[4] = {col, heads > 1 ? static_cast<cuuint64_t>(v.shead) : col,
                                 rows > 1 ? static_cast<cuuint64_t>(v.srow) : col,
                                 static_cast<cuuint64_t>(v.skv)};
  for (int i = 0; i < 4; ++i)
    if (strides[i] == 0 || strides[i] % 16 || strides[i] >= (1ull << 40)) return false;
  const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(box_cols), 1, 1, 1};
  const cuuint32_t step[5] = {1, 1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, v.base, dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shape of the tensor-core kernel for R query rows per K/V head.
void attn_tc_shape(int R, int* M, int* MT) {
  *M = 2 * kRows;
  *MT = (R + 2 * kRows - 1) / (2 * kRows);
}

int launch_attn_tc(const AttnParams& p, int rows, int grid, cudaStream_t stream) {
  CUtensorMap map;
  if (!kv_tensor_map(&map, p.cache, p.hd, p.cap, p.H, rows, kCols)) return SPECDEC_ERR_UNSUPPORTED;
  return p.hd == 64 ? launch_tc<64>(p, map, grid, stream) : launch_tc<128>(p, map, grid, stream);
}

}  // namespace specdec
