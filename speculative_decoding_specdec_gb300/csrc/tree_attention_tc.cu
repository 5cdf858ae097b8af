// Attention of a draft tree over the cache on the tensor cores: bf16, head sizes 64 and 128.
//
// One CTA per SM, two accumulators of 128 query rows each, A and B.  With more than 128 rows in an
// M-tile pair, A and B are different rows over the same columns; with at most 128, they are the
// same rows over alternate column tiles and are merged at the end.  Either way one accumulator's
// softmax runs while the tensor cores work for the other.
//   warps 0-3, 4-7  softmax of A, B: one thread per row reads its 128 scores from tensor memory,
//                   keeps maximum and sum, writes the weights back as bf16 over the scores;
//   warps 8, 10     TMA: K, V tiles of 128 columns into two stages or three (128-byte swizzle);
//   warp 9          one thread issues S = Q K^T (both operands in shared memory) and
//                   O += P V (P from tensor memory, V as it lies: MN-major).
// Tensor memory (512 columns): S/P of A and B, O of A and B, 128 columns each.
// The running maximum is only followed when it grows by more than 2^32 in weight (and from the
// first columns on): until then weights, their sum and O are that much larger, which neither fp32
// nor bf16 minds.  O is then rescaled by the row's thread, when no product of that accumulator is
// in flight.
//
// What bounds it.  512 rows over 4600 columns (32 trees of 32 nodes, 16 query heads per K/V head):
// 86 us, 0.79 PFLOP/s; 256 rows over 131071 columns: 124 us, 1.10 PFLOP/s and 4.3 TB/s.  In the latter
// a CTA takes 54 tile pairs in 212000 active cycles, 3900 a pair where its products take 2048 at the
// peak rate (the tensor pipe is busy for 52 %): an accumulator's softmax stands between its two
// products.  In the former the pipe is busy for 43 %: more segments are opened and closed.
//
// A tile that holds nodes' columns or the end of a row needs care: its V columns behind the nodes
// and of unused nodes are zeroed in shared memory (0 * NaN is NaN in a matrix product), and so is
// what is not finite of the used nodes'; the rows that see such a node get it back from the cache
// when they are written.
#include <cmath>

#include "tcgen05.cuh"
#include "tree_attention.cuh"

namespace specdec {

namespace {

constexpr int kThreads = 384;  // (the last warp only completes the third warpgroup)
// Registers per thread: 384 x 168 at launch; 2 x 128 x 224 + 128 x 56 = those 64512.
constexpr int kRegsSoftmax = 224, kRegsOther = 56;
constexpr int kCols = 128;     // columns of a K/V tile
constexpr int kRows = 128;     // rows of an accumulator
constexpr int kStages = 2;      // of V, and of K where A and B are different rows; else K has one more
constexpr int kMaxKStages = 3;
constexpr uint32_t kTries = 1u << 18;  // polls after which a wait gives up
constexpr float kGrow = 32.f;  // log2 of the growth of the maximum that is let pass

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
  return mbar_wait_bounded(bar, parity, kTries);
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
  uint64_t k_full[kMaxKStages], k_empty[kMaxKStages], v_full[kStages], v_empty[kStages];
  uint64_t q_full, v_clean, s_full[2], p_ready[2], o_done[2], drained;
};

// Tiles of a unit that are of its prefix (they come first).
template <bool kBoth> __device__ __forceinline__ int prefix_tiles(const AttnSegment& s) {
  return kBoth ? (s.plen + kCols - 1) / kCols : 0;
}

template <int HD> struct Smem {
  static constexpr int kQ = kRows * HD * 2, kTile = kCols * HD * 2;
  static constexpr int q = 0;                          // A's rows, then B's
  static constexpr int k = 2 * kQ, v = k + kStages * kTile;
  static constexpr int bytes = v + kStages * kTile + 1024;  // and alignment to 1024
  // K's stage i: the third is where B's rows of Q would be
  __host__ __device__ static constexpr int k_stage(int i) { return i < kStages ? k + i * kTile : kQ; }
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

// kMode: over the rows' own columns, alone or behind a prefix pass, a prefix pass, or both parts in one
// (map2: the prefixes').
template <int HD, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const AttnParams p, const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map2) {
  using S = Smem<HD>;
  constexpr bool kPrefix = kMode == kPrefixPass, kBoth = kMode == kBothParts, kHasPrior = kMode == kBehind;
  constexpr int kSteps = HD / 16, kPanels = HD / 64;
  extern __shared__ char raw[];
  __shared__ Bars bar;
  __shared__ uint32_t s_tmem;
  __shared__ int s_par[kMaxTree], s_bad;
  __shared__ unsigned long long s_anc[kMaxTree], s_poison;
  __shared__ float2 s_ml[kRows];
  char* smem = raw + (1024 - smem_addr(raw) % 1024) % 1024;
  const AttnPlan plan = attn_plan_at(smem + S::bytes - 1024, kPrefix ? p.P : p.B);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.x / p.MT, mt = blockIdx.x % p.MT;
  int nrows = min(2 * kRows, p.T * p.G - mt * 2 * kRows);  // query rows of this pair (prefix pass: of the unit)
  const bool two = kPrefix ? p.two != 0 : nrows > kRows;   // A and B are different rows, else alternate tiles
  if (warp == 0) attn_plan<kMode>(p, kCols, plan);
  if (warp == 9) tmem_alloc(&s_tmem, 512);
  if (tid == 32) {
    for (int i = 0; i < kMaxKStages; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.v_full[i], 1);
      mbar_init(&bar.v_empty[i], 1);
    }
    mbar_init(&bar.q_full, 256);
    mbar_init(&bar.v_clean, 1);
    mbar_init(&bar.drained, 1);
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
  pdl_launch_dependents();  // the merge of cut units may be set up
  const uint32_t tmem = s_tmem;
  const AttnShares sh = attn_shares<kMode>(p, plan);
  const bool work = sh.total > 0 && g < sh.groups;
  const int x0 = work ? sh.start(g) : 0, x1 = work ? sh.start(g + 1) : 0;
  const int nk = two ? kStages : kMaxKStages;
  bool ok = true;

  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
  if (warp == 8 || warp == 10) {
    // ------------------------------------------------------------------------------- TMA
    // Warp 8 for K, warp 10 for V: one for both would hold K back until a stage of V is free.
    if (lane == 0) {
      const bool is_v = warp == 10;
      const int stages = is_v ? kStages : nk;
      uint64_t *full = is_v ? bar.v_full : bar.k_full, *empty = is_v ? bar.v_empty : bar.k_empty;
      int n = 0;  // tiles so far
      AttnSegment seg;
      for (int x = x0; ok && attn_next<kMode>(p, plan, x, x1, seg); x = seg.next) {
        const int crow = p.one_row ? 0 : seg.b, pt = prefix_tiles<kBoth>(seg);
        for (int tile = seg.tile0; tile < seg.tile1; ++tile, ++n) {
          const bool of_prefix = kBoth && tile < pt;
          const int st = n % stages, col = of_prefix ? seg.pfirst + tile * kCols : seg.first + (tile - pt) * kCols;
          // the first product needs K and Q: what comes after must not stand before Q in the queue
          if (n == (is_v ? 0 : 1) && !(ok = wait(&bar.q_full, 0))) break;
          if (!(ok = wait(&empty[st], ((n / stages) & 1) ^ 1))) break;
          mbar_arrive_expect_tx(&full[st], S::kTile);
          char* to = smem + (is_v ? S::v + st * S::kTile : S::k_stage(st));
          for (int j = 0; j < kPanels; ++j)
            tma_load_5d(to + j * kCols * 128, of_prefix ? &map2 : &map, j * 64, col, seg.h, of_prefix ? seg.prow : crow, is_v, &full[st]);
        }
      }
      // no copy outlives the CTA: the last ones issued have landed (their tiles were used) unless
      // a wait gave up
      if (!ok)
        for (int i = max(0, n - stages); i < n; ++i) (void)wait(&full[i % stages], (i / stages) & 1);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------------------- MMA
    // The whole warp follows the jobs, A's and B's in turn, and one elected lane issues.  In turn,
    // so that one accumulator's softmax runs beside the other's products: with a warp for each, the
    // two fell into step, and both waited while both computed.  A wait costs this warp time even
    // where there is nothing to wait for, with the tensor cores idle, so it has one per job: the
    // softmax's threads see to V and the next K before they release the weights.  What an MMA's operands are made of
    // is the same in all lanes and made so for the compiler to see (the shuffles): an MMA takes
    // its descriptors from uniform registers, and moving them there lane by lane took longer than
    // the products.
    constexpr uint32_t id_s = mma_idesc(kRows, kCols, false), id_o = mma_idesc(kRows, HD, true);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t sm = __shfl_sync(0xffffffffu, smem_addr(smem), 0);
    const bool pair = __shfl_sync(0xffffffffu, two ? 1 : 0, 0) != 0;
    const uint64_t q_desc = mma_desc(sm + S::q, 16, 1024), k_desc = mma_desc(sm, 16, 1024),
                   v_desc = mma_desc(sm + S::v, kCols * 128, 1024);
    int kv = 0, seg_no = 0, done[2] = {0, 0};  // tiles, segments, jobs of A and B so far
    AttnSegment seg;
    for (int x = x0; ok && attn_next<kMode>(p, plan, x, x1, seg); x = seg.next, ++seg_no) {
      const int n = __shfl_sync(0xffffffffu, seg.tile1 - seg.tile0, 0), jobs = pair ? 2 * n : n;
      const int pt = prefix_tiles<kBoth>(seg);
      const int clean = pt + seg.old / kCols - seg.tile0;  // the first tile that needs care
      const int ragged = kBoth && seg.plen % kCols ? pt - 1 - seg.tile0 : -1;  // and the prefix's last
      // Job i is tile i / 2 for A or B (pair), or tile i for one of them.
      auto tile_of = [&](int i) { return pair ? i >> 1 : i; };
      auto full = [&](uint64_t* bars, int stages, int i) {  // K or V of job i
        const int t = kv + tile_of(i);
        if (!pair || !(i & 1)) ok = ok && warp_wait(&bars[t % stages], (t / stages) & 1);
      };
      auto scores = [&](int i) {  // S = Q K^T
        const int a = i & 1, st = pair ? (kv + (i >> 1)) % kStages : (kv + i) % kMaxKStages;
        const uint64_t qa = q_desc + (pair ? a : 0) * (S::kQ / 16), ka = k_desc + S::k_stage(st) / 16;
        const uint32_t d = tm + a * kCols;
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < kSteps; ++s)
            mma_ss(d, qa + ((s >> 2) * kRows * 128 + (s & 3) * 32) / 16,
                   ka + ((s >> 2) * kCols * 128 + (s & 3) * 32) / 16, id_s, s > 0);
          mma_commit(&bar.s_full[a]);
          if (!pair || a == 1) mma_commit(&bar.k_empty[st]);
        }
        __syncwarp();
      };
      ok = warp_wait(&bar.q_full, seg_no & 1);
      tmem_fence_after();
      for (int i = 0; i < 2 && i < jobs; ++i) {
        full(bar.k_full, nk, i);
        if (ok) scores(i);
      }
      for (int i = 0; i < jobs && ok; ++i) {
        const int a = i & 1, tile = tile_of(i), st = (kv + tile) % kStages;
        const bool of_prefix = kBoth && seg.tile0 + tile < pt;
        const int col0 = (seg.tile0 + tile - (of_prefix ? 0 : pt)) * kCols;
        const int steps = min(kCols / 16, ((of_prefix ? seg.plen : seg.cols) - col0 + 15) >> 4);
        if ((tile >= clean || (kBoth && tile == ragged)) && (!pair || a == 0)) {
          full(bar.v_full, kStages, i);
          if (!ok) break;
          // clean V where it may hold anything: a lane per column (steps of 16 columns behind the
          // last are left out of the product)
          char* vt = smem + S::v + st * S::kTile;
          for (int c = max(0, (of_prefix ? seg.plen : seg.old) - col0) + lane; c < steps * 16; c += 32) {
            const int node = col0 + c - seg.old;
            const bool drop = kPrefix || of_prefix || node >= p.T || s_anc[node] == 0;
            auto at = [&](int k) { return reinterpret_cast<uint4*>(vt + swizzled(c, k, kCols)); };
            if (!drop) {
              bool bad = false;
#pragma unroll
              for (int k = 0; k < HD / 8; ++k) bad |= inf_or_nan(*at(k));
              if (bad) {
                atomicOr(&s_poison, 1ull << node);
                attn_make_finite(vt, c, kCols, 0, HD / 8);
              }
            } else {
#pragma unroll
              for (int k = 0; k < HD / 8; ++k) *at(k) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_async_smem();
          __syncwarp();
        }
        if (i == jobs - 1 && lane == 0) arrive(&bar.v_clean);  // the segment's V has been seen
        const uint64_t va = v_desc + st * (S::kTile / 16);
        const uint32_t d = tm + (2 + a) * kCols, w = tm + a * kCols;
        // weights, and with them V and the next K: one wait per job
        if (!(ok = warp_wait(&bar.p_ready[a], done[a] & 1))) break;
        ++done[a];
        tmem_fence_after();
        if (elect_one()) {
          mma_ts(d, w, va, id_o, i >= 2);
#pragma unroll
          for (int s = 1; s < kCols / 16; ++s)
            if (s < steps) mma_ts(d, w + s * 8, va + s * (2048 / 16), id_o, true);
          if (!pair || a == 1) mma_commit(&bar.v_empty[st]);
          if (i + 2 >= jobs) mma_commit(&bar.o_done[a]);
        }
        __syncwarp();
        if (i + 2 < jobs) scores(i + 2);
      }
      kv += n;
    }
    // where a wait gave up, products may still be on their way to tensor memory, which is freed below
    if (!ok) {
      if (elect_one()) mma_commit(&bar.drained);
      (void)warp_wait(&bar.drained, 0);
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------------------------- softmax
    const int a = warp >> 2, r = tid & (kRows - 1);       // accumulator, row of it
    const int pr = two ? a * kRows + r : r;               // row of the pair
    const int rr = mt * 2 * kRows + pr;                   // query row of the unit
    bool mine = pr < nrows;
    bool idle = (two ? a * kRows : 0) + (warp & 3) * 32 >= nrows;  // a warp without rows
    const int t_of = !kPrefix && mine ? rr / p.G : 0;
    const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // lane 32 * (warp % 4)
    const uint32_t t_s = tmem + lane_base + a * kCols, t_o = tmem + lane_base + (2 + a) * kCols;
    // a scale of zero as the smallest one: hidden scores are -infinity and have to stay so
    const float scale = fmaxf(fabsf(p.scale_log2), 1.2e-38f);
    int seg_no = 0, seen = 0, ends = 0, kv = 0;  // segments, jobs, accumulations, tiles so far
    // A thread copies its 16-byte chunk of every kPer-th Q row straight to shared memory (rows that
    // do not exist are zero): holding them in registers over the segment before made the compiler
    // spill them, one round trip to memory each.
    constexpr int kChunks = HD / 8, kPer = 256 / kChunks, kLoads = 2 * kRows / kPer;
    const int qc = tid % kChunks, q0 = tid / kChunks, nq = two ? kLoads : kLoads / 2;
    auto ask = [&](const AttnSegment& sg) {
      const char* base = p.q + (kPrefix ? 0 : sg.b) * p.qr + static_cast<long long>(sg.h) * p.G * HD * 2 + qc * 16;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int q = q0 + k * kPer, qq = mt * 2 * kRows + q;
        if (kPrefix && k < nq) {
          const AttnQuery at = attn_query<true>(p, sg, q < sg.rows ? q : 0);
          cp_async16(smem + S::q + (q / kRows) * S::kQ + swizzled(q % kRows, qc, kRows),
                     p.q + at.b * p.qr + at.t * p.qt + at.h * (HD * 2) + qc * 16, q < sg.rows);
        } else if (k < nq) {
          const int t = p.g_shift >= 0 ? qq >> p.g_shift : qq / p.G;
          cp_async16(smem + S::q + (q / kRows) * S::kQ + swizzled(q % kRows, qc, kRows),
                     q < nrows ? base + t * p.qt + (qq - t * p.G) * (HD * 2) : p.q, q < nrows);
        }
      }
      if (!kPrefix && p.parents && tid < p.T) s_par[tid] = __ldg(p.parents + sg.b * p.T + tid);
    };
    // Q has arrived: ancestors, and the products may begin
    auto open = [&] {
      if (!kPrefix && tid < p.T) {
        bool bad = false;
        s_anc[tid] = tree_ancestors(p.parents ? s_par : nullptr, tid, bad);
        if (bad) {
          s_bad = 1;
          set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
        }
      }
      cp_async_wait_all();
      if (p.scale_log2 < 0.f)  // a negative scale turns Q (each thread what it copied)
        for (int k = 0; k < nq; ++k) {
          const int q = q0 + k * kPer;
          uint4* v = reinterpret_cast<uint4*>(smem + S::q + (q / kRows) * S::kQ + swizzled(q % kRows, qc, kRows));
          *v = make_uint4(v->x ^ 0x80008000u, v->y ^ 0x80008000u, v->z ^ 0x80008000u, v->w ^ 0x80008000u);
        }
      fence_async_smem();
      arrive(&bar.q_full);
    };
    AttnSegment seg;
    bool more = attn_next<kMode>(p, plan, x0, x1, seg);
    if (more) {
      ask(seg);
      if (tid == 0) s_bad = 0;
      named_bar_sync(1, 256);
      open();
      named_bar_sync(1, 256);
    }
    // What the merge has to know of the border before this share, if it is the first one that cuts
    // a unit: the unit, its parts' first slot and how many there are.
    if (mt == 0 && tid == 0) {
      int4 cut = make_int4(0, 0, 0, 0);
      if (more && !s_bad && x0 > seg.unit0 && sh.owner(seg.unit0) == g - 1)
        cut = make_int4(kPrefix ? seg.row0 : seg.b, seg.h,
                        (sh.start(g - 1) >= seg.unit0 ? 0 : 1) | (kPrefix ? seg.rows << 1 : 0),
                        sh.owner(seg.unit0 + seg.tiles - 1) - g + 2);
      p.cuts[g] = cut;
    }
    for (; more; ++seg_no) {
      const int n = seg.tile1 - seg.tile0;
      if constexpr (kPrefix) {
        nrows = seg.rows;
        mine = pr < nrows;
        idle = (two ? a * kRows : 0) + (warp & 3) * 32 >= nrows;
      }
      const unsigned long long anc = mine ? (kPrefix ? ~0ull : s_anc[t_of]) : 0ull;
      const int jobs = two ? n : (n - a + 1) >> 1;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < jobs; ++j, ++seen) {
        if (!(ok = warp_wait(&bar.s_full[a], seen & 1))) break;
        if (!idle) {
          tmem_fence_after();
          const int at = seg.tile0 + (two ? j : 2 * j + a), pt = prefix_tiles<kBoth>(seg);
          const bool of_prefix = kBoth && at < pt;
          const int base = of_prefix ? at * kCols - seg.plen : (at - pt) * kCols - seg.old;
          // One pass with the maximum so far: weights are taken against it while the tile's own
          // maximum is found, and only where that is too large are they taken again.
          uint32_t w[4][16];
          uint64_t sum[2];
          float mx;
          auto weigh = [&] {
            const float off = m == -INFINITY ? 0.f : m;
            const uint64_t scale2 = pack2(scale, scale), off2 = pack2(-off, -off);
            float top[2] = {-INFINITY, -INFINITY};
            sum[0] = sum[1] = 0;
            uint32_t s[2][32];
            tmem_ld32(t_s, s[0]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t(&v)[32] = s[c & 1];
              tmem_wait_ld32(v);
              if (c < 3) tmem_ld32(t_s + (c + 1) * 32, s[(c + 1) & 1]);
              if (base + kCols > 0) {
                const uint32_t vis = visible32(kPrefix || of_prefix ? 0ull : anc, base + c * 32);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (!(vis >> k & 1)) v[k] = __float_as_uint(-INFINITY);
              }
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                top[k & 1] = fmaxf(top[k & 1], fmaxf(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])));
                const float2 z = unpack2(fma2(pack2u(v[2 * k], v[2 * k + 1]), scale2, off2));
                const float e0 = ex2(z.x), e1 = ex2(z.y);
                sum[k & 1] = add2(sum[k & 1], pack2(e0, e1));
                // rounded to bf16: with V in bf16 the product takes nothing wider
                w[c][k] = bf16_pack(e0, e1);
              }
            }
            mx = fmaxf(top[0], top[1]) * scale;
          };
          weigh();
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
                tmem_wait_ld16(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st16(t_o + c * 16, o);
              }
            }
            weigh();
          }
          // the weights go over scores that have been read
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_st16(t_s + c * 16, w[c]);
          const float2 both = unpack2(add2(sum[0], sum[1]));
          l += both.x + both.y;
        }
        {  // this tile's V, and the K of this accumulator's next one
          const int t = kv + (two ? j : 2 * j + a), next = t + (two ? 1 : 2);
          if (r == 0) ok = wait(&bar.v_full[t % kStages], (t / kStages) & 1);
          if (r == 32 && j + 1 < jobs) ok = wait(&bar.k_full[next % nk], (next / nk) & 1);
          ok = __all_sync(0xffffffffu, ok);
        }
        if (!idle) {
          tmem_wait_st();
          tmem_fence_before();
        }
        arrive(&bar.p_ready[a]);
      }
      kv += n;
      // ----------------------------------------------------------------------------- output
      // Every score of both accumulators has been read, so Q may be replaced: the next segment is
      // opened, and its first products run, before this one is written out.
      const AttnSegment now = seg;
      if (!(ok = named_bar_all(1, 256, ok))) break;
      more = attn_next<kMode>(p, plan, seg.next, x1, seg);
      if (more) ask(seg);
      if (jobs > 0) ok = warp_wait(&bar.o_done[a], ends++ & 1);
      ok = ok && warp_wait(&bar.v_clean, seg_no & 1);
      tmem_fence_after();
      const unsigned long long poison = kPrefix ? 0ull : anc & s_poison;  // nodes it sees whose V is not finite somewhere
      if (kHasPrior) pdl_wait();
      const int state = kHasPrior && mine ? p.prior[now.b] : 0;  // of a prefix pass
      const bool write = mine && !s_bad && state >= 0;
      if (!(ok = named_bar_all(1, 256, ok))) break;  // all have read s_poison and s_bad
      if (tid == 0) s_bad = 0;
      if (tid == 0) s_poison = 0;
      named_bar_sync(1, 256);
      if (more) open();
      // this row's sums, B's merged into A's where both hold parts of one row
      float fa = 1.f, fb = 0.f;
      auto part = [&](uint32_t from, int c, float (&o)[32]) {  // columns 32c .. of an accumulator's O
        uint32_t u[32];
        tmem_ld32(from + c * 32, u);
        tmem_wait_ld32(u);
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = __uint_as_float(u[k]);
      };
      const bool whole = now.tile0 == 0 && now.tile1 == now.tiles;
      const int slot = whole ? 0 : attn_slot(p, sh, g, mt, now.unit0);
      char* y = p.out + now.b * p.outr + t_of * p.outt +
                static_cast<long long>(now.h * p.G + (mine ? rr % p.G : 0)) * HD * 2;
      long long prior = 0;  // where this row's part of a prefix is or goes
      float f_own = 1.f, f_prior = 0.f;
      if (kPrefix && mine) {
        const AttnQuery at = attn_query<kPrefix>(p, now, pr);
        prior = attn_prior_at(p, at.b, at.t, at.h);
      } else if (kHasPrior && state > 0) {
        prior = attn_prior_at(p, now.b, t_of, now.h * p.G + rr % p.G);
      }
      auto store_out = [&](int c, float (&o)[32]) {  // (zeros for an unused node, whatever o is)
        if constexpr (kPrefix) {
          float4* to = reinterpret_cast<float4*>(p.prior_o + prior * HD + c * 32);
#pragma unroll
          for (int k = 0; k < 8; ++k) to[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          return;
        }
        if (kHasPrior && state > 0) {
          const float4* from = reinterpret_cast<const float4*>(p.prior_o + prior * HD + c * 32);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 v = __ldcg(from + k);
            o[4 * k] = o[4 * k] * f_own + v.x * f_prior;
            o[4 * k + 1] = o[4 * k + 1] * f_own + v.y * f_prior;
            o[4 * k + 2] = o[4 * k + 2] * f_own + v.z * f_prior;
            o[4 * k + 3] = o[4 * k + 3] * f_own + v.w * f_prior;
          }
        }
        const float inv = 1.f / l;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(y + c * 64 + k * 16) =
              anc ? make_uint4(bf16_pack(o[8 * k] * inv, o[8 * k + 1] * inv),
                               bf16_pack(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                               bf16_pack(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                               bf16_pack(o[8 * k + 6] * inv, o[8 * k + 7] * inv))
                  : make_uint4(0, 0, 0, 0);
      };
      auto store_lse = [&](float mm, float ll) {
        if (kPrefix) p.prior_ml[prior] = make_float2(mm, ll);
        else if (p.lse)
          p.lse[(static_cast<long long>(now.b) * p.T + t_of) * p.Hq + now.h * p.G + rr % p.G] =
              anc ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
      };
      // one chunk of the row's merged sums goes to the output, or to the partial results
      auto emit = [&](int c, float (&o)[32]) {
        if (!write) return;
        if (whole) {
          store_out(c, o);
        } else {
          float4* w = reinterpret_cast<float4*>(p.part_o) +
                      (static_cast<long long>(slot) * (HD / 4) + c * 8) * 2 * kRows + pr;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            w[k * 2 * kRows] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      };
      // Tensor memory's lanes are a warp's by its place in the warpgroup, so A's threads reach B's O
      // of the same rows themselves; only (m, l) has to be passed.
      if (!two) {
        if (a == 1) s_ml[r] = make_float2(m, l);
        named_bar_sync(2, 256);
        tmem_fence_after();
        if (a == 0 && n > 1) {
          const float2 b = s_ml[r];
          const float mn = fmaxf(m, b.x), off = mn == -INFINITY ? 0.f : mn;
          fa = ex2(m - off);
          fb = ex2(b.x - off);
          l = l * fa + b.y * fb;
          m = mn;
        }
      }
      if (kHasPrior && whole && state > 0) {
        const float2 ml = attn_join(m, l, __ldcg(p.prior_ml + prior), f_own, f_prior);
        m = ml.x;
        l = ml.y;
      }
      if ((two || a == 0) && !idle)
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          float o[32];
          part(t_o, c, o);
          if (!two && n > 1) {
            float q[32];
            part(t_o + kCols, c, q);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = o[k] * fa + q[k] * fb;
          }
          emit(c, o);
        }
      const bool owner = write && (two || a == 0);
      if (poison && owner)
        attn_add_not_finite(poison, attn_node_v(p, now), HD, 0, 4, whole ? y : nullptr,
                            reinterpret_cast<float4*>(p.part_o) + static_cast<long long>(slot) * (HD / 4) * 2 * kRows + pr, 2 * kRows);
      if (whole) {
        if (owner) store_lse(m, l);
      } else if (owner) {
        // (a row without a used node is told by an infinite sum)
        p.part_ml[static_cast<long long>(slot) * 2 * kRows + pr] = make_float2(m, anc ? l : INFINITY);
      }
      named_bar_sync(1, 256);  // the next segment's ancestors are there
    }
    if (!ok) cp_async_wait_all();  // (Q of a segment that was not opened)
  }
  if (!ok) set_status(p.status, SPECDEC_ERR_TIMEOUT);
  if (kHasPrior) pdl_wait();  // no CTA ends before the prefix pass: the next kernel waits for this one alone
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == 9) {
    tmem_fence_after();
    tmem_free(tmem, 512);
  }
}

// Units that share borders cut, merged by a launch of their own: it spreads the parts over the GPU
// and needs no tickets, where the CTA that came last would add parts of 128 KB one after the other
// behind the last share.  CTA = border and 32 rows; thread = row and 4 * kPer of its values.
// Measured alone and cold (ncu), 75 borders of 512 rows: 14.7 us for 30 MB, the loads' latency.
// A prefix pass has few units of many parts: there kSlices CTAs share a row's values (8 units of 256 rows
// in 19 parts: 11.3 us, 17.4 us with one).
template <int HD, int kMode>
__global__ void __launch_bounds__(256) attn_merge_kernel(const AttnParams p) {
  constexpr bool kPrefix = kMode == kPrefixPass;
  constexpr int kSlices = kPrefix ? HD / 32 : 1, kPer = HD / 32 / kSlices;  // float4 a thread holds
  constexpr int kBlock = 64;     // parts at a time
  __shared__ float2 s_ml[kBlock][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slice = blockIdx.y % kSlices, by = blockIdx.y / kSlices;
  const int g0 = blockIdx.x, block = by & 7, mt = by >> 3;
  const int pr = block * 32 + lane, rr = mt * 2 * kRows + pr, t = rr / p.G;
  if (kPrefix) pdl_launch_dependents();  // the pass over own columns may be set up
  pdl_wait();
  const int4 cut = __ldcg(p.cuts + g0 + 1);
  const int b = cut.x, qh = cut.y * p.G + rr - t * p.G, parts = cut.w;
  if (parts < 2 || (kPrefix && block * 32 >= cut.z >> 1)) return;
  auto slot = [&](int i) { return 2ll * ((g0 + i) * p.MT + mt) + (i == 0 ? cut.z & 1 : 0); };
  // the parts in blocks: their rows' (m, l) into shared memory at once, then the sums
  const int d0 = (slice * 8 + warp) * kPer;  // first float4
  bool live = true;
  float m = -INFINITY, l = 0.f;
  float4 o[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* base = reinterpret_cast<const float4*>(p.part_o) + d0 * 2 * kRows + pr;
  for (int i0 = 0; i0 < parts; i0 += kBlock) {
    const int n = min(kBlock, parts - i0);
    __syncthreads();
    for (int i = warp; i < n; i += 8)
      s_ml[i][lane] = p.part_ml[slot(i0 + i) * 2 * kRows + pr];
    __syncthreads();
    live &= s_ml[0][lane].y != INFINITY;
    float mn = m;
    for (int i = 0; i < n; ++i) mn = fmaxf(mn, s_ml[i][lane].x);
    const float off = mn == -INFINITY ? 0.f : mn, f0 = ex2(m - off);
    m = mn;
    l *= f0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      o[k].x *= f0;
      o[k].y *= f0;
      o[k].z *= f0;
      o[k].w *= f0;
    }
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float4* w = base + slot(i0 + i) * (HD / 4 * 2 * kRows);
      const float2 ml = s_ml[i][lane];
      const float f = ex2(ml.x - off);
      l += ml.y * f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const float4 v = w[k * 2 * kRows];
        o[k].x += v.x * f;
        o[k].y += v.y * f;
        o[k].z += v.z * f;
        o[k].w += v.w * f;
      }
    }
  }
  if constexpr (kPrefix) {
    if (pr >= cut.z >> 1) return;
    AttnSegment s = {};
    s.row0 = cut.x;
    s.h = cut.y;
    const AttnQuery row = attn_query<true>(p, s, pr);
    const long long at = attn_prior_at(p, row.b, row.t, row.h);
    if (d0 == 0) p.prior_ml[at] = make_float2(m, l);
    float4* to = reinterpret_cast<float4*>(p.prior_o + at * HD) + d0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) to[k] = o[k];
    return;
  }
  if (rr >= p.T * p.G) return;
  if constexpr (kMode == kBehind) {
    const int state = p.prior[b];
    if (state < 0) return;
    if (state > 0) {
      const long long at = attn_prior_at(p, b, t, qh);
      float f0, f1;
      const float2 ml = attn_join(m, l, __ldcg(p.prior_ml + at), f0, f1);
      m = ml.x;
      l = ml.y;
      const float4* from = reinterpret_cast<const float4*>(p.prior_o + at * HD) + d0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const float4 v = __ldcg(from + k);
        o[k].x = o[k].x * f0 + v.x * f1;
        o[k].y = o[k].y * f0 + v.y * f1;
        o[k].z = o[k].z * f0 + v.z * f1;
        o[k].w = o[k].w * f0 + v.w * f1;
      }
    }
  }
  const float inv = 1.f / l;
  char* y = p.out + b * p.outr + t * p.outt + static_cast<long long>(qh) * HD * 2 + d0 * 8;
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    *reinterpret_cast<uint2*>(y + k * 8) = live ? make_uint2(bf16_pack(o[k].x * inv, o[k].y * inv), bf16_pack(o[k].z * inv, o[k].w * inv))
                                                : make_uint2(0, 0);
  if (p.lse && d0 == 0)
    p.lse[(static_cast<long long>(b) * p.T + t) * p.Hq + qh] =
        live ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <int HD, int kMode>
int launch_tc(const AttnParams& p, const CUtensorMap& map, const CUtensorMap& map2, int grid, cudaStream_t stream) {
  auto kernel = attn_tc_kernel<HD, kMode>;
  constexpr int smem = Smem<HD>::bytes;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             smem + (kMode == kBothParts ? both_plan_bytes(kAttnMaxRows) : attn_plan_bytes(kAttnMaxRows)));
  if (e != cudaSuccess) return map_cuda_error(e);
  const int plan = kMode == kBothParts ? both_plan_bytes(p.B) : kMode == kPrefixPass ? prefix_plan_bytes(p.P) : attn_plan_bytes(p.B);
  const cudaError_t e2 = attn_launch(kernel, grid, kThreads, smem + plan, kMode == kBehind, stream, p, map, map2);
  if (e2 != cudaSuccess || p.groups == 1) return map_cuda_error(e2);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(p.groups - 1, p.MT * 8 * (kMode == kPrefixPass ? HD / 32 : 1));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return map_cuda_error(cudaLaunchKernelEx(&cfg, attn_merge_kernel<HD, kMode>, p));
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

int launch_attn_tc(const AttnParams& p, int rows, int grid, bool prefix, cudaStream_t stream) {
  CUtensorMap map;
  if (!kv_tensor_map(&map, p.cache, p.hd, p.cap, p.H, rows, kCols)) return SPECDEC_ERR_UNSUPPORTED;
  if (prefix)
    return p.hd == 64 ? launch_tc<64, kPrefixPass>(p, map, map, grid, stream) : launch_tc<128, kPrefixPass>(p, map, map, grid, stream);
  if (p.prior)
    return p.hd == 64 ? launch_tc<64, kBehind>(p, map, map, grid, stream) : launch_tc<128, kBehind>(p, map, map, grid, stream);
  return p.hd == 64 ? launch_tc<64, kOwn>(p, map, map, grid, stream) : launch_tc<128, kOwn>(p, map, map, grid, stream);
}

int launch_attn_tc_both(const AttnParams& p, int rows, const ByteView& prefix, int prefix_rows, int grid, cudaStream_t stream) {
  CUtensorMap map, map2;
  if (!kv_tensor_map(&map, p.cache, p.hd, p.cap, p.H, rows, kCols) ||
      !kv_tensor_map(&map2, prefix, p.hd, p.prefix_cap, p.H, prefix_rows, kCols))
    return SPECDEC_ERR_UNSUPPORTED;
  return p.hd == 64 ? launch_tc<64, kBothParts>(p, map, map2, grid, stream) : launch_tc<128, kBothParts>(p, map, map2, grid, stream);
}

}  // namespace specdec
