// Tokens from score rows: temperature, top-k, top-p, min-p, and the draw from a given uniform.
//
// The mathematics.  With z(x) = (max - x) log2(e) / T a token of score x has the mass 2^-z, its
// probability up to the row's sum.  In order of score (lowest index first among equals) top-k keeps
// the first k tokens, top-p those of them before which less than top_p of their mass lies, and min-p
// cuts at x = max + T ln(min_p).  Every setting keeps a beginning of that order, so a cut is one token,
// the last that is kept, and the kept set is told by its (score, index).  The draw is the first token
// by index whose running mass exceeds u times the sum.
//
// A cluster holds a row in its CTAs' shared memory, read once from HBM; everything after is on chip:
//   1. the highest score (and whether there is NaN);
//   2. only where top-k or top-p is set: a histogram of counts over 2048 bins of z (64 an octave),
//      each CTA's merged over the cluster by parts.  Where the tokens up to the cut are few they are listed
//      and sorted.  Otherwise: the bin that holds a cut; its tokens, listed in every
//      CTA and ranked by comparing all pairs.  Which bin holds top-p's cut is guessed from the counts
//      and the bins' middles, and settled by a pass that sums what lies before and in it, which also
//      moves the next guess: a pass or two, and no sums by atomics.  A bin of more tokens than the
//      list has room for is split by key until it has few, or equal ones, which are counted by index;
//   3. the kept masses' sums by warp, CTA and cluster, and in the warp that owns the draw the token.
// Masses are fp32 exponentials, added up within a 16-byte vector and then as whole numbers of 2^-42 of
// the highest: the sums depend on no order and no number of CTAs, so a row repeats bit for bit.
#include <algorithm>
#include <cmath>

#include "tree.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBins = 2048, kPer = kBins / kThreads, kList = 1024, kEach = kList / kThreads;
constexpr int kMaxCluster = 16;
constexpr int kMassBits = 42;
constexpr long long kMaxRow = 1400 << 10;  // bytes
constexpr uint32_t kTries = 1u << 17, kNs = 20000;  // a wait gives up after about 2.6 s

struct SampleParams {
  const char* x;
  long long stride;  // bytes
  int V, pv, bounds_stride;
  const float *temperature, *top_p, *min_p, *uniforms;
  const int32_t* top_k;
  int32_t* token;
  float* logprob;
  specdec_keep_bound* bounds;
  int32_t* status;
};

__device__ __forceinline__ void remote_store(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void remote_store(uint32_t a, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t remote_load(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row's scale: its highest score, and log2(e) / T in two floats (the second at most 1: times a
// difference of scores it is finite, or the difference is not).
struct Scale {
  float top, sh, sl;
  // Never falling as x falls.
  __device__ __forceinline__ float z(float x) const { return (top - x) * sh; }
  __device__ __forceinline__ float exponent(float x) const {  // -z
    const float d = x - top;
    return fmaf(d, sh, d * sl);
  }
  // (a score of -infinity makes the exponent NaN or -infinity, either of which the maximum drops)
  __device__ __forceinline__ float mass(float x) const { return ex2(fmaxf(exponent(x), -200.f)); }
};
__device__ __forceinline__ int bin_of(float z) { return static_cast<int>(fminf(z * 64.f, kBins - 1.f)); }
// A sum of masses, at most 8, as a whole number of 2^-42 (what is less is dropped).
__device__ __forceinline__ unsigned long long whole(float v) {
  const uint32_t bits = __float_as_uint(v), e = bits >> 23;
  const unsigned long long m = static_cast<unsigned long long>((bits & 0x7FFFFFu) | 0x800000u) << 22;
  return e < 70 ? 0 : m >> (130 - e);  // v = m 2^(e - 172)
}

// The natural logarithm of 0 < f <= 1 in two floats, to about 2^-40: f = 2^k m, ln m = 2 artanh(r) with
// r = (m - 1) / (m + 1), |r| <= 0.2, whose first term alone needs both.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two log_two(float f) {
  int k;
  float m = frexpf(f, &k);
  if (m < 0.75f) {
    m *= 2.f;
    --k;
  }
  const float n = m - 1.f, d = m + 1.f, d_lo = m - (d - 1.f);  // m - 1 is exact
  const float r = __fdiv_rn(n, d), r_lo = __fdiv_rn(fmaf(-r, d, n) - r * d_lo, d);
  const float q = r * r, series = r * q * fmaf(q, fmaf(q, fmaf(q, fmaf(q, fmaf(q, 1.f / 13, 1.f / 11), 1.f / 9), 1.f / 7), 1.f / 5), 1.f / 3);
  // k ln 2: the first float has few enough bits for an exact product
  const float kf = static_cast<float>(k), base = kf * 0.693359375f;
  const float hi = base + 2.f * r, back = hi - base;
  const float lo = ((base - (hi - back)) + (2.f * r - back)) + fmaf(kf, -2.12194440e-4f, 2.f * (series + r_lo));
  const float sum = hi + lo;
  return Two{sum, lo - (sum - hi)};
}

// floor(f * x) and ceil(f * x) for 0 <= f < 1.
__device__ __forceinline__ unsigned long long times(float f, unsigned long long x, bool up) {
  int e;
  const float m = frexpf(f, &e);  // f = m 2^e, 24 bits
  const unsigned long long i = static_cast<unsigned long long>(static_cast<uint32_t>(ldexpf(m, 24)));
  const int s = 24 - e;  // > 23
  const unsigned long long hi = __umul64hi(i, x), lo = i * x;
  if (s >= 128) return up && (hi | lo) ? 1 : 0;
  const unsigned long long q = s >= 64 ? hi >> (s - 64) : lo >> s | hi << (64 - s);
  const bool rest = s >= 64 ? lo != 0 || (s > 64 && hi << (128 - s)) : lo << (64 - s) != 0;
  return q + (up && rest ? 1 : 0);
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

struct Shared {
  unsigned long long slot[2][3][kMaxCluster];  // what the cluster's CTAs tell each other, in turn
  unsigned long long warp_a[kWarps], warp_b[kWarps], warp_c[kWarps];
  uint64_t bar[kWarps];
  float warp_f[kWarps];
  uint32_t best, listed, lo, hi;
  uint32_t count_before, count;
  float est_before, est;
  int found;
};

// One thread's bins: how many tokens they hold, and of all before them how many those are and what they
// weigh by the bins' middles.
struct Bins {
  uint32_t count[kPer], count_before;
  float est_before;
};

// kCuts: whether there may be top-k or top-p.
template <typename T, bool kCuts>
__global__ void __launch_bounds__(kThreads, kCuts ? 3 : 4) sample_kernel(const SampleParams p) {
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(16) char smem[];
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_rank(), C = [] {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return static_cast<int>(n);
  }();
  const int r = blockIdx.x / C;
  uint4* s_x = reinterpret_cast<uint4*>(smem);
  uint32_t* s_hist = reinterpret_cast<uint32_t*>(smem + static_cast<size_t>(p.pv) * 16);  // [kBins], or this CTA's list
  uint32_t* s_all = s_hist + kBins;                                                        // merged, or the cluster's list
  int turn = 0;
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (waited for before the first remote store)
  auto together = [&] {
    __syncwarp();
    if (C == 1) __syncthreads();
    else cluster_sync_all();
  };
  // Every CTA's values, the same in all its threads: s.slot[..][i][rank] in each.
  using Slots = const unsigned long long (*)[kMaxCluster];
  auto gather = [&](unsigned long long a, unsigned long long b, unsigned long long c) -> Slots {
    Slots got = s.slot[turn];
    if (tid < 3 * C) {
      const int i = tid / C;
      remote_store(cluster_map(&s.slot[turn][i][rank], tid - i * C), i == 0 ? a : i == 1 ? b : c);
    }
    together();
    turn ^= 1;
    return got;
  };
  // Sums of three values over the warp, the CTA and the cluster, in all threads.
  auto sum_all = [&](unsigned long long& a, unsigned long long& b, unsigned long long& c) {
    a = warp_sum(a);
    b = warp_sum(b);
    c = warp_sum(c);
    __syncthreads();
    if (lane == 0) {
      s.warp_a[warp] = a;
      s.warp_b[warp] = b;
      s.warp_c[warp] = c;
    }
    __syncthreads();
    a = warp_sum(lane < kWarps ? s.warp_a[lane] : 0);
    b = warp_sum(lane < kWarps ? s.warp_b[lane] : 0);
    c = warp_sum(lane < kWarps ? s.warp_c[lane] : 0);
    const Slots all = gather(a, b, c);
    a = b = c = 0;
    for (int i = 0; i < C; ++i) {
      a += all[0][i];
      b += all[1][i];
      c += all[2][i];
    }
  };

  // ---------------------------------------------------------------------- the row, once
  const char* row = p.x + static_cast<long long>(r) * p.stride;
  const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));  // elements before it in its first vector
  const int pw = (p.pv + kWarps - 1) / kWarps, v0 = warp * pw, v1 = min(p.pv, v0 + pw);  // a warp's vectors are consecutive
  const int base = rank * p.pv;
  const float temperature = p.temperature ? p.temperature[r] : 1.f, u = p.uniforms[r];
  const int top_k = p.top_k ? p.top_k[r] : 0;
  const float top_p = p.top_p ? p.top_p[r] : 1.f, min_p = p.min_p ? p.min_p[r] : 0.f;
  auto index_of = [&](int v) { return (base + v) * N - skew; };  // of a vector's first element
  float top = -INFINITY;
  bool odd = false;  // NaN or +infinity
  const uint4 none = sizeof(T) == 2 ? make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u)
                                    : make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
  // A warp fetches its own vectors: those that lie in the row whole by one bulk copy, all of a CTA's in
  // flight together; the others by element.
  const int whole0 = max(v0, min(v1, (skew > 0 ? 1 : 0) - base)), whole1 = max(whole0, min(v1, (p.V + skew) / N - base));
  if (lane == 0) {
    mbar_init(&s.bar[warp], 1);
    fence_mbar_init();
    if (whole1 > whole0) {
      mbar_arrive_expect_tx(&s.bar[warp], (whole1 - whole0) * 16);
      bulk_g2s(s_x + whole0, row + static_cast<long long>(index_of(whole0)) * static_cast<int>(sizeof(T)), (whole1 - whole0) * 16, &s.bar[warp]);
    }
  }
  for (int v = v0 + lane; v < v1; v += 32) {
    if (v >= whole0 && v < whole1) continue;
    uint4 w = none;
    T* q = reinterpret_cast<T*>(&w);
    const int e = index_of(v);
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (e + k >= 0 && e + k < p.V) q[k] = reinterpret_cast<const T*>(row)[e + k];
    s_x[v] = w;
  }
  __syncwarp();
  const bool late = whole1 > whole0 && !mbar_wait_sleep(&s.bar[warp], 0, kTries, kNs);
#pragma unroll 4
  for (int v = v0 + lane; v < v1; v += 32) {
    float f[N];
    Vec<T>::unpack(s_x[v], f);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      top = fmaxf(top, f[k]);
      odd |= !(f[k] < INFINITY);
    }
  }
  if (late) (void)mbar_wait_sleep(&s.bar[warp], 0, kTries, kNs);  // (no copy outlives the CTA)
  const bool bad_setting = !(temperature >= 0.f && temperature < INFINITY) || top_k < 0 || !(top_p > 0.f && top_p <= 1.f) ||
                           !(min_p >= 0.f && min_p <= 1.f) || !(u >= 0.f && u < 1.f);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  odd = __any_sync(0xffffffffu, odd);
  if (lane == 0) s.warp_a[warp] = static_cast<unsigned long long>(order_bits(top)) << 1 | (odd ? 1 : 0);
  const bool gave_up = __syncthreads_or(late);
  unsigned long long mine;
  {
    const unsigned long long one = s.warp_a[lane % kWarps];
    mine = static_cast<unsigned long long>(__reduce_max_sync(0xffffffffu, static_cast<uint32_t>(one >> 1))) << 1 |
           (__any_sync(0xffffffffu, one & 1) ? 1 : 0);
  }
  if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster runs
  {
    const Slots all = gather(mine, gave_up, 0);
    mine = all[0][0];
    unsigned long long any = all[1][0];
    for (int i = 1; i < C; ++i) {
      mine = max(mine, all[0][i]) | ((mine | all[0][i]) & 1);
      any |= all[1][i];
    }
    if (any) {  // every CTA leaves: nothing is sent any more
      if (rank == 0 && tid == 0) set_status(p.status, SPECDEC_ERR_TIMEOUT);
      return;
    }
  }
  const uint32_t top_key = static_cast<uint32_t>(mine >> 1);
  auto score_of = [](uint32_t key) { return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key); };
  top = score_of(top_key);
  if (bad_setting || (mine & 1) || top == -INFINITY) {
    if (rank == 0 && tid == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
    return;
  }
  auto each = [&](auto f) {  // this thread's elements: f(score, index)
    for (int v = v0 + lane; v < v1; v += 32) {
      float x[N];
      Vec<T>::unpack(s_x[v], x);
      const int e = index_of(v);
#pragma unroll
      for (int k = 0; k < N; ++k) f(x[k], e + k);
    }
  };
  auto write = [&](int token, float logprob, uint32_t key, int last) {
    p.token[r] = token;
    if (p.logprob) p.logprob[r] = logprob;
    if (p.bounds) p.bounds[static_cast<long long>(r) * p.bounds_stride] = specdec_keep_bound{key, last};
  };
  if (temperature == 0.f) {  // the first of the highest
    int at = INT32_MAX;
    each([&](float x, int e) {
      if (x == top) at = min(at, e);
    });
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) s.warp_b[warp] = at;
    __syncthreads();
    unsigned long long least = s.warp_b[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) least = min(least, s.warp_b[w]);
    const Slots all = gather(least, 0, 0);
    for (int i = 0; i < C; ++i) least = min(least, all[0][i]);
    if (rank == 0 && tid == 0) write(static_cast<int>(least), 0.f, top_key, static_cast<int>(least));
    return;
  }
  Scale sc;
  sc.top = top;
  constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.92596303e-8f;  // log2(e) in two floats
  sc.sh = fminf(__fdiv_rn(kLog2eHi, temperature), 1e30f);
  sc.sl = sc.sh < 1e7f ? __fdiv_rn(fmaf(-sc.sh, temperature, kLog2eHi) + kLog2eLo, temperature) : 0.f;

  // The least key that min-p keeps: of the first float that is not below max + T ln(min_p), in two floats
  // (64 bits are so slow here that one logarithm in them took 5 us).
  auto min_p_key = [&] {
    const Two l = log_two(min_p);
    const float a = temperature * l.hi, b = fmaf(temperature, l.hi, -a) + temperature * l.lo;
    float hi = top + a;
    const float back = hi - top, rest = (top - (hi - back)) + (a - back) + b;
    const float sum = hi + rest, over = rest - (sum - hi);
    if (!(sum > -INFINITY)) return 0u;  // (below every score: all are kept)
    uint32_t key = order_bits(sum);
    if (over > 0.f) ++key;              // the next float
    return min(key, top_key);
  };
  // The drawn token, of a sum of kept masses.
  auto finish = [&](int token, float score, unsigned long long total, uint32_t key, int last) {
    // the highest mass is 1 and among the kept: the sum's logarithm from what it is above 1
    const float above = static_cast<float>(total - (1ull << kMassBits)) * (1.f / (1ull << kMassBits));
    write(token, fmaf(sc.exponent(score), 0.693147181f, -log1pf(above)), key, last);
  };

  // ---------------------------------------------------------------------- the cuts
  uint32_t cut_key = 0;       // kept: a larger key, or this one up to index cut_last
  int cut_last = INT32_MAX;
  float cut = -INFINITY;      // its score
  auto in_row = [&](int e) { return e >= 0 && e < p.V; };
  auto is_kept = [&](float x, int e) { return x > cut || (x == cut && e <= cut_last); };
  const bool by_mass = top_p < 1.f, by_count = top_k > 0 && top_k < p.V;
  if (kCuts && (by_mass || by_count)) {
    // Counts by place (place(x): -1 for none), merged over the cluster; middle(b): what a token of bin
    // b weighs, roughly.
    auto histogram = [&](auto place, auto middle) {
      for (int i = tid; i < kBins; i += kThreads) s_hist[i] = 0;
      __syncthreads();
      uint32_t far = 0;  // (the last place is counted apart: it may hold nearly all of a row)
      each([&](float x, int e) {
        const int at = in_row(e) ? place(x) : -1;
        if (at == kBins - 1) ++far;
        else if (at >= 0) atomicAdd(&s_hist[at], 1u);
      });
      far = __reduce_add_sync(0xffffffffu, far);
      if (lane == 0 && far) atomicAdd(&s_hist[kBins - 1], far);
      together();
      if (C > 1) {  // a CTA adds up its part of the bins over all, and tells all
        const int part = kBins / C;
        for (int i = tid; i < part; i += kThreads) {
          const int b = rank * part + i;
          uint32_t count = 0;
          for (int c = 0; c < C; ++c) count += remote_load(cluster_map(&s_hist[b], c));
          for (int c = 0; c < C; ++c) remote_store(cluster_map(&s_all[b], c), count);
        }
        together();
      }
      Bins g;
      uint32_t count = 0;
      float est = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        g.count[i] = (C > 1 ? s_all : s_hist)[kPer * tid + i];
        count += g.count[i];
        est += static_cast<float>(g.count[i]) * middle(kPer * tid + i);
      }
      uint32_t ca = count;
      float ea = est;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t oc = __shfl_up_sync(0xffffffffu, ca, d);
        const float oe = __shfl_up_sync(0xffffffffu, ea, d);
        if (lane >= d) {
          ca += oc;
          ea += oe;
        }
      }
      if (lane == 31) {
        s.warp_a[warp] = ca;
        s.warp_f[warp] = ea;
      }
      __syncthreads();
      g.count_before = ca - count;
      g.est_before = ea - est;
      for (int w = 0; w < warp; ++w) {
        g.count_before += static_cast<uint32_t>(s.warp_a[w]);
        g.est_before += s.warp_f[w];
      }
      return g;
    };
    // The last bin in [lo, hi) that is not empty and begins before `tokens` tokens, or before `est`; -1
    // if there is none.  What it holds and what comes before it are left in s.
    auto bin_with = [&](const Bins& g, auto middle, bool mass, uint32_t tokens, float est, int lo, int hi) {
      __syncthreads();
      if (tid == 0) s.best = 0;
      __syncthreads();
      uint32_t cb = g.count_before;
      float eb = g.est_before;
      int at = -1;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int b = kPer * tid + i;
        if (g.count[i] > 0 && b >= lo && b < hi && (mass ? eb < est : cb < tokens)) at = i;
        cb += g.count[i];
        if (mass) eb += static_cast<float>(g.count[i]) * middle(b);
      }
      if (at >= 0) atomicMax(&s.best, kPer * tid + at + 1);
      __syncthreads();
      const int best = static_cast<int>(s.best) - 1;
      if (best >= 0 && tid == best / kPer) {
        cb = g.count_before;
        eb = g.est_before;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const float est_in = static_cast<float>(g.count[i]) * middle(kPer * tid + i);
          if (kPer * tid + i == best) {
            s.count_before = cb;
            s.est_before = eb;
            s.count = g.count[i];
            s.est = est_in;
          }
          cb += g.count[i];
          eb += est_in;
        }
      }
      __syncthreads();
      return best;
    };
    // The bin with the cut of a target of mass, what is left of it there (in `target`), and in s what
    // the bin holds.  kind(b) gives a test of scores: 1 before bin b (of what the histogram counted),
    // 2 in it, 0 neither.  With `fraction` the target is that much of what is kept so far, which the
    // first pass finds and est_total guesses.
    auto mass_bin = [&](const Bins& g, auto middle, auto kind, float fraction, float est_total, unsigned long long& target) {
      int lo = 0, hi = kBins, low = -1;  // low: the last bin that was found to begin before the target
      unsigned long long low_before = 0;
      float want = fraction > 0.f ? fraction * est_total : static_cast<float>(target) * (1.f / (1ull << kMassBits));
      for (int round = 0; round < 48 && lo < hi; ++round) {
        // a guess; after a few the middle (so the bounds meet within the rounds there are)
        const int mid = lo + 1 + (hi - lo) / 2;
        int b = round < 5 ? bin_with(g, middle, true, 0, want, lo, hi) : -1;
        if (b < 0) b = bin_with(g, middle, true, 0, INFINITY, lo, min(mid, hi));
        if (b < 0) {
          lo = mid;
          continue;
        }
        const float est_before = s.est_before;
        const auto test = kind(b);
        unsigned long long before = 0, in = 0, all = 0;
        const bool first = fraction > 0.f;
        for (int v = v0 + lane; v < v1; v += 32) {
          float x[N];
          Vec<T>::unpack(s_x[v], x);
          float vb = 0.f, vi = 0.f, va = 0.f;
          const int e = index_of(v);
#pragma unroll
          for (int k = 0; k < N; ++k) {  // (places outside the row weigh nothing)
            const float m = sc.mass(x[k]);
            const int c = test(x[k]);
            vb += c == 1 ? m : 0.f;
            vi += c == 2 ? m : 0.f;
            if (first) va += is_kept(x[k], e + k) ? m : 0.f;
          }
          before += whole(vb);
          in += whole(vi);
          all += whole(va);
        }
        sum_all(before, in, all);
        if (first) {
          target = max(1ull, times(fraction, all, true));
          fraction = 0.f;
        }
        if (before >= target) {
          hi = b;
        } else {
          low = b;
          low_before = before;
          if (target <= before + in) break;
          lo = b + 1;  // (where rounding has put the target between two bins, the earlier one is taken whole)
        }
        // the next guess: as much further as the target is from what has been summed
        want = est_before + (static_cast<float>(target) - static_cast<float>(before)) * (1.f / (1ull << kMassBits));
      }
      (void)bin_with(g, middle, true, 0, INFINITY, low, low + 1);  // (the last one tried may be another)
      target -= low_before;
      return low;
    };
    auto middle = [](int b) { return ex2((b + 0.5f) * (-1.f / 64)); };
    const Bins bins = histogram([&](float x) { return bin_of(sc.z(x)); }, middle);

    // Most settings keep few tokens.  Where the bins up to the cut's hold no more than the list, one pass
    // counts them (and, for top-p alone, sums the row), another sends them to the first CTA in order of
    // index, and that does the rest.  For top-p the bin is guessed from the bins' middles (2 % beyond
    // what they say); the listed mass shows whether it was far enough.
    (void)bin_with(bins, middle, true, 0, INFINITY, 0, kBins);
    float est_kept = s.est_before + s.est;
    const int enough = by_count ? bin_with(bins, middle, false, top_k, 0.f, 0, kBins) : bin_with(bins, middle, true, 0, 1.02f * top_p * est_kept, 0, kBins);
    const uint32_t count_before = s.count_before;
    if (count_before + s.count <= kList) {
      unsigned long long* list = reinterpret_cast<unsigned long long*>(s_all);  // (key, ~index): larger is earlier in the order
      unsigned long long* few = reinterpret_cast<unsigned long long*>(s_hist);
      unsigned long long total = 0, in_list = 0, listed = 0;
      const bool alone = !by_count;
      auto takes = [&](float x, int e) { return in_row(e) && bin_of(sc.z(x)) <= enough; };
      for (int v = v0 + lane; v < v1; v += 32) {
        float x[N];
        Vec<T>::unpack(s_x[v], x);
        const int e = index_of(v);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const float m = alone ? sc.mass(x[k]) : 0.f;
          sum += m;
          if (takes(x[k], e + k)) {
            ++listed;
            if (alone) in_list += whole(m);
          }
        }
        if (alone) total += whole(sum);
      }
      const unsigned long long in_warp = warp_sum(listed);
      sum_all(total, in_list, listed);
      // where this warp's begin: its CTA's are those of the sums before
      unsigned long long to = 0, cta = 0;
      __syncthreads();
      if (lane == 0) s.warp_a[warp] = in_warp;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        to += w < warp ? s.warp_a[w] : 0;
        cta += s.warp_a[w];
      }
      const unsigned long long target = alone ? max(1ull, times(top_p, total, true)) : 0;
      if (in_list >= target) {
        const Slots all = gather(cta, 0, 0);  // (and all are done with the histograms)
        for (int i = 0; i < rank; ++i) to += all[0][i];
        if (in_warp > 0) {
          const uint32_t first = cluster_map(list, 0);
          for (int vv = v0; vv < v1; vv += 32) {
            const int v = vv + lane;
            float x[N];
            Vec<T>::unpack(v < v1 ? s_x[v] : none, x);
            const int e = index_of(v);
            uint32_t has = 0;
#pragma unroll
            for (int k = 0; k < N; ++k) has |= v < v1 && takes(x[k], e + k) ? 1u << k : 0;
            if (!__any_sync(0xffffffffu, has != 0)) continue;
            const uint32_t here = __popc(has), scan = static_cast<uint32_t>(warp_scan(here));
            uint32_t at = static_cast<uint32_t>(to) + scan - here;
#pragma unroll
            for (int k = 0; k < N; ++k)
              if (has >> k & 1)
                remote_store(first + 8 * at++, static_cast<unsigned long long>(order_bits(x[k])) << 32 | ~static_cast<uint32_t>(e + k));
            to += __shfl_sync(0xffffffffu, scan, 31);
          }
        }
        together();
        if (rank != 0) return;
        // ------------------------------------------------------------- one CTA from here on
        const int n = static_cast<int>(listed);
        unsigned long long token[kEach], mass[kEach];  // consecutive ones of the list (0: none)
        int bin[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          token[i] = kEach * tid + i < n ? list[kEach * tid + i] : 0;
          const float x = token[i] ? score_of(static_cast<uint32_t>(token[i] >> 32)) : -INFINITY;
          mass[i] = token[i] ? whole(sc.mass(x)) : 0;
          bin[i] = token[i] ? bin_of(sc.z(x)) : kBins;
        }
        auto block_sum = [&](unsigned long long v) {
          v = warp_sum(v);
          __syncthreads();
          if (lane == 0) s.warp_a[warp] = v;
          __syncthreads();
          v = 0;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) v += s.warp_a[w];
          return v;
        };
        // The last token of bin b before which, in the bin, there are fewer than `left` tokens, or less mass.
        auto last_in = [&](int b, bool by_sum, unsigned long long left) {
          __syncthreads();
          if (tid == 0) s.listed = s.best = 0;
          __syncthreads();
#pragma unroll
          for (int i = 0; i < kEach; ++i)
            if (bin[i] == b) few[atomicAdd(&s.listed, 1u)] = token[i];
          __syncthreads();
          const int m = static_cast<int>(s.listed);
          for (int i = warp; i < m; i += kWarps) {
            const unsigned long long me = few[i];
            uint32_t tokens = 0;
            unsigned long long sum = 0;
            for (int j = lane; j < m; j += 32)
              if (few[j] > me) {
                ++tokens;
                if (by_sum) sum += whole(sc.mass(score_of(static_cast<uint32_t>(few[j] >> 32))));
              }
            tokens = __reduce_add_sync(0xffffffffu, tokens);
            if (by_sum) sum = warp_sum(sum);
            if (lane == 0 && (by_sum ? sum : tokens) < left) atomicMax(&s.best, tokens << 16 | (i + 1));
          }
          __syncthreads();
          return m ? few[max(0, static_cast<int>(s.best & 0xFFFF) - 1)] : 0ull;
        };
        unsigned long long end = 0;  // the last that is kept
        if (by_count) end = last_in(enough, false, top_k - count_before);
        if (by_mass) {
          unsigned long long own = 0;
          if (by_count) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) own += token[i] >= end ? mass[i] : 0;
            own = block_sum(own);
          }
          const unsigned long long below = by_count ? max(1ull, times(top_p, own, true)) : target;
          // the last bin that begins before `below`
          int lo = 0, hi = enough + 1;
          unsigned long long at_lo = 0;
          while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            unsigned long long v = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) v += bin[i] < mid ? mass[i] : 0;
            v = block_sum(v);
            if (v < below) {
              lo = mid;
              at_lo = v;
            } else {
              hi = mid;
            }
          }
          end = max(end, last_in(lo, true, below - at_lo));
        }
        uint32_t end_key = static_cast<uint32_t>(end >> 32);
        int end_index = static_cast<int>(~static_cast<uint32_t>(end));
        if (min_p > 0.f) {
          const uint32_t least = min_p_key();
          if (least > end_key) {
            end = static_cast<unsigned long long>(least) << 32;
            end_key = least;
            end_index = INT32_MAX;
          }
        }
        // the draw, in order of index
        unsigned long long own = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) own += token[i] >= end ? mass[i] : 0;
        const unsigned long long inc = warp_scan(own);
        __syncthreads();
        if (lane == 31) s.warp_a[warp] = inc;
        __syncthreads();
        unsigned long long at = inc - own, sum = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          at += w < warp ? s.warp_a[w] : 0;
          sum += s.warp_a[w];
        }
        const unsigned long long want = times(u, sum, false);
        if (want < at || want >= at + own) return;
        bool got = false;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          at += token[i] >= end ? mass[i] : 0;
          if (!got && at > want) {
            got = true;
            finish(static_cast<int>(~static_cast<uint32_t>(token[i])), score_of(static_cast<uint32_t>(token[i] >> 32)), sum, end_key, end_index);
          }
        }
        return;
      }
    }

    // The cut: the last token of the order before which there are fewer than `target` tokens, or less
    // than `fraction` of the mass kept so far.  Sets cut_key, cut and cut_last.
    auto find_cut = [&](bool mass, unsigned long long target, float fraction) {
      int bin;
      if (mass) {
        bin = mass_bin(bins, middle, [&](int b) {
          return [&sc, b](float x) {
            const float z = sc.z(x) * 64.f;
            return z < b ? 1 : (z < b + 1 || b == kBins - 1 ? 2 : 0);
          };
        }, fraction, est_kept, target);
      } else {
        bin = bin_with(bins, middle, false, static_cast<uint32_t>(target), 0.f, 0, kBins);
        target -= s.count_before;
        est_kept = s.est_before + s.est;
      }
      uint32_t count = s.count, klo = 0, khi = 0;
      bool by_key = false;
      auto inside = [&](float x) {
        const uint32_t key = order_bits(x);
        return by_key ? key >= klo && key <= khi : bin_of(sc.z(x)) == bin;
      };
      for (int round = 0; count > kList && round < 8; ++round) {  // (each leaves a two-thousandth of the keys)
        __syncthreads();
        if (tid == 0) {
          s.lo = 0xFFFFFFFFu;
          s.hi = 0;
        }
        __syncthreads();
        uint32_t lo = 0xFFFFFFFFu, hi = 0;
        each([&](float x, int e) {
          if (in_row(e) && inside(x)) {
            lo = min(lo, order_bits(x));
            hi = max(hi, order_bits(x));
          }
        });
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
          atomicMin(&s.lo, lo);
          atomicMax(&s.hi, hi);
        }
        __syncthreads();
        const Slots all = gather(s.lo, s.hi, 0);
        klo = 0xFFFFFFFFu;
        khi = 0;
        for (int i = 0; i < C; ++i) {
          klo = min(klo, static_cast<uint32_t>(all[0][i]));
          khi = max(khi, static_cast<uint32_t>(all[1][i]));
        }
        by_key = true;
        if (klo == khi) break;
        const int shift = max(0, 21 - __clz(khi - klo));
        const uint32_t a = klo, z = khi;
        auto first_of = [=](int b) { return z - (static_cast<uint32_t>(b) << shift); };  // a bin's highest key
        auto middle = [&](int b) { return b <= static_cast<int>((z - a) >> shift) ? sc.mass(score_of(max(a, first_of(b)))) : 0.f; };
        const Bins g = histogram([&](float x) { return inside(x) ? static_cast<int>((z - order_bits(x)) >> shift) : -1; }, middle);
        int at;
        if (mass) {
          at = mass_bin(g, middle, [&](int b) {
            const uint32_t h = first_of(b);
            return [=](float x) {
              const uint32_t key = order_bits(x);
              return key > z || key < a ? 0 : key > h ? 1 : h - key < (1u << shift) ? 2 : 0;
            };
          }, 0.f, 0.f, target);
        } else {
          at = bin_with(g, middle, false, static_cast<uint32_t>(target), 0.f, 0, kBins);
          target -= s.count_before;
        }
        count = s.count;
        khi = first_of(at);
        if (khi - klo >= 1u << shift) klo = khi - ((1u << shift) - 1);
      }
      if (count > kList) {
        // equal scores: the last one by index
        const uint32_t key = klo;
        const float score = score_of(key);
        const unsigned long long one = whole(sc.mass(score));
        const unsigned long long want = !mass ? target : one == 0 ? count : min(static_cast<unsigned long long>(count), (target + one - 1) / one);
        unsigned long long n = 0;
        each([&](float x, int e) { n += in_row(e) && x == score; });
        n = warp_sum(n);
        __syncthreads();
        if (lane == 0) s.warp_a[warp] = n;
        if (tid == 0) s.found = 0;
        __syncthreads();
        unsigned long long before = 0, total = 0;
        for (int w = 0; w < kWarps; ++w) {
          before += w < warp ? s.warp_a[w] : 0;
          total += s.warp_a[w];
        }
        const Slots all = gather(total, 0, 0);
        for (int i = 0; i < rank; ++i) before += all[0][i];
        if (before < want && want <= before + n) {  // this warp has it
          for (int vv = v0; vv < v1; vv += 32) {
            const int v = vv + lane;
            float x[N];
            Vec<T>::unpack(v < v1 ? s_x[v] : none, x);
            const int e = index_of(v);
            unsigned long long here = 0;
#pragma unroll
            for (int k = 0; k < N; ++k) here += v < v1 && in_row(e + k) && x[k] == score;
            const unsigned long long scan = warp_scan(here);
            unsigned long long at = before + scan - here;
#pragma unroll
            for (int k = 0; k < N; ++k)
              if (v < v1 && in_row(e + k) && x[k] == score && ++at == want) s.found = e + k + 1;
            before += __shfl_sync(0xffffffffu, scan, 31);
          }
        }
        __syncthreads();
        const Slots who = gather(s.found, 0, 0);
        unsigned long long last = 0;
        for (int i = 0; i < C; ++i) last = max(last, who[0][i]);
        cut_key = key;
        cut_last = static_cast<int>(last) - 1;
      } else {
        // this CTA's tokens in question, then everyone's in every CTA, in order of rank
        uint32_t *l_key = s_hist, *l_index = s_hist + kList, *a_key = s_all, *a_index = s_all + kList;
        together();  // all are done with the histograms
        if (tid == 0) {
          s.listed = 0;
          s.best = 0;
        }
        __syncthreads();
        each([&](float x, int e) {
          if (in_row(e) && inside(x)) {
            const uint32_t i = atomicAdd(&s.listed, 1u);
            l_key[i] = order_bits(x);
            l_index[i] = e;
          }
        });
        __syncthreads();
        const Slots all = gather(s.listed, 0, 0);
        int n = 0;
        for (int c = 0; c < C; ++c) {
          const int m = static_cast<int>(all[0][c]);
          for (int i = tid; i < 2 * m; i += kThreads) {
            const int f = i >= m ? 1 : 0, j = i - f * m;
            s_all[f * kList + n + j] = remote_load(cluster_map(&s_hist[f * kList + j], c));
          }
          n += m;
        }
        __syncthreads();
        // a warp ranks a token: what is before it, and whether it is kept
        for (int i = rank * kWarps + warp; i < n; i += C * kWarps) {
          const unsigned long long me = static_cast<unsigned long long>(a_key[i]) << 32 | ~a_index[i];
          uint32_t tokens = 0;
          unsigned long long sum = 0;
          for (int j = lane; j < n; j += 32) {
            const uint32_t key = a_key[j];
            if ((static_cast<unsigned long long>(key) << 32 | ~a_index[j]) > me) {
              ++tokens;
              if (mass) sum += whole(sc.mass(score_of(key)));
            }
          }
          tokens = __reduce_add_sync(0xffffffffu, tokens);
          if (mass) sum = warp_sum(sum);
          if (lane == 0 && (mass ? sum : tokens) < target) atomicMax(&s.best, tokens << 16 | (i + 1));
        }
        __syncthreads();
        const Slots who = gather(s.best, 0, 0);  // (and the lists may be written again)
        unsigned long long best = 0;
        for (int i = 0; i < C; ++i) best = max(best, who[0][i]);
        const int at = max(0, static_cast<int>(best & 0xFFFF) - 1);  // (the first token is always kept)
        cut_key = a_key[at];
        cut_last = static_cast<int>(a_index[at]);
      }
      cut = score_of(cut_key);
    };
    if (by_count) find_cut(false, top_k, 0.f);
    if (by_mass) find_cut(true, 0, top_p);
  }
  if (min_p > 0.f) {
    const uint32_t key = min_p_key();
    if (key > cut_key) {
      cut_key = key;
      cut_last = INT32_MAX;
      cut = score_of(key);
    }
  }

  // ---------------------------------------------------------------------- the draw
  const bool cuts = cut_key != 0;
  // the running masses of a vector's tokens, as sums of floats: the last is what the vector adds
  auto running = [&](int v, float (&m)[N], float (&x)[N]) {
    Vec<T>::unpack(s_x[v], x);
    const int e = index_of(v);
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float mass = sc.mass(x[k]);
      sum += !cuts || is_kept(x[k], e + k) ? mass : 0.f;
      m[k] = sum;
    }
  };
  unsigned long long sum = 0;
  if (cuts) {
    for (int v = v0 + lane; v < v1; v += 32) {
      float m[N], x[N];
      running(v, m, x);
      sum += whole(m[N - 1]);
    }
  } else {
#pragma unroll 4
    for (int v = v0 + lane; v < v1; v += 32) {
      float x[N], vector = 0.f;
      Vec<T>::unpack(s_x[v], x);
#pragma unroll
      for (int k = 0; k < N; ++k) vector += sc.mass(x[k]);
      sum += whole(vector);
    }
  }
  sum = warp_sum(sum);
  __syncthreads();
  if (lane == 0) s.warp_a[warp] = sum;
  __syncthreads();
  unsigned long long before = 0, cta = 0;
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? s.warp_a[w] : 0;
    cta += s.warp_a[w];
  }
  const Slots all = gather(cta, 0, 0);
  unsigned long long total = 0;
  for (int i = 0; i < C; ++i) {
    before += i < rank ? all[0][i] : 0;
    total += all[0][i];
  }
  const unsigned long long want = times(u, total, false);  // the first whose running mass is above it
  if (want < before || want >= before + sum) return;
  for (int vv = v0; vv < v1; vv += 32) {
    const int v = vv + lane;
    float m[N], x[N];
    unsigned long long here = 0;
    if (v < v1) {
      running(v, m, x);
      here = whole(m[N - 1]);
    }
    const unsigned long long scan = warp_scan(here), at = before + scan - here;
    if (want >= at && want < at + here) {
      int token = 0;
      float score = 0.f;
      bool got = false;
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (!got && at + whole(m[k]) > want) {
          got = true;
          token = index_of(v) + k;
          score = x[k];
        }
      finish(token, score, total, cut_key, cut_last);
    }
    const unsigned long long step = __shfl_sync(0xffffffffu, scan, 31);
    if (want < before + step) return;
    before += step;
  }
}

template <typename T>
int launch_sample(SampleParams p, int R, cudaStream_t stream) {
  constexpr int N = Vec<T>::N;
  const int vectors = (p.V + 2 * N - 2) / N;  // whatever the row's alignment
  const size_t extra = p.top_k || p.top_p ? 2 * kBins * 4 : 0;
  constexpr size_t kRoom = 200 << 10;
  const int sms = std::max(1, sm_count());
  // CTAs that an SM holds at once, and of a row: what its scores need, then more while all rows' run at once
  auto bytes = [&](int c) { return static_cast<size_t>((vectors - 1) / c + 1) * 16 + extra; };
  auto resident = [&](int c) { return std::min<long long>(4, (220 << 10) / (bytes(c) + (2 << 10))) * sms; };
  int C = 1;
  while (C < kMaxCluster && (bytes(C) > (112 << 10) || (R * 2LL * C <= resident(2 * C) && vectors > C * 256))) C *= 2;
  p.pv = (vectors - 1) / C + 1;
  const size_t smem = static_cast<size_t>(p.pv) * 16 + extra;
  if (smem > kRoom) return SPECDEC_ERR_UNSUPPORTED;
  auto kernel = extra ? sample_kernel<T, true> : sample_kernel<T, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRoom));
  if (e != cudaSuccess) return map_cuda_error(e);
  if (C > 8) {
    const cudaError_t e2 = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e2 != cudaSuccess) return map_cuda_error(e2);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(R * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return map_cuda_error(cudaLaunchKernelEx(&cfg, kernel, p));
}

}  // namespace
}  // namespace specdec

extern "C" int specdec_sample(const specdec_sample_args* a, void* stream) {
  using namespace specdec;
  if (!a) return SPECDEC_ERR_INVALID_ARG;
  const int es = elem_size(a->dtype);
  if (!es || a->R < 0 || a->V < 1 || a->row_stride < a->V || a->bounds_stride < 0) return SPECDEC_ERR_INVALID_ARG;
  if (a->R == 0) return SPECDEC_OK;
  if (!a->logits || !a->uniforms || !a->token || !a->dev_status) return SPECDEC_ERR_INVALID_ARG;
  auto off = [](const void* p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
  if (off(a->logits, es) || off(a->uniforms, 4) || off(a->token, 4) || off(a->dev_status, 4) || off(a->temperature, 4) ||
      off(a->top_k, 4) || off(a->top_p, 4) || off(a->min_p, 4) || off(a->logprob, 4) || off(a->keep_bounds, 4))
    return SPECDEC_ERR_INVALID_ARG;
  if (a->keep_bounds && a->R > 1 && a->bounds_stride < 1) return SPECDEC_ERR_INVALID_ARG;
  if (a->R >= (1 << 24) || static_cast<long long>(a->V) * es > kMaxRow || a->bounds_stride >= (1 << 30)) return SPECDEC_ERR_UNSUPPORTED;
  SampleParams p = {};
  p.x = static_cast<const char*>(a->logits);
  p.stride = a->row_stride * es;
  p.V = a->V;
  p.bounds_stride = static_cast<int>(a->bounds_stride);
  p.temperature = a->temperature;
  p.top_k = a->top_k;
  p.top_p = a->top_p;
  p.min_p = a->min_p;
  p.uniforms = a->uniforms;
  p.token = a->token;
  p.logprob = a->logprob;
  p.bounds = static_cast<specdec_keep_bound*>(a->keep_bounds);
  p.status = a->dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return es == 2 ? launch_sample<uint16_t>(p, a->R, s) : launch_sample<float>(p, a->R, s);
}
