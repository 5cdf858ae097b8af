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
//   2. only where top-k or top-p is set: a histogram of the scores, each CTA's merged over the cluster by
//      parts, and from it the bin that holds the cut.  A bf16 row has a bin for every score from 2^-8 to
//      128 and of either sign, so that counts give the masses, and the cut is a score of which so many
//      are kept, by index.  An fp32 row has 32 bins an octave, with the masses' sums; the cut's bin is listed
//      in every CTA and searched there, or where it holds more than the list, split by key first;
//   3. the kept masses' sums by warp, CTA and cluster, and in the warp that owns the draw the token.
// Masses are fp32 exponentials, added up within a 16-byte vector, counted from the row's first score, and
// then as whole numbers of 2^-42 of the highest: the sums depend on no order, no number of CTAs and no
// address, so a row repeats bit for bit.
//
// Measured (rows whose scores fit L2 come from there).  No cuts: 256 rows of 151552, fp32 47 us (3.3
// TB/s), bf16 25 us; one bf16 row of 151936 5.8 us.  There instructions issue in 49 % of the cycles and
// DRAM is at 42 %: a row's steps follow each other, with three CTAs on an SM to fill the gaps (of 192 or
// 384 threads 47 and 53 us against 49 before sums in two parts, bf16 27 and 28 against 26).  With cuts,
// bf16 rows of 151936 with eight likely tokens over a long tail, 64: top-k 24 us, top-p 36; 256: top-k 81; one
// with top-p 21.  Shared-memory atomics and exchanges over the cluster, one after the other, are what is left.
// fp32, 64 rows of 151936: top-k 51, top-p 71 us (three more atomics a token, and the list).  2 rows of 1000:
// 14 us, all latency.
// One bin a score for bf16 against 32 an octave and the list, on other rows: 64 with top-k 24 us against 36,
// with top-p 33 against 58; one with top-p 20 against 28.
#include <algorithm>
#include <cmath>

#include "tree.cuh"

namespace specdec {
namespace {

constexpr int kNarrow = 1024, kWide = 4096;  // bins
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kList = 1024, kEach = kList / kThreads;
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

__device__ __forceinline__ void remote_store(uint32_t a, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void remote_store4(uint32_t a, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 remote_load4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
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
  __device__ __forceinline__ float exponent(float x) const {  // -z
    const float d = x - top;
    return fmaf(d, sh, d * sl);
  }
  // (a score of -infinity or NaN makes the exponent NaN or -infinity, either of which the maximum drops)
  __device__ __forceinline__ float mass(float x) const { return ex2(fmaxf(exponent(x), -200.f)); }
  // Of N scores, two at a time: the same roundings.
  template <int N> __device__ __forceinline__ void masses(const float* x, float* m) const {
    const uint64_t t2 = pack2(-top, -top), h2 = pack2(sh, sh), l2 = pack2(sl, sl);
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      const uint64_t d = add2(pack2(x[k], x[k + 1]), t2);
      const float2 e = unpack2(fma2(d, h2, mul2(d, l2)));
      m[k] = ex2(fmaxf(e.x, -200.f));
      m[k + 1] = ex2(fmaxf(e.y, -200.f));
    }
  }
};

// The larger of two words' scores, NaN where either is (of bf16 in both halves).
template <typename T> __device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
  uint32_t y;
  if constexpr (sizeof(T) == 2) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  else asm("max.NaN.f32 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
// A sum of masses, at most 8, as a whole number of 2^-42 (what is less is dropped).
__device__ __forceinline__ unsigned long long whole(float v) {
  const uint32_t bits = __float_as_uint(v), e = bits >> 23;
  const unsigned long long m = static_cast<unsigned long long>((bits & 0x7FFFFFu) | 0x800000u) << 22;
  return e < 70 ? 0 : m >> (130 - e);  // v = m 2^(e - 172)
}

// The sum of whole(v) over up to 2^8 such v, in half the instructions (256 rows without cuts: fp32 46 us
// against 49, bf16 25 against 27; by conversions of floats to 64 bits 51, 27): v rounded to 2^-19 is the last bits of
// v + 24, and what that left (exact, at most 2^-20 of either sign) in 2^-42, rounded down, those of its sum with
// 1.5 * 2^23.
struct WholeSum {
  uint32_t high = 0;
  int low = 0;
  __device__ __forceinline__ void add(float v) {
    const float h = v + 24.f, l = __fmaf_rd(v - (h - 24.f), 1ll << kMassBits, 12582912.f);
    high += __float_as_uint(h) - __float_as_uint(24.f);
    low += __float_as_int(l) - __float_as_int(12582912.f);
  }
  __device__ __forceinline__ unsigned long long value() const { return (static_cast<unsigned long long>(high) << (kMassBits - 19)) + low; }
};

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
  // k ln 2, ln 2 in two parts as Cody and Waite split it ("Software Manual for the Elementary Functions"):
  // the first has few enough bits for an exact product
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

// (in three parts of 26 bits, whose sums of 32 fit: three instructions in the place of ten shuffles)
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
  const uint32_t a = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v) & 0x3FFFFFFu),
                 b = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 26) & 0x3FFFFFFu),
                 c = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 52));
  return a + (static_cast<unsigned long long>(b) << 26) + (static_cast<unsigned long long>(c) << 52);
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

// (without cuts as small as can be: a few hundred bytes decide whether an SM holds a third CTA of a row of
// 151552 fp32 scores in eight parts, 54 us for 256 rows against 63)
template <bool kCuts> struct Shared {
  static constexpr int kTold = kCuts ? 3 : 2;
  unsigned long long slot[2][kTold][kMaxCluster];  // what the cluster's CTAs tell each other, in turn
  unsigned long long warp_a[kWarps], warp_b[kWarps], warp_c[kCuts ? kWarps : 1];
  uint64_t bar[kWarps];
  unsigned long long count_before, mass_before;
  uint32_t listed, count;
  int bin, found;
};

// A score's place among the wide bins, which fall: scores of 128 and more; the values of bf16 (to which
// other scores are cut off) down to 2^-8; what is nearer to zero; the values from -2^-8 to above -128; the
// rest.  The first, the middle and the last bin hold more than one score of bf16.
constexpr uint32_t kSmall = 119u << 7, kLarge = 134u << 7;  // upper halves of 2^-8 and 2^7
constexpr uint32_t kValues = kLarge - kSmall;
constexpr int kWidePlaces = 2 * kValues + 3;
static_assert(kWidePlaces <= kWide - 32 && (kWidePlaces - 1) / 4 < kNarrow - 32, "room for the masked tokens' counts");
__device__ __forceinline__ int wide_place(float x) {
  const uint32_t bits = __float_as_uint(x), size = (bits & 0x7FFFFFFFu) >> 16;
  const int off = static_cast<int>(min(max(size, kSmall - 1), kLarge) - kSmall);  // -1: near zero; kValues: far
  return bits >> 31 ? kValues + 2 + off : kValues - off;
}
__device__ __forceinline__ int mixed(int b) { return b == 0 ? 0 : b == kValues + 1 ? 1 : b == kWidePlaces - 1 ? 2 : -1; }
__device__ __forceinline__ float wide_score(int b) {  // of a bin of one score
  return b <= kValues ? __uint_as_float((kSmall + kValues - b) << 16) : __uint_as_float(0x80000000u | (kSmall + b - kValues - 2) << 16);
}
// Keys of a bin: the highest and the lowest.
__device__ __forceinline__ uint32_t wide_high(int b) {
  if (b == 0) return 0xFFFFFFFFu;
  if (b <= kValues + 1) return 0x80000000u | ((kSmall + kValues + 1 - b) << 16) - 1;
  return ~(0x80000000u | (kSmall + b - kValues - 2) << 16);
}
__device__ __forceinline__ uint32_t wide_low(int b) { return b == kWidePlaces - 1 ? 0u : wide_high(b + 1) + 1; }

// kCuts: whether there may be top-k or top-p.  (Without, in the same kernel: 256 rows of 151552 fp32 58 us
// against 46, bf16 33 against 25: the histograms' room and registers.)
template <typename T, bool kCuts>
__global__ void __launch_bounds__(kThreads, kCuts ? 2 : 4) sample_kernel(const SampleParams p) {
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(16) char smem[];
  using Sh = Shared<kCuts>;
  __shared__ Sh s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_rank(), C = [] {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return static_cast<int>(n);
  }();
  const int r = blockIdx.x / C;
  uint4* s_x = reinterpret_cast<uint4*>(smem);
  uint32_t* s_hist = reinterpret_cast<uint32_t*>(smem + static_cast<size_t>(p.pv) * 16);  // this CTA's counts, or lists
  uint32_t* s_all = s_hist + kWide;                                                        // the cluster's counts
  int turn = 0;
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (waited for before the first remote store)
  auto together = [&] {
    __syncwarp();
    if (C == 1) __syncthreads();
    else cluster_sync_all();
  };
  // Every CTA's values, the same in all its threads: s.slot[..][i][rank] in each.
  using Slots = const unsigned long long (*)[kMaxCluster];
  auto gather = [&](unsigned long long a, unsigned long long b = 0, unsigned long long c = 0) -> Slots {
    Slots got = s.slot[turn];
    if (tid < Sh::kTold * C) {
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
  const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));  // elements before it in memory's 16 bytes
  // a warp's vectors are consecutive, and of them a lane's in the draw (an odd number, so that the lanes'
  // reads fall into different banks)
  const int run = ((p.pv - 1) / (32 * kWarps) + 1) | 1, v0 = min(p.pv, warp * 32 * run), v1 = min(p.pv, v0 + 32 * run);
  const int run0 = min(v1, v0 + lane * run), run1 = min(v1, run0 + run);
  const int base = rank * p.pv;
  const float temperature = p.temperature ? p.temperature[r] : 1.f, u = p.uniforms[r];
  const int top_k = p.top_k ? p.top_k[r] : 0;
  const float top_p = p.top_p ? p.top_p[r] : 1.f, min_p = p.min_p ? p.min_p[r] : 0.f;
  auto index_of = [&](int v) { return (base + v) * N; };  // of a vector's first element
  float top = -INFINITY;
  bool odd = false;  // NaN or +infinity
  // (places outside the row are NaN, which no comparison below takes and which weighs nothing)
  const uint32_t nan = sizeof(T) == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
  const uint4 none = make_uint4(nan, nan, nan, nan);
  // A warp fetches its own vectors by one bulk copy, all of a CTA's in flight together, and what lies in the row in
  // part by element.  Vectors are counted from the row's first element, so that what is added up in one
  // does not follow from where the row lies: where it begins inside memory's 16 bytes, the copy brings
  // those that lie in it whole, `skew` elements too far on, and the warp moves them to their places (128 rows
  // of 50257 without cuts, most of them so: fp32 11.1 us, bf16 10.4; left where memory puts them 8.9, 8.8).
  const int copy0 = max(v0, min(v1, (skew > 0 ? 1 : 0) - base)), copy1 = max(copy0, min(v1, (p.V + skew) / N - base));
  const int whole1 = max(v0, min(v1, p.V / N - base));  // vectors from v0 on that lie in the row whole
  if (lane == 0) {
    mbar_init(&s.bar[warp], 1);
    fence_mbar_init();
    if (copy1 > copy0) {
      mbar_arrive_expect_tx(&s.bar[warp], (copy1 - copy0) * 16);
      bulk_g2s(s_x + copy0, row + static_cast<long long>(index_of(copy0) - skew) * static_cast<int>(sizeof(T)), (copy1 - copy0) * 16, &s.bar[warp]);
    }
  }
  auto by_element = [&](int v) {
    uint4 w = none;
    T* q = reinterpret_cast<T*>(&w);
    const int e = index_of(v);
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (e + k < p.V) q[k] = reinterpret_cast<const T*>(row)[e + k];
    return w;
  };
  for (int v = v0 + lane; v < v1; v += 32)
    if (v < copy0 || v >= copy1) s_x[v] = by_element(v);
  // (moved: the last copied vector's second part lies in one that was not copied, or for another warp)
  const bool moves = skew > 0 && copy1 > copy0;
  const uint4 last = moves && lane == 0 ? by_element(copy1 - 1) : none;
  __syncwarp();
  const bool late = copy1 > copy0 && !mbar_wait_sleep(&s.bar[warp], 0, kTries, kNs);
  if (moves) {
    const int words = skew * static_cast<int>(sizeof(T)) / 4, bits = skew * static_cast<int>(sizeof(T)) % 4 * 8;
    for (int vv = copy0; vv < copy1 - 1; vv += 32) {
      const int v = vv + lane;
      const uint4 a = v < copy1 - 1 ? s_x[v] : none, b = v < copy1 - 1 ? s_x[v + 1] : none;
      uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      __syncwarp();  // all have read
#pragma unroll
      for (int k = 0; k < 6; ++k) w[k] = words & 2 ? w[k + 2] : w[k];
#pragma unroll
      for (int k = 0; k < 5; ++k) w[k] = words & 1 ? w[k + 1] : w[k];
      if (v < copy1 - 1)
        s_x[v] = make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                            __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
    }
    if (lane == 0) s_x[copy1 - 1] = last;
    __syncwarp();
  }
  {
    // (-infinity is a word of its own for each type; NaN stays, and so does +infinity)
    const uint32_t least = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
    uint32_t most[4] = {least, least, least, least};
    auto edge = [&](int v) {  // a vector that lies in the row in part
      float f[N];
      Vec<T>::unpack(s_x[v], f);
      for (int k = 0; k < N; ++k) {
        top = fmaxf(top, f[k]);
        odd |= index_of(v) + k < p.V && !(f[k] < INFINITY);
      }
    };
#pragma unroll 4
    for (int v = v0 + lane; v < whole1; v += 32) {
      const uint4 w = s_x[v];
      most[0] = max_nan<T>(most[0], w.x);
      most[1] = max_nan<T>(most[1], w.y);
      most[2] = max_nan<T>(most[2], w.z);
      most[3] = max_nan<T>(most[3], w.w);
    }
    for (int v = whole1 + lane; v < v1; v += 32) edge(v);
    const uint32_t word = max_nan<T>(max_nan<T>(most[0], most[1]), max_nan<T>(most[2], most[3]));
    const float a = __uint_as_float(sizeof(T) == 2 ? word << 16 : word), b = __uint_as_float(word & 0xFFFF0000u);
    top = fmaxf(top, sizeof(T) == 2 ? fmaxf(a, b) : a);
    odd |= !(a < INFINITY) || (sizeof(T) == 2 && !(b < INFINITY));
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
    const Slots all = gather(mine, gave_up);
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
  auto each = [&](auto f) {  // this thread's scores of the row
    for (int v = v0 + lane; v < v1; v += 32) {
      float x[N];
      Vec<T>::unpack(s_x[v], x);
      if (v < whole1) {
#pragma unroll
        for (int k = 0; k < N; ++k) f(x[k]);
      } else {
        const int e = index_of(v);
        for (int k = 0; k < N; ++k)
          if (e + k < p.V) f(x[k]);
      }
    }
  };
  auto write = [&](int token, float logprob) {
    p.token[r] = token;
    if (p.logprob) p.logprob[r] = logprob;
  };
  if (temperature == 0.f) {  // the first of the highest
    int at = INT32_MAX;
    for (int v = v0 + lane; v < v1; v += 32) {
      float x[N];
      Vec<T>::unpack(s_x[v], x);
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (x[k] == top) at = min(at, index_of(v) + k);
    }
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) s.warp_b[warp] = at;
    __syncthreads();
    unsigned long long least = s.warp_b[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) least = min(least, s.warp_b[w]);
    const Slots all = gather(least);
    for (int i = 0; i < C; ++i) least = min(least, all[0][i]);
    if (rank == 0 && tid == 0) {
      write(static_cast<int>(least), 0.f);
      if (p.bounds) p.bounds[static_cast<long long>(r) * p.bounds_stride] = specdec_keep_bound{top_key, static_cast<int>(least)};
    }
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
  auto finish = [&](int token, float score, unsigned long long total) {
    // the highest mass is 1 and among the kept: the sum's logarithm from what it is above 1
    const float above = static_cast<float>(total - (1ull << kMassBits)) * (1.f / (1ull << kMassBits));
    write(token, fmaf(sc.exponent(score), 0.693147181f, -log1pf(above)));
  };

  // ---------------------------------------------------------------------- the cuts
  uint32_t cut_key = 0;        // kept: a larger key, and the first `ties` tokens of this one
  uint32_t ties = 0xFFFFFFFFu;  // (all)
  float cut = -INFINITY;       // its score
  auto in_row = [&](int e) { return e < p.V; };
  const bool by_mass = top_p < 1.f, by_count = top_k > 0 && top_k < p.V;
  if (kCuts && (by_mass || by_count)) {
    uint32_t* all_count = s_all;                                                       // of the cluster
    unsigned long long* all_mass = reinterpret_cast<unsigned long long*>(s_all + kNarrow);  // (not with kWide bins)
    unsigned long long mixed_mass[3] = {0, 0, 0};  // of the wide bins that hold more than one score
    // Counts, and with `sums` masses, of tokens by place, added up over the cluster: pass(add) calls
    // add(place) for each.  hot: the place of the lowest scores, where masked tokens are, perhaps nearly all:
    // they are counted in the last 32 bins, by lane (negative: it is a place like the others).  Nothing here
    // branches for a token: branches were most of what a token cost.
    auto histogram = [&](int bins, bool sums, int hot, auto pass) {
      for (int i = tid; i < bins * (sums ? 4 : 1); i += kThreads) s_hist[i] = 0;
      __syncthreads();
      pass([&](int at) { atomicAdd(&s_hist[at == hot ? bins - 32 + lane : at], 1u); });
      if (hot >= 0) {
        __syncthreads();
        if (warp == 0) {
          const uint32_t n = __reduce_add_sync(0xffffffffu, s_hist[bins - 32 + lane]);
          s_hist[bins - 32 + lane] = 0;
          if (lane == 0) s_hist[hot] += n;
        }
      }
      together();
      // a CTA adds up its part of the bins over all (four lanes to four bins, a quarter of the CTAs each), and
      // tells all
      const int part = bins / C, b0 = rank * part;
      for (int i = tid; i < part; i += kThreads) {
        const int b = b0 + (i & ~3);
        uint4 n = make_uint4(0, 0, 0, 0);
        unsigned long long m[4] = {0, 0, 0, 0};
        auto add = [](uint4& a, uint4 v) {
          a.x += v.x;
          a.y += v.y;
          a.z += v.z;
          a.w += v.w;
        };
#pragma unroll
        for (int k = 0; k < kMaxCluster / 4; ++k) {
          const int c = 4 * k + (i & 3);
          if (c >= C) break;
          const uint32_t a = cluster_map(&s_hist[b], c);
          add(n, remote_load4(a));
          if (sums)
#pragma unroll
            for (int h = 0; h < 3; ++h) {
              const uint4 v = remote_load4(a + 4 * (h + 1) * bins);
              m[0] += static_cast<unsigned long long>(v.x) << (28 - 14 * h);
              m[1] += static_cast<unsigned long long>(v.y) << (28 - 14 * h);
              m[2] += static_cast<unsigned long long>(v.z) << (28 - 14 * h);
              m[3] += static_cast<unsigned long long>(v.w) << (28 - 14 * h);
            }
        }
#pragma unroll
        for (int d = 1; d < 4; d *= 2) {
          add(n, make_uint4(__shfl_xor_sync(0xffffffffu, n.x, d), __shfl_xor_sync(0xffffffffu, n.y, d),
                            __shfl_xor_sync(0xffffffffu, n.z, d), __shfl_xor_sync(0xffffffffu, n.w, d)));
          if (sums)
#pragma unroll
            for (int k = 0; k < 4; ++k) m[k] += __shfl_xor_sync(0xffffffffu, m[k], d);
        }
        const int k = i & 3;  // (each lane has all four)
        all_count[b + k] = k == 0 ? n.x : k == 1 ? n.y : k == 2 ? n.z : n.w;
        if (sums) all_mass[b + k] = k == 0 ? m[0] : k == 1 ? m[1] : k == 2 ? m[2] : m[3];
      }
      __syncthreads();
      for (int i = tid; i < part / 4 * C; i += kThreads) {
        const int c = i / (part / 4), b = b0 + 4 * (i - c * (part / 4));
        if (c == rank) continue;
        remote_store4(cluster_map(&all_count[b], c), *reinterpret_cast<const uint4*>(&all_count[b]));
        if (sums) {
          remote_store4(cluster_map(&all_mass[b], c), *reinterpret_cast<const uint4*>(&all_mass[b]));
          remote_store4(cluster_map(&all_mass[b + 2], c), *reinterpret_cast<const uint4*>(&all_mass[b + 2]));
        }
      }
      together();
    };
    // A pass for fp32 and for what one bin holds: place(x) < 0 is none.
    auto by_place = [&](int bins, auto place) {
      return [&, bins, place](auto add) {
        each([&](float x) {
          const int at = place(x);
          if (at < 0) return;
          add(at);
          if (by_mass) {  // 14 bits at a time, so that 2^17 tokens' fit 32
            const unsigned long long m = whole(sc.mass(x));
            const uint32_t hi = static_cast<uint32_t>(m >> 28);
            if (hi) atomicAdd(&s_hist[bins + at], hi);  // (few)
            atomicAdd(&s_hist[2 * bins + at], static_cast<uint32_t>(m >> 14) & 0x3FFFu);
            atomicAdd(&s_hist[3 * bins + at], static_cast<uint32_t>(m) & 0x3FFFu);
          }
        });
      };
    };
    // The last bin that is not empty and begins before `target` tokens, or that much mass (in `wide` bins a
    // score's mass times its count): it, what it holds and what is before it are left in s.  With target 0
    // all of the mass, in s.mass_before.
    auto bin_with = [&](int bins, bool wide, bool by_sum, unsigned long long target) {
      auto mass_in = [&](int b, uint32_t n) -> unsigned long long {
        if (n == 0 || !by_mass) return 0;
        if (!wide) return all_mass[b];
        const int m = mixed(b);
        return m < 0 ? n * whole(sc.mass(wide_score(b))) : m == 0 ? mixed_mass[0] : m == 1 ? mixed_mass[1] : mixed_mass[2];
      };
      // a warp has neighbouring bins, of which a lane has every 32nd
      const int per = bins / kWarps, b0 = warp * per + lane;
      uint32_t count = 0;
      unsigned long long mass = 0;
#pragma unroll 4
      for (int i = 0; i < per; i += 32) {
        const uint32_t n = all_count[b0 + i];
        count += n;
        mass += mass_in(b0 + i, n);
      }
      count = __reduce_add_sync(0xffffffffu, count);
      mass = warp_sum(mass);
      __syncthreads();
      if (lane == 0) {
        s.warp_a[warp] = count;
        s.warp_b[warp] = mass;
      }
      __syncthreads();
      unsigned long long cb = 0, mb = 0, c_at = 0, m_at = 0;
      int owner = 0;  // the last warp with tokens that begins before the target
      for (int w = 0; w < kWarps; ++w) {
        const unsigned long long c = s.warp_a[w], m = s.warp_b[w];
        if (c > 0 && (by_sum ? mb : cb) < target) {
          owner = w;
          c_at = cb;
          m_at = mb;
        }
        cb += c;
        mb += m;
      }
      if (target == 0) {
        if (tid == 0) s.mass_before = mb;
        __syncthreads();
        return;
      }
      if (warp == owner) {
        for (int i = 0; i < per; i += 32) {
          const uint32_t n = all_count[b0 + i];
          const unsigned long long m = mass_in(b0 + i, n), ci = warp_scan(n), mi = warp_scan(m);
          const unsigned long long c0 = c_at + ci - n, m0 = m_at + mi - m;
          const uint32_t could = __ballot_sync(0xffffffffu, n > 0 && (by_sum ? m0 : c0) < target);
          if (could && lane == 31 - __clz(could)) {  // (a later one takes its place)
            s.bin = b0 + i;
            s.count_before = c0;
            s.mass_before = m0;
            s.count = n;
          }
          c_at += __shfl_sync(0xffffffffu, ci, 31);
          m_at += __shfl_sync(0xffffffffu, mi, 31);
          if ((by_sum ? m_at : c_at) >= target) break;
          __syncwarp();
        }
      }
      __syncthreads();
    };
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

    // The first histogram: 32 bins an octave, or for bf16 one a score.
    constexpr bool kWideBins = sizeof(T) == 2;
    bool first_there = false;
    auto first = [&] {
      if (kWideBins) {
        unsigned long long m[3] = {0, 0, 0};
        histogram(kWide, false, kWidePlaces - 1, [&](auto add) {
          for (int v = v0 + lane; v < v1; v += 32) {
            const uint4 q = s_x[v];
            const uint32_t word[4] = {q.x, q.y, q.z, q.w};
            const bool full = v < whole1;
            uint32_t apart = full ? 0u : 0xFFu;  // bits of those to be seen one by one (few, or weighing nothing)
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // wide_place of two scores at once
              const uint32_t w = word[k];
              const uint32_t size = __vminu2(__vmaxu2(w & 0x7FFF7FFFu, (kSmall - 1) * 0x10001u), kLarge * 0x10001u) - (kSmall - 1) * 0x10001u;
              const uint32_t minus = (w >> 15 & 0x10001u) * 0xFFFFu, middle = (kValues + 1) * 0x10001u;
              const uint32_t b = ((middle + size) & minus) | ((middle - size) & ~minus);
              if (full) {
                add(static_cast<int>(b & 0xFFFFu));
                add(static_cast<int>(b >> 16));
              }
              if (by_mass) {  // in bins of several scores
                if ((size & 0xFFFFu) - 1 >= kValues) apart |= 1u << (2 * k);
                if ((size >> 16) - 1 >= kValues) apart |= 2u << (2 * k);
              }
            }
            for (; apart; apart &= apart - 1) {
              const int k = __ffs(apart) - 1;
              const uint32_t w = k < 4 ? (k < 2 ? q.x : q.y) : (k < 6 ? q.z : q.w);
              if (!full && !in_row(index_of(v) + k)) continue;
              const float x = __uint_as_float(k & 1 ? w & 0xFFFF0000u : w << 16);
              const int b = wide_place(x), of = mixed(b);
              if (!full) add(b);
              if (!by_mass || of < 0) continue;
              const unsigned long long weight = whole(sc.mass(x));
              m[0] += of == 0 ? weight : 0;
              m[1] += of == 1 ? weight : 0;
              m[2] += of == 2 ? weight : 0;
            }
          }
        });
        if (by_mass) {
          sum_all(m[0], m[1], m[2]);
#pragma unroll
          for (int k = 0; k < 3; ++k) mixed_mass[k] = m[k];
        }
      } else {
        histogram(kNarrow, by_mass, (kWidePlaces - 1) >> 2, by_place(kNarrow, [](float x) { return wide_place(x) >> 2; }));
      }
      first_there = true;
    };

    // The cut: the last token of the order before which there are fewer than `target` tokens, or less mass.
    // Sets cut_key, cut and ties; returns the mass up to and with it (where masses are counted).
    auto find_cut = [&](bool by_sum, unsigned long long target) -> unsigned long long {
      if (!first_there) first();
      bin_with(kWideBins ? kWide : kNarrow, kWideBins, by_sum, target);
      int b = s.bin;
      uint32_t klo = kWideBins ? wide_low(b) : wide_low(min(4 * b + 3, kWidePlaces - 1)), khi = wide_high(kWideBins ? b : 4 * b);
      bool one_score = kWideBins && mixed(b) < 0;
      uint32_t count = s.count;
      unsigned long long sum = s.mass_before;
      target -= by_sum ? s.mass_before : s.count_before;
      for (int round = 0; !one_score && klo < khi && count > kList && round < 4; ++round) {  // (each leaves a thousandth of the keys)
        const int shift = max(0, 22 - __clz(khi - klo));
        const uint32_t a = klo, z = khi;
        first_there = false;
        histogram(kNarrow, by_mass, -1, by_place(kNarrow, [=](float x) {
          const uint32_t key = order_bits(x);
          return key >= a && key <= z ? static_cast<int>((z - key) >> shift) : -1;
        }));
        bin_with(kNarrow, false, by_sum, target);
        b = s.bin;
        khi = z - (static_cast<uint32_t>(b) << shift);
        if (khi - a >= 1u << shift) klo = khi - ((1u << shift) - 1);
        count = s.count;
        sum += s.mass_before;
        target -= by_sum ? s.mass_before : s.count_before;
      }
      if (one_score || klo == khi) {
        const float score = one_score ? wide_score(b) : score_of(klo);
        const unsigned long long one = by_mass ? whole(sc.mass(score)) : 0;
        const unsigned long long want = !by_sum ? target : one == 0 ? count : min(static_cast<unsigned long long>(count), (target + one - 1) / one);
        cut_key = order_bits(score);
        cut = score;
        ties = want >= count ? 0xFFFFFFFFu : static_cast<uint32_t>(want);
        return sum + want * one;
      }
      // this CTA's tokens in question, then everyone's in every CTA, in order of rank
      uint32_t *l_list = s_hist, *list = l_list + kList;  // keys
      together();  // all are done with the histograms
      if (tid == 0) s.listed = 0;
      __syncthreads();
      {
        const uint32_t a = klo, z = khi;
        for (int v = v0 + lane; v < v1; v += 32) {
          float x[N];
          Vec<T>::unpack(s_x[v], x);
          const int e = index_of(v);
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const uint32_t key = order_bits(x[k]);
            if (key >= a && key <= z && in_row(e + k)) l_list[atomicAdd(&s.listed, 1u)] = key;
          }
        }
      }
      __syncthreads();
      const Slots all = gather(s.listed);
      int n = 0;
      for (int c = 0; c < C; ++c) {
        const int m = static_cast<int>(all[0][c]);
        for (int i = tid; i < m; i += kThreads) list[n + i] = remote_load(cluster_map(&l_list[i], c));
        n += m;
      }
      __syncthreads();
      uint32_t key[kEach];
      unsigned long long weight[kEach], mass[kEach];  // what is counted, and the mass
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const bool have = kThreads * i + tid < n;
        key[i] = have ? list[kThreads * i + tid] : 0;
        mass[i] = have && by_mass ? whole(sc.mass(score_of(key[i]))) : 0;
        weight[i] = by_sum ? mass[i] : have ? 1 : 0;
      }
      // the least key before which (among larger ones) there is less than the target
      uint32_t k0 = klo, k1 = khi;
      while (k0 < k1) {
        const uint32_t mid = k0 + (k1 - k0) / 2;
        unsigned long long v = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) v += key[i] > mid ? weight[i] : 0;
        if (block_sum(v) < target) k1 = mid;
        else k0 = mid + 1;
      }
      // (that may be a key below the last kept one where nothing is between: the least that is there)
      uint32_t least = 0xFFFFFFFFu;
      unsigned long long larger = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (key[i] >= k1 && kThreads * i + tid < n) least = min(least, key[i]);
        larger += key[i] > k1 ? weight[i] : 0;
      }
      least = __reduce_min_sync(0xffffffffu, least);
      __syncthreads();
      if (lane == 0) s.warp_b[warp] = least;
      larger = block_sum(larger);
      for (int w = 0; w < kWarps; ++w) least = min(least, static_cast<uint32_t>(s.warp_b[w]));
      unsigned long long equal = 0, above = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const bool have = kThreads * i + tid < n;
        equal += have && key[i] == least ? 1 : 0;
        above += have && key[i] > least ? mass[i] : 0;
      }
      equal = block_sum(equal);
      if (by_mass) above = block_sum(above);
      together();  // the lists may be written again
      cut_key = least;
      cut = score_of(least);
      const unsigned long long one = by_mass ? whole(sc.mass(cut)) : 0;
      unsigned long long want = equal;
      if (least == k1) want = min(equal, !by_sum ? target - larger : one == 0 ? equal : (target - larger + one - 1) / one);
      ties = want == equal ? 0xFFFFFFFFu : static_cast<uint32_t>(want);
      return sum + above + want * one;
    };
    unsigned long long kept = 0;
    if (by_count) kept = find_cut(false, top_k);
    if (by_mass) {
      if (!by_count) {
        first();
        bin_with(kWideBins ? kWide : kNarrow, kWideBins, true, 0);
        kept = s.mass_before;
      }
      (void)find_cut(true, max(1ull, times(top_p, kept, true)));
    }
  }
  if (min_p > 0.f) {
    const uint32_t key = min_p_key();
    if (key > cut_key) {
      cut_key = key;
      ties = 0xFFFFFFFFu;
      cut = score_of(key);
    }
  }

  // ---------------------------------------------------------------------- the draw
  // Of a vector: the running masses of what is kept above the cut (as sums of floats: the last is what the
  // vector adds; with all ties kept, them too) and how many tokens are at it.
  const bool cuts = cut_key != 0, some = ties != 0xFFFFFFFFu;
  const unsigned long long one = some ? whole(sc.mass(cut)) : 0;
  WholeSum masses;
  uint32_t equal = 0;
  if (cuts) {
    for (int v = run0; v < run1; ++v) {
      float x[N], vector = 0.f;
      Vec<T>::unpack(s_x[v], x);
      bool any = false;
#pragma unroll
      for (int k = 0; k < N; ++k) any |= x[k] >= cut;
      if (!any) continue;
      float mass[N];
      sc.masses<N>(x, mass);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        vector += x[k] > cut || (!some && x[k] == cut) ? mass[k] : 0.f;
        equal += x[k] == cut;
      }
      masses.add(vector);
    }
  } else {
#pragma unroll 4
    for (int v = run0; v < run1; ++v) {
      float x[N], mass[N], vector = 0.f;
      Vec<T>::unpack(s_x[v], x);
      sc.masses<N>(x, mass);
#pragma unroll
      for (int k = 0; k < N; ++k) vector += mass[k];
      masses.add(vector);
    }
  }
  unsigned long long sum = masses.value();
  const unsigned long long of_lane = sum;
  const uint32_t equal_of_lane = equal;
  sum = warp_sum(sum);
  if (some) equal = __reduce_add_sync(0xffffffffu, equal);
  __syncthreads();
  if (lane == 0) {
    s.warp_a[warp] = sum;
    s.warp_b[warp] = equal;
  }
  __syncthreads();
  unsigned long long before = 0, cta = 0, ties_before = 0, ties_cta = 0;
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? s.warp_a[w] : 0;
    cta += s.warp_a[w];
    if (some) {
      ties_before += w < warp ? s.warp_b[w] : 0;
      ties_cta += s.warp_b[w];
    }
  }
  const Slots all = gather(cta, ties_cta);
  unsigned long long total = 0;
  for (int i = 0; i < C; ++i) {
    before += i < rank ? all[0][i] : 0;
    total += all[0][i];
    if (some) ties_before += i < rank ? all[1][i] : 0;
  }
  // (of the ties the first `ties` in the row)
  auto of_ties = [&](unsigned long long n) { return some ? min(n, static_cast<unsigned long long>(ties)) * one : 0; };
  if (some) total += ties * one;
  const unsigned long long want = times(u, total, false);  // the first whose running mass is above it
  const unsigned long long begin = before + of_ties(ties_before), end = before + sum + of_ties(ties_before + equal);
  // the warp of the last kept tie tells its index, where a bound is wanted
  const bool tells = some && p.bounds && ties_before < ties && ties <= ties_before + equal, draws = want >= begin && want < end;
  if (p.bounds && !some && rank == 0 && tid == 0)
    p.bounds[static_cast<long long>(r) * p.bounds_stride] = specdec_keep_bound{cut_key, INT32_MAX};
  if (!tells && !draws) return;
  // the run that has the token, or the tie, then the place in it: a vector a lane
  const unsigned long long lane_before = before + warp_scan(of_lane) - of_lane;
  const unsigned long long lane_ties = some ? ties_before + warp_scan(equal_of_lane) - equal_of_lane : 0;
  for (const bool tie : {false, true}) {
    if (tie ? !tells : !draws) continue;
    const bool here = tie ? lane_ties < ties && ties <= lane_ties + equal_of_lane
                          : want >= lane_before + of_ties(lane_ties) && want < lane_before + of_lane + of_ties(lane_ties + equal_of_lane);
    const int owner = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    if (owner < 0) continue;
    unsigned long long at = __shfl_sync(0xffffffffu, lane_before, owner), t_at = __shfl_sync(0xffffffffu, lane_ties, owner);
    const int first = __shfl_sync(0xffffffffu, run0, owner), last = __shfl_sync(0xffffffffu, run1, owner);
    for (int vv = first; vv < last; vv += 32) {
      const int v = vv + lane;
      float m[N], x[N], vector = 0.f;
      Vec<T>::unpack(v < last ? s_x[v] : none, x);
      uint32_t t = 0;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float mass = sc.mass(x[k]);
        vector += !cuts || x[k] > cut || (!some && x[k] == cut) ? mass : 0.f;
        m[k] = vector;
        t += some && x[k] == cut;
      }
      const unsigned long long add = whole(vector), scan = warp_scan(add), mine = at + scan - add;
      const unsigned long long t_scan = some ? warp_scan(t) : 0;
      unsigned long long n = t_at + t_scan - t;
      const bool has = want >= mine + of_ties(n) && want < mine + add + of_ties(n + t);
      bool got = false;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (some && x[k] == cut && ++n == ties && tie)
          p.bounds[static_cast<long long>(r) * p.bounds_stride] = specdec_keep_bound{cut_key, index_of(v) + k};
        if (!tie && has && !got && mine + whole(m[k]) + of_ties(n) > want) {
          got = true;
          finish(index_of(v) + k, x[k], total);
        }
      }
      at += __shfl_sync(0xffffffffu, scan, 31);
      t_at += __shfl_sync(0xffffffffu, t_scan, 31);
    }
  }
}

template <typename T>
int launch_sample(SampleParams p, int R, cudaStream_t stream) {
  constexpr int N = Vec<T>::N;
  const int vectors = (p.V + N - 1) / N;
  const size_t extra = p.top_k || p.top_p ? 2 * kWide * 4 : 0;
  constexpr size_t kRoom = 200 << 10;
  const int sms = std::max(1, sm_count());
  // CTAs that an SM holds at once, and of a row: what its scores need, then more while all rows' run at once.
  // (A CTA's part is as large as lets two be on an SM: of 60 KB at most, with more CTAs to a row, 256 bf16 rows
  // of 151936 with top-k took 292 us against 88, 256 fp32 rows without cuts 72 against 49.  More while all
  // run at once, of 8 KB of scores each and from 8 CTAs to 16 of 16 KB: bf16 with top-p, one row of 151936
  // 20 us against 27 with what it needs, or 23 with 8; of 4 KB, or of 16: 8 rows of 32000 18.3, 21.0, 19.1; of
  // 16000 20.3, 19.8, 21.3; 16 CTAs of 8 KB in place of 8: 8 rows of 64000 22.0 against 19.7.)
  auto bytes = [&](int c) { return static_cast<size_t>((vectors - 1) / c + 1) * 16 + extra; };
  auto resident = [&](int c) { return std::min<long long>(extra ? 2 : 4, (220 << 10) / (bytes(c) + (2 << 10))) * sms; };
  int C = 1;
  while (C < kMaxCluster && (bytes(C) > (112 << 10) || (R * 2LL * C <= resident(2 * C) && vectors > C * (C < 8 ? 512 : 1024)))) C *= 2;
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
