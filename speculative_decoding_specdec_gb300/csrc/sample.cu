// Tokens from score rows: temperature, top-k, top-p, min-p, and the draw from a given uniform.
//
// The mathematics.  With z(x) = (max - x) log2(e) / T a token of score x has the mass 2^-z, its
// probability up to the row's sum.  In order of score (lowest index first among equals) top-k keeps
// the first k tokens, top-p those of them before which less than top_p of their mass lies, and min-p
// cuts at x = max + T ln(min_p).  Every setting keeps a beginning of that order, so a cut is one token,
// the last that is kept, and the kept set is told by its (score, index).  The draw is the first token
// by index whose running mass exceeds u times the sum.
//
// Masses are integers (2^-42 of the highest), so sums do not depend on their order and rows repeat
// bit for bit.  A mass is off by about 2^-27 of itself: z is held in two floats, split into eighths
// with a table of 2^(-i/8) and a Taylor polynomial of e^w, |w| < 0.044.  fp32 exponentials, off by
// 2^-22 in one direction for every token of one bf16 score, would move the borders between tokens
// enough to turn a draw in some ten thousand.
//
// A cluster holds a row in its CTAs' shared memory, read once from HBM; everything after is on chip:
//   1. the highest score (and whether there is NaN);
//   2. only where top-k or top-p is set: a histogram of 1024 bins of z (32 an octave down to 2^-16, 16 an
//      octave down to 2^-48) with counts and masses, each CTA's merged over the cluster by parts; the
//      bin that holds a cut; its tokens, listed in every CTA and ranked by comparing all pairs.  A bin
//      of more tokens than the list has room for is split by key until it has few, or equal ones,
//      which are counted by index;
//   3. the kept masses' sums by warp, CTA and cluster, and in the warp that owns the draw the token.
#include <algorithm>
#include <cmath>

#include "tree.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024, kList = 1024;
constexpr int kMaxCluster = 8;
constexpr int kMassBits = 42;
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number

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

// 2^-(i/8) as an integer of 30 bits and, times 2^26, as a float.
struct Entry {
  uint32_t whole;
  float f26;
};

// A row's scale: its highest score and log2(e) / T in two floats.
struct Scale {
  float top, sh, sl;
  const Entry* table;
  // z, to a float's precision and never falling as x falls
  __device__ __forceinline__ float z(float x) const { return (top - x) * sh; }
  // The mass as m * 2^(-30 - n); 0 beyond 2^-60.
  __device__ __forceinline__ uint32_t mass(float x, int& n) const {
    const float d = top - x, back = d - top, lost = (top - (d - back)) - (x + back);  // d and what it lost
    const float zh = d * sh, zl = fmaf(d, sh, -zh) + fmaf(d, sl, lost * sh);
    const float qm = fmaf(zh, 8.f, kMagic);
    const int q = __float_as_int(qm) - __float_as_int(kMagic);
    const float w = (fmaf(qm - kMagic, -0.125f, zh) + zl) * -0.693147181f;
    const float e = w * fmaf(w, fmaf(w, fmaf(w, fmaf(w, 1.f / 120, 1.f / 24), 1.f / 6), 0.5f), 1.f);  // e^w - 1
    const bool in = zh < 60.f;
    const Entry t = table[q & 7];
    n = in ? q >> 3 : 0;
    return in ? t.whole + ((__float_as_int(fmaf(e, t.f26, kMagic)) - __float_as_int(kMagic)) << 4) : 0u;
  }
  __device__ __forceinline__ unsigned long long mass42(float x) const {
    int n;
    const unsigned long long m = mass(x, n);
    return m << (kMassBits - 30) >> n;
  }
};
__device__ __forceinline__ int bin_of(float z) {
  const float b = z < 16.f ? z * 32.f : fminf(fmaf(z, 16.f, 256.f), kBins - 1.f);
  return static_cast<int>(b);
}
__device__ __forceinline__ int octave_of(int bin) { return bin < 512 ? bin >> 5 : 16 + ((bin - 512) >> 4); }
// A mass in units of 2^-30 of its bin's octave (at most 1 of those).
__device__ __forceinline__ uint32_t in_octave(uint32_t m, int n, int octave) { return n > octave ? m >> (n - octave) : m; }

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
  unsigned long long slot[2][kMaxCluster];  // what the cluster's CTAs tell each other, in turn
  unsigned long long warp_a[kWarps], warp_b[kWarps];
  unsigned long long found[4];
  uint32_t best, listed;
  uint32_t lo, hi;
  Entry table[8];
};

// Counts and masses of one thread's two bins and of all before them.
struct Bins {
  unsigned long long count[2], mass[2], rel[2], count_before[2], mass_before[2];
};

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p) {
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
  uint32_t* s_hist = reinterpret_cast<uint32_t*>(smem + static_cast<size_t>(p.pv) * 16);  // [3][kBins], or this CTA's list
  uint32_t* s_all = s_hist + 3 * kBins;                                                    // merged, or the cluster's list
  int turn = 0;
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (waited for before the first remote store)
  // Every CTA's value, in s.slot[..][rank] of each.
  auto gather = [&](unsigned long long v) -> const unsigned long long* {
    const unsigned long long* got = s.slot[turn];
    if (C == 1) {
      if (tid == 0) s.slot[turn][0] = v;
      __syncthreads();
    } else {
      if (tid < C) remote_store(cluster_map(&s.slot[turn][rank], tid), v);
      __syncwarp();
      cluster_sync_all();
    }
    turn ^= 1;
    return got;
  };
  auto together = [&] {
    __syncwarp();
    if (C == 1) __syncthreads();
    else cluster_sync_all();
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
  if (tid == 0) s.listed = 0;
  if (tid < 8) {
    const double f = exp2(-tid / 8.0);
    s.table[tid] = Entry{static_cast<uint32_t>(f * 1073741824.0 + 0.5), static_cast<float>(f * 67108864.0)};
  }
  const uint4 none = sizeof(T) == 2 ? make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u)
                                    : make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
#pragma unroll 4
  for (int v = v0 + lane; v < v1; v += 32) {
    const int e = index_of(v);
    uint4 w = none;
    if (e >= 0 && e + N <= p.V) {
      w = ldg_stream(row + static_cast<long long>(e) * static_cast<int>(sizeof(T)));
    } else {
      T* q = reinterpret_cast<T*>(&w);
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (e + k >= 0 && e + k < p.V) q[k] = reinterpret_cast<const T*>(row)[e + k];
    }
    s_x[v] = w;
    float f[N];
    Vec<T>::unpack(w, f);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      top = fmaxf(top, f[k]);
      odd |= !(f[k] < INFINITY);
    }
  }
  const bool bad_setting = !(temperature >= 0.f && temperature < INFINITY) || top_k < 0 || !(top_p > 0.f && top_p <= 1.f) ||
                           !(min_p >= 0.f && min_p <= 1.f) || !(u >= 0.f && u < 1.f);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  odd = __any_sync(0xffffffffu, odd);
  if (lane == 0) s.warp_a[warp] = static_cast<unsigned long long>(order_bits(top)) << 1 | (odd ? 1 : 0);
  __syncthreads();
  unsigned long long mine = s.warp_a[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) mine = max(mine, s.warp_a[w]) | ((mine | s.warp_a[w]) & 1);
  if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster runs
  {
    const unsigned long long* all = gather(mine);
    mine = all[0];
    for (int i = 1; i < C; ++i) mine = max(mine, all[i]) | ((mine | all[i]) & 1);
  }
  const uint32_t top_key = static_cast<uint32_t>(mine >> 1);
  auto score_of = [](uint32_t key) { return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key); };
  top = score_of(top_key);
  if (bad_setting || (mine & 1) || top == -INFINITY) {
    if (rank == 0 && tid == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
    together();  // no CTA leaves while another may write to it
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
    const unsigned long long* all = gather(least);
    for (int i = 0; i < C; ++i) least = min(least, all[i]);
    if (rank == 0 && tid == 0) write(static_cast<int>(least), 0.f, top_key, static_cast<int>(least));
    return;
  }
  const double per = fmin(1.4426950408889634 / static_cast<double>(temperature), 1e30);
  Scale sc;
  sc.top = top;
  sc.sh = static_cast<float>(per);
  sc.sl = static_cast<float>(per - static_cast<double>(sc.sh));
  sc.table = s.table;

  // ---------------------------------------------------------------------- the cuts
  uint32_t cut_key = 0;       // kept: a larger key, or this one up to index cut_last
  int cut_last = INT32_MAX;
  const bool by_mass = top_p < 1.f, by_count = top_k > 0 && top_k < p.V;
  if (by_mass || by_count) {
    // Histogram of what `in` accepts, merged over the cluster, with the sums before each bin.
    // in(x): the element's place, or -1; oct(place): the octave that its masses are in units of;
    // down(place): what takes those, times 2^(kMassBits - 30), to the sums' unit.
    auto histogram = [&](auto in, auto oct, auto down) {
      for (int i = tid; i < 3 * kBins; i += kThreads) s_hist[i] = 0;
      __syncthreads();
      uint32_t far = 0;  // (the last place, of most elements in a peaked row, is counted by itself)
      each([&](float x, int e) {
        const int place = e >= 0 && e < p.V ? in(x) : -1;
        if (place == kBins - 1) {
          ++far;
        } else if (place >= 0) {
          atomicAdd(&s_hist[place], 1u);
        }
        if (by_mass && place >= 0) {
          int n;
          const uint32_t m = sc.mass(x, n), rel = in_octave(m, n, oct(place));
          if (m != 0) {  // in two halves, so that sums of 2^16 of them and more fit 32 bits
            atomicAdd(&s_hist[kBins + place], rel >> 15);
            atomicAdd(&s_hist[2 * kBins + place], rel & 0x7FFFu);
          }
        }
      });
      far = __reduce_add_sync(0xffffffffu, far);
      if (lane == 0 && far) atomicAdd(&s_hist[kBins - 1], far);
      together();
      // a CTA adds up its part of the bins over all, 4 threads a bin, and tells all
      unsigned long long* all_rel = reinterpret_cast<unsigned long long*>(s_all);
      uint32_t* all_count = s_all + 2 * kBins;
      const int part = kBins / C;
      for (int i = tid; i < part * 4; i += kThreads) {
        const int b = rank * part + (i >> 2), q = i & 3;
        unsigned long long count = 0, rel = 0;
        for (int c = q; c < C; c += 4) {
          const uint32_t a = cluster_map(&s_hist[b], c);
          count += remote_load(a);
          rel += (static_cast<unsigned long long>(remote_load(a + 4 * kBins)) << 15) + remote_load(a + 8 * kBins);
        }
        count += __shfl_xor_sync(0xffffffffu, count, 1);
        rel += __shfl_xor_sync(0xffffffffu, rel, 1);
        count += __shfl_xor_sync(0xffffffffu, count, 2);
        rel += __shfl_xor_sync(0xffffffffu, rel, 2);
        for (int c = q; c < C; c += 4) {
          remote_store(cluster_map(&all_rel[b], c), rel);
          remote_store(cluster_map(&all_count[b], c), static_cast<uint32_t>(count));
        }
      }
      together();
      Bins g;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        g.count[i] = all_count[2 * tid + i];
        g.rel[i] = all_rel[2 * tid + i];
        g.mass[i] = g.rel[i] << (kMassBits - 30) >> down(2 * tid + i);
      }
      const unsigned long long ca = warp_scan(g.count[0] + g.count[1]), ma = warp_scan(g.mass[0] + g.mass[1]);
      if (lane == 31) {
        s.warp_a[warp] = ca;
        s.warp_b[warp] = ma;
      }
      __syncthreads();
      unsigned long long cb = ca - g.count[0] - g.count[1], mb = ma - g.mass[0] - g.mass[1];
      for (int w = 0; w < warp; ++w) {
        cb += s.warp_a[w];
        mb += s.warp_b[w];
      }
      g.count_before[0] = cb;
      g.count_before[1] = cb + g.count[0];
      g.mass_before[0] = mb;
      g.mass_before[1] = mb + g.mass[0];
      return g;
    };
    // The last bin that is not empty and begins before `target` tokens, or that much mass: its place,
    // and in s.found what is before it and in it (tokens, mass, tokens, relative mass).
    auto bin_with = [&](const Bins& g, bool mass, unsigned long long target) {
      __syncthreads();
      if (tid == 0) s.best = 0;
      __syncthreads();
      bool have[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        have[i] = g.count[i] > 0 && (mass ? g.mass_before[i] : g.count_before[i]) < target;
        if (have[i]) atomicMax(&s.best, 2 * tid + i + 1);
      }
      __syncthreads();
      const int at = static_cast<int>(s.best) - 1;
      if (tid == at >> 1) {
        const int i = at & 1;
        s.found[0] = i ? g.count_before[1] : g.count_before[0];
        s.found[1] = i ? g.mass_before[1] : g.mass_before[0];
        s.found[2] = i ? g.count[1] : g.count[0];
        s.found[3] = i ? g.rel[1] : g.rel[0];
      }
      __syncthreads();
      return at;
    };
    const Bins bins = histogram([&](float x) { return bin_of(sc.z(x)); }, octave_of, octave_of);

    // The cut: the last token of the order before which there are fewer than `target` tokens, or less
    // mass.  Sets cut_key and cut_last; returns the mass up to and with it (if masses are counted).
    auto find_cut = [&](bool mass, unsigned long long target) -> unsigned long long {
      const int bin = bin_with(bins, mass, target);
      const int oct = octave_of(bin);
      const unsigned long long mass_before = s.found[1];
      unsigned long long count = s.found[2], rel = s.found[3], left;  // of the tokens still in question, and what is left of the target
      if (mass) {
        const unsigned long long want = target - mass_before, whole = rel << (kMassBits - 30) >> oct;
        left = want >= whole ? rel : min(rel, ((want << oct) + ((1ull << (kMassBits - 30)) - 1)) >> (kMassBits - 30));
        left = max(left, 1ull);
      } else {
        left = target - s.found[0];
      }
      unsigned long long rel_before = 0;  // in the bin, of what is kept for certain
      uint32_t klo = 0, khi = 0xFFFFFFFFu;
      auto inside = [&](float x) {
        const uint32_t key = order_bits(x);
        return key >= klo && key <= khi && bin_of(sc.z(x)) == bin;
      };
      auto rel_of = [&](float x) {
        int n;
        const uint32_t m = sc.mass(x, n);
        return in_octave(m, n, oct);
      };
      for (int round = 0; count > kList && round < 8; ++round) {  // (each leaves a thousandth of the keys)
        __syncthreads();
        if (tid == 0) {
          s.lo = 0xFFFFFFFFu;
          s.hi = 0;
        }
        __syncthreads();
        uint32_t lo = 0xFFFFFFFFu, hi = 0;
        each([&](float x, int e) {
          if (e >= 0 && e < p.V && inside(x)) {
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
        const unsigned long long* all = gather(static_cast<unsigned long long>(s.hi) << 32 | s.lo);
        klo = 0xFFFFFFFFu;
        khi = 0;
        for (int i = 0; i < C; ++i) {
          klo = min(klo, static_cast<uint32_t>(all[i]));
          khi = max(khi, static_cast<uint32_t>(all[i] >> 32));
        }
        if (klo == khi) break;
        const int shift = max(0, 22 - __clz(khi - klo));
        const Bins g = histogram([&](float x) { return inside(x) ? static_cast<int>((khi - order_bits(x)) >> shift) : -1; },
                                 [&](int) { return oct; }, [](int) { return kMassBits - 30; });  // (sums in the bin's unit)
        const int at = bin_with(g, mass, left);
        const uint32_t first = khi - (static_cast<uint32_t>(at) << shift);
        khi = first;
        if (first - klo >= 1u << shift) klo = first - ((1u << shift) - 1);
        left -= mass ? s.found[1] : s.found[0];
        rel_before += s.found[1];
        count = s.found[2];
        rel = s.found[3];
      }
      if (count > kList) {
        // equal scores: the last one by index
        const uint32_t key = klo;
        const uint32_t one = rel_of(score_of(key));
        const unsigned long long want = !mass ? left : one == 0 ? count : min(count, (left + one - 1) / one);
        unsigned long long n = 0;
        each([&](float x, int e) { n += e >= 0 && e < p.V && order_bits(x) == key; });
        n = warp_sum(n);
        __syncthreads();
        if (lane == 0) s.warp_a[warp] = n;
        __syncthreads();
        unsigned long long before = 0, total = 0;
        for (int w = 0; w < kWarps; ++w) {
          before += w < warp ? s.warp_a[w] : 0;
          total += s.warp_a[w];
        }
        const unsigned long long* all = gather(total);
        for (int i = 0; i < rank; ++i) before += all[i];
        __syncthreads();
        if (tid == 0) s.found[0] = 0;
        __syncthreads();
        if (before < want && want <= before + n) {  // this warp has it
          for (int vv = v0; vv < v1; vv += 32) {
            const int v = vv + lane;
            float x[N];
            if (v < v1) Vec<T>::unpack(s_x[v], x);
            const int e = index_of(v);
            unsigned long long here = 0;
#pragma unroll
            for (int k = 0; k < N; ++k) here += v < v1 && e + k >= 0 && e + k < p.V && order_bits(x[k]) == key;
            const unsigned long long scan = warp_scan(here);
            unsigned long long at = before + scan - here;
#pragma unroll
            for (int k = 0; k < N; ++k)
              if (v < v1 && e + k >= 0 && e + k < p.V && order_bits(x[k]) == key && ++at == want) s.found[0] = e + k + 1;
            before += __shfl_sync(0xffffffffu, scan, 31);
          }
        }
        __syncthreads();
        const unsigned long long* who = gather(s.found[0]);
        unsigned long long last = 0;
        for (int i = 0; i < C; ++i) last = max(last, who[i]);
        cut_key = key;
        cut_last = static_cast<int>(last) - 1;
        rel_before += want * one;
      } else {
        // this CTA's tokens in question, then everyone's in every CTA, in order of rank
        uint32_t *l_key = s_hist, *l_index = s_hist + kList, *l_rel = s_hist + 2 * kList;
        uint32_t *a_key = s_all, *a_index = s_all + kList, *a_rel = s_all + 2 * kList;
        together();  // all are done with the histograms
        if (tid == 0) s.listed = 0;
        __syncthreads();
        each([&](float x, int e) {
          if (e >= 0 && e < p.V && inside(x)) {
            const uint32_t i = atomicAdd(&s.listed, 1u);
            l_key[i] = order_bits(x);
            l_index[i] = e;
            l_rel[i] = by_mass ? rel_of(x) : 0;
          }
        });
        __syncthreads();
        const unsigned long long* all = gather(s.listed);
        int n = 0;
        for (int c = 0; c < C; ++c) {
          const int m = static_cast<int>(all[c]);
          for (int i = tid; i < 3 * m; i += kThreads) {
            const int f = i / m, j = i - f * m;
            s_all[f * kList + n + j] = remote_load(cluster_map(&s_hist[f * kList + j], c));
          }
          n += m;
        }
        if (tid == 0) s.best = 0;
        __syncthreads();
        // a warp ranks a token: what is before it, and whether it is kept
        auto before_of = [&](int i, unsigned long long& tokens, unsigned long long& sum) {
          const unsigned long long me = static_cast<unsigned long long>(a_key[i]) << 32 | ~a_index[i];
          tokens = sum = 0;
          for (int j = lane; j < n; j += 32)
            if ((static_cast<unsigned long long>(a_key[j]) << 32 | ~a_index[j]) > me) {
              ++tokens;
              sum += a_rel[j];
            }
          tokens = warp_sum(tokens);
          sum = warp_sum(sum);
        };
        for (int i = rank * kWarps + warp; i < n; i += C * kWarps) {
          unsigned long long tokens, sum;
          before_of(i, tokens, sum);
          if (lane == 0 && (mass ? sum : tokens) < left) atomicMax(&s.best, static_cast<uint32_t>(tokens) << 16 | (i + 1));
        }
        __syncthreads();
        const unsigned long long* who = gather(s.best);
        unsigned long long best = 0;
        for (int i = 0; i < C; ++i) best = max(best, who[i]);
        const int at = static_cast<int>(best & 0xFFFF) - 1;
        cut_key = a_key[at];
        cut_last = static_cast<int>(a_index[at]);
        unsigned long long tokens, sum;
        before_of(at, tokens, sum);
        rel_before += sum + a_rel[at];
        together();  // the lists may be written again
      }
      return mass_before + (rel_before << (kMassBits - 30) >> oct);
    };
    unsigned long long kept = 0;
    if (by_count) {
      kept = find_cut(false, top_k);
    } else if (by_mass) {  // all of it
      const unsigned long long end = bins.mass_before[1] + bins.mass[1];
      __syncthreads();
      if (tid == kThreads - 1) s.found[0] = end;
      __syncthreads();
      kept = s.found[0];
    }
    if (by_mass) (void)find_cut(true, max(1ull, times(top_p, kept, true)));
  }
  if (min_p > 0.f) {
    const double cut = static_cast<double>(top) + static_cast<double>(temperature) * log(static_cast<double>(min_p));
    const float least = __double2float_ru(fmax(cut, -3.4028234663852886e38));
    const uint32_t key = order_bits(least);  // (the highest score's own at most)
    if (key > cut_key) {
      cut_key = key;
      cut_last = INT32_MAX;
    }
  }

  // ---------------------------------------------------------------------- the draw
  const bool cuts = cut_key != 0;
  const float cut = score_of(cut_key);
  auto kept_mass = [&](float x, int e) -> unsigned long long {
    if (cuts && !(x > cut || (x == cut && e <= cut_last))) return 0;
    return sc.mass42(x);
  };
  unsigned long long sum = 0;
  each([&](float x, int e) { sum += kept_mass(x, e); });
  sum = warp_sum(sum);
  __syncthreads();
  if (lane == 0) s.warp_a[warp] = sum;
  __syncthreads();
  unsigned long long before = 0, mine_all = 0;
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? s.warp_a[w] : 0;
    mine_all += s.warp_a[w];
  }
  const unsigned long long* all = gather(mine_all);
  unsigned long long total = 0;
  for (int i = 0; i < C; ++i) {
    before += i < rank ? all[i] : 0;
    total += all[i];
  }
  const unsigned long long want = times(u, total, false);  // the first whose running mass is above it
  if (want < before || want >= before + sum) return;
  for (int vv = v0; vv < v1; vv += 32) {
    const int v = vv + lane;
    float x[N];
    Vec<T>::unpack(v < v1 ? s_x[v] : none, x);
    const int e = index_of(v);
    unsigned long long here = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) here += kept_mass(x[k], e + k);
    const unsigned long long scan = warp_scan(here);
    unsigned long long at = before + scan - here;
    if (want >= at && want < at + here) {
      int token = 0;
      float score = 0.f;
      bool got = false;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        at += kept_mass(x[k], e + k);
        if (!got && at > want) {
          got = true;
          token = e + k;
          score = x[k];
        }
      }
      const double lp = (static_cast<double>(score) - static_cast<double>(top)) / static_cast<double>(temperature) -
                        log(static_cast<double>(total) * (1.0 / (1ull << kMassBits)));
      write(token, static_cast<float>(lp), cut_key, cut_last);
    }
    const unsigned long long step = __shfl_sync(0xffffffffu, scan, 31);
    if (want < before + step) return;
    before += step;
  }
}

// CTAs of a row: as many as one wave has room for, at least what its scores need.
template <typename T>
int launch_sample(SampleParams p, int R, cudaStream_t stream) {
  constexpr int N = Vec<T>::N;
  const int vectors = (p.V + 2 * N - 2) / N;  // whatever the row's alignment
  const size_t extra = p.top_k || p.top_p ? 6 * kBins * 4 : 0;
  constexpr size_t kRoom = 200 << 10;
  const int sms = std::max(1, sm_count());
  int C = 1;
  while (C < kMaxCluster && (static_cast<size_t>((vectors - 1) / C + 1) * 16 > (96 << 10) || (static_cast<long long>(R) * C * 2 <= 2 * sms && vectors > C * 256)))
    C *= 2;
  p.pv = (vectors - 1) / C + 1;
  const size_t smem = static_cast<size_t>(p.pv) * 16 + extra;
  if (smem > kRoom) return SPECDEC_ERR_UNSUPPORTED;
  auto kernel = sample_kernel<T>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRoom));
  if (e != cudaSuccess) return map_cuda_error(e);
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
  if (a->R >= (1 << 24) || a->V >= (1 << 24) || a->bounds_stride >= (1 << 30)) return SPECDEC_ERR_UNSUPPORTED;
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
