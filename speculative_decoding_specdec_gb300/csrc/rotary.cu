// Rotary positions of new tokens' queries and keys, fused with the append of their K/V columns.
//
// The mathematics.  Position p turns pair i of a head, (x1, x2), by the angle p * f_i:
//   (x1 c - x2 s, x1 s + x2 c),  c = cos(p f_i), s = sin(p f_i),
// so that the dot product of a turned query and a turned key depends on the difference of their
// positions alone.  c and s come from a table made once per model in 64 bits: p * f_i in fp32
// would be off by 4e-3 radians at p = 65536, and any scaling of f_i for long contexts costs
// nothing here.
//
// What bounds it.  Every value is read and written once (three flops per value): HBM for a
// prefill, the launch and one dependent chain of loads (parents or position, table, values) for
// a verification pass.  The unit of work is one 16-byte vector of a head, or a pair of them in
// the half layout, whose mates lie rot_dim / 2 values apart; consecutive threads take consecutive
// vectors.  Measured: 8 prompts of up to 1024 tokens, 32 heads of 128 each of q, k and v: 48 us
// (5.4 TB/s); 32 trees of 32 nodes, 32 query and 2 K/V heads: 6.9 us.
#include <algorithm>
#include <cmath>

#include "tree.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // heads in flight per thread

struct RotaryParams {
  ByteView cache;  // of the layer
  const char *q, *k, *v;
  char* qo;
  long long qr, qt, kr, kt, vr, vt, or_, ot;  // bytes between rows and tokens
  const float2* table;
  const int32_t *n_committed, *width, *parents, *positions, *columns, *start;
  int32_t* status;
  int T, Hq, H, hd, rot, interleaved, table_len, cap, one_row;
};

// Norms of the heads: nullptr where q or k has none.
struct NormParams {
  const char *q_weight, *k_weight;
  float eps, offset, inv_hd;
  int f32, same;  // the weights' type; whether it is q's and 16-byte loads reach them
};

// Position and column of token t of row b; false if nothing is to be written to the cache for it:
// it is padding (col < 0) or an unused node (pos = 0), whose q_out is zero, or an error was recorded
// (pos < 0 <= col).  All threads of the CTA get the same answer.
__device__ bool locate(const RotaryParams& p, int b, int t, int& pos, int& col) {
  if (p.positions) {
    pos = p.positions[static_cast<long long>(b) * p.T + t];
    col = p.columns[static_cast<long long>(b) * p.T + t];
    if (col < 0) return false;
  } else {
    __shared__ int s_par[kMaxTree];
    const int n = p.n_committed[b], W = *p.width;
    int depth = t;
    bool bad = n < 1 || n > W;
    if (p.parents) {
      if (threadIdx.x < p.T) s_par[threadIdx.x] = p.parents[b * p.T + threadIdx.x];
      __syncthreads();
      // the whole row's tree is checked, as the attention of the same pass does
      bool off = false;
      if (threadIdx.x < p.T) (void)tree_ancestors(s_par, threadIdx.x, off);
      bad |= __syncthreads_or(off);
      if (!bad) {
        bool unused = false;
        const unsigned long long m = tree_ancestors(s_par, t, unused);
        if (m == 0) return false;
        depth = __popcll(m) - 1;
      }
    }
    if (bad) {
      if (threadIdx.x == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
      pos = -1;
      return false;
    }
    // (a width near the integers' end is beyond every cache, and its columns must not wrap around)
    if (W > p.cap - t) {
      if (threadIdx.x == 0) set_status(p.status, SPECDEC_ERR_CAPACITY);
      pos = -1;
      return false;
    }
    pos = n - 1 + depth;  // at most W - 1 + t
    col = W - 1 + t;
  }
  if (pos < 0 || pos >= p.table_len || col >= p.cap) {
    if (threadIdx.x == 0)
      set_status(p.status, col >= p.cap ? SPECDEC_ERR_CAPACITY : SPECDEC_ERR_INPUT_RANGE);
    pos = -1;
    return false;
  }
  return true;
}

// N consecutive values as they lie, as floats, and back: one 16-byte access (N = Vec<T>::N) or one
// scalar.
template <typename T, int N> struct Values {
  using Raw = uint4;
  __device__ __forceinline__ static Raw load(const T* x) { return *reinterpret_cast<const uint4*>(x); }
  __device__ __forceinline__ static Raw zero() { return make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ static void unpack(Raw r, float* f) { Vec<T>::unpack(r, f); }
  __device__ __forceinline__ static Raw pack(const float* f) {
    if constexpr (sizeof(T) == 2)
      return make_uint4(bf16_pack(f[0], f[1]), bf16_pack(f[2], f[3]), bf16_pack(f[4], f[5]), bf16_pack(f[6], f[7]));
    else
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  __device__ __forceinline__ static void store(T* y, Raw r) { *reinterpret_cast<uint4*>(y) = r; }
};
template <typename T> struct Values<T, 1> {
  using Raw = T;
  __device__ __forceinline__ static Raw load(const T* x) { return *x; }
  __device__ __forceinline__ static Raw zero() { return T(0); }
  __device__ __forceinline__ static void unpack(Raw r, float* f) { f[0] = Vec<T>::scalar(&r); }
  __device__ __forceinline__ static Raw pack(const float* f) {
    if constexpr (sizeof(T) == 2) return bf16_bits(f[0]);
    else return f[0];
  }
  __device__ __forceinline__ static void store(T* y, Raw r) { *y = r; }
};

// A unit is two runs of N values of a head: N pairs to turn (the runs are rot_dim / 2 apart in
// the half layout, and one behind the other when interleaved), or 2N values to copy.  One thread
// reads both runs before it writes either, so q_out may be q.
template <typename T, int N, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const RotaryParams p) {
  const int b = blockIdx.x / p.T, t = blockIdx.x % p.T;
  int pos = 0, col = 0;
  const bool write = locate(p, b, t, pos, col);
  if (!write && pos < 0 && col >= 0) return;  // an error was recorded
  // A thread keeps its place in the head, so its cosines and sines are read once for all heads.
  const int half = p.rot / 2, per_head = p.hd / (2 * N), turned = half / N;
  const int step = kThreads / per_head, j = threadIdx.x % per_head;
  if (threadIdx.x >= step * per_head) return;
  const long long row = p.one_row ? 0 : b;
  const bool turns = j < turned;
  float2 c[N];
  if (turns && write) {
    const float2* cs = p.table + static_cast<long long>(pos) * half + j * N;
#pragma unroll
    for (int k = 0; k < N; ++k) c[k] = __ldg(cs + k);
  }
  const bool far = turns && !kInterleaved;  // the two runs lie rot_dim / 2 apart
  const int e0 = far ? j * N : 2 * j * N, e1 = far ? e0 + half : e0 + N;
  const int heads = write ? p.Hq + 2 * p.H : p.Hq;
  const char *q = p.q + b * p.qr + t * p.qt, *k = p.k + b * p.kr + t * p.kt,
             *v = p.v + b * p.vr + t * p.vt;
  char *qo = p.qo + b * p.or_ + t * p.ot,
       *to = p.cache.base + row * p.cache.srow + static_cast<long long>(col) * p.hd * sizeof(T);
  for (int h0 = blockIdx.y * step + threadIdx.x / per_head; h0 < heads; h0 += gridDim.y * step * kHeads) {
    typename Values<T, N>::Raw r0[kHeads], r1[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {  // loads first: they wait for memory together
      const int h = h0 + i * gridDim.y * step;
      r0[i] = r1[i] = Values<T, N>::zero();
      if (h < heads && write) {
        const T* x = reinterpret_cast<const T*>(h < p.Hq ? q : h < p.Hq + p.H ? k : v) +
                     (h < p.Hq ? h : h < p.Hq + p.H ? h - p.Hq : h - p.Hq - p.H) * p.hd;
        r0[i] = Values<T, N>::load(x + e0);
        r1[i] = Values<T, N>::load(x + e1);
      }
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = h0 + i * gridDim.y * step;
      if (h >= heads) break;
      const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.H;
      T* y = is_q ? reinterpret_cast<T*>(qo) + h * p.hd
                  : reinterpret_cast<T*>(to + (is_v ? p.cache.skv : 0) + (h - p.Hq - (is_v ? p.H : 0)) * p.cache.shead);
      if (turns && !is_v && write) {
        // pairs: neighbours of the 2N values, or one of each run
        float w[2 * N];
        Values<T, N>::unpack(r0[i], w);
        Values<T, N>::unpack(r1[i], w + N);
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const int a = kInterleaved ? 2 * n : n, b = kInterleaved ? 2 * n + 1 : N + n;
          const float x1 = w[a], x2 = w[b];
          w[a] = x1 * c[n].x - x2 * c[n].y;
          w[b] = x1 * c[n].y + x2 * c[n].x;
        }
        r0[i] = Values<T, N>::pack(w);
        r1[i] = Values<T, N>::pack(w + N);
      }
      Values<T, N>::store(y + e0, r0[i]);
      Values<T, N>::store(y + e1, r1[i]);
    }
  }
}

// Norms of q's and k's heads in the same pass.  y = x / sqrt(mean of x^2 + eps) * (offset + w) over the
// whole head, then the rotation, rounded once.  A head belongs to `lanes` neighbouring lanes of a warp
// (a power of two; U units each), so its sum of squares is a few shuffles and its values are read
// once, all of them before any is written (q_out may be q).
//
// A warp takes an item, a token's heads or a part of them, by itself.  What a token costs besides its
// values (its place, addresses, cosines) is spent once per warp: with a CTA per token eight warps
// spent it, and instructions bounded it (47 us for the prompts below at 2.3 instructions a cycle and
// SM, 3600 of them a token).  A thread keeps its place in the head and with it its weights (kSame: of q's
// type, N values in a vector), asks for the next item's place before this one's values, and has three
// heads in flight: two CTAs per SM with room for that in registers (32 us; three CTAs, spilling: 56).
// Bulk copies into a ring of shared memory, with a CTA's barrier per token, were slower (50 us).
// Measured: 8 prompts of up to 1024 tokens, 32 query and 8 K/V heads of 128 (145 MB): 32 us (4.5 TB/s);
// 16 trees of 32 nodes, the same heads: 6.4 us.
struct Place {
  int pos, col;
};
__device__ __forceinline__ Place given(const RotaryParams& p, unsigned token) {
  return p.positions ? Place{p.positions[token], p.columns[token]} : Place{0, 0};
}
// As locate, by a warp; s_par: room for its row's parents.
__device__ __forceinline__ bool warp_locate(const RotaryParams& p, int b, int t, Place& at, int* s_par) {
  const int lane = threadIdx.x & 31;
  int code = 0;
  if (!p.positions) {
    const int n = p.n_committed[b], W = *p.width;
    int depth = t;
    bool bad = n < 1 || n > W;
    if (p.parents) {
      __syncwarp();  // the item before is done with it
      for (int i = lane; i < p.T; i += 32) s_par[i] = p.parents[b * p.T + i];
      __syncwarp();
      for (int i = lane; i < p.T; i += 32) (void)tree_ancestors(s_par, i, bad);
      bad = __any_sync(0xffffffffu, bad);
      if (!bad) {
        const unsigned long long m = tree_ancestors(s_par, t, bad);
        if (m == 0) {
          at.col = -1;
          return false;
        }
        depth = __popcll(m) - 1;
      }
    }
    if (bad) code = SPECDEC_ERR_INPUT_RANGE;
    else if (W > p.cap - t) code = SPECDEC_ERR_CAPACITY;  // (a width near the integers' end must not wrap around)
    at = Place{n - 1 + depth, W - 1 + t};
  } else if (at.col < 0) {
    return false;
  }
  if (!code) {
    const long long pos = at.pos < 0 ? -1 : static_cast<long long>(at.pos) + (p.start ? p.start[b] : 0);
    if (at.col >= p.cap) code = SPECDEC_ERR_CAPACITY;
    else if (pos < 0 || pos >= p.table_len || (p.start && p.start[b] < 0)) code = SPECDEC_ERR_INPUT_RANGE;
    at.pos = static_cast<int>(pos);
  }
  if (code) {
    if (lane == 0) set_status(p.status, code);
    at = Place{-1, 0};
    return false;
  }
  return true;
}

template <typename T, int N, bool kInterleaved, int U, bool kSame>
__global__ void __launch_bounds__(kThreads, U == 1 ? 2 : 1)
norm_rotary_kernel(const RotaryParams p, const NormParams w, unsigned items, unsigned parts, int part) {
  constexpr int kFlight = U == 1 ? 3 : 1;  // heads in flight per thread
  using V = Values<T, N>;
  __shared__ int s_par[kThreads / 32][kMaxTree];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int half = p.rot / 2, units = p.hd / (2 * N), turned = half / N, all = p.Hq + 2 * p.H;
  const int lanes = units >= 32 ? 32 : 1 << (32 - __clz(max(units - 1, 0)));
  const int step = 32 / lanes, j0 = lane % lanes, mine = lane / lanes;
  // where the runs of unit j begin
  auto run0 = [&](int j) { return j < turned && !kInterleaved ? j * N : 2 * j * N; };
  auto run1 = [&](int j) { return j < turned && !kInterleaved ? j * N + half : 2 * j * N + N; };
  auto weights = [&](const char* from, int e, float* f) {  // N of any type from value e on
#pragma unroll
    for (int n = 0; n < N; ++n)
      f[n] = w.f32 ? __ldg(reinterpret_cast<const float*>(from) + e + n)
                   : __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(from) + e + n)) << 16);
  };
  typename V::Raw wq[2], wk[2];
  if constexpr (kSame) {
    const int j = min(j0, units - 1);
    const T *a = reinterpret_cast<const T*>(w.q_weight), *z = reinterpret_cast<const T*>(w.k_weight);
    wq[0] = a ? V::load(a + run0(j)) : V::zero();
    wq[1] = a ? V::load(a + run1(j)) : V::zero();
    wk[0] = z ? V::load(z + run0(j)) : V::zero();
    wk[1] = z ? V::load(z + run1(j)) : V::zero();
  }
  const unsigned stride = gridDim.x * (kThreads / 32);
  auto token_of = [&](unsigned item) { return parts == 1 ? item : item / parts; };
  unsigned item = blockIdx.x * (kThreads / 32) + warp;
  Place ahead{0, 0};
  if (item < items) ahead = given(p, token_of(item));
  for (; item < items; item += stride) {
    const unsigned token = token_of(item);
    const int b = token / static_cast<unsigned>(p.T), t = token - static_cast<unsigned>(b) * p.T;
    const int h0 = (item - token * parts) * part, h1 = min(all, h0 + part);
    Place at = ahead;
    const bool write = warp_locate(p, b, t, at, s_par[warp]);
    if (item + stride < items) ahead = given(p, token_of(item + stride));
    T* qo = reinterpret_cast<T*>(p.qo + b * p.or_ + t * p.ot);
    if (!write) {
      if (at.col < 0) {  // padding or an unused node (otherwise an error was recorded)
        const int end = min(h1, p.Hq) * p.hd / N;
        for (int i = h0 * p.hd / N + lane; i < end; i += 32) V::store(qo + i * N, V::zero());
      }
      continue;
    }
    const T *q = reinterpret_cast<const T*>(p.q + b * p.qr + t * p.qt),
            *k = reinterpret_cast<const T*>(p.k + b * p.kr + t * p.kt) - p.Hq * p.hd,
            *v = reinterpret_cast<const T*>(p.v + b * p.vr + t * p.vt) - (p.Hq + p.H) * p.hd;
    char* to = p.cache.base + (p.one_row ? 0 : b) * p.cache.srow + static_cast<long long>(at.col) * p.hd * sizeof(T);
    const float2* cs = p.table + static_cast<long long>(at.pos) * half;
    float2 c[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j0 + u * lanes < turned)
#pragma unroll
        for (int n = 0; n < N; ++n) c[u][n] = __ldg(cs + (j0 + u * lanes) * N + n);
    for (int first = h0; first < h1; first += step * kFlight) {
      typename V::Raw r0[kFlight][U], r1[kFlight][U];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {  // loads first: they wait for memory together
        const int h = first + i * step + mine;
        const T* x = (h < p.Hq ? q : h < p.Hq + p.H ? k : v) + h * p.hd;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * lanes;
          r0[i][u] = r1[i][u] = V::zero();
          if (h < h1 && j < units) {
            r0[i][u] = V::load(x + run0(j));
            r1[i][u] = V::load(x + run1(j));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int h = first + i * step + mine;
        const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.H;
        T* y = is_q ? qo + h * p.hd
                    : reinterpret_cast<T*>(to + (is_v ? p.cache.skv : 0) + (h - p.Hq - (is_v ? p.H : 0)) * p.cache.shead);
        if (first + i * step < p.Hq + p.H) {  // (not all of the warp's heads are v's)
          const char* weight = is_v ? nullptr : is_q ? w.q_weight : w.k_weight;
          uint64_t sums = 0;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float f[2 * N];
            V::unpack(r0[i][u], f);
            V::unpack(r1[i][u], f + N);
#pragma unroll
            for (int n = 0; n < 2 * N; n += 2) {
              const uint64_t x = pack2(f[n], f[n + 1]);
              sums = fma2(x, x, sums);
            }
          }
          const float2 two = unpack2(sums);
          float sum = two.x + two.y;
          for (int d = lanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          const float inv = rsqrtf(fmaf(sum, w.inv_hd, w.eps));
          const uint64_t inv2 = pack2(inv, inv), off2 = pack2(w.offset, w.offset);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int j = j0 + u * lanes;
            float f[2 * N];
            V::unpack(r0[i][u], f);
            V::unpack(r1[i][u], f + N);
            if (weight && j < units) {
              float g[2 * N];
              if constexpr (kSame) {
                V::unpack(is_q ? wq[0] : wk[0], g);
                V::unpack(is_q ? wq[1] : wk[1], g + N);
              } else {
                weights(weight, run0(j), g);
                weights(weight, run1(j), g + N);
              }
#pragma unroll
              for (int n = 0; n < 2 * N; n += 2) {
                const float2 x = unpack2(mul2(mul2(pack2(f[n], f[n + 1]), inv2), add2(pack2(g[n], g[n + 1]), off2)));
                f[n] = x.x;
                f[n + 1] = x.y;
              }
            }
            const bool turns = j < turned && !is_v;
            if (turns) {  // pairs: neighbours of the 2N values, or one of each run
#pragma unroll
              for (int n = 0; n < N; ++n) {
                const int e0 = kInterleaved ? 2 * n : n, e1 = kInterleaved ? 2 * n + 1 : N + n;
                const float x1 = f[e0], x2 = f[e1];
                f[e0] = x1 * c[u][n].x - x2 * c[u][n].y;
                f[e1] = x1 * c[u][n].y + x2 * c[u][n].x;
              }
            }
            if (weight || turns) {  // (what is only copied stays as it is, NaN's bits too)
              r0[i][u] = V::pack(f);
              r1[i][u] = V::pack(f + N);
            }
          }
        }
        if (h < h1)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int j = j0 + u * lanes;
            if (j >= units) continue;
            V::store(y + run0(j), r0[i][u]);
            V::store(y + run1(j), r1[i][u]);
          }
      }
    }
  }
}

// Whether 16-byte vectors reach every run.
template <typename T> bool vectors(const RotaryParams& p) {
  constexpr int N = Vec<T>::N;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                         reinterpret_cast<uintptr_t>(p.v) | reinterpret_cast<uintptr_t>(p.qo) |
                         p.qr | p.qt | p.kr | p.kt | p.vr | p.vt | p.or_ | p.ot;
  return bits % 16 == 0 && p.rot % (2 * N) == 0 && p.hd % (2 * N) == 0;
}

template <typename T>
int launch_rotary(const RotaryParams& p, int B, cudaStream_t s) {
  constexpr int N = Vec<T>::N;
  const bool vec = vectors<T>(p);
  // few tokens: a token's heads over several CTAs
  const int per_pass = kThreads / (p.hd / (2 * (vec ? N : 1))), passes = (p.Hq + 2 * p.H + per_pass - 1) / per_pass;
  const int want = (4 * std::max(1, sm_count()) - 1) / (B * p.T) + 1;
  const dim3 grid(B * p.T, std::max(1, std::min(want, passes)));
  if (vec && p.interleaved) rotary_kernel<T, N, true><<<grid, kThreads, 0, s>>>(p);
  else if (vec) rotary_kernel<T, N, false><<<grid, kThreads, 0, s>>>(p);
  else if (p.interleaved) rotary_kernel<T, 1, true><<<grid, kThreads, 0, s>>>(p);
  else rotary_kernel<T, 1, false><<<grid, kThreads, 0, s>>>(p);
  return map_cuda_error(cudaGetLastError());
}

template <typename T, int N, int U, bool kSame>
int launch_norm_rotary(const RotaryParams& p, const NormParams& w, int B, cudaStream_t s) {
  constexpr int kWarps = kThreads / 32, kPerSm = U == 1 ? 2 : 1;
  // heads a warp takes at once, and a token's heads over as many warps as fill the GPU
  const int units = p.hd / (2 * N), all = p.Hq + 2 * p.H;
  int lanes = 1;
  while (lanes < units && lanes < 32) lanes *= 2;
  const int step = 32 / lanes, tokens = B * p.T, room = std::max(1, sm_count()) * kPerSm * kWarps;
  const int want = std::max(1, std::min((all - 1) / step + 1, room / tokens));
  const int part = ((all - 1) / want / step + 1) * step, parts = (all - 1) / part + 1;
  const long long items = static_cast<long long>(tokens) * parts;
  if (items >= (1LL << 31)) return SPECDEC_ERR_UNSUPPORTED;  // (then parts is 1: as many tokens are refused before)
  const int grid = static_cast<int>(std::min<long long>((items - 1) / kWarps + 1, room / kWarps));
  if (p.interleaved) norm_rotary_kernel<T, N, true, U, kSame><<<grid, kThreads, 0, s>>>(p, w, static_cast<unsigned>(items), parts, part);
  else norm_rotary_kernel<T, N, false, U, kSame><<<grid, kThreads, 0, s>>>(p, w, static_cast<unsigned>(items), parts, part);
  return map_cuda_error(cudaGetLastError());
}
template <typename T>
int launch_norm_rotary(const RotaryParams& p, const NormParams& w, int B, cudaStream_t s) {
  constexpr int N = Vec<T>::N;
  const bool vec = vectors<T>(p);
  const int units = p.hd / (2 * (vec ? N : 1));  // of heads of 512 values: 32 of bf16 vectors, 64 of fp32's
  if constexpr (N == 4)
    if (vec && units > 32) return launch_norm_rotary<T, N, 2, false>(p, w, B, s);
  if (vec && w.same) return launch_norm_rotary<T, N, 1, true>(p, w, B, s);
  if (vec) return launch_norm_rotary<T, N, 1, false>(p, w, B, s);
  return units <= 32 ? launch_norm_rotary<T, 1, 1, false>(p, w, B, s) : launch_norm_rotary<T, 1, 8, false>(p, w, B, s);
}

// Checks the arguments and fills what the kernels take.
int rotary_params(const specdec_rotary_args* a, RotaryParams& p) {
  if (a->B < 0 || a->T < 1 || a->heads_q < 1 || a->layer < 0 || a->table_len < 1)
    return SPECDEC_ERR_INVALID_ARG;
  if (a->B == 0) return SPECDEC_OK;
  const int st = check_view(a->cache, 0);
  if (st) return st;
  const specdec_kv_view& c = a->cache;
  const long long es = elem_size(c.dtype);
  if (a->layer >= c.layers || !(c.rows >= a->B || c.rows == 1)) return SPECDEC_ERR_INVALID_ARG;
  if (a->rot_dim < 2 || a->rot_dim % 2 || a->rot_dim > c.head_dim) return SPECDEC_ERR_INVALID_ARG;
  const bool pass = a->n_committed || a->width || a->parents;
  if (pass ? !a->n_committed || !a->width || a->positions || a->columns
           : !a->positions || !a->columns)
    return SPECDEC_ERR_INVALID_ARG;
  // (in one cache row the batch rows' nodes would go to the same columns)
  if (pass && c.rows == 1 && a->B > 1) return SPECDEC_ERR_INVALID_ARG;
  if (!a->q || !a->k || !a->v || !a->q_out || !a->table || !a->dev_status)
    return SPECDEC_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(a->q) % es || reinterpret_cast<uintptr_t>(a->k) % es ||
      reinterpret_cast<uintptr_t>(a->v) % es || reinterpret_cast<uintptr_t>(a->q_out) % es ||
      reinterpret_cast<uintptr_t>(a->table) % sizeof(float2))
    return SPECDEC_ERR_INVALID_ARG;
  if ((pass && a->T > SPECDEC_MAX_TREE) || static_cast<long long>(a->B) * a->T >= (1LL << 31) ||
      static_cast<long long>(a->heads_q + 2LL * c.heads) * c.head_dim >= (1LL << 30) ||
      c.head_dim > 2 * kThreads)
    return SPECDEC_ERR_UNSUPPORTED;
  p = {};
  p.cache = to_bytes(c);
  p.cache.base += a->layer * p.cache.sl;
  p.q = static_cast<const char*>(a->q);
  p.k = static_cast<const char*>(a->k);
  p.v = static_cast<const char*>(a->v);
  p.qo = static_cast<char*>(a->q_out);
  p.qr = a->q_stride_row * es;
  p.qt = a->q_stride_token * es;
  p.kr = a->k_stride_row * es;
  p.kt = a->k_stride_token * es;
  p.vr = a->v_stride_row * es;
  p.vt = a->v_stride_token * es;
  p.or_ = a->q_out_stride_row * es;
  p.ot = a->q_out_stride_token * es;
  p.table = reinterpret_cast<const float2*>(a->table);
  p.n_committed = a->n_committed;
  p.width = a->width;
  p.parents = a->parents;
  p.positions = a->positions;
  p.columns = a->columns;
  p.status = a->dev_status;
  p.T = a->T;
  p.Hq = a->heads_q;
  p.H = c.heads;
  p.hd = c.head_dim;
  p.rot = a->rot_dim;
  p.interleaved = a->interleaved ? 1 : 0;
  p.table_len = a->table_len;
  p.cap = c.cap_cols;
  p.one_row = c.rows == 1 ? 1 : 0;
  return SPECDEC_OK;
}

}  // namespace
}  // namespace specdec

extern "C" int specdec_rotary_append(const specdec_rotary_args* a, void* stream) {
  using namespace specdec;
  if (!a) return SPECDEC_ERR_INVALID_ARG;
  RotaryParams p = {};
  const int rc = rotary_params(a, p);
  if (rc || a->B == 0) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a->cache.dtype == SPECDEC_BF16 ? launch_rotary<uint16_t>(p, a->B, s) : launch_rotary<float>(p, a->B, s);
}

extern "C" int specdec_norm_rotary_append(const specdec_norm_rotary_args* args, void* stream) {
  using namespace specdec;
  if (!args) return SPECDEC_ERR_INVALID_ARG;
  const specdec_rotary_args* a = &args->rotary;
  RotaryParams p = {};
  const int rc = rotary_params(a, p);
  if (rc || a->B == 0) return rc;
  const int ws = elem_size(args->weight_dtype);
  const uintptr_t bits = reinterpret_cast<uintptr_t>(args->q_weight) | reinterpret_cast<uintptr_t>(args->k_weight);
  if (!ws || bits % ws || reinterpret_cast<uintptr_t>(args->start) % 4 || !std::isfinite(args->eps) ||
      args->eps < 0.f || !std::isfinite(args->weight_offset))
    return SPECDEC_ERR_INVALID_ARG;
  p.start = args->start;
  NormParams w = {};
  w.q_weight = static_cast<const char*>(args->q_weight);
  w.k_weight = static_cast<const char*>(args->k_weight);
  w.eps = args->eps;
  w.offset = args->weight_offset;
  w.inv_hd = 1.f / a->cache.head_dim;
  w.f32 = args->weight_dtype == SPECDEC_F32 ? 1 : 0;
  w.same = bits % 16 == 0 && args->weight_dtype == a->cache.dtype ? 1 : 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a->cache.dtype == SPECDEC_BF16 ? launch_norm_rotary<uint16_t>(p, w, a->B, s)
                                        : launch_norm_rotary<float>(p, w, a->B, s);
}
