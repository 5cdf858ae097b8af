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
// vectors.  One grid row of CTAs serves a token.
#include "tree.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 256;

struct RotaryParams {
  ByteView cache;  // of the layer
  const char *q, *k, *v;
  char* qo;
  long long qr, qt, kr, kt, vr, vt, or_, ot;  // bytes between rows and tokens
  const float2* table;
  const int32_t *n_committed, *width, *parents, *positions, *columns;
  int32_t* status;
  int T, Hq, H, hd, rot, interleaved, table_len, cap, one_row;
};

// Position and column of token t of row b; false if nothing is to be written for it.  All
// threads of the CTA get the same answer.
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
    pos = n - 1 + depth;
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

// N consecutive values as floats, and back, by one 16-byte access (N = Vec<T>::N) or one scalar.
template <typename T, int N>
__device__ __forceinline__ void load_values(const T* x, float* f) {
  if constexpr (N == 1) f[0] = Vec<T>::scalar(x);
  else Vec<T>::unpack(*reinterpret_cast<const uint4*>(x), f);
}
template <typename T, int N>
__device__ __forceinline__ void store_values(T* y, const float* f) {
  if constexpr (N == 1) {
    if constexpr (sizeof(T) == 2) *y = bf16_bits(f[0]);
    else *y = f[0];
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(y) = make_uint4(bf16_pack(f[0], f[1]), bf16_pack(f[2], f[3]),
                                              bf16_pack(f[4], f[5]), bf16_pack(f[6], f[7]));
  } else {
    *reinterpret_cast<float4*>(y) = make_float4(f[0], f[1], f[2], f[3]);
  }
}

// A unit is two runs of N values of a head: N pairs to turn (the runs are rot_dim / 2 apart in
// the half layout, and one behind the other when interleaved), or 2N values to copy.  One thread
// reads both runs before it writes either, so q_out may be q.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p) {
  const int b = blockIdx.x / p.T, t = blockIdx.x % p.T;
  int pos = 0, col = 0;
  const bool write = locate(p, b, t, pos, col);
  if (!write && pos < 0) return;  // an error was recorded
  const long long row = p.one_row ? 0 : b;
  const int half = p.rot / 2;
  const float2* cs = p.table + static_cast<long long>(pos) * half;
  const int per_head = p.hd / (2 * N), turned = half / N;
  const int total = (p.Hq + 2 * p.H) * per_head;
  for (int u = blockIdx.y * kThreads + threadIdx.x; u < total; u += gridDim.y * kThreads) {
    const int h = u / per_head, j = u % per_head;
    const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.H;
    if (!is_q && !write) break;
    const int hk = is_q ? h : is_v ? h - p.Hq - p.H : h - p.Hq;
    const char* src = is_q ? p.q + b * p.qr + t * p.qt
                           : is_v ? p.v + b * p.vr + t * p.vt : p.k + b * p.kr + t * p.kt;
    const T* x = reinterpret_cast<const T*>(src) + hk * p.hd;
    T* y = is_q ? reinterpret_cast<T*>(p.qo + b * p.or_ + t * p.ot) + hk * p.hd
                : reinterpret_cast<T*>(p.cache.base + (is_v ? p.cache.skv : 0) +
                                       row * p.cache.srow + hk * p.cache.shead) +
                      static_cast<long long>(col) * p.hd;
    const bool turn = j < turned && !is_v;
    const int e0 = turn && !p.interleaved ? j * N : 2 * j * N;
    const int e1 = turn && !p.interleaved ? e0 + half : e0 + N;
    float f0[N], f1[N];
    load_values<T, N>(x + e0, f0);
    load_values<T, N>(x + e1, f1);
    if (turn && p.interleaved) {  // pairs are neighbours in the 2N values
      float v[2 * N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        v[k] = f0[k];
        v[N + k] = f1[k];
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float2 c = cs[j * N + k];
        const float a = v[2 * k], m = v[2 * k + 1];
        v[2 * k] = a * c.x - m * c.y;
        v[2 * k + 1] = a * c.y + m * c.x;
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        f0[k] = v[k];
        f1[k] = v[N + k];
      }
    } else if (turn) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float2 c = cs[j * N + k];
        const float a = f0[k], m = f1[k];
        f0[k] = a * c.x - m * c.y;
        f1[k] = a * c.y + m * c.x;
      }
    }
    if (!write) {
#pragma unroll
      for (int k = 0; k < N; ++k) f0[k] = f1[k] = 0.f;
    }
    store_values<T, N>(y + e0, f0);
    store_values<T, N>(y + e1, f1);
  }
}

template <typename T>
int launch_rotary(const RotaryParams& p, int B, cudaStream_t s) {
  constexpr int N = Vec<T>::N;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                         reinterpret_cast<uintptr_t>(p.v) | reinterpret_cast<uintptr_t>(p.qo) |
                         p.qr | p.qt | p.kr | p.kt | p.vr | p.vt | p.or_ | p.ot;
  const bool vec = bits % 16 == 0 && p.rot % (2 * N) == 0 && p.hd % (2 * N) == 0;
  const dim3 grid(B * p.T);
  if (vec) rotary_kernel<T, N><<<grid, kThreads, 0, s>>>(p);
  else rotary_kernel<T, 1><<<grid, kThreads, 0, s>>>(p);
  return map_cuda_error(cudaGetLastError());
}

}  // namespace
}  // namespace specdec

extern "C" int specdec_rotary_append(const specdec_rotary_args* a, void* stream) {
  using namespace specdec;
  if (!a) return SPECDEC_ERR_INVALID_ARG;
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
  if (!a->q || !a->k || !a->v || !a->q_out || !a->table || !a->dev_status)
    return SPECDEC_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(a->q) % es || reinterpret_cast<uintptr_t>(a->k) % es ||
      reinterpret_cast<uintptr_t>(a->v) % es || reinterpret_cast<uintptr_t>(a->q_out) % es ||
      reinterpret_cast<uintptr_t>(a->table) % sizeof(float2))
    return SPECDEC_ERR_INVALID_ARG;
  if ((pass && a->T > SPECDEC_MAX_TREE) || static_cast<long long>(a->B) * a->T >= (1LL << 31) ||
      static_cast<long long>(a->heads_q + 2LL * c.heads) * c.head_dim >= (1LL << 30))
    return SPECDEC_ERR_UNSUPPORTED;
  RotaryParams p = {};
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return es == 2 ? launch_rotary<uint16_t>(p, a->B, s) : launch_rotary<float>(p, a->B, s);
}
