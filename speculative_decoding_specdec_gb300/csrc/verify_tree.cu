// Verification of a tree of drafted tokens against the target's scores: greedy and sampled.
//
// "Inference Engineering: Part 5/8: When Speculative Decoding Backfires": the acceptance rules
// are those of "Exactness Means Different Things For Greedy And Sampled Output", applied from the
// root down: at a node the children are candidates for the same position.
//   Greedy: the choice is the row's argmax; go on at the first child that carries it.
//   Sampled: children in order; child x is accepted with probability min(1, p(x)/q(x)), else
//   p <- normalize(max(0, p - q)) and, for siblings drawn without replacement, q <- q without x,
//   normalised.  Then P(next token = y) = p(y): each test accepts x ~ q with mass min(p, q), and
//   what it leaves, max(0, p - q), is what the next test or the draw starts from.
//
// GB300 mapping.  A walk visits few of the T rows (one more than it accepts), and which ones is
// known only on the way, so one thread-block cluster walks one batch row and reads the visited
// rows alone (greedy: all used rows at once where they are small, see launch_greedy).  Its CTAs split
// the vocabulary; every step ends in one exchange: each warp stores its record into every CTA's
// shared memory, by stores that count their bytes on a barrier there, and every warp reduces all
// records in rank order.  All threads of the cluster then hold the same decision and no result has to
// be sent back.  Two record buffers alternate.  A buffer is written again by exchange n + 2, which a
// warp sends after it has received all of exchange n + 1, and every warp sends its part of that after
// it has read exchange n: no record is overwritten before it was read.
// What bounds it: the chain of dependent steps (row latency, reduction, exchange); the visited rows
// are a few hundred KB per step.  Measured: greedy, 8 trees of 16 nodes, V 32000: 9.5 us; 16 trees of
// 64 nodes, V 151936: 21 us; sampled, 32 trees of 16 nodes, V 151552: 45 us (67000 cycles, of which
// the special-function unit is busy for 16 %, issue 47 %; barriers and loads are waited for most).
#include <algorithm>
#include <climits>
#include <cmath>

#include "tree.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
static_assert(kMaxCluster <= kWarps, "a warp per CTA sums its records");
constexpr int kUnroll = 4;  // 16-byte loads in flight per thread

struct TreeParams {
  const void *target, *draft_scores;
  int T, V, D, C, replacement, vec;  // vec: rows are 16-byte aligned
  long long row_stride;
  float c2;  // log2(e) / temperature
  const int32_t *tokens, *parents;
  const float* uniforms;
  int32_t *accept_len, *out_token, *path, *draft, *status;
};

// A batch row's tree in shared memory, and the walk along it.
struct Walk {
  int par[kMaxTree], tok[kMaxTree];
  int path[SPECDEC_MAX_DRAFT];
};

// First child of `cur` above `last` for which want(i) holds; T if there is none.  Every warp of
// the cluster computes the same answer.
template <typename F>
__device__ __forceinline__ int next_child(const Walk& w, int T, int cur, int last, F want) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i0 = 0; i0 < kMaxTree; i0 += 32) {
    const int i = i0 + lane;
    const bool yes = i < T && i > last && w.par[i] == cur && want(i);
    const unsigned m = __ballot_sync(0xffffffffu, yes);
    if (m) return i0 + __ffs(m) - 1;
  }
  return T;
}

// A node's parent and token on their way from memory (thread = node).
struct NodeLoad {
  int par, tok;
};
__device__ __forceinline__ NodeLoad ask_tree(const TreeParams& p, int b) {
  const int i = threadIdx.x;
  NodeLoad n{i - 1, 0};
  if (i < p.T) {
    if (p.parents) n.par = __ldg(p.parents + b * p.T + i);
    n.tok = __ldg(p.tokens + b * p.T + i);
  }
  return n;
}
// The tree in shared memory, checked.  Returns false (in every CTA of the cluster) where it is bad.
__device__ __forceinline__ bool place_tree(const TreeParams& p, NodeLoad n, Walk& w) {
  const int i = threadIdx.x;
  if (i < p.T) {
    w.par[i] = n.par;
    w.tok[i] = n.tok;
  }
  __syncthreads();
  bool bad = false;
  if (i < p.T) (void)tree_ancestors(w.par, i, bad);
  return !__syncthreads_or(bad);
}

// Rank 0 writes the walk's results.
__device__ void write_walk(const TreeParams& p, int b, const Walk& w, int a, int token) {
  const int i = threadIdx.x;
  if (i < p.D) {
    p.path[b * p.D + i] = i < a ? w.path[i] : -1;
    p.draft[b * p.D + i] = i < a ? w.tok[w.path[i]] : 0;
  }
  if (i == 0) {
    p.accept_len[b] = a;
    p.out_token[b] = token;
  }
}

// One 16-byte vector of a row: elements [v * VN, v * VN + VN), minus infinity behind V.  `vec`: rows
// are 16-byte aligned.  Rows with another stride or start take single elements.
template <typename T>
__device__ __forceinline__ uint4 load_scores(const T* row, int v, int V, bool vec) {
  constexpr int VN = Vec<T>::N;
  if (vec && (v + 1) * VN <= V) return ldg_stream(row + static_cast<long long>(v) * VN);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) {
      const int e = v * VN + k;
      w[k] = e < V ? __float_as_uint(__ldg(reinterpret_cast<const float*>(row) + e)) : 0xFF800000u;
    } else {
      const int e = v * VN + 2 * k;
      const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
      w[k] = (e < V ? __ldg(r + e) : 0xFF80u) | (e + 1 < V ? __ldg(r + e + 1) : 0xFF80u) << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ int slice_start(int vecs, int rank, int C) {
  return static_cast<int>(static_cast<long long>(vecs) * rank / C);
}

// The barriers of the exchanges.  Exchange n uses buffer n & 1; `bytes` arrive from the cluster.
struct Exchange {
  uint64_t bar[2];
};
constexpr uint32_t kExchangeTries = 1u << 22;

__device__ __forceinline__ void exchange_expect(Exchange& x, int n, uint32_t bytes) {
  if (threadIdx.x == 0) mbar_arrive_expect_tx(&x.bar[n & 1], bytes);
}
__device__ __forceinline__ bool exchange_wait(Exchange& x, int n) {
  return mbar_wait_bounded(&x.bar[n & 1], (n >> 1) & 1, kExchangeTries);
}

// The largest key of a warp, in every lane: scores first, then, among those that tie, the complemented
// index (two integer reductions in place of five 64-bit shuffles).
__device__ __forceinline__ unsigned long long warp_max(unsigned long long key) {
  const uint32_t hi = static_cast<uint32_t>(key >> 32);
  const uint32_t top = __reduce_max_sync(0xffffffffu, hi);
  const uint32_t lo = __reduce_max_sync(0xffffffffu, hi == top ? static_cast<uint32_t>(key) : 0u);
  return static_cast<unsigned long long>(top) << 32 | lo;
}

// ------------------------------------------------------------------------------------- greedy

// kAll: every row is read before the walk, a warp per row; else the walk's rows, one by one.
template <typename T, bool kAll>
__global__ void __launch_bounds__(kThreads) tree_greedy_kernel(const TreeParams p) {
  constexpr int VN = Vec<T>::N;
  __shared__ Walk w;
  __shared__ Exchange x;
  __shared__ unsigned long long s_rec[2][kAll ? 1 : kMaxCluster * kWarps];  // a key of every warp of the cluster
  __shared__ unsigned long long s_all[kAll ? kMaxTree : 1][kMaxCluster];
  __shared__ int s_choice[kMaxTree];
  const int rank = static_cast<int>(cluster_rank()), b = blockIdx.x / p.C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    mbar_init(&x.bar[0], 1);
    mbar_init(&x.bar[1], 1);
    fence_mbar_init();
  }
  const NodeLoad node = ask_tree(p, b);
  const T* rows = static_cast<const T*>(p.target) + static_cast<long long>(b) * p.T * p.row_stride;
  const int vecs = (p.V + VN - 1) / VN, v0 = slice_start(vecs, rank, p.C), v1 = slice_start(vecs, rank + 1, p.C);
  // the best of a row's vectors [v0, v1), taken `step` apart from v0 + first by this thread
  auto best = [&](const T* row, int first, int step) {
    float bv = 0.f;
    int bi = -1;
    for (int v = v0 + first; v < v1; v += step * kUnroll) {
      uint4 r[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (v + k * step < v1) r[k] = load_scores(row, v + k * step, p.V, p.vec);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (v + k * step < v1) {
          float f[VN];
          Vec<T>::unpack(r[k], f);
          take_vector<VN>(f, (v + k * step) * VN, bv, bi);
        }
    }
    return warp_max(bi >= 0 && bi < p.V ? make_key(bv, bi) : 0ull);
  };
  unsigned long long key = 0;
  if (!kAll) key = best(rows, tid, kThreads);  // the root's row, while the tree is on its way
  const bool ok = place_tree(p, node, w);
  cluster_sync_all();  // every CTA of the cluster has started: its shared memory may be written
  bool alive = true;
  int a = 0, token = -1;
  if (ok && w.par[0] != kUnusedNode) {
    if (kAll) {
      exchange_expect(x, 0, p.T * p.C * 8);
      for (int i = warp; i < p.T; i += kWarps) {
        const unsigned long long mine = w.par[i] == kUnusedNode ? 0ull : best(rows + i * p.row_stride, lane, 32);
        if (lane < p.C) cluster_send(cluster_map(&s_all[i][rank], lane), mine, cluster_map(&x.bar[0], lane));
      }
      alive = exchange_wait(x, 0);
      if (alive && tid < p.T) {
        key = s_all[tid][0];
        for (int r = 1; r < p.C; ++r) key = max(key, s_all[tid][r]);
        s_choice[tid] = key ? static_cast<int>(~static_cast<uint32_t>(key)) : -1;
      }
      alive = __syncthreads_and(alive) != 0;  // (a wait that gave up did so for all)
    }
    for (int cur = 0, n = 0; alive; ++n) {
      int choice;
      if (kAll) {
        choice = s_choice[cur];
      } else {
        // every warp's key to every CTA, and all of them reduced by every warp
        exchange_expect(x, n, p.C * kWarps * 8);
        if (n > 0) key = best(rows + cur * p.row_stride, tid, kThreads);
        if (lane < p.C)
          cluster_send(cluster_map(&s_rec[n & 1][rank * kWarps + warp], lane), key, cluster_map(&x.bar[n & 1], lane));
        if (!(alive = __all_sync(0xffffffffu, exchange_wait(x, n)))) break;
        key = 0;
        for (int i = lane; i < p.C * kWarps; i += 32) key = max(key, s_rec[n & 1][i]);
        key = warp_max(key);
        choice = key ? static_cast<int>(~static_cast<uint32_t>(key)) : -1;
      }
      if (choice < 0) {  // only NaN
        if (rank == 0 && tid == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
        break;
      }
      const int next = a < p.D ? next_child(w, p.T, cur, cur, [&](int i) { return w.tok[i] == choice; })
                               : p.T;
      if (next == p.T) {
        token = choice;
        break;
      }
      if (tid == 0) w.path[a] = next;
      ++a;
      cur = next;
    }
  }
  alive = __syncthreads_and(alive) != 0;
  if (!ok || !alive) {
    if (rank == 0 && tid == 0) set_status(p.status, ok ? SPECDEC_ERR_TIMEOUT : SPECDEC_ERR_INPUT_RANGE);
  } else if (rank == 0) {
    write_walk(p, b, w, a, token);
  }
  cluster_sync_all();  // no CTA leaves while another might still write to it
}

// ------------------------------------------------------------------------------------ sampled

// 2^x by the PTX instruction ex2.approx.ftz.f32 (relative error below 2^-21).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The smallest normal number.  A residual below it counts as none: its inverse may be infinite, and
// infinity times the zeros of the residual NaN.
constexpr float kLeastMass = 1.17549435e-38f;

// p and q at the current node after `k` rejections: softmaxes of the two rows, then one step
// max(0, p - q) / R and q without the rejected token, over Q, per rejection.
struct Stage {
  float mt, it, mq, iq;        // maximum (times c2) and inverse sum of the target's, draft's row
  int k;
  int tok[kMaxTree];           // rejected tokens
  float ir[kMaxTree];          // 1 / R, 0 where the residual was empty (p then stays)
  float iqs[kMaxTree];         // 1 / Q
};

__device__ __forceinline__ void probabilities(const Stage& s, float c2, int replacement, int e,
                                              float zt, float zq, float& pv, float& qv) {
  pv = ex2(fmaf(zt, c2, -s.mt)) * s.it;
  qv = ex2(fmaf(zq, c2, -s.mq)) * s.iq;
  for (int i = 0; i < s.k; ++i) {
    const float ir = s.ir[i];
    if (ir > 0.f) pv = fmaxf(pv - qv, 0.f) * ir;
    if (!replacement) qv = e == s.tok[i] ? 0.f : qv * s.iqs[i];
  }
}

// The same of a vector's elements e0 .. e0 + N - 1 (a stage's numbers are read once for all).
template <int N>
__device__ __forceinline__ void probabilities(const Stage& s, float c2, int replacement, int e0,
                                              const float* zt, const float* zq, float* pv, float* qv) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    pv[k] = ex2(fmaf(zt[k], c2, -s.mt)) * s.it;
    qv[k] = ex2(fmaf(zq[k], c2, -s.mq)) * s.iq;
  }
  for (int i = 0; i < s.k; ++i) {
    const float ir = s.ir[i], iqs = s.iqs[i];
    const int at = s.tok[i] - e0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (ir > 0.f) pv[k] = fmaxf(pv[k] - qv[k], 0.f) * ir;
      if (!replacement) qv[k] = at == k ? 0.f : qv[k] * iqs;
    }
  }
}

// (m, l): maximum of x * c2 and the sum of 2^(x * c2 - m).
struct MaxSum {
  float m, l;
};
__device__ __forceinline__ MaxSum merged(MaxSum a, MaxSum b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return MaxSum{m, a.l + b.l};  // nothing yet (or NaN, which has to stay)
  return MaxSum{m, a.l * ex2(a.m - m) + b.l * ex2(b.m - m)};
}
// A warp's: the maximum by one integer reduction of its order-preserving bits, then the sums to it.
__device__ __forceinline__ MaxSum warp_merged(MaxSum s) {
  const uint32_t top = __reduce_max_sync(0xffffffffu, order_bits(s.m));
  const float m = __uint_as_float(top & 0x80000000u ? top ^ 0x80000000u : ~top);
  s.l *= s.m == -INFINITY ? 1.f : ex2(s.m - m);  // (nothing yet, or NaN, which has to stay)
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) s.l += __shfl_xor_sync(0xffffffffu, s.l, k);
  return MaxSum{m, s.l};
}
template <int N> __device__ __forceinline__ float tree_sum(float* t) {
#pragma unroll
  for (int h = N / 2; h > 0; h >>= 1)
#pragma unroll
    for (int k = 0; k < h; ++k) t[k] += t[k + h];
  return t[0];
}
template <int N> __device__ __forceinline__ void fold(MaxSum& s, const float* x, float c2) {
  float mx = x[0];
#pragma unroll
  for (int k = 1; k < N; ++k) mx = fmaxf(mx, x[k]);
  mx *= c2;
  if (mx > s.m) {
    s.l *= ex2(s.m - mx);
    s.m = mx;
  }
  // all -infinity so far: every term is zero (a NaN still shows)
  const float off = s.m == -INFINITY ? 0.f : s.m;
  float t[N];
#pragma unroll
  for (int k = 0; k < N; ++k) t[k] = ex2(fmaf(x[k], c2, -off));
  s.l += tree_sum<N>(t);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  return v;
}
__device__ __forceinline__ float2 warp_sum(float2 v) {
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, k);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, k);
  }
  return v;
}

constexpr int kRuns = 6;                      // runs of kThreads vectors that are held of a row
constexpr int kHold = kRuns * kThreads;       // 48 KB of each row: two CTAs per SM

// kKeep: the slices of both rows stay in shared memory while a node is worked on (loaded once, all
// at once; every test and the draw go over them); else each pass loads them again, from L2.
// (In registers they took a code so long that fetching it was most of a small batch's time.)
template <typename T, bool kKeep>
__global__ void __launch_bounds__(kThreads, 2) tree_sample_kernel(const TreeParams p) {
  constexpr int VN = Vec<T>::N;
  __shared__ Walk w;
  __shared__ Stage st;
  __shared__ Exchange x;
  __shared__ float s_u[kMaxTree], s_zt[kMaxTree], s_zq[kMaxTree];
  __shared__ float4 s_rec[2][kMaxCluster * kWarps];  // a record of every warp of the cluster
  __shared__ float s_mass[kMaxCluster];  // each CTA's share of p's mass, not normalised
  __shared__ float s_entry[kRuns * kWarps];
  extern __shared__ uint4 hold[];  // kKeep: [2][kHold]
  __shared__ int s_token;
  const int rank = static_cast<int>(cluster_rank()), b = blockIdx.x / p.C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* target = static_cast<const T*>(p.target) + static_cast<long long>(b) * p.T * p.row_stride;
  const T* drafts = static_cast<const T*>(p.draft_scores) + static_cast<long long>(b) * p.T * p.row_stride;
  if (tid == 0) {
    mbar_init(&x.bar[0], 1);
    mbar_init(&x.bar[1], 1);
    fence_mbar_init();
  }
  const NodeLoad node = ask_tree(p, b);
  const int vecs = (p.V + VN - 1) / VN, v0 = slice_start(vecs, rank, p.C), v1 = slice_start(vecs, rank + 1, p.C);
  const T *zt = target, *zq = drafts;
  bool inner = p.T > 1;
  auto load = [&] {  // a thread copies what it will read
    for (int v = v0 + tid; v < v1; v += kThreads) {
      const int i = v - v0;
      if (p.vec && (v + 1) * VN <= p.V) {
        cp_async16(hold + i, zt + static_cast<long long>(v) * VN, true);
        if (inner) cp_async16(hold + kHold + i, zq + static_cast<long long>(v) * VN, true);
      } else {
        hold[i] = load_scores(zt, v, p.V, p.vec);
        if (inner) hold[kHold + i] = load_scores(zq, v, p.V, p.vec);
      }
    }
  };
  if (kKeep) load();  // the root's rows, while the tree is on its way
  bool ok = place_tree(p, node, w);
  // every child's scores at its parent, fetched once (the tests need no exchange of them)
  bool bad_u = false;
  if (ok && tid < p.T && w.par[tid] != kUnusedNode) {
    s_u[tid] = p.uniforms[b * p.T + tid];
    bad_u = !(s_u[tid] >= 0.f && s_u[tid] < 1.f);
    if (tid > 0 && w.tok[tid] >= 0 && w.tok[tid] < p.V) {
      const long long at = w.par[tid] * p.row_stride + w.tok[tid];
      s_zt[tid] = Vec<T>::scalar(target + at);
      s_zq[tid] = Vec<T>::scalar(drafts + at);
    }
  }
  ok &= !__syncthreads_or(bad_u);
  cluster_sync_all();  // every CTA of the cluster has started: its shared memory may be written
  const bool walking = ok && w.par[0] != kUnusedNode;
  bool draw = walking, alive = true;
  int cur = 0, a = 0, n = 0, token = -1;
  auto get = [&](int v, float* t, float* q) {  // a vector's scores in both rows
    Vec<T>::unpack(kKeep ? hold[v - v0] : load_scores(zt, v, p.V, p.vec), t);
    if (inner) Vec<T>::unpack(kKeep ? hold[kHold + v - v0] : load_scores(zq, v, p.V, p.vec), q);
  };
  // f(v, target's values, draft's) over this thread's vectors
  auto over = [&](auto f) {
#pragma unroll 2
    for (int v = v0 + tid; v < v1; v += kThreads) {
      float t[VN], q[VN];
      get(v, t, q);
      f(v, t, q);
    }
  };
  // This warp's record to every CTA, and all warps' of the cluster.
  auto exchange = [&](float4 r) {
    if (lane < p.C)
      cluster_send4(cluster_map(&s_rec[n & 1][rank * kWarps + warp], lane), r, cluster_map(&x.bar[n & 1], lane));
    alive = __all_sync(0xffffffffu, exchange_wait(x, n));
    return s_rec[n++ & 1];
  };
  const int records = p.C * kWarps;
  // Each CTA's share of p's mass, from the records of the exchange that gave p (before the next one
  // is sent: its buffer may then be written to).  Warp r sums rank r's.
  auto sum_masses = [&](const float4* rec, float top) {  // top: what softmax sums are relative to
    if (warp < p.C) {
      float m = 0.f;
      if (lane < kWarps) {
        const float4 y = rec[warp * kWarps + lane];
        // (near 2^-126, where ex2 gives zero, the roundings of y.x and of a score decide whether its
        // probability is zero: a CTA counts only where some of its probabilities surely are not)
        m = top == -INFINITY ? y.x : y.x - top < -125.f ? 0.f : y.y * ex2(y.x - top);
      }
      m = warp_sum(m);
      if (lane == 0) s_mass[warp] = m;
    }
  };
  while (walking) {
    zt = target + cur * p.row_stride;
    zq = drafts + cur * p.row_stride;
    int child = a < p.D ? next_child(w, p.T, cur, cur, [](int) { return true; }) : p.T;
    inner = child < p.T;
    exchange_expect(x, n, records * 16);
    if (kKeep) {
      if (n > 0) load();
      cp_async_wait_all();
    }
    MaxSum t{-INFINITY, 0.f}, q{-INFINITY, 0.f};
    over([&](int, const float* ft, const float* fq) {
      fold<VN>(t, ft, p.c2);
      if (inner) fold<VN>(q, fq, p.c2);
    });
    t = warp_merged(t);
    if (inner) q = warp_merged(q);
    const float4* rec = exchange(make_float4(t.m, t.l, q.m, q.l));
    MaxSum tt{-INFINITY, 0.f}, qq{-INFINITY, 0.f};
    for (int i = lane; i < records; i += 32) {
      const float4 y = rec[i];
      tt = merged(tt, MaxSum{y.x, y.y});
      if (inner) qq = merged(qq, MaxSum{y.z, y.w});
    }
    tt = warp_merged(tt);
    if (inner) qq = warp_merged(qq);
    const bool fine = tt.l > 0.f && tt.l < INFINITY && tt.m < INFINITY &&
                      (!inner || (qq.l > 0.f && qq.l < INFINITY && qq.m < INFINITY));
    if (tid == 0) {
      st.mt = tt.m;
      st.it = 1.f / tt.l;
      st.mq = inner ? qq.m : 0.f;
      st.iq = inner ? 1.f / qq.l : 0.f;
      st.k = 0;
    }
    sum_masses(rec, tt.m);
    // One warp's wait may give up where another's does not: all leave together, or barriers would wait
    // for those that have left.
    if (!(alive = __syncthreads_and(alive) != 0)) break;
    if (!fine) {
      if (rank == 0 && tid == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
      draw = false;
      break;
    }
    bool accepted = false;
    while (child < p.T) {
      const int c = w.tok[child];
      if (c < 0 || c >= p.V) {
        if (rank == 0 && tid == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
      } else {
        float pc, qc;
        probabilities(st, p.c2, p.replacement, c, s_zt[child], s_zq[child], pc, qc);
        if (s_u[child] * qc < pc) {
          accepted = true;
          break;
        }
        // rejected: the residual's mass and what is left of q
        exchange_expect(x, n, records * 16);
        float2 sum = make_float2(0.f, 0.f);
        over([&](int v, const float* ft, const float* fq) {
          float pe[VN], qe[VN];
          probabilities<VN>(st, p.c2, p.replacement, v * VN, ft, fq, pe, qe);
#pragma unroll
          for (int k = 0; k < VN; ++k) {
            pe[k] = fmaxf(pe[k] - qe[k], 0.f);
            if (v * VN + k == c) qe[k] = 0.f;
          }
          sum.x += tree_sum<VN>(pe);
          sum.y += tree_sum<VN>(qe);
        });
        sum = warp_sum(sum);
        rec = exchange(make_float4(sum.x, sum.y, 0.f, 0.f));
        sum = make_float2(0.f, 0.f);
        for (int i = lane; i < records; i += 32) {
          sum.x += rec[i].x;
          sum.y += rec[i].y;
        }
        sum = warp_sum(sum);
        const float R = sum.x, Q = sum.y;
        const bool left = R >= kLeastMass;
        if (left) sum_masses(rec, -INFINITY);
        if (tid == 0) {
          st.tok[st.k] = c;
          st.ir[st.k] = left ? 1.f / R : 0.f;
          st.iqs[st.k] = Q > 0.f ? 1.f / Q : 0.f;
          ++st.k;
        }
        if (!(alive = __syncthreads_and(alive) != 0)) break;
      }
      child = next_child(w, p.T, cur, child, [](int) { return true; });
    }
    if (!alive || !accepted) break;
    if (tid == 0) w.path[a] = child;
    ++a;
    cur = child;
    __syncthreads();  // the stage is rewritten for the next node
  }
  // The draw: the CTA whose slice holds u * total finds the token (rank order, so ascending).
  alive = __syncthreads_and(alive) != 0;
  if (!ok || !alive) {
    if (rank == 0 && tid == 0) set_status(p.status, ok ? SPECDEC_ERR_TIMEOUT : SPECDEC_ERR_INPUT_RANGE);
  } else if (draw) {
    // Every warp finds the same owner, a lane per CTA; the last one with any mass takes what rounding
    // leaves.
    const float share = lane < p.C ? s_mass[lane] : 0.f;
    float upto = share;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const float o = __shfl_up_sync(0xffffffffu, upto, k);
      if (lane >= k) upto += o;
    }
    const float total = __shfl_sync(0xffffffffu, upto, 31);
    const unsigned past = __ballot_sync(0xffffffffu, share > 0.f && upto > s_u[0] * total),
                   some_mass = __ballot_sync(0xffffffffu, share > 0.f);
    const int owner = past ? __ffs(past) - 1 : 31 - __clz(some_mass);
    const float before = __shfl_sync(0xffffffffu, upto - share, owner);
    if (rank == owner) {
      const float goal = s_u[0];  // probabilities() are masses over the total
      // Masses of 32 consecutive vectors (a warp's in one run), kRuns runs at a time; the entry
      // where the running sum passes the goal, then the vector in it, then the element.
      float run = before / total;
      int pick = -1, last_v = -1;  // first vector of the chosen entry, of the last with any mass
      float start = 0.f, last_start = 0.f;
      for (int first = v0; first < v1 && pick < 0; first += kHold) {
        const int runs = min(kRuns, (v1 - first + kThreads - 1) / kThreads);
#pragma unroll 2
        for (int k = 0; k < runs; ++k) {
          const int v = first + k * kThreads + tid;
          float m = 0.f;
          if (v < v1) {
            float ft[VN], fq[VN], pe[VN], qe[VN];
            get(v, ft, fq);
            probabilities<VN>(st, p.c2, p.replacement, v * VN, ft, fq, pe, qe);
            m = tree_sum<VN>(pe);
          }
          m = warp_sum(m);
          if (lane == 0) s_entry[k * kWarps + warp] = m;
        }
        __syncthreads();
        constexpr int kEach = kRuns * kWarps / 32;  // entries per lane; every warp finds the same
        float e[kEach], sum = 0.f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          e[i] = lane * kEach + i < runs * kWarps ? s_entry[lane * kEach + i] : 0.f;
          sum += e[i];
        }
        float inc = sum;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
          const float o = __shfl_up_sync(0xffffffffu, inc, k);
          if (lane >= k) inc += o;
        }
        float at = run + inc - sum;  // before this lane's entries
        int mine = -1, some = -1;
        float mine_at = 0.f, some_at = 0.f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          if (e[i] > 0.f) {
            some = i;
            some_at = at;
            if (mine < 0 && at + e[i] > goal) {
              mine = i;
              mine_at = at;
            }
          }
          at += e[i];
        }
        auto vector_of = [&](int l, int i) {
          const int entry = l * kEach + i;
          return first + entry / kWarps * kThreads + entry % kWarps * 32;
        };
        const unsigned over = __ballot_sync(0xffffffffu, mine >= 0), any = __ballot_sync(0xffffffffu, some >= 0);
        if (over) {
          const int l = __ffs(over) - 1;
          pick = vector_of(l, __shfl_sync(0xffffffffu, mine, l));
          start = __shfl_sync(0xffffffffu, mine_at, l);
        } else if (any) {
          const int l = 31 - __clz(any);
          last_v = vector_of(l, __shfl_sync(0xffffffffu, some, l));
          last_start = __shfl_sync(0xffffffffu, some_at, l);
        }
        run += __shfl_sync(0xffffffffu, inc, 31);
        __syncthreads();
      }
      if (pick < 0) {
        pick = last_v;
        start = last_start;
      }
      if (warp == 0) {
        const int v = pick + lane;
        float pe[VN], m = 0.f;
#pragma unroll
        for (int k = 0; k < VN; ++k) pe[k] = 0.f;
        if (v < v1) {
          float ft[VN], fq[VN], qe[VN], sum[VN];
          get(v, ft, fq);
          probabilities<VN>(st, p.c2, p.replacement, v * VN, ft, fq, pe, qe);
#pragma unroll
          for (int k = 0; k < VN; ++k) sum[k] = pe[k];
          m = tree_sum<VN>(sum);
        }
        float inc = m;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
          const float o = __shfl_up_sync(0xffffffffu, inc, k);
          if (lane >= k) inc += o;
        }
        const unsigned over = __ballot_sync(0xffffffffu, m > 0.f && start + inc > goal),
                       any = __ballot_sync(0xffffffffu, m > 0.f);
        if (lane == (over ? __ffs(over) - 1 : 31 - __clz(any))) {
          float at = start + inc - m;
          int found = -1, some = 0;
#pragma unroll
          for (int k = 0; k < VN; ++k)
            if (pe[k] > 0.f) {
              at += pe[k];
              some = k;
              if (found < 0 && at > goal) found = k;
            }
          s_token = v * VN + (found >= 0 ? found : some);
        }
      }
      __syncthreads();
      token = s_token;
      write_walk(p, b, w, a, token);
    }
  } else if (rank == 0) {
    __syncthreads();
    write_walk(p, b, w, a, -1);
  }
  cluster_sync_all();  // no CTA leaves while another might still write to it
}

// Clusters that read their rows' slices with a few vectors per thread, all rows' clusters at once if
// they fit.  Returns the CTAs per cluster.
template <typename K>
int tree_cluster(K kernel, int B, int V, int es, size_t smem, int* cache) {
  const long long vecs = static_cast<long long>(V) * es / 16;
  const int most = static_cast<int>(std::min<long long>(kMaxCluster, vecs / kThreads + 1));
  return cluster_for_one_wave(reinterpret_cast<const void*>(kernel), B, 1, most, kThreads, smem, cache);
}

template <typename K>
int launch_tree(K kernel, const TreeParams& p, int B, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(B * p.C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.C > 8) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return map_cuda_error(e);
  }
  return map_cuda_error(cudaLaunchKernelEx(&cfg, kernel, p));
}

template <typename T>
int launch_greedy(TreeParams& p, int B, cudaStream_t s) {
  static int caches[2][64 * 17];
  // All rows at once where a CTA's share of them takes it less time than the steps of a walk do:
  // about 2 us a step against 25 KB a us and CTA, and 30 MB in all.  bf16, 8 rows, about two accepted
  // nodes, all at once against one by one: V 4000, 16 nodes 8.1 | 10.4 us, 32 nodes (256 KB a CTA)
  // 11.1 | 8.3; V 32000, 16 nodes 8.4 | 11.2, 32 nodes 11.6 | 9.2; V 151936, 4 nodes 10.4 | 9.1 (the
  // rule's loss), 8 nodes 12.7 | 11.8; 32 rows, V 32000, 16 nodes (31 MB) 11.6 | 13.6.  A walk that
  // accepts nothing is ahead one by one throughout (V 32000, 16 nodes, one row: 7.6 | 5.5).
  p.C = tree_cluster(tree_greedy_kernel<T, true>, B, p.V, sizeof(T), 0, caches[0]);
  const long long bytes = static_cast<long long>(p.T) * p.V * sizeof(T);
  if (bytes / p.C <= (128 << 10) && bytes * B <= (30 << 20))
    return launch_tree(tree_greedy_kernel<T, true>, p, B, 0, s);
  p.C = tree_cluster(tree_greedy_kernel<T, false>, B, p.V, sizeof(T), 0, caches[1]);
  return launch_tree(tree_greedy_kernel<T, false>, p, B, 0, s);
}

template <typename T>
int launch_sample(TreeParams& p, int B, cudaStream_t s) {
  static int caches[2][64 * 17];
  constexpr size_t kSmem = 2 * kHold * 16;
  const cudaError_t e = cudaFuncSetAttribute(tree_sample_kernel<T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kSmem));
  if (e != cudaSuccess) return map_cuda_error(e);
  // the slices held, if need be by more CTAs per row than one wave has room for
  const int vecs = (p.V + Vec<T>::N - 1) / Vec<T>::N, least = (vecs + kHold - 1) / kHold;
  if (least <= kMaxCluster) {
    p.C = std::max(least, tree_cluster(tree_sample_kernel<T, true>, B, p.V, sizeof(T), kSmem, caches[0]));
    return launch_tree(tree_sample_kernel<T, true>, p, B, kSmem, s);
  }
  p.C = tree_cluster(tree_sample_kernel<T, false>, B, p.V, sizeof(T), 0, caches[1]);
  return launch_tree(tree_sample_kernel<T, false>, p, B, 0, s);
}

int check_tree(const void* logits, int dtype, int B, int T, int V, long long row_stride,
               const int32_t* tokens, int D, const int32_t* accept_len, const int32_t* out_token,
               const int32_t* path, const int32_t* draft, const int32_t* status) {
  const int es = elem_size(dtype);
  if (es == 0 || B < 0 || T < 1 || D < 1 || V < 1 || row_stride < V)
    return SPECDEC_ERR_INVALID_ARG;
  if (T > SPECDEC_MAX_TREE || D > SPECDEC_MAX_DRAFT) return SPECDEC_ERR_UNSUPPORTED;
  if (B == 0) return SPECDEC_OK;
  if (!logits || !tokens || !accept_len || !out_token || !path || !draft || !status)
    return SPECDEC_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % es) return SPECDEC_ERR_INVALID_ARG;
  if (B > (1 << 20) || row_stride > (1LL << 40) / es / T / B) return SPECDEC_ERR_UNSUPPORTED;
  return SPECDEC_OK;
}

}  // namespace
}  // namespace specdec

extern "C" int specdec_verify_tree_greedy(const void* logits, int dtype, int B, int T, int V,
                                          long long row_stride, const int32_t* tokens,
                                          const int32_t* parents, int D, int32_t* accept_len,
                                          int32_t* out_token, int32_t* path, int32_t* draft,
                                          int32_t* dev_status, void* stream) {
  using namespace specdec;
  const int rc = check_tree(logits, dtype, B, T, V, row_stride, tokens, D, accept_len, out_token,
                            path, draft, dev_status);
  if (rc != SPECDEC_OK || B == 0) return rc;
  TreeParams p = {};
  p.target = logits;
  p.T = T;
  p.V = V;
  p.D = D;
  p.row_stride = row_stride;
  p.tokens = tokens;
  p.parents = parents;
  p.accept_len = accept_len;
  p.out_token = out_token;
  p.path = path;
  p.draft = draft;
  p.status = dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long es = elem_size(dtype);
  p.vec = reinterpret_cast<uintptr_t>(logits) % 16 == 0 && row_stride * es % 16 == 0;
  return dtype == SPECDEC_BF16 ? launch_greedy<uint16_t>(p, B, s) : launch_greedy<float>(p, B, s);
}

extern "C" int specdec_verify_tree_sample(const void* target_logits, const void* draft_logits,
                                          int dtype, int B, int T, int V, long long row_stride,
                                          float temperature, const int32_t* tokens,
                                          const int32_t* parents, const float* uniforms,
                                          int replacement, int D, int32_t* accept_len,
                                          int32_t* out_token, int32_t* path, int32_t* draft,
                                          int32_t* dev_status, void* stream) {
  using namespace specdec;
  const int rc = check_tree(target_logits, dtype, B, T, V, row_stride, tokens, D, accept_len,
                            out_token, path, draft, dev_status);
  if (rc != SPECDEC_OK) return rc;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return SPECDEC_ERR_INVALID_ARG;
  if (B == 0) return SPECDEC_OK;
  if (!draft_logits || !uniforms || reinterpret_cast<uintptr_t>(draft_logits) % elem_size(dtype))
    return SPECDEC_ERR_INVALID_ARG;
  TreeParams p = {};
  p.target = target_logits;
  p.draft_scores = draft_logits;
  p.T = T;
  p.V = V;
  p.D = D;
  p.replacement = replacement ? 1 : 0;
  p.row_stride = row_stride;
  p.c2 = 1.4426950408889634f / temperature;
  p.tokens = tokens;
  p.parents = parents;
  p.uniforms = uniforms;
  p.accept_len = accept_len;
  p.out_token = out_token;
  p.path = path;
  p.draft = draft;
  p.status = dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long es = elem_size(dtype);
  p.vec = reinterpret_cast<uintptr_t>(target_logits) % 16 == 0 &&
          reinterpret_cast<uintptr_t>(draft_logits) % 16 == 0 && row_stride * es % 16 == 0;
  return dtype == SPECDEC_BF16 ? launch_sample<uint16_t>(p, B, s) : launch_sample<float>(p, B, s);
}
