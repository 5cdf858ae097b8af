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
// rows alone.  Its CTAs split the vocabulary; every step ends in one exchange (each CTA writes its
// record into every CTA's shared memory, a cluster barrier, everyone reduces the records in rank
// order), after which all threads of the cluster hold the same decision and no result has to be
// sent back.  Two record buffers alternate: the barrier between two exchanges separates a
// record's readers from its next writer.
// What bounds it: the chain of dependent steps (row latency, block reduction, cluster barrier);
// the visited rows are a few hundred KB per step.
#include <algorithm>
#include <climits>
#include <cmath>

#include "tree.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kUnroll = 4;  // 16-byte loads in flight per thread and row

struct TreeParams {
  const void *target, *draft_scores;
  int T, V, D, C, replacement;
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

// Load and check the tree.  Returns false (in every CTA of the cluster) where it is bad.
__device__ bool load_tree(const TreeParams& p, int b, Walk& w) {
  const int i = threadIdx.x;
  if (i < p.T) {
    w.par[i] = p.parents ? p.parents[b * p.T + i] : i - 1;
    w.tok[i] = p.tokens[b * p.T + i];
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

// Elements [lo, hi) of a row: fv(first index, values, VN) for whole 16-byte vectors and
// fs(index, value) for the few elements around them.  Threads take consecutive vectors.
template <typename T, typename FV, typename FS>
__device__ __forceinline__ void scan_slice(const T* row, int lo, int hi, FV fv, FS fs) {
  constexpr int VN = Vec<T>::N;
  const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(row + lo) % 16 / sizeof(T));
  const int head = min(hi - lo, mis ? VN - mis : 0);
  const int nv = (hi - lo - head) / VN;
  const int tid = threadIdx.x;
  if (tid < head) fs(lo + tid, Vec<T>::scalar(row + lo + tid));
  const T* body = row + lo + head;
  for (int v0 = 0; v0 < nv; v0 += kThreads * kUnroll) {
    uint4 r[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int v = v0 + k * kThreads + tid;
      if (v < nv) r[k] = ldg_stream(body + static_cast<long long>(v) * VN);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int v = v0 + k * kThreads + tid;
      if (v < nv) {
        float x[VN];
        Vec<T>::unpack(r[k], x);
        fv(lo + head + v * VN, x);
      }
    }
  }
  const int tail = lo + head + nv * VN + tid;
  if (tail < hi) fs(tail, Vec<T>::scalar(row + tail));
}

__device__ __forceinline__ int slice_start(int V, int rank, int C) {
  return static_cast<int>(static_cast<long long>(V) * rank / C);
}

// ------------------------------------------------------------------------------------- greedy

template <typename T>
__global__ void __launch_bounds__(kThreads) tree_greedy_kernel(const TreeParams p) {
  constexpr int VN = Vec<T>::N;
  __shared__ Walk w;
  __shared__ unsigned long long s_warp[kWarps];
  __shared__ unsigned long long s_rec[2][kMaxCluster];
  const int rank = static_cast<int>(cluster_rank()), b = blockIdx.x / p.C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool ok = load_tree(p, b, w);
  cluster_sync_all();  // every CTA of the cluster has started: its shared memory may be written
  if (!ok) {
    if (rank == 0 && tid == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
    return;
  }
  const int lo = slice_start(p.V, rank, p.C), hi = slice_start(p.V, rank + 1, p.C);
  int cur = 0, a = 0, token = -1, buf = 0;
  while (w.par[0] != kUnusedNode) {
    const T* row = static_cast<const T*>(p.target) +
                   (static_cast<long long>(b) * p.T + cur) * p.row_stride;
    float bv = 0.f;
    int bi = -1;
    unsigned long long key = 0;
    scan_slice(row, lo, hi,
               [&](int e, const float* x) { take_vector<VN>(x, e, bv, bi); },
               [&](int e, float x) { if (x == x) key = max(key, make_key(x, e)); });
    if (bi >= 0) key = max(key, make_key(bv, bi));
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, k));
    if (lane == 0) s_warp[warp] = key;
    __syncthreads();
    if (warp == 0) {
      key = lane < kWarps ? s_warp[lane] : 0ull;
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, k));
      if (lane < p.C) cluster_st_u64(cluster_map(&s_rec[buf][rank], lane), key);
    }
    cluster_sync_all();
    key = s_rec[buf][0];
    for (int r = 1; r < p.C; ++r) key = max(key, s_rec[buf][r]);
    buf ^= 1;
    if (key == 0) {  // only NaN
      if (rank == 0 && tid == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
      break;
    }
    const int choice = static_cast<int>(~static_cast<uint32_t>(key));
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
  __syncthreads();
  if (rank == 0) write_walk(p, b, w, a, token);
}

// ------------------------------------------------------------------------------------ sampled

// 2^x by the PTX instruction ex2.approx.ftz.f32 (relative error below 2^-21).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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

struct Record {
  float a, b, c, d;
};

// Sum of (x, y) over the CTA, in every thread of warp 0.
__device__ __forceinline__ float2 block_sum(float2 v, float2* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, k);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, k);
  }
  if (lane == 0) s_warp[warp] = v;
  __syncthreads();
  v = make_float2(0.f, 0.f);
  if (warp == 0) {
    if (lane < kWarps) v = s_warp[lane];
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, k);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, k);
    }
  }
  return v;
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
#pragma unroll
  for (int h = N / 2; h > 0; h >>= 1)
#pragma unroll
    for (int k = 0; k < h; ++k) t[k] += t[k + h];
  s.l += t[0];
}
template <typename T>
__device__ __forceinline__ MaxSum slice_max_sum(const T* row, int lo, int hi, float c2,
                                                MaxSum* s_warp) {
  constexpr int VN = Vec<T>::N;
  MaxSum s{-INFINITY, 0.f};
  scan_slice(row, lo, hi, [&](int, const float* x) { fold<VN>(s, x, c2); },
             [&](int, float x) { fold<1>(s, &x, c2); });
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 16; k > 0; k >>= 1)
    s = merged(s, MaxSum{__shfl_xor_sync(0xffffffffu, s.m, k),
                         __shfl_xor_sync(0xffffffffu, s.l, k)});
  if (lane == 0) s_warp[warp] = s;
  __syncthreads();
  s = MaxSum{-INFINITY, 0.f};
  if (warp == 0) {
    if (lane < kWarps) s = s_warp[lane];
#pragma unroll
    for (int k = 16; k > 0; k >>= 1)
      s = merged(s, MaxSum{__shfl_xor_sync(0xffffffffu, s.m, k),
                           __shfl_xor_sync(0xffffffffu, s.l, k)});
  }
  return s;
}

// Warp 0 writes this CTA's record into every CTA of the cluster.
__device__ __forceinline__ void send(Record* slot, int C, Record r) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32 && lane < C) {
    const uint32_t a = cluster_map(slot, lane);
    cluster_st_f32(a, r.a);
    cluster_st_f32(a + 4, r.b);
    cluster_st_f32(a + 8, r.c);
    cluster_st_f32(a + 12, r.d);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) tree_sample_kernel(const TreeParams p) {
  constexpr int VN = Vec<T>::N;
  __shared__ Walk w;
  __shared__ Stage st;
  __shared__ float s_u[kMaxTree], s_zt[kMaxTree], s_zq[kMaxTree];
  __shared__ MaxSum s_ms[2][kWarps];
  __shared__ float2 s_sum[kWarps];
  __shared__ Record s_rec[2][kMaxCluster];
  __shared__ float s_mass[kMaxCluster];  // each CTA's share of p's mass, not normalised
  __shared__ int s_token;
  const int rank = static_cast<int>(cluster_rank()), b = blockIdx.x / p.C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* target = static_cast<const T*>(p.target) + static_cast<long long>(b) * p.T * p.row_stride;
  const T* drafts = static_cast<const T*>(p.draft_scores) + static_cast<long long>(b) * p.T * p.row_stride;
  bool ok = load_tree(p, b, w);
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
  if (!ok) {
    if (rank == 0 && tid == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
    return;
  }
  const int lo = slice_start(p.V, rank, p.C), hi = slice_start(p.V, rank + 1, p.C);
  int cur = 0, a = 0, token = -1, buf = 0;
  const bool walking = w.par[0] != kUnusedNode;
  bool draw = walking;
  while (walking) {
    const T* zt = target + cur * p.row_stride;
    const T* zq = drafts + cur * p.row_stride;
    int child = a < p.D ? next_child(w, p.T, cur, cur, [](int) { return true; }) : p.T;
    const bool inner = child < p.T;
    MaxSum t = slice_max_sum(zt, lo, hi, p.c2, s_ms[0]);
    MaxSum q{0.f, 1.f};
    if (inner) q = slice_max_sum(zq, lo, hi, p.c2, s_ms[1]);
    send(&s_rec[buf][rank], p.C, Record{t.m, t.l, q.m, q.l});
    cluster_sync_all();
    MaxSum tt{-INFINITY, 0.f}, qq{-INFINITY, 0.f};
    for (int r = 0; r < p.C; ++r) {
      const Record x = s_rec[buf][r];
      tt = merged(tt, MaxSum{x.a, x.b});
      qq = merged(qq, MaxSum{x.c, x.d});
    }
    if (!(tt.l > 0.f && tt.l < INFINITY && tt.m < INFINITY) ||
        (inner && !(qq.l > 0.f && qq.l < INFINITY && qq.m < INFINITY))) {
      if (rank == 0 && tid == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
      draw = false;
      break;
    }
    if (tid == 0) {
      st.mt = tt.m;
      st.it = 1.f / tt.l;
      st.mq = qq.m;
      st.iq = inner ? 1.f / qq.l : 0.f;
      st.k = 0;
    }
    if (tid < p.C) {
      const Record x = s_rec[buf][tid];
      s_mass[tid] = x.a == -INFINITY ? 0.f : x.b * ex2(x.a - tt.m);
    }
    buf ^= 1;
    __syncthreads();
    bool accepted = false;
    while (child < p.T) {
      const int x = w.tok[child];
      if (x < 0 || x >= p.V) {
        if (rank == 0 && tid == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
      } else {
        float pv, qv;
        probabilities(st, p.c2, p.replacement, x, s_zt[child], s_zq[child], pv, qv);
        if (s_u[child] * qv < pv) {
          accepted = true;
          break;
        }
        // rejected: the residual's mass and what is left of q
        float2 sum = make_float2(0.f, 0.f);
        auto one = [&](int e, float z1, float z2) {
          float pe, qe;
          probabilities(st, p.c2, p.replacement, e, z1, z2, pe, qe);
          sum.x += fmaxf(pe - qe, 0.f);
          sum.y += e == x ? 0.f : qe;
        };
        // the draft row may be aligned otherwise than the target's: read element by element there
        scan_slice(zt, lo, hi,
                   [&](int e, const float* v) {
#pragma unroll
                     for (int k = 0; k < VN; ++k) one(e + k, v[k], Vec<T>::scalar(zq + e + k));
                   },
                   [&](int e, float v) { one(e, v, Vec<T>::scalar(zq + e)); });
        sum = block_sum(sum, s_sum);
        send(&s_rec[buf][rank], p.C, Record{sum.x, sum.y, 0.f, 0.f});
        cluster_sync_all();
        float R = 0.f, Q = 0.f;
        for (int r = 0; r < p.C; ++r) {
          R += s_rec[buf][r].a;
          Q += s_rec[buf][r].b;
        }
        if (tid < p.C && R > 0.f) s_mass[tid] = s_rec[buf][tid].a;
        buf ^= 1;
        if (tid == 0) {
          st.tok[st.k] = x;
          st.ir[st.k] = R > 0.f ? 1.f / R : 0.f;
          st.iqs[st.k] = Q > 0.f ? 1.f / Q : 0.f;
          ++st.k;
        }
        __syncthreads();
      }
      child = next_child(w, p.T, cur, child, [](int) { return true; });
    }
    if (!accepted) break;
    if (tid == 0) w.path[a] = child;
    ++a;
    cur = child;
    __syncthreads();  // the stage is rewritten for the next node
  }
  // The draw: the CTA whose slice holds u * total finds the token (rank order, so ascending).
  if (draw) {
    // Every thread finds the same owner; the last CTA with any mass takes what rounding leaves.
    float total = 0.f, before = 0.f, run0 = 0.f;
    for (int r = 0; r < p.C; ++r) total += s_mass[r];
    int owner = -1, last = 0;
    for (int r = 0; r < p.C; ++r) {
      const float m = s_mass[r];
      if (m > 0.f) {
        if (owner < 0) before = run0;
        if (owner < 0 && run0 + m > s_u[0] * total) owner = r;
        last = r;
      }
      run0 += m;
    }
    if (owner < 0) owner = last;
    if (rank == owner) {
      const float goal = s_u[0];           // probabilities() are masses over the total
      const T* zt = target + cur * p.row_stride;
      const T* zq = drafts + cur * p.row_stride;
      const bool inner = st.iq > 0.f;
      auto mass = [&](int e) {
        float pe, qe;
        probabilities(st, p.c2, p.replacement, e, Vec<T>::scalar(zt + e),
                      inner ? Vec<T>::scalar(zq + e) : 0.f, pe, qe);
        return pe;
      };
      // warps take consecutive chunks
      const int n = hi - lo, c0 = lo + static_cast<int>(static_cast<long long>(n) * warp / kWarps),
                c1 = lo + static_cast<int>(static_cast<long long>(n) * (warp + 1) / kWarps);
      float s = 0.f;
      for (int e = c0 + lane; e < c1; e += 32) s += mass(e);
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
      if (lane == 0) s_sum[warp] = make_float2(s, 0.f);
      if (tid == 0) s_token = -1;
      __syncthreads();
      float run = before / total;
      int pick = -1, end = -1;
      float start = 0.f;
      for (int k = 0; k < kWarps; ++k) {
        const float v = s_sum[k].x;
        if (v > 0.f) {
          end = k;
          if (pick < 0 && run + v > goal) {
            pick = k;
            start = run;
          }
          if (pick < 0) start = run;
        }
        run += v;
      }
      if (pick < 0) pick = end;
      if (warp == pick) {
        int found = -1, some = -1;
        float at = start;
        for (int e0 = c0; e0 < c1 && found < 0; e0 += 32) {
          const int e = e0 + lane;
          const float v = e < c1 ? mass(e) : 0.f;
          float inc = v;
#pragma unroll
          for (int k = 1; k < 32; k <<= 1) {
            const float o = __shfl_up_sync(0xffffffffu, inc, k);
            if (lane >= k) inc += o;
          }
          const unsigned over = __ballot_sync(0xffffffffu, v > 0.f && at + inc > goal);
          const unsigned pos = __ballot_sync(0xffffffffu, v > 0.f);
          if (over) found = e0 + __ffs(over) - 1;
          if (pos) some = e0 + 31 - __clz(pos);
          at += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) s_token = found >= 0 ? found : some;
      }
      __syncthreads();
      token = s_token;
      write_walk(p, b, w, a, token);
    }
  } else {
    __syncthreads();
    if (rank == 0) write_walk(p, b, w, a, -1);
  }
}

template <typename K>
int launch_tree(K kernel, TreeParams& p, int B, int es, int* cache, cudaStream_t s) {
  // CTAs that each have a few vectors per thread to read, and all rows' clusters at once if they fit
  const long long vecs = static_cast<long long>(p.V) * es / 16;
  const int most = static_cast<int>(std::min<long long>(kMaxCluster, vecs / kThreads + 1));
  p.C = cluster_for_one_wave(reinterpret_cast<const void*>(kernel), B, 1, most, kThreads, 0, cache);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(B * p.C);
  cfg.blockDim = dim3(kThreads);
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

int g_active_greedy[2][64 * 17], g_active_sample[2][64 * 17];

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
  if (dtype == SPECDEC_BF16)
    return launch_tree(tree_greedy_kernel<uint16_t>, p, B, 2, g_active_greedy[0], s);
  return launch_tree(tree_greedy_kernel<float>, p, B, 4, g_active_greedy[1], s);
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
  if (dtype == SPECDEC_BF16)
    return launch_tree(tree_sample_kernel<uint16_t>, p, B, 2, g_active_sample[0], s);
  return launch_tree(tree_sample_kernel<float>, p, B, 4, g_active_sample[1], s);
}
