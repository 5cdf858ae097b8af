// Commit of a tree's accepted path: K/V columns of the accepted nodes, made contiguous.
//
// For every (layer, k/v, row, head) the columns of nodes path[0] < path[1] < .. go one after the
// other behind the committed ones.  Path nodes increase and path[i-1] >= i, so moving them in
// ascending order within one thread never overwrites a column that is still to be read: the call
// works in place.  One thread owns one 16-byte vector of a column and moves it for every accepted
// node; a batch of loads is in flight before the first store.
//
// What bounds it: a few hundred bytes per head, so the launch and two dependent loads (path, then
// columns); the bytes are 2 * 2 * sum(a_b) * layers * heads * head_dim elements.  Measured: 32 layers,
// 8 rows, 32 heads (16 accepted nodes): 5.2 us; 40 layers, 32 rows, 2 heads: 3.7 us.
#include "tree.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 256;

struct CommitParams {
  ByteView src, dst;
  const int32_t *width, *width_dst, *accept_len, *path, *n_committed, *rows, *first_col;
  int32_t* status;
  int B, T, D, src_cap, dst_cap, src_one_row;
  unsigned L, H, col_vecs;
};

__global__ void __launch_bounds__(kThreads) commit_kernel(const CommitParams p) {
  __shared__ int s_path[SPECDEC_MAX_DRAFT];
  const int b = blockIdx.x;
  const int a = p.accept_len[b];
  bool bad = a < 0 || a > p.D;
  if (!bad && threadIdx.x < a) {
    const int node = p.path[b * p.D + threadIdx.x];
    const int before = threadIdx.x ? p.path[b * p.D + threadIdx.x - 1] : 0;
    s_path[threadIdx.x] = node;
    bad = node <= before || node >= p.T;
  }
  // first: column of node 0; to: column of the first accepted node in dst, less one
  long long first, to;
  if (p.first_col) {
    const int r = p.rows ? p.rows[b] : b;
    if (r < 0) {
      bad = true;
      first = 0;
    } else {
      const int n = p.n_committed[r];
      bad |= n < 1;
      first = static_cast<long long>(p.first_col[r]) + n - 1;
    }
    to = first;
  } else {
    const int W = *p.width;
    bad |= W < 1;
    first = W - 1;
    to = p.width_dst ? static_cast<long long>(*p.width_dst) - 2 - a : first;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && blockIdx.y == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
    return;
  }
  if (a == 0) return;
  if (first < 0 || first + s_path[a - 1] >= p.src_cap || to < -1 || to + a >= p.dst_cap) {
    if (threadIdx.x == 0 && blockIdx.y == 0) set_status(p.status, SPECDEC_ERR_CAPACITY);
    return;
  }
  const long long row = p.src_one_row ? 0 : b;
  // (unsigned: below 2^31 vectors, and a step more, which is below 2^24, does not wrap around)
  const unsigned total = 2u * p.L * p.H * p.col_vecs, step = gridDim.y * kThreads;
  for (unsigned u = blockIdx.y * kThreads + threadIdx.x; u < total; u += step) {
    const int vec = u % p.col_vecs;
    unsigned q = u / p.col_vecs;
    const int h = q % p.H;
    q /= p.H;
    const int kv = q & 1, l = q >> 1;
    const uint4* s = reinterpret_cast<const uint4*>(p.src.base + l * p.src.sl + kv * p.src.skv +
                                                    row * p.src.srow + h * p.src.shead) + vec;
    uint4* d = reinterpret_cast<uint4*>(p.dst.base + l * p.dst.sl + kv * p.dst.skv +
                                        row * p.dst.srow + h * p.dst.shead) + vec;
    constexpr int kBatch = 8;
    for (int i0 = 0; i0 < a; i0 += kBatch) {
      uint4 x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i0 + i < a) x[i] = s[(first + s_path[i0 + i]) * p.col_vecs];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i0 + i < a) d[(to + 1 + i0 + i) * p.col_vecs] = x[i];
    }
  }
}

}  // namespace
}  // namespace specdec

extern "C" int specdec_tree_commit(const specdec_tree_commit_args* a, void* stream) {
  using namespace specdec;
  if (!a) return SPECDEC_ERR_INVALID_ARG;
  if (a->B < 0 || a->T < 1 || a->D < 1) return SPECDEC_ERR_INVALID_ARG;
  if (a->T > SPECDEC_MAX_TREE || a->D > SPECDEC_MAX_DRAFT || a->B > 1024)
    return SPECDEC_ERR_UNSUPPORTED;
  if (a->B == 0) return SPECDEC_OK;
  int st = check_view(a->src, 0);
  if (st) return st;
  st = check_view(a->dst, elem_size(a->src.dtype));
  if (st) return st;
  const specdec_kv_view &s = a->src, &d = a->dst;
  if (s.layers != d.layers || s.heads != d.heads || s.head_dim != d.head_dim ||
      s.rows != d.rows || !(s.rows >= a->B || s.rows == 1))
    return SPECDEC_ERR_INVALID_ARG;
  const bool same = s.base == d.base && s.stride_layer == d.stride_layer &&
                    s.stride_kv == d.stride_kv && s.stride_row == d.stride_row &&
                    s.stride_head == d.stride_head && s.cap_cols == d.cap_cols;
  if (!same) {
    uintptr_t slo, shi, dlo, dhi;
    view_span(s, slo, shi);
    view_span(d, dlo, dhi);
    if (slo < dhi && dlo < shi) return SPECDEC_ERR_INVALID_ARG;
  }
  if (!a->accept_len || !a->path || !a->dev_status) return SPECDEC_ERR_INVALID_ARG;
  if (a->first_col ? !same || !a->n_committed || a->width_dst : !a->width || a->rows)
    return SPECDEC_ERR_INVALID_ARG;
  if (!a->first_col && (a->width_dst ? same : false)) return SPECDEC_ERR_INVALID_ARG;
  if (!a->first_col && s.rows == 1 && a->B > 1) return SPECDEC_ERR_INVALID_ARG;
  const long long vecs = static_cast<long long>(s.head_dim) * elem_size(s.dtype) / 16;
  const long long total = 2LL * s.layers * s.heads * vecs;
  if (total >= (1LL << 31)) return SPECDEC_ERR_UNSUPPORTED;
  const int sms = sm_count();
  if (sms <= 0) return SPECDEC_ERR_CUDA;
  CommitParams p = {};
  p.src = to_bytes(s);
  p.dst = to_bytes(d);
  p.width = a->width;
  p.width_dst = a->width_dst;
  p.accept_len = a->accept_len;
  p.path = a->path;
  p.n_committed = a->n_committed;
  p.rows = a->rows;
  p.first_col = a->first_col;
  p.status = a->dev_status;
  p.B = a->B;
  p.T = a->T;
  p.D = a->D;
  p.L = s.layers;
  p.H = s.heads;
  p.src_cap = s.cap_cols;
  p.dst_cap = d.cap_cols;
  p.col_vecs = static_cast<unsigned>(vecs);
  p.src_one_row = s.rows == 1 ? 1 : 0;
  // every thread one vector where the grid's second dimension allows it
  const int slices = static_cast<int>((total + kThreads - 1) / kThreads);
  const dim3 grid(a->B, slices < 65535 ? slices : 65535);
  commit_kernel<<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return map_cuda_error(cudaGetLastError());
}
