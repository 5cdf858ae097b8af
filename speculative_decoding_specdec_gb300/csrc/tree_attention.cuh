// What the tree attention kernels share: parameters, the split of the work, the partial results.
//
// The mathematics.  For a query row r (node t, query head) with scores z_c = scale * (q . k_c):
//   m = max z_c, l = sum 2^((z_c - m) log2 e), o = sum 2^((z_c - m) log2 e) v_c,  out = o / l,
// over any order of the columns in one pass: a larger maximum m' rescales l and o by 2^(m - m'),
// and two parts of a row's columns merge the same way.
//
// The split.  A unit is one K/V head of one batch row: its columns are those of the row's
// committed tokens and then of the T nodes, contiguous in the cache, cut into tiles.  All query
// rows (node, query head of the group) of the unit use the same columns; M of them make an M-tile.
// The tiles of all units, in order, are cut into equal contiguous shares, one per group of
// MT CTAs (MT M-tiles), so ragged lengths leave no CTA idle and the MT CTAs that stream the same
// columns do so at the same time (one DRAM read, the rest from L2).  A unit that lies in one share
// is finished by its CTA; one cut by share borders is written as partial results (m, l, o) to the
// workspace and merged in share order, so that results do not depend on which CTA came last: by the
// CTA that takes the unit's last ticket, or (tensor-core kernel, whose parts are larger) by a launch
// of its own.  A share has at most two cut units (its first and last).
//
// A shared prefix.  Rows that share a prefix attend it in a pass of its own, before the pass over their
// own columns, by the same kernels (kPrefix): a unit is then one K/V head of one prefix and up to M of
// the query rows of all batch rows of its group, which see all its columns.  That pass leaves (m, l, o)
// of every query row, and the pass over the rows' own columns merges them where it writes its results.
// Where a batch row's own query rows fill the tensor cores' tiles by themselves, nothing is gained by
// taking several together: then (kBoth) one pass has units of one batch row whose tiles are those of its
// prefix and then those of its own columns.
#pragma once

#include "tree.cuh"

namespace specdec {

constexpr int kAttnMaxRows = 1024;
constexpr int kAttnMaxPrefixes = 512;
constexpr float kLog2e = 1.4426950408889634f;

struct AttnParams {
  ByteView cache;  // of the layer, bytes
  const char* q;
  char* out;
  float* lse;
  long long qr, qt, outr, outt;  // bytes between rows and tokens
  const int32_t *n_committed, *width, *parents, *rows, *first_col;
  int32_t* status;
  unsigned* ticket;  // [groups * MT], zero between calls
  float2* part_ml;   // [grid * 2][M]
  float* part_o;     // [grid * 2][M][hd]
  int4* cuts;        // [groups], tensor-core kernel: the units that borders cut
  float scale_log2;  // scale * log2(e)
  int B, T, Hq, H, G, hd, cap, one_row, MT, groups, min_tiles, open, g_shift;  // g_shift: log2 G, or -1
  // A shared prefix (the prefix pass has its cache as `cache`): the rows' state (1: what the prefix pass
  // left is to be merged; 0: there is no prefix; -1: an error), nullptr if there is none at all, and what
  // it left, by (row, node, query head).
  int32_t* prior;
  float2* prior_ml;
  float* prior_o;
  const int32_t *prefix_len, *prefix_first, *group_start;
  int P, M, two, prefix_cap, prefix_one_row;  // prefixes; query rows of a unit; whether some group may have more than 128
};

// One batch row's columns.
struct AttnRow {
  int first, old, cols;  // first column, committed columns N - 1, all columns N - 1 + T (0: error)
};

__device__ __forceinline__ AttnRow attn_row(const AttnParams& p, int b, int* err) {
  const int r = p.rows ? p.rows[b] : b;
  *err = 0;
  if (r < 0) {
    *err = SPECDEC_ERR_INPUT_RANGE;
    return AttnRow{0, 0, 0};
  }
  const int n = p.n_committed[r];
  long long first;
  bool bad = n < 1;
  if (p.first_col) {
    first = p.first_col[r];
    bad |= first < 0;
  } else {
    const int W = *p.width;
    bad |= n > W;
    first = static_cast<long long>(W) - n;
  }
  if (bad) {
    *err = SPECDEC_ERR_INPUT_RANGE;
    return AttnRow{0, 0, 0};
  }
  if (first + n - 1 + p.T > p.cap) {
    *err = SPECDEC_ERR_CAPACITY;
    return AttnRow{0, 0, 0};
  }
  return AttnRow{static_cast<int>(first), n - 1, n - 1 + p.T};
}

// The plan in shared memory: tiles of the rows before row b, per K/V head, and the rows.
// (a prefix pass: of the prefixes, with their first query row (b T + t) G + g and number of query rows)
// (kBoth: also each row's prefix: its columns, -1 for an error, first column and cache row)
struct AttnPlan {
  int *pre, *first, *old, *row0, *rows;  // [B + 1], [B], [B]; prefix pass: [P + 1] and [P]
  int *plen, *pfirst, *prow;             // [B]
};
enum AttnMode { kOwn = 0, kPrefixPass = 1, kBothParts = 2, kBehind = 3 };  // kBehind: own columns behind a prefix pass
__host__ __device__ constexpr int attn_plan_bytes(int B) { return (3 * B + 1) * 4; }
__host__ __device__ constexpr int prefix_plan_bytes(int P) { return (5 * P + 1) * 4; }
static_assert(prefix_plan_bytes(kAttnMaxPrefixes) <= attn_plan_bytes(kAttnMaxRows), "one room for either plan");
__device__ __forceinline__ AttnPlan attn_plan_at(void* smem, int n) {
  int* p = static_cast<int*>(smem);
  return AttnPlan{p, p + n + 1, p + 2 * n + 1, p + 3 * n + 1, p + 4 * n + 1, p + 3 * n + 1, p + 4 * n + 1, p + 5 * n + 1};
}
__host__ __device__ constexpr int both_plan_bytes(int B) { return (6 * B + 1) * 4; }

// A unit counts `p.open` tiles more than it has, for what a CTA spends on opening and closing it,
// so that shares with many short units take no longer than others.
// Built by warp 0 of every CTA (the caller synchronises); CTA 0 records errors.
template <int kMode = kOwn>
__device__ __forceinline__ void attn_plan(const AttnParams& p, int tile, const AttnPlan& plan) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  if constexpr (kMode == kBothParts) {
    bool bad = false;
    for (int i = lane; i < p.P; i += 32) {
      const int b0 = p.group_start[i], b1 = p.group_start[i + 1];
      bad |= b0 < 0 || b1 < b0 || b1 > p.B;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (bad && blockIdx.x == 0 && lane == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
    for (int b = lane; b < p.B; b += 32) plan.plen[b] = bad ? -1 : 0;
    for (int i0 = 0; i0 < p.P && !bad; i0 += 32) {
      const int i = i0 + lane;
      int b0 = 0, b1 = 0, len = 0, first = 0;
      if (i < p.P) {
        b0 = p.group_start[i];
        b1 = p.group_start[i + 1];
        len = p.prefix_len[i];
        first = p.prefix_first ? p.prefix_first[i] : 0;
        const int err = len < 0 || first < 0 ? SPECDEC_ERR_INPUT_RANGE
                        : len > p.prefix_cap || first > p.prefix_cap - len ? SPECDEC_ERR_CAPACITY : 0;
        if (err) {
          len = -1;
          if (blockIdx.x == 0) set_status(p.status, err);
        }
      }
      __syncwarp();
      for (int k = 0; k < min(32, p.P - i0); ++k) {
        const int g0 = __shfl_sync(0xffffffffu, b0, k), g1 = __shfl_sync(0xffffffffu, b1, k);
        const int l = __shfl_sync(0xffffffffu, len, k), f = __shfl_sync(0xffffffffu, first, k);
        for (int b = g0 + lane; b < g1; b += 32) {
          plan.plen[b] = l;
          plan.pfirst[b] = f;
          plan.prow[b] = p.prefix_one_row ? 0 : i0 + k;
        }
      }
    }
    __syncwarp();
  }
  if constexpr (kMode == kPrefixPass) {
    // rows of no group, or of one of a prefix without columns, are 0; where the groups' bounds are not
    // ascending within the batch nothing is known of any row
    bool bad = false;
    for (int i = lane; i < p.P; i += 32) {
      const int b0 = p.group_start[i], b1 = p.group_start[i + 1];
      bad |= b0 < 0 || b1 < b0 || b1 > p.B;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (blockIdx.x == 0) {
      for (int b = lane; b < p.B; b += 32) p.prior[b] = bad ? -1 : 0;
      __syncwarp();
      if (bad && lane == 0) set_status(p.status, SPECDEC_ERR_INPUT_RANGE);
    }
    for (int i0 = 0; i0 < p.P; i0 += 32) {
      const int i = i0 + lane;
      int tiles = 0;
      if (i < p.P) {
        const int b0 = p.group_start[i], b1 = p.group_start[i + 1], len = p.prefix_len[i];
        const int first = p.prefix_first ? p.prefix_first[i] : 0;
        const int err = bad ? 0 : len < 0 || first < 0 ? SPECDEC_ERR_INPUT_RANGE
                                : len > p.cap || first > p.cap - len ? SPECDEC_ERR_CAPACITY : 0;
        const bool live = !bad && !err && len > 0 && b1 > b0;
        const int rows = live ? (b1 - b0) * p.T * p.G : 0;
        tiles = live ? ((rows + p.M - 1) / p.M) * ((len + tile - 1) / tile + p.open) : 0;
        plan.first[i] = first;
        plan.old[i] = len;
        plan.row0[i] = live ? b0 * p.T * p.G : 0;
        plan.rows[i] = rows;
        if (blockIdx.x == 0 && (err || live)) {
          if (err) set_status(p.status, err);
          for (int b = b0; b < b1; ++b) p.prior[b] = err ? -1 : 1;
        }
      }
      int inc = tiles;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, k);
        if (lane >= k) inc += o;
      }
      if (i < p.P) plan.pre[i] = carry + inc - tiles;
      carry += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) plan.pre[p.P] = carry;
    return;
  }
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    int tiles = 0, first = 0, old = 0;
    if (b < p.B) {
      int err;
      const AttnRow r = attn_row(p, b, &err);
      if (err && blockIdx.x == 0) set_status(p.status, err);
      tiles = r.cols > 0 ? (r.cols + tile - 1) / tile + p.open : 0;
      if (kMode == kBothParts && tiles > 0) {
        const int len = plan.plen[b];
        tiles = len < 0 ? 0 : tiles + (len + tile - 1) / tile;
      }
      first = r.first;
      old = r.old;
    }
    int inc = tiles;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, inc, k);
      if (lane >= k) inc += o;
    }
    if (b < p.B) {
      plan.pre[b] = carry + inc - tiles;
      plan.first[b] = first;
      plan.old[b] = old;
    }
    carry += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) plan.pre[p.B] = carry;
}

// Shares of the tile sequence: group g has [start(g), start(g + 1)); the first `rem` have one tile
// more than the others.  (32-bit: the host checks that the longest sequence fits.)
struct AttnShares {
  int total, groups, base, rem;
  __device__ int start(int g) const { return g * base + min(g, rem); }
  __device__ int owner(int x) const {  // the group whose share holds tile x
    const int more = rem * (base + 1);
    return x < more ? x / (base + 1) : rem + (x - more) / base;
  }
};
template <int kMode = kOwn>
__device__ __forceinline__ AttnShares attn_shares(const AttnParams& p, const AttnPlan& plan) {
  AttnShares s;
  s.total = plan.pre[kMode == kPrefixPass ? p.P : p.B] * p.H;
  const int most = s.total / p.min_tiles;
  s.groups = most < 1 ? 1 : min(most, p.groups);
  s.base = s.total / s.groups;
  s.rem = s.total - s.base * s.groups;
  return s;
}

// A contiguous run of tiles of one unit inside a share (it may have none, if the share ends in what
// the unit counts for being opened).
struct AttnSegment {
  int b, h, tile0, tile1, tiles;  // unit (its cache row), its tiles [tile0, tile1) of `tiles`
  int unit0;                      // place of the unit's first tile in the sequence
  int next;                       // place behind the segment
  int first, old, cols;           // its columns: AttnRow
  int row0, rows;                 // prefix pass: its first query row, and how many it has
  int plen, pfirst, prow;         // kBoth: the columns of the prefix, whose tiles come first
};
template <int kMode = kOwn>
__device__ __forceinline__ AttnSegment attn_segment(const AttnParams& p, const AttnPlan& plan,
                                                    int x, int end) {
  constexpr bool kPrefix = kMode == kPrefixPass;
  int lo = 0, hi = (kPrefix ? p.P : p.B) - 1;  // the last row with pre * H <= x: it has tiles
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (plan.pre[mid] * p.H <= x) lo = mid;
    else hi = mid - 1;
  }
  AttnSegment s;
  s.b = lo;
  int span = plan.pre[lo + 1] - plan.pre[lo];
  const int rem = x - plan.pre[lo] * p.H;
  if constexpr (kPrefix) {  // a head's units are neighbours: they use the same columns
    const int units = (plan.rows[lo] + p.M - 1) / p.M;
    span /= units;
    const int unit = rem / span;
    s.h = unit / units;
    const int k = unit - s.h * units;
    s.row0 = plan.row0[lo] + k * p.M;
    s.rows = min(p.M, plan.rows[lo] - k * p.M);
  } else {
    s.h = rem / span;
  }
  const int at = kPrefix ? rem % span : rem - s.h * span;
  s.next = min(end, x - at + span);
  s.tiles = span - p.open;
  s.tile0 = max(0, at - p.open);
  s.tile1 = max(0, s.next - x + at - p.open);
  s.unit0 = x - at + p.open;
  s.first = plan.first[lo];
  s.old = plan.old[lo];
  s.cols = s.old + (kPrefix ? 0 : p.T);
  if constexpr (kMode == kBothParts) {
    s.plen = plan.plen[lo];
    s.pfirst = plan.pfirst[lo];
    s.prow = plan.prow[lo];
  }
  return s;
}

// The next segment with tiles at or behind x; false at the share's end.
template <int kMode = kOwn>
__device__ __forceinline__ bool attn_next(const AttnParams& p, const AttnPlan& plan, int x, int end,
                                          AttnSegment& s) {
  while (x < end) {
    s = attn_segment<kMode>(p, plan, x, end);
    if (s.tile1 > s.tile0) return true;
    x = s.next;
  }
  return false;
}

// Takes a ticket of a cut unit's M-tile mt; true in every thread for the CTA that took the last one
// (the partial results of all are then visible to it).  n: CTAs that share the unit, the first of
// them of share g0, which names the ticket: a share is the first of one cut unit at most.
__device__ __forceinline__ bool attn_last(const AttnParams& p, int g0, int mt, int n, int* s_flag) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned* t = &p.ticket[g0 * p.MT + mt];
    const unsigned old = atomicAdd(t, 1u);
    *s_flag = old + 1 == static_cast<unsigned>(n);
    if (*s_flag) *t = 0;
    __threadfence();
  }
  __syncthreads();
  return *s_flag != 0;
}

// Slot of the partial result that share g's CTA of M-tile mt wrote for the unit that begins at
// unit0 (its first tile's place): 0 if its segment starts the share, else 1.
__device__ __forceinline__ int attn_slot(const AttnParams& p, const AttnShares& sh, int g, int mt,
                                         int unit0) {
  return 2 * (g * p.MT + mt) + (sh.start(g) >= unit0 ? 0 : 1);
}

// V of nodes that is not finite, in the kernels of matrix products.  There a hidden column has the
// weight 0, and 0 * NaN is NaN, so such values of a node's V are zero in shared memory, and the rows
// that see the node get them added from the cache to what has been written (attn_add_not_finite):
// their weight is not zero, and whatever it is the result in that place of the head is an infinity
// or NaN.  Both out of line: among the loops they cost every call 1.5 to 2.5 %.
__device__ __forceinline__ bool inf_or_nan(uint32_t w) {  // either of two bf16 values
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ bool inf_or_nan(uint4 v) {
  return inf_or_nan(v.x) || inf_or_nan(v.y) || inf_or_nan(v.z) || inf_or_nan(v.w);
}
// Zeros in the place of what is not finite in the 16-byte chunks [c0, c1) of row r of a tile of
// `rows` rows in panels of 64 values (the 128-byte swizzle).
inline __device__ __noinline__ void attn_make_finite(char* tile, int r, int rows, int c0, int c1) {
  auto of = [](uint32_t w) {
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
    return w;
  };
  for (int c = c0; c < c1; ++c) {
    uint4* at = reinterpret_cast<uint4*>(tile + (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    *at = make_uint4(of(at->x), of(at->y), of(at->z), of(at->w));
  }
}
// V of a segment's first node (the columns of the others follow).
__device__ __forceinline__ const char* attn_node_v(const AttnParams& p, const AttnSegment& s) {
  return p.cache.base + p.cache.skv + (p.one_row ? 0 : s.b) * p.cache.srow + s.h * p.cache.shead +
         (static_cast<long long>(s.first) + s.old) * p.hd * 2;
}
// Groups of 4 values d0, d0 + step, .. of a row that this thread has written, as bf16 to `out` or
// (out == nullptr) as partial sums, part + 4-value group * part_step; nodes: those that the row sees
// and whose V, from `v` on, is not finite somewhere.
inline __device__ __noinline__ void attn_add_not_finite(unsigned long long nodes, const char* v, int hd, int d0, int step,
                                                 char* out, float4* part, int part_step) {
  for (; nodes; nodes &= nodes - 1) {
    const char* from = v + (__ffsll(nodes) - 1) * hd * 2;
    for (int d = d0; d < hd; d += step) {
      const uint2 w = *reinterpret_cast<const uint2*>(from + d * 2);
      auto of = [](float x) { return fabsf(x) < INFINITY ? 0.f : x; };  // (an infinity or NaN)
      const float4 x = make_float4(of(bf16_lo(w.x)), of(bf16_hi(w.x)), of(bf16_lo(w.y)), of(bf16_hi(w.y)));
      if (out) {
        uint2* at = reinterpret_cast<uint2*>(out + d * 2);
        const uint2 y = *at;
        *at = make_uint2(bf16_pack(bf16_lo(y.x) + x.x, bf16_hi(y.x) + x.y), bf16_pack(bf16_lo(y.y) + x.z, bf16_hi(y.y) + x.w));
      } else {
        float4* at = part + static_cast<long long>(d / 4) * part_step;
        const float4 y = *at;
        *at = make_float4(y.x + x.x, y.y + x.y, y.z + x.z, y.w + x.w);
      }
    }
  }
}

// Query row r of a unit: its batch row, node and query head.  (Prefix pass: rows of a unit are counted
// through its group's batch rows.)
struct AttnQuery {
  int b, t, h;
};
template <bool kPrefix>
__device__ __forceinline__ AttnQuery attn_query(const AttnParams& p, const AttnSegment& s, int r) {
  const int row = kPrefix ? s.row0 + r : r;
  const int node = p.g_shift >= 0 ? row >> p.g_shift : row / p.G, h = s.h * p.G + row - node * p.G;
  if constexpr (!kPrefix) return AttnQuery{s.b, node, h};
  const int b = node / p.T;
  return AttnQuery{b, node - b * p.T, h};
}
// Where the prefix pass leaves (m, l) and o / hd of a query row.
__device__ __forceinline__ long long attn_prior_at(const AttnParams& p, int b, int t, int h) {
  return (static_cast<long long>(b) * p.T + t) * p.Hq + h;
}
// The pass over own columns may start while the prefix pass before it still runs: what that left is read
// behind this, and no CTA ends before (the next kernel waits for this one alone).
__device__ __forceinline__ void attn_wait_prior(const AttnParams& p) {
  if (p.prior) pdl_wait();
}
// Merging two parts of a row: the factors of the first's and the second's sums, and (m, l) of both.
__device__ __forceinline__ float2 attn_join(float m0, float l0, float2 part, float& f0, float& f1) {
  const float m = fmaxf(m0, part.x), off = m == -INFINITY ? 0.f : m;
  f0 = exp2f(m0 - off);
  f1 = exp2f(part.x - off);
  return make_float2(m, l0 * f0 + part.y * f1);
}

// Launch of a pass, behind a prefix pass as its programmatic dependent.
template <typename... Params, typename... Args>
cudaError_t attn_launch(void (*kernel)(Params...), int grid, int threads, size_t smem, bool behind, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = behind ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The tensor-core kernel (tree_attention_tc.cu): rows per M-tile and M-tiles for R query rows per
// K/V head, and its launch (rows: of the cache).
void attn_tc_shape(int R, int* M, int* MT);
int launch_attn_tc(const AttnParams& p, int rows, int grid, bool prefix, cudaStream_t stream);
// Both parts in one pass; prefix: the prefixes' cache layer and its rows.
int launch_attn_tc_both(const AttnParams& p, int rows, const ByteView& prefix, int prefix_rows, int grid, cudaStream_t stream);
// The kernel for few rows (tree_attention_mma.cu).
void attn_mma_shape(int R, int hd, int* M, int* MT, int* tile, int* per_sm);
int launch_attn_mma(const AttnParams& p, int M, int rows, int grid, bool prefix, cudaStream_t stream);

}  // namespace specdec
