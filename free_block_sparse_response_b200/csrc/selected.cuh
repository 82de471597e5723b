// Launch interface of the rotary and selected-block attention kernels (internal).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include "common.cuh"

namespace spr {

// A [batch, heads, rows, d] tensor with contiguous rows; strides in elements.
struct View {
  void* p;
  long long sb, sh, sn;
};

struct RotaryArgs {
  View x[2], y[2];  // q and k (h[1] = 0: no second tensor)
  int h[2];
  int Bt, n, d;
  int first, rot;   // the rotated dims [first, first + rot)
  bool half, f32, inverse;
  int axes, pairs[4];
  float factor;
  const double* freqs;  // [rot / 2] radians per position
  const int* positions;
  long long pos_sb, pos_sn;
  bool copy_rest;        // set by the launcher
  int heads_per_thread;  // set by the launcher
};
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t st);

// Tokens of one sub-slice of the selection lists (one CTA's bit masks).
constexpr int kSub = 512;
// Blocks per head that the lists' shared-memory masks hold.
constexpr int kMaxBlocks = 2048;

// CTAs of the tensor-core kernels: one per SM.
constexpr int kTcShares = 148;

// One work item of the attention kernels: rows [r0, r0 + rows) of the entries of key block g,
// whose first entry is `off` of its region's list; row r is query head r % group of entry r / group.
// rows = 0: none.  live, qs: the length and the position of query 0, both from the block's first
// key on.  total: the block's rows in this region.  k: a.range of the block.
struct __align__(16) Unit {
  int g, off, r0, rows, live, qs, b, kh, total;
  float k;
  int pad[2];
};

struct SelArgs {
  bool f32, causal;
  int Bt, Hq, Hk, group, n, nk, d, block, nb, top;
  int n_first, n_local;
  int q_start0;          // position of query 0 where q_start is null
  const int* kv_len;     // [Bt] or null (nk)
  const int* q_start;    // [Bt] or null
  float scale;
  View q, k, v, o, go, gq, gk, gv;
  const int* sel;        // [Bt, Hk, n, top]
  float* lse;            // [Bt, Hq, n]
  const float* means;    // [Bt, Hk, nb, d]
  int* status;
  // number of rows that a call leaves to a second kernel, then the rows: select, [Bt, Hk, n] to
  // select_row_kernel; attention in bf16, [Bt, Hq, n] to mend_kernel
  int* slow;
  void* mean_parts;      // select: bf16 [Bt, Hk, nb][2][d], the means' hi and lo parts
  float* mean_norm2;     // select: [Bt, Hk, nb] squared norms of the means
  // lists: per region (batch, key head, slice of `slice` tokens), `slices` regions per head
  int slice, slices;
  int subs;              // sub-slices of a slice
  int* offs;             // [regions][nb][subs]: counts, then first entries
  int* list;             // [regions][slice * top] tokens, block by block, ascending
  int* inv;              // [Bt, Hk, n, top] entry of (token, slot) in its region, or -1
  int unit_rows, unit_cap;
  Unit* units;           // [regions][unit_cap], the last ones empty
  int* n_units;          // [regions]
  int4* blk;             // [regions][nb] {units, first slot of their sums where there are more, first unit, -}
  // partial rows of one chunk of regions, [chunk regions][slice * top * group][d]: fp32, or fp16
  // with the columns of part_column() (selected_tc.cuh)
  float* part;
  // statistics of each partial row.  fp32: its maximum (log2 units) and sum; fp16 forward: its
  // log-sum-exp and the exponent that its values are to be multiplied by 2^ of; fp16 dQ: -, scale
  float2* ml;
  // bf16, [Bt * Hk][nb]: not finite where a block is wide (its parts take store_wide), else, forward, the
  // power of two that the parts of rows which see all of it are divided by; forward, [Bt * Hk][nb *
  // block]: the power for rows that see the block up to this key
  float* range;
  signed char* key_range;
  float* delta;          // backward: sum of o * go per query row
  __nv_bfloat16* rest;   // [Bt, Hq, n, d] what the rounding of o left off, or null
  float* seg;            // backward: [chunk regions][seg_cap][2][block][d] sums of split blocks
  int seg_cap;
  // backward, a head of several slices: [2][nk][d] sums of dV and of dK over the slices so
  // far of the head at work, or null (the launches write a.gk and a.gv)
  float* acc;
};

// Device limits of one batch element.
__device__ __forceinline__ int kv_len_of(const SelArgs& a, int b) {
  return a.kv_len == nullptr ? a.nk : min(max(a.kv_len[b], 0), a.nk);
}
__device__ __forceinline__ int q_start_of(const SelArgs& a, int b) {
  return a.q_start == nullptr ? a.q_start0 : min(max(a.q_start[b], -(1 << 29)), 1 << 29);
}

cudaError_t launch_key_means(const SelArgs& a, const int* kv_start, int max_new, float* means, cudaStream_t st);
cudaError_t launch_select(const SelArgs& a, int* sel, cudaStream_t st);
cudaError_t launch_lists(const SelArgs& a, cudaStream_t st);
// a.range (forward: and a.key_range) from the blocks of V (backward: K), whose sums the parts are; before
// the lists.
cudaError_t launch_ranges(const SelArgs& a, bool backward, cudaStream_t st);
// One chunk of `count` regions starting at region `first`.
cudaError_t launch_selected_forward(const SelArgs& a, int first, int count, cudaStream_t st);
cudaError_t launch_selected_backward(const SelArgs& a, int first, int count, cudaStream_t st);
// The single-token form: whether it takes this call, and the whole of it in one launch.
bool use_decode(const SelArgs& a);
cudaError_t launch_decode(const SelArgs& a, cudaStream_t st);
cudaError_t launch_delta(const SelArgs& a, cudaStream_t st);
// a.acc to rows of a.gk and a.gv, (batch, key head) z.
cudaError_t launch_slice_sums(const SelArgs& a, int z, cudaStream_t st);
// The elements of the listed rows of a.o, or (grad) a.gq, that their parts could not hold.
cudaError_t launch_mend(const SelArgs& a, bool grad, cudaStream_t st);

}  // namespace spr
