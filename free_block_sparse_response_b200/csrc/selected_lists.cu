// Selected-block attention: from each query's selected blocks to each block's queries.
//
// The attention kernels work block by block: one key block against 128 of the queries that
// selected it, so that a key tile is read once for many queries although every query has its
// own selection.  This file turns the selection [token][slot] -> block around.  Tokens are
// cut into slices (regions: batch x key head x slice), slices into sub-slices of 512 tokens:
//   count    one CTA per sub-slice sets one bit per (block, token) in shared memory and counts
//            each block's bits;
//   scan     one CTA per region turns the counts into first entries, block by block, and
//            cuts every block's rows into work units;
//   scatter  one CTA per sub-slice sets the bits again; an entry's place is the block's first
//            entry plus the set bits before its token.
// Bits make the order independent of the threads' timing: entries of a block ascend by token,
// so every sum over a block's queries is formed in the same order in each run.  All three are
// bound by latency, of memory and of the bits' atomics (the selection is 4 bytes per query and
// slot, read four times): 16 heads x 32,760 tokens x 16 slots, 256 blocks, 42, 21 and 78 us.
#include <cuda_runtime.h>

#include "common.cuh"
#include "selected.cuh"

namespace spr {
namespace {

constexpr int kWords = kSub / 32;

// The valid entries of the sub-slice's rows: ascending, in [0, nb), up to the first negative
// one.  An entry out of range or not above all earlier ones is reported and skipped; a block with
// no key that the token may attend to is skipped (f gets -1).  The lanes of a warp take the slots
// of one or more rows (a power of two of at least 4 lanes a row).  Rows that only ascend need one
// comparison with the neighbour; a prefix maximum sorts out the others.  Bound by instructions.
template <typename F>
__device__ __forceinline__ void each_selected(const SelArgs& a, int z, int t0, F f) {
  const int b = z / a.Hk, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int width = 4;
  while (width < 32 && width < a.top) width *= 2;
  const int per = 32 / width, slot = lane & (width - 1), sub = lane / width;
  const int len = kv_len_of(a, b), qs = q_start_of(a, b), shift = a.block == 128 ? 7 : 6;
  const int* row0 = a.sel + static_cast<size_t>(z) * a.n * a.top;
  const int rows = min(kSub, a.n - t0);
  bool bad = false;
  // the first chunk of a row is read two steps ahead
  auto entry = [&](int i, int j) {
    return i < rows && j < a.top ? __ldg(row0 + static_cast<size_t>(t0 + i) * a.top + j) : -1;
  };
  int ahead = entry(warp * per + sub, slot), ahead2 = entry((warp + warps) * per + sub, slot);
  for (int i0 = warp * per; i0 < rows; i0 += warps * per) {
    const int i = i0 + sub;
    const int head = ahead;
    ahead = ahead2;
    ahead2 = entry(i + 2 * warps * per, slot);
    // last block that holds a key the token may attend to (negative: none)
    const int last = (a.causal ? min(len - 1, qs + t0 + i) : len - 1) >> shift;
    int above = -1;  // largest entry of the chunks before
    bool ended = false;
    for (int j0 = 0; j0 < a.top; j0 += width) {
      const int j = j0 + slot;
      const int g = j0 == 0 ? head : entry(i, j);
      int prev = __shfl_up_sync(0xffffffffu, g, 1, width);
      if (slot == 0) prev = ended ? -1 : above;
      bool take = g >= 0;
      const bool plain = g < 0 || (g < a.nb && g > prev && (prev >= 0 || (j == 0)));
      if (__all_sync(0xffffffffu, plain)) {
        if (j0 + width < a.top) {
          const int end = __shfl_sync(0xffffffffu, g, width - 1, width);
          above = max(above, end);
          ended = end < 0;
        }
      } else {
        // entries from the row's first negative one on do not count
        const unsigned neg = __ballot_sync(0xffffffffu, g < 0) >> (sub * width);
        const bool past = ended || g < 0 || (neg & ((1u << slot) - 1u)) != 0;
        const int v = past || g >= a.nb ? -1 : g;
        int mx = v;  // inclusive prefix maximum over the row's lanes
        for (int o = 1; o < width; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, mx, o, width);
          if (slot >= o) mx = max(mx, y);
        }
        const int y = __shfl_up_sync(0xffffffffu, mx, 1, width);
        prev = max(above, slot > 0 ? y : -1);
        if (!past && (g >= a.nb || g <= prev)) bad = true;
        take = v >= 0 && v > prev;
        above = max(above, __shfl_sync(0xffffffffu, mx, width - 1, width));
        ended = ended || (neg & (width == 32 ? 0xffffffffu : (1u << width) - 1u)) != 0;
      }
      if (i < rows && j < a.top) f(i, (static_cast<size_t>(z) * a.n + t0 + i) * a.top + j, take && g <= last ? g : -1);
    }
  }
  if (bad) record_error(a.status, kErrInvalidArg);
}

__device__ __forceinline__ void set_bits(const SelArgs& a, uint32_t* mask, int z, int t0) {
  for (int i = threadIdx.x; i < a.nb * kWords; i += blockDim.x) mask[i] = 0;
  __syncthreads();
  each_selected(a, z, t0, [&](int i, size_t, int g) {
    if (g >= 0) atomicOr(&mask[g * kWords + (i >> 5)], 1u << (i & 31));
  });
  __syncthreads();
}

__global__ void __launch_bounds__(512) count_kernel(const SelArgs a) {
  extern __shared__ __align__(16) uint32_t mask[];  // [nb][kWords]
  const int z = blockIdx.y, s = blockIdx.x;  // sub-slice s of the head's tokens
  set_bits(a, mask, z, s * kSub);
  const int region = z * a.slices + s / a.subs, ls = s % a.subs;
  for (int g = threadIdx.x; g < a.nb; g += blockDim.x) {
    int c = 0;
#pragma unroll
    for (int w = 0; w < kWords; w += 4) {  // (16-byte reads: a quarter of the bank conflicts)
      const uint4 x = *reinterpret_cast<const uint4*>(mask + g * kWords + w);
      c += __popc(x.x) + __popc(x.y) + __popc(x.z) + __popc(x.w);
    }
    a.offs[(static_cast<size_t>(region) * a.nb + g) * a.subs + ls] = c;
  }
}

// Exclusive prefix sum of one value per thread over a block of 512 threads; total in `sum`.
__device__ __forceinline__ int block_scan(int v, int& sum, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < 16 ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    if (lane < 16) s_warp[lane] = w;
  }
  __syncthreads();
  const int before = warp > 0 ? s_warp[warp - 1] : 0;
  sum = s_warp[15];
  __syncthreads();
  return before + x - v;
}

// A warp a block adds the block's counts, the CTA's threads form the prefix sums over blocks,
// then a warp a block writes its sub-slices' first entries and its units.
__global__ void __launch_bounds__(512) scan_kernel(const SelArgs a) {
  extern __shared__ int4 s_blk[];  // [nb] {entries, then first entry | units | first slot | first unit}
  __shared__ int s_warp[16];
  const int region = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = region % a.slices, z = region / a.slices, b = z / a.Hk;
  const int len = kv_len_of(a, b), qs = q_start_of(a, b);
  // sub-slices of this region that hold tokens
  const int live = min(a.subs, ceil_div(a.n - s * a.slice, kSub));
  int* offs = a.offs + static_cast<size_t>(region) * a.nb * a.subs;
  // (eight blocks' counts under way: one at a time each costs a memory latency)
  constexpr int kBatch = 8;
  for (int g0 = warp; g0 < a.nb; g0 += 16 * kBatch) {
    int cnt[kBatch] = {};
    for (int i = lane; i < live; i += 32) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (g0 + 16 * k < a.nb) cnt[k] += offs[static_cast<size_t>(g0 + 16 * k) * a.subs + i];
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int sum = __reduce_add_sync(0xffffffffu, cnt[k]);
      if (lane == 0 && g0 + 16 * k < a.nb) s_blk[g0 + 16 * k].x = sum;
    }
  }
  __syncthreads();
  int entry0 = 0, unit0 = 0, slot0 = 0;
  for (int g0 = 0; g0 < a.nb; g0 += 512) {
    const int g = g0 + threadIdx.x;
    const int cnt = g < a.nb ? s_blk[g].x : 0;
    const int nu = ceil_div(cnt * a.group, a.unit_rows);
    int sum;
    const int off = entry0 + block_scan(cnt, sum, s_warp);
    entry0 += sum;
    const int u = unit0 + block_scan(nu, sum, s_warp);
    unit0 += sum;
    const int slot = slot0 + block_scan(nu > 1 ? nu : 0, sum, s_warp);
    slot0 += sum;
    if (g < a.nb) {
      s_blk[g] = make_int4(off, cnt, slot, u);
      a.blk[static_cast<size_t>(region) * a.nb + g] = make_int4(nu, slot, u, 0);
    }
  }
  __syncthreads();
  for (int g0 = warp; g0 < a.nb; g0 += 16 * kBatch) {
    int off[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) off[k] = g0 + 16 * k < a.nb ? s_blk[g0 + 16 * k].x : 0;
    for (int i0 = 0; i0 < live; i0 += 32) {
      const int i = i0 + lane;
      int c[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        c[k] = i < live && g0 + 16 * k < a.nb ? offs[static_cast<size_t>(g0 + 16 * k) * a.subs + i] : 0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        int x = c[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (i < live && g0 + 16 * k < a.nb) offs[static_cast<size_t>(g0 + 16 * k) * a.subs + i] = off[k] + x - c[k];
        off[k] += __shfl_sync(0xffffffffu, x, 31);
      }
    }
  }
  for (int g0 = warp; g0 < a.nb; g0 += 16 * 32) {
    // (the ranges of the warp's next 32 blocks at once)
    const int gl = g0 + 16 * lane;
    const float ranges = a.f32 || gl >= a.nb ? 0.f : __ldg(a.range + static_cast<size_t>(z) * a.nb + gl);
    for (int j = 0; j < 32 && g0 + 16 * j < a.nb; ++j) {
      const int g = g0 + 16 * j;
      const float range = __shfl_sync(0xffffffffu, ranges, j);
      const int4 k = s_blk[g];
      const int rows = k.y * a.group, nu = ceil_div(rows, a.unit_rows);
      for (int i = lane; i < nu; i += 32)
        a.units[static_cast<size_t>(region) * a.unit_cap + k.w + i] =
            Unit{g, k.x, i * a.unit_rows, min(a.unit_rows, rows - i * a.unit_rows), len - g * a.block, qs - g * a.block, b,
                 z % a.Hk, rows, range, {}};
    }
  }
  if (threadIdx.x == 0) a.n_units[region] = unit0;
  if (threadIdx.x == 0 && region == 0) *a.slow = 0;
  // the kernels on the fp32 pipes launch a CTA for every unit there may be
  if (a.f32)
    for (int u = unit0 + threadIdx.x; u < a.unit_cap; u += 512)
      a.units[static_cast<size_t>(region) * a.unit_cap + u] = Unit{};
}

__global__ void __launch_bounds__(512) scatter_kernel(const SelArgs a) {
  // bits [nb][kWords], the words' first entries [nb][kWords] from the blocks' first entries [nb]
  extern __shared__ __align__(16) uint32_t mask[];
  const int z = blockIdx.y, s = blockIdx.x, t0 = s * kSub;
  const int region = z * a.slices + s / a.subs, ls = s % a.subs;
  uint16_t* before = reinterpret_cast<uint16_t*>(mask + a.nb * kWords);
  int* first = reinterpret_cast<int*>(before + a.nb * kWords);
  const int* offs = a.offs + static_cast<size_t>(region) * a.nb * a.subs + ls;
  for (int g = threadIdx.x; g < a.nb; g += blockDim.x) first[g] = __ldg(offs + static_cast<size_t>(g) * a.subs);
  set_bits(a, mask, z, t0);
  for (int g = threadIdx.x; g < a.nb; g += blockDim.x) {
    uint32_t c = 0, at[kWords / 2];
#pragma unroll
    for (int w = 0; w < kWords; w += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(mask + g * kWords + w);
      const uint32_t y = c + __popc(x.x), u = y + __popc(x.y), v = u + __popc(x.z);
      at[w / 2] = c | y << 16, at[w / 2 + 1] = u | v << 16;
      c = v + __popc(x.w);
    }
#pragma unroll
    for (int w = 0; w < kWords / 2; w += 4)
      *reinterpret_cast<uint4*>(before + g * kWords + 2 * w) = make_uint4(at[w], at[w + 1], at[w + 2], at[w + 3]);
  }
  __syncthreads();
  int* list = a.list + static_cast<size_t>(region) * a.slice * a.top;
  each_selected(a, z, t0, [&](int i, size_t at, int g) {
    int e = -1;
    if (g >= 0) {
      const int w = g * kWords + (i >> 5);
      e = first[g] + before[w] + __popc(mask[w] & ((1u << (i & 31)) - 1u));
      list[e] = t0 + i;
    }
    a.inv[at] = e;
  });
}

}  // namespace

cudaError_t launch_lists(const SelArgs& a, cudaStream_t st) {
  const int heads = a.Bt * a.Hk, subs = ceil_div(a.n, kSub);
  if (heads > 65535) return cudaErrorInvalidValue;
  const size_t mask = sizeof(uint32_t) * a.nb * kWords, both = mask + sizeof(int) * a.nb + sizeof(uint16_t) * a.nb * kWords;
  if (both > 227 * 1024) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(count_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(scatter_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
  count_kernel<<<dim3(subs, heads), 512, mask, st>>>(a);
  if ((e = counted(cudaGetLastError(), 1)) != cudaSuccess) return e;
  scan_kernel<<<heads * a.slices, 512, sizeof(int4) * a.nb, st>>>(a);
  if ((e = counted(cudaGetLastError(), 1)) != cudaSuccess) return e;
  scatter_kernel<<<dim3(subs, heads), 512, both, st>>>(a);
  return counted(cudaGetLastError(), 1);
}

}  // namespace spr
