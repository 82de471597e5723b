// Mean key of every key block, and the blocks that each query selects.
//
// A block's mean key is summed in 64 bits (exact for bf16 keys) and rounded once to 32.  The
// score of a query and a block is (sum of the group's queries) . mean; the selection is
// decided on scores in 64 bits, so it is the definition's whatever the types.
#include <cuda_runtime.h>

#include "common.cuh"
#include "selected.cuh"

namespace spr {
namespace {

// One CTA per (block, key head, batch).  16-byte loads: D / V threads cover a row.
template <typename T, int D>
__global__ void __launch_bounds__(256) key_means_kernel(const SelArgs a, const int* __restrict__ kv_start,
                                                        float* __restrict__ means) {
  constexpr int V = 16 / sizeof(T), kCols = D / V, kRows = 256 / kCols;
  __shared__ double part[kRows][D];
  const int b = blockIdx.z, h = blockIdx.y, len = kv_len_of(a, b);
  int g = blockIdx.x;
  if (kv_start != nullptr) {  // only blocks that hold keys [kv_start, kv_len)
    const int start = max(kv_start[b], 0);
    g += start / a.block;
    if (start >= len || g * a.block >= len) return;
  }
  const int cnt = min(a.block, len - g * a.block);
  const int c = threadIdx.x % kCols * V, r0 = threadIdx.x / kCols;
  double acc[V] = {};
  const T* row = static_cast<const T*>(a.k.p) + b * a.k.sb + h * a.k.sh + static_cast<long long>(g) * a.block * a.k.sn + c;
#pragma unroll 4
  for (int r = r0; r < cnt; r += kRows) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + r * a.k.sn);
    const T* x = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += static_cast<double>(to_f32<T>(x[i]));
  }
#pragma unroll
  for (int i = 0; i < V; ++i) part[r0][c + i] = acc[i];
  __syncthreads();
  if (threadIdx.x < D) {
    double s = 0.0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) s += part[r][threadIdx.x];
    means[((static_cast<size_t>(b) * a.Hk + h) * a.nb + g) * D + threadIdx.x] =
        cnt > 0 ? static_cast<float>(s / cnt) : 0.f;
  }
}

// Order of a candidate block's score as an unsigned key: forced blocks above every number,
// a NaN below; 0 is no candidate.
__device__ __forceinline__ unsigned long long score_key(double s) {
  if (s != s) return 1ull;
  if (s == 0.0) s = 0.0;  // -0 ties with +0
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(s));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

// One warp per (batch, key head, token): every block's score in 64 bits, then the `top`
// largest keys by binary search over the key's bits, ties to the lower block.
template <typename T, int D>
__global__ void __launch_bounds__(256) select_exact_kernel(const SelArgs a, int* __restrict__ sel) {
  extern __shared__ unsigned long long keys_smem[];
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long w = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp;
  if (w >= static_cast<long long>(a.Bt) * a.Hk * a.n) return;
  unsigned long long* keys = keys_smem + static_cast<size_t>(warp) * a.nb;
  const int t = static_cast<int>(w % a.n), z = static_cast<int>(w / a.n), b = z / a.Hk, kh = z % a.Hk;
  int* out = sel + w * a.top;
  double q[C] = {};
  for (int h = 0; h < a.group; ++h) {
    const T* p = static_cast<const T*>(a.q.p) + b * a.q.sb + (kh * a.group + h) * a.q.sh + t * a.q.sn + lane * C;
#pragma unroll
    for (int c = 0; c < C; ++c) q[c] += static_cast<double>(to_f32<T>(p[c]));
  }
  const int len = kv_len_of(a, b), pos = q_start_of(a, b) + t;
  int last = len - 1;
  if (a.causal) last = min(last, pos);
  const int cand = last < 0 ? 0 : last / a.block + 1;  // candidates are blocks [0, cand)
  const int mine = a.causal && pos >= 0 ? pos / a.block : -1;
  const float* m = a.means + (static_cast<size_t>(z) * a.nb) * D + lane * C;
  for (int g = 0; g < cand; ++g) {
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) s = fma(q[c], static_cast<double>(m[static_cast<size_t>(g) * D + c]), s);
    s = warp_sum_d(s);
    const bool forced = g < a.n_first || (a.causal && g <= mine && g > mine - a.n_local);
    if (lane == 0) {
      if (!forced && s != s) record_error(a.status, kErrNonFinite);
      keys[g] = forced ? ~0ull : score_key(s);
    }
  }
  __syncwarp();
  const int want = min(a.top, cand);
  // largest key value v with at least `want` keys >= v
  unsigned long long v = 0;
  if (want < cand) {
    for (int bit = 63; bit >= 0; --bit) {
      const unsigned long long tryv = v | (1ull << bit);
      int c = 0;
      for (int g = lane; g < cand; g += 32) c += keys[g] >= tryv;
      if (__reduce_add_sync(0xffffffffu, c) >= want) v = tryv;
    }
  }
  int above = 0;
  for (int g = lane; g < cand; g += 32) above += keys[g] > v;
  int ties = want - __reduce_add_sync(0xffffffffu, above);  // keys equal to v that are taken
  int n_out = 0;
  for (int g0 = 0; g0 < cand; g0 += 32) {
    const int g = g0 + lane;
    const bool eq = g < cand && keys[g] == v, gt = g < cand && keys[g] > v;
    const unsigned eqm = __ballot_sync(0xffffffffu, eq);
    const bool take = gt || (eq && __popc(eqm & ((1u << lane) - 1u)) < ties);
    const unsigned tm = __ballot_sync(0xffffffffu, take);
    if (take) out[n_out + __popc(tm & ((1u << lane) - 1u))] = g;
    n_out += __popc(tm);
    ties -= min(ties, __popc(eqm));
  }
  for (int j = n_out + lane; j < a.top; j += 32) out[j] = -1;
}

template <typename T, int D>
cudaError_t select_blocks(const SelArgs& a, int* sel, cudaStream_t st) {
  // eight warps' keys in shared memory while they fit, fewer warps past that
  int warps = 8;
  while (warps > 1 && sizeof(unsigned long long) * a.nb * warps > 96 * 1024) warps /= 2;
  const size_t smem = sizeof(unsigned long long) * a.nb * warps;
  cudaError_t e = cudaFuncSetAttribute(select_exact_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(a.Bt) * a.Hk * a.n;
  select_exact_kernel<T, D><<<static_cast<unsigned>((rows + warps - 1) / warps), 32 * warps, smem, st>>>(a, sel);
  return counted(cudaGetLastError(), 1);
}

}  // namespace

cudaError_t launch_key_means(const SelArgs& a, const int* kv_start, int max_new, float* means, cudaStream_t st) {
  const int blocks = kv_start == nullptr ? a.nb : min(a.nb, (max_new + a.block - 2) / a.block + 1);
  if (a.Hk > 65535 || a.Bt > 65535) return cudaErrorInvalidValue;
  const dim3 grid(blocks, a.Hk, a.Bt);
  if (a.f32)
    a.d == 128 ? key_means_kernel<float, 128><<<grid, 256, 0, st>>>(a, kv_start, means)
               : key_means_kernel<float, 64><<<grid, 256, 0, st>>>(a, kv_start, means);
  else
    a.d == 128 ? key_means_kernel<__nv_bfloat16, 128><<<grid, 256, 0, st>>>(a, kv_start, means)
               : key_means_kernel<__nv_bfloat16, 64><<<grid, 256, 0, st>>>(a, kv_start, means);
  return counted(cudaGetLastError(), 1);
}

cudaError_t launch_select(const SelArgs& a, int* sel, cudaStream_t st) {
  if (a.f32) return a.d == 128 ? select_blocks<float, 128>(a, sel, st) : select_blocks<float, 64>(a, sel, st);
  return a.d == 128 ? select_blocks<__nv_bfloat16, 128>(a, sel, st) : select_blocks<__nv_bfloat16, 64>(a, sel, st);
}

}  // namespace spr
