// Mean key of every key block, and the blocks that each query selects.
//
// A block's mean key is summed in 64 bits (exact for bf16 keys) and rounded once to 32.  The
// score of a query and a block is (sum of the group's queries) . mean, and the selection is the
// one that scores in 64 bits give.  Prompts (select_tile_kernel) do not compute them all:
//
//   1. Scores s~ of a tile of queries from bf16 hi + lo parts on the tensor cores.  With
//      x = hi + lo + r, |lo| <= 2^-9 |x| and |r| <= 2^-18 |x|, the products hi hi + hi lo + lo hi
//      leave out at most 3 * 2^-18 sum |q||m| (single bf16 queries have no lo part: two products, 2 *
//      2^-18).  A product of 16 columns adds 17 numbers in an order and with an internal rounding
//      that are not specified; cutting each off 2^-23 below the largest, eight of them in a row lose at
//      most 8 * 17 * 2^-23, and 2^-8 of that twice in the lo products.  In all 2.8e-5, and 2^-15 is
//      3.05e-5.  The sum of a group's G queries in fp32 adds G - 1 roundings, 2^-24 each, of their
//      magnitudes: |s~ - s| <= e = (2^-15 + (G - 1) 2^-23) |q| max |m_g| (Cauchy-Schwarz; |q| is the
//      norm of the group's sum of magnitudes, the second term twice what it has to be, which covers
//      the rounding of that sum).
//   2. The k-th and (k+1)-th largest s~, a and b.  Scores above b + 2e are in and scores below
//      a - 2e are out whatever the rounding; with a - b > 2e nothing is left between.
//   3. The few blocks between are compared by their scores in 64 bits.
//
// Rows that leave more than 32 blocks open (equal keys, zero or non-finite queries) go to a
// list that select_row_kernel works off, one CTA a row, all scores in 64 bits; it also takes
// the calls of a few rows.  Bound by instructions (8 heads x 8,192 tokens: issue slots 61% busy,
// tensor pipe 6%), step 2 the larger part: 276 us for 2 x 8 key heads x 16,383 tokens in groups of
// 4, 128 blocks; the bytes would take 55.
#include <cuda_runtime.h>

#include "common.cuh"
#include "selected.cuh"
#include "warp_mma.cuh"

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

// What a token may select from: blocks [0, cand), of which the forced ones come first.
struct Scope {
  int cand, mine;
};
__device__ __forceinline__ Scope scope_of(const SelArgs& a, int b, int t) {
  const int pos = q_start_of(a, b) + t;
  int last = kv_len_of(a, b) - 1;
  if (a.causal) last = min(last, pos);
  const int sh = a.block == 128 ? 7 : 6;
  return Scope{last < 0 ? 0 : (last >> sh) + 1, a.causal && pos >= 0 ? pos >> sh : -1};
}
__device__ __forceinline__ bool is_forced(const SelArgs& a, const Scope& s, int g) {
  return g < a.n_first || (a.causal && g <= s.mine && g > s.mine - a.n_local);
}

// Writes the `want` largest of the keys of blocks [0, cand), ties to the lower block, ascending,
// then -1.  One warp; the threshold by binary search over the key's bits.
__device__ __forceinline__ void pick(const unsigned long long* keys, int cand, int top, int* out) {
  const int lane = threadIdx.x & 31;
  const int want = min(top, cand);
  // largest key value v with at least `want` keys >= v
  unsigned long long v = 0;
  int have = cand;
  for (int bit = 63; bit >= 0 && have != want; --bit) {
    const unsigned long long tryv = v | (1ull << bit);
    int c = 0;
    for (int g = lane; g < cand; g += 32) c += keys[g] >= tryv;
    c = __reduce_add_sync(0xffffffffu, c);
    if (c >= want) v = tryv, have = c;
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
  for (int j = n_out + lane; j < top; j += 32) out[j] = -1;
}

// One CTA per row (batch, key head, token): eight lanes per block form its score in 64 bits,
// then one warp picks.  Rows [0, rows), or those of `list` (its length at list[-1]).
template <typename T, int D>
__global__ void __launch_bounds__(256) select_row_kernel(const SelArgs a, int* __restrict__ sel, const int* __restrict__ list,
                                                         long long rows) {
  extern __shared__ unsigned long long keys[];  // [nb]
  constexpr int C = D / 8;
  const int part = threadIdx.x & 7, grp = threadIdx.x >> 3;
  if (list != nullptr) rows = __ldg(list - 1);
  for (long long i = blockIdx.x; i < rows; i += gridDim.x) {
    const long long w = list != nullptr ? list[i] : i;
    const int t = static_cast<int>(w % a.n), z = static_cast<int>(w / a.n), b = z / a.Hk, kh = z % a.Hk;
    const Scope sc = scope_of(a, b, t);
    double q[C] = {};
    for (int h = 0; h < a.group; ++h) {
      const T* p = static_cast<const T*>(a.q.p) + b * a.q.sb + (kh * a.group + h) * a.q.sh + t * a.q.sn;
#pragma unroll
      for (int c = 0; c < C; ++c) q[c] += static_cast<double>(to_f32<T>(p[(c / 4) * 32 + part * 4 + c % 4]));
    }
    const float* m = a.means + static_cast<size_t>(z) * a.nb * D + part * 4;
    // the means of kBatch blocks a lane under way
    constexpr int kBatch = 4;
    for (int g0 = 0; g0 < sc.cand; g0 += 32 * kBatch) {
      float4 x[kBatch][C / 4];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int g = min(g0 + 32 * k + grp, sc.cand - 1);
#pragma unroll
        for (int c = 0; c < C; c += 4)
          x[k][c / 4] = __ldg(reinterpret_cast<const float4*>(m + static_cast<size_t>(g) * D + c * 8));
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int g = g0 + 32 * k + grp;
        double s = 0.0;
#pragma unroll
        for (int c = 0; c < C; c += 4) {
          s = fma(q[c], static_cast<double>(x[k][c / 4].x), s);
          s = fma(q[c + 1], static_cast<double>(x[k][c / 4].y), s);
          s = fma(q[c + 2], static_cast<double>(x[k][c / 4].z), s);
          s = fma(q[c + 3], static_cast<double>(x[k][c / 4].w), s);
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (part == 0 && g < sc.cand) {
          const bool forced = is_forced(a, sc, g);
          if (!forced && s != s) record_error(a.status, kErrNonFinite);
          keys[g] = forced ? ~0ull : score_key(s);
        }
      }
    }
    __syncthreads();
    if (threadIdx.x < 32) pick(keys, sc.cand, a.top, sel + w * a.top);
    __syncthreads();
  }
}

__device__ __forceinline__ float warp_min_f(float x) {
  float y;
  asm("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_max_f(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// The means' hi and lo parts, [rows][2][D], and their norms squared (infinite for a NaN), for the
// tiles, which would each split them again.  Eight values a thread.
template <int D>
__global__ void __launch_bounds__(256) split_means_kernel(const SelArgs a, int rows) {
  constexpr int kPer = D / 8;
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const int row = static_cast<int>(min(i / kPer, static_cast<long long>(rows) - 1)), c = static_cast<int>(i % kPer) * 8;
  const float4* p = reinterpret_cast<const float4*>(a.means + static_cast<size_t>(row) * D + c);
  const float4 u = __ldg(p), v = __ldg(p + 1);
  const float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  uint32_t h[4], l[4];
  float y = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) split_bf16x2(x[2 * k], x[2 * k + 1], h[k], l[k]);
#pragma unroll
  for (int k = 0; k < 8; ++k) y = fmaf(x[k], x[k], y);
#pragma unroll
  for (int o = kPer / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
  if (i / kPer >= rows) return;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.mean_parts) + static_cast<size_t>(row) * 2 * D + c;
  *reinterpret_cast<uint4*>(out) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4*>(out + D) = make_uint4(l[0], l[1], l[2], l[3]);
  if (c == 0) a.mean_norm2[row] = y != y ? __builtin_huge_valf() : y;
}

// Tiles of ROWS tokens of one (batch, key head) against 64 blocks at a time.
constexpr int kMostSmem = 227 * 1024;
constexpr int kChunk = 64, kTileWarps = 16, kTileThreads = 32 * kTileWarps;

template <int D, int ROWS, bool QLO = true>
size_t tile_smem(int nb) {
  const int ld = (nb + kChunk - 1) / kChunk * kChunk + 4;
  return 2 * static_cast<size_t>(D) * ((QLO ? 2 : 1) * ROWS + 2 * kChunk) + sizeof(float) * ld * ROWS + sizeof(float) * ROWS +
         kTileWarps * 32 * sizeof(int) + 16;
}

// VPL: a lane's scores of a row in registers (32 VPL blocks and more), 0: read from shared memory.
template <typename T, int D, int ROWS, int VPL, bool QLO>
__global__ void __launch_bounds__(kTileThreads) select_tile_kernel(const SelArgs a, int* __restrict__ sel, int* __restrict__ list) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kTileQ = ROWS * D * 2, kTileM = kChunk * D * 2, kQ = QLO ? 2 * kTileQ : kTileQ;
  constexpr int RG = ROWS / 16, CG = kTileWarps / RG < 8 ? kTileWarps / RG : 8, NT = kChunk / CG / 8;  // warps over rows, columns; column tiles a warp
  constexpr float kInf = __builtin_huge_valf();
  const int ld = ceil_div(a.nb, kChunk) * kChunk + 4;
  const uint32_t sqh = smem_u32(smem), sql = sqh + kTileQ, smh = sqh + kQ, sml = smh + kTileM;
  float* score = reinterpret_cast<float*>(smem + kQ + 2 * kTileM);  // [ROWS][ld]
  float* qn = score + static_cast<size_t>(ROWS) * ld;
  int* open = reinterpret_cast<int*>(qn + ROWS);                    // [warp][32]
  int* mmax = open + kTileWarps * 32;                               // bits of the largest mean norm squared
  const int z = blockIdx.y, b = z / a.Hk, kh = z % a.Hk, t0 = blockIdx.x * ROWS;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the tile's last token sees the most
  const int most = scope_of(a, b, min(t0 + ROWS, a.n) - 1).cand;
  const __nv_bfloat16* parts = static_cast<const __nv_bfloat16*>(a.mean_parts) + static_cast<size_t>(z) * a.nb * 2 * D;
  auto load_chunk = [&](int g0) {
#pragma unroll
    for (int i = tid; i < 2 * kChunk * (D / 8); i += kTileThreads) {
      const int c = i % (2 * D / 8), r = i / (2 * D / 8);  // hi, then lo columns of a mean
      const bool in = g0 + r < a.nb;
      cp_async_16((c < D / 8 ? smh : sml) + swz<D>(r, c % (D / 8)), parts + static_cast<size_t>(in ? g0 + r : 0) * 2 * D + c * 8,
                  in ? 16 : 0);
    }
    cp_async_commit();
  };
  if (most > 0) load_chunk(0);
  if (tid == 0) *mmax = 0;
  __syncthreads();
  {
    float y = 0.f;
    for (int g = tid; g < most; g += kTileThreads) y = fmaxf(y, __ldg(a.mean_norm2 + static_cast<size_t>(z) * a.nb + g));
    y = warp_max_f(y);
    if (lane == 0 && y > 0.f) atomicMax(mmax, __float_as_int(y));  // order of nonnegative floats
  }
  // the group's query sums and the norms of their sums of magnitudes: D / 8 threads a row
#pragma unroll 1
  for (int i = tid; i < ROWS * (D / 8); i += kTileThreads) {
    const int r = i / (D / 8), c = i % (D / 8) * 8;
    float x[8] = {}, y = 0.f, mag[8] = {};
    if (t0 + r < a.n) {
      const T* p = static_cast<const T*>(a.q.p) + b * a.q.sb + static_cast<long long>(kh * a.group) * a.q.sh + (t0 + r) * a.q.sn + c;
      for (int h = 0; h < a.group; ++h, p += a.q.sh) {
        uint4 v[sizeof(T) / 2];
#pragma unroll
        for (int k = 0; k < static_cast<int>(sizeof(T) / 2); ++k) v[k] = reinterpret_cast<const uint4*>(p)[k];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float f = to_f32<T>(reinterpret_cast<const T*>(v)[k]);
          x[k] += f;
          mag[k] += fabsf(f);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) y = fmaf(mag[k], mag[k], y);
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (c == 0) qn[r] = sqrtf(y);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) split_bf16x2(x[2 * k], x[2 * k + 1], hi[k], lo[k]);
    const uint32_t at = swz<D>(r, c / 8);
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(sqh + at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
    if (QLO)
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(sql + at), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
  }
  const int rg = warp % RG, cg = warp / RG;
  for (int g0 = 0; g0 < most; g0 += kChunk) {
    cp_async_wait<0>();
    __syncthreads();
    if (cg < CG) {  // (more warps than 8-column strips)
      float hh[NT][4], rest[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) hh[n][k] = rest[n][k] = 0.f;
#pragma unroll
      for (int k2 = 0; k2 < D / 32; ++k2) {  // two 16-column steps
        uint32_t ah[2][4], al[2][4];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t at = swz<D>(rg * 16 + (lane & 15), (2 * k2 + s) * 2 + (lane >> 4));
          ldmatrix_x4(ah[s], sqh + at);
          if (QLO) ldmatrix_x4(al[s], sql + at);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t bh[4], bl[4];
          const uint32_t at = swz<D>((cg * NT + n) * 8 + (lane & 7), 4 * k2 + (lane >> 3));
          ldmatrix_x4(bh, smh + at);
          ldmatrix_x4(bl, sml + at);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            mma_bf16_16816(hh[n], ah[s], bh + 2 * s);
            mma_bf16_16816(rest[n], ah[s], bl + 2 * s);
            if (QLO) mma_bf16_16816(rest[n], al[s], bh + 2 * s);
          }
        }
      }
      float* out = score + static_cast<size_t>(rg * 16 + (lane >> 2)) * ld + g0 + cg * NT * 8 + (lane & 3) * 2;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        *reinterpret_cast<float2*>(out + n * 8) = make_float2(hh[n][0] + rest[n][0], hh[n][1] + rest[n][1]);
        *reinterpret_cast<float2*>(out + 8 * ld + n * 8) = make_float2(hh[n][2] + rest[n][2], hh[n][3] + rest[n][3]);
      }
    }
    __syncthreads();  // the chunk is read
    if (g0 + kChunk < most) load_chunk(g0 + kChunk);
  }
  __syncthreads();
  const float mnorm = sqrtf(__int_as_float(*mmax));
  const float margin = 0x1p-14f + 0x1p-22f * static_cast<float>(a.group - 1);
  int* my_open = open + warp * 32;
  for (int r = warp; r < ROWS && t0 + r < a.n; r += kTileWarps) {
    const long long w = static_cast<long long>(z) * a.n + t0 + r;
    int* out = sel + w * a.top;
    const Scope sc = scope_of(a, b, t0 + r);
    const float* sr = score + r * ld;
    const float e2 = margin * qn[r] * mnorm;  // 2e
    // forced: [0, f0) and [l0, l0 + local)
    const int f0 = min(a.n_first, sc.cand), l0 = max(f0, sc.mine - a.n_local + 1);
    const int local = max(0, min(sc.mine + 1, sc.cand) - l0), forced = f0 + local;
    const int want = min(a.top, sc.cand);
    const bool split = forced < want && want < sc.cand;  // some of the others, not all or none
    // The bound holds where nothing in it or in the products overflows or drops out of the normal range.
    // A score may be a NaN only where a norm is not finite: the row kernel looks, whether it decides or not.
    const bool odd = forced < sc.cand && !(qn[r] < kInf && mnorm < kInf);
    if (odd || (split && !(e2 < 0x1p100f && qn[r] > 0x1p-60f && mnorm > 0x1p-60f && e2 > 0x1p-90f))) {
      if (lane == 0) list[atomicAdd(list - 1, 1)] = static_cast<int>(w);
      continue;
    }
    // What to choose from: infinite where a block is in, -infinite where it is out (the finite
    // bound rules out such scores); in registers where they fit.
    auto score_of = [&](int g) {
      const bool in = g < f0 || static_cast<unsigned>(g - l0) < static_cast<unsigned>(local) || (!split && want == sc.cand);
      return g >= sc.cand ? -kInf : in ? kInf : split ? sr[g] : -kInf;
    };
    float val[VPL > 0 ? VPL : 1];
#pragma unroll
    for (int i = 0; i < VPL; ++i) val[i] = score_of(32 * i + lane);
    auto each_score = [&](auto f) {  // f(x, first block of the 32)
      if (VPL > 0) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) f(val[i], 32 * i);
      } else {
        for (int g0 = 0; g0 < sc.cand; g0 += 32) f(score_of(g0 + lane), g0);
      }
    };
    // scores above hi are in, scores in [lo, hi] open; bit j of `chosen`: the j-th open block is in
    float lo = kInf, hi = 0.f;
    unsigned chosen = 0;
    if (split) {
      auto count = [&](float v) {
        int c = 0;
        each_score([&](float x, int) { c += x >= v; });
        return __reduce_add_sync(0xffffffffu, c);
      };
      // Halving the range of the values finds a threshold between the want-th and the next one in
      // about log2(range / gap) steps (seven for 16 of 128 normal scores; over the keys' bits the
      // sign and exponent alone take nine).
      float vlo = kInf, vhi = -kInf;
      each_score([&](float x, int) {
        vhi = fmaxf(vhi, x == kInf ? vhi : x);
        vlo = fminf(vlo, x == -kInf ? vlo : x);
      });
      vlo = warp_min_f(vlo), vhi = warp_max_f(vhi);
      float v = vlo;
      int have = sc.cand;  // scores >= v
      for (int step = 0; step < 24 && have != want; ++step) {
        const float mid = 0.5f * vlo + 0.5f * vhi;
        if (!(mid > vlo && mid < vhi)) break;
        const int c = count(mid);
        if (c >= want)
          v = vlo = mid, have = c;
        else
          vhi = mid;
      }
      if (have != want) {  // (nearly) equal scores: the exact one by its bits
        uint32_t bits = 0;
        have = sc.cand;
        for (int bit = 31; bit >= 0 && have != want; --bit) {
          const uint32_t next = bits | (1u << bit);
          int c = 0;
          each_score([&](float x, int) { c += x > -kInf && float_order_key(x) >= next; });
          c = __reduce_add_sync(0xffffffffu, c);
          if (c >= want) bits = next, have = c;
        }
        v = float_from_order_key(bits);
      }
      // the want-th largest, and the one after it
      float fa = kInf, fb = -kInf;
      each_score([&](float x, int) {
        if (x >= v)
          fa = fminf(fa, x);
        else
          fb = fmaxf(fb, x);
      });
      fa = warp_min_f(fa);
      fb = have > want ? fa : warp_max_f(fb);
      hi = fb;
      if (!(fa - fb > e2)) {
        lo = fa - e2, hi = fb + e2;
        int in = 0, mid = 0;
        each_score([&](float x, int g0) {
          in += __popc(__ballot_sync(0xffffffffu, x > hi));
          const bool o = x >= lo && x <= hi;
          const unsigned om = __ballot_sync(0xffffffffu, o);
          const int at = mid + __popc(om & ((1u << lane) - 1u));
          if (o && at < 32) my_open[at] = g0 + lane;
          mid += __popc(om);
        });
        __syncwarp();
        if (mid > 32) {
          if (lane == 0) list[atomicAdd(list - 1, 1)] = static_cast<int>(w);
          continue;
        }
        // the open blocks' scores in 64 bits: lane j keeps the j-th's
        constexpr int C = D / 32;
        double q[C] = {};
        for (int h = 0; h < a.group; ++h) {
          const T* p = static_cast<const T*>(a.q.p) + b * a.q.sb + (kh * a.group + h) * a.q.sh + (t0 + r) * a.q.sn + lane * C;
#pragma unroll
          for (int c = 0; c < C; ++c) q[c] += static_cast<double>(to_f32<T>(p[c]));
        }
        double mine = 0.0;
        for (int j = 0; j < mid; ++j) {
          const float* m = a.means + (static_cast<size_t>(z) * a.nb + my_open[j]) * D + lane * C;
          double s = 0.0;
#pragma unroll
          for (int c = 0; c < C; ++c) s = fma(q[c], static_cast<double>(__ldg(m + c)), s);
          s = warp_sum_d(s);
          if (lane == j) mine = s;
        }
        int before = 0;  // open blocks that come before this lane's
        for (int j = 0; j < mid; ++j) {
          const double s = __shfl_sync(0xffffffffu, mine, j);
          before += s > mine || (s == mine && j < lane);
        }
        chosen = __ballot_sync(0xffffffffu, lane < mid && before < want - in);
        __syncwarp();
      }
    }
    int n_out = 0, n_open = 0;
    const unsigned below = (1u << lane) - 1u;
    each_score([&](float x, int g0) {
      bool take = x > hi;
      if (chosen != 0) {
        const bool o = x >= lo && x <= hi;
        const unsigned om = __ballot_sync(0xffffffffu, o);
        if (o) take = (chosen >> (n_open + __popc(om & below))) & 1u;
        n_open += __popc(om);
      }
      const unsigned tm = __ballot_sync(0xffffffffu, take);
      if (take) out[n_out + __popc(tm & below)] = g0 + lane;
      n_out += __popc(tm);
    });
    for (int j = n_out + lane; j < a.top; j += 32) out[j] = -1;
  }
}

template <typename T, int D>
cudaError_t row_select(const SelArgs& a, int* sel, const int* list, cudaStream_t st) {
  const size_t smem = sizeof(unsigned long long) * a.nb;
  const long long rows = static_cast<long long>(a.Bt) * a.Hk * a.n;
  const unsigned grid = static_cast<unsigned>(list != nullptr ? 2 * 148 : rows < 8 * 148 ? rows : 8 * 148);
  select_row_kernel<T, D><<<grid, 256, smem, st>>>(a, sel, list, rows);
  return counted(cudaGetLastError(), 1);
}

template <typename T, int D, int ROWS, int VPL, bool QLO>
cudaError_t tile_select(const SelArgs& a, int* sel, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(a.slow, 0, sizeof(int), st);
  if (e != cudaSuccess) return e;
  const int means = a.Bt * a.Hk * a.nb;
  split_means_kernel<D><<<static_cast<unsigned>((static_cast<long long>(means) * (D / 8) + 255) / 256), 256, 0, st>>>(a, means);
  if ((e = counted(cudaGetLastError(), 1)) != cudaSuccess) return e;
  const size_t smem = tile_smem<D, ROWS, QLO>(a.nb);
  auto kern = select_tile_kernel<T, D, ROWS, VPL, QLO>;
  // (the same in every call: the limit is the kernel's, and another host thread may be about to launch it)
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
  if (e != cudaSuccess) return e;
  kern<<<dim3(ceil_div(a.n, ROWS), a.Bt * a.Hk), kTileThreads, smem, st>>>(a, sel, a.slow + 1);
  if ((e = counted(cudaGetLastError(), 1)) != cudaSuccess) return e;
  return row_select<T, D>(a, sel, a.slow + 1, st);
}

template <typename T, int D, int ROWS, int VPL>
cudaError_t tile_select(const SelArgs& a, int* sel, cudaStream_t st) {
  if (sizeof(T) == 2 && a.group == 1) return tile_select<T, D, ROWS, VPL, sizeof(T) != 2>(a, sel, st);
  return tile_select<T, D, ROWS, VPL, true>(a, sel, st);
}

// Few rows: a CTA each.  Otherwise tiles, the tallest whose scores fit in shared memory (a mean is
// read once per tile); a row's scores stay in registers up to 640 blocks (20 a lane).  Measured,
// row and tile kernels in us: 512 rows of 64 blocks, groups of 4, 13 and 21, 1,024 rows 21 and 21;
// 512 rows, single heads, 10.6 and 10.6, 1,024 rows 17 and 14; 256 rows of 512 blocks 23 and 43.
template <typename T, int D>
cudaError_t select_blocks(const SelArgs& a, int* sel, cudaStream_t st) {
  if (static_cast<long long>(a.Bt) * a.Hk * a.n <= 4 * 148) return row_select<T, D>(a, sel, nullptr, st);
  if (a.nb <= 640 && tile_smem<D, 64>(a.nb) <= kMostSmem) {
    if (a.nb <= 128) return tile_select<T, D, 64, 4>(a, sel, st);
    return a.nb <= 256 ? tile_select<T, D, 64, 8>(a, sel, st) : tile_select<T, D, 64, 20>(a, sel, st);
  }
  if (tile_smem<D, 32>(a.nb) <= kMostSmem)
    return a.nb <= 640 ? tile_select<T, D, 32, 20>(a, sel, st) : tile_select<T, D, 32, 0>(a, sel, st);
  return tile_select<T, D, 16, 0>(a, sel, st);
}

}  // namespace

cudaError_t launch_key_means(const SelArgs& a, const int* kv_start, int max_new, float* means, cudaStream_t st) {
  // max_new keys from any place in a block touch at most this many
  const int blocks = kv_start == nullptr ? a.nb : min(a.nb, (min(max_new, a.nk) + a.block - 2) / a.block + 1);
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
