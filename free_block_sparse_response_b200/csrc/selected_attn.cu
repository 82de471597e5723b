// Selected-block attention and its backward pass in fp32 (on the fp32 pipes), and the passes that
// join their partial rows.
//
// Mathematics: query row i attends to the keys of its selected blocks.  With block g's
//   m_ig = max_j s_ij,  l_ig = sum_j exp(s_ij - m_ig),  o_ig = sum_j exp(s_ij - m_ig) v_j
// over the keys j of block g that i may see, the row is joined from its blocks' parts:
//   m = max_g m_ig,  l = sum_g exp(m_ig - m) l_ig,  O_i = sum_g exp(m_ig - m) o_ig / l,
//   lse_i = m + log l.
// Backward, with P_ij = exp(s_ij - lse_i) and delta_i = sum_c O_ic dO_ic:
//   dV_j = sum_i P_ij dO_i,  dS_ij = P_ij (dO_i . v_j - delta_i) tau,
//   dQ_i = sum_j dS_ij k_j,  dK_j = sum_i dS_ij q_i;
// a work unit (one block, some of its queries) forms its part of dK and dV in registers and
// one partial dQ row per query; split blocks' parts and the dQ rows are summed in order.
#include <cuda_runtime.h>

#include "common.cuh"
#include "selected.cuh"
#include "selected_tc.cuh"

namespace spr {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T>
__device__ __forceinline__ float4 load4(const T* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v) {
  *reinterpret_cast<float4*>(p) = v;
}

template <typename T>
__device__ __forceinline__ T* row_ptr(const View& v, int b, int h, int t) {
  return static_cast<T*>(v.p) + b * v.sb + h * v.sh + t * v.sn;
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
__device__ __forceinline__ void axpy4(float s, float4 x, float4& y) {
  y.x = fmaf(s, x.x, y.x), y.y = fmaf(s, x.y, y.y), y.z = fmaf(s, x.z, y.z), y.w = fmaf(s, x.w, y.w);
}

// Rows of a key block in shared memory (row stride D + 4 floats); keys at or past the
// batch element's length are zero and never read.
template <typename T, int D, int B, int THREADS>
__device__ __forceinline__ void load_block(float* dst, const View& v, int b, int h, int j0, int len) {
  for (int i = threadIdx.x; i < B * (D / 4); i += THREADS) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j0 + r < len) x = load4<T>(row_ptr<const T>(v, b, h, j0 + r) + c);
    *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = x;
  }
}

// ------------------------------------------------------------------------------ rows formed again

// A query row straight from the inputs in fp32:
//   sum_j P_j v_j, or (GRAD) sum_j dS_j k_j, over the visible keys of its selected blocks.
// Keys that the row does not see are not touched, so that whatever they hold (a NaN times a weight of
// 0 is a NaN) does not reach it.  D / V lanes take a key, V columns each; warp `warp` of `warps` takes
// its share of the keys, kBatch at a time in flight, and x gets its sums of columns V (lane % (D / V)) ..
template <typename T, int D, bool GRAD>
__device__ __noinline__ void sum_again(const SelArgs& a, int z, int t, int h, float lse2, float delta, int warp, int warps,
                                       float* x) {
  constexpr int V = 16 / sizeof(T), L = D / V, kKeys = 32 / L, kBatch = 4;
  const int lane = threadIdx.x & 31, ch = lane % L, b = z / a.Hk, kh = z % a.Hk, hq = kh * a.group + h;
  auto piece = [&](const View& v, int hv, int j) { return *reinterpret_cast<const uint4*>(row_ptr<const T>(v, b, hv, j) + ch * V); };
  auto at = [](const uint4& v, int c) { return to_f32<T>(reinterpret_cast<const T*>(&v)[c]); };
  const uint4 q = piece(a.q, hq, t), go = GRAD ? piece(a.go, hq, t) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int c = 0; c < V; ++c) x[c] = 0.f;
  const size_t slots = (static_cast<size_t>(z) * a.n + t) * a.top;
  const int last = a.causal ? min(kv_len_of(a, b) - 1, q_start_of(a, b) + t) : kv_len_of(a, b) - 1;
  const int keys = lse2 == -__builtin_huge_valf() ? 0 : a.top * a.block;  // (a zero row of the forward pass)
  const float scale2 = a.scale * kLog2e;
  for (int i0 = warp * kKeys * kBatch; i0 < keys; i0 += warps * kKeys * kBatch) {
    uint4 k[kBatch], v[kBatch];
    bool live[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kKeys + lane / L, s = i / a.block;
      const int j = i < keys && a.inv[slots + s] >= 0 ? a.sel[slots + s] * a.block + i % a.block : last + 1;
      live[u] = j <= last;
      k[u] = live[u] ? piece(a.k, kh, j) : make_uint4(0, 0, 0, 0);
      v[u] = live[u] ? piece(a.v, kh, j) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      float s = 0.f, dp = 0.f;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        s = fmaf(at(q, c), at(k[u], c), s);
        if (GRAD) dp = fmaf(at(go, c), at(v[u], c), dp);
      }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        if (GRAD) dp += __shfl_xor_sync(0xffffffffu, dp, o);
      }
      if (!live[u]) continue;
      const float p = exp2f(fmaf(s, scale2, -lse2)), w = GRAD ? p * (dp - delta) * a.scale : p;
#pragma unroll
      for (int c = 0; c < V; ++c) x[c] = fmaf(w, GRAD ? at(k[u], c) : at(v[u], c), x[c]);
    }
  }
#pragma unroll
  for (int o = L; o < 32; o <<= 1)
#pragma unroll
    for (int c = 0; c < V; ++c) x[c] += __shfl_xor_sync(0xffffffffu, x[c], o);
}

// fp32: the NaNs of a row (columns D / 32 lane ..) in place of which it has a value, by the row's warp.
template <int D, bool GRAD>
__device__ __forceinline__ void mend_row(const SelArgs& a, int z, int t, int h, float lse2, float delta, float (&y)[D / 32]) {
  bool open = false;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) open = open || y[c] != y[c];
  if (!__any_sync(0xffffffffu, open)) return;
  const int lane = threadIdx.x & 31;
  float x[4];
  sum_again<float, D, GRAD>(a, z, t, h, lse2, delta, 0, 1, x);
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float w = x[c];
    if (D == 64) {  // four columns a lane there, two here
      const float u = __shfl_sync(0xffffffffu, x[c], lane / 2), v = __shfl_sync(0xffffffffu, x[c + 2], lane / 2);
      w = lane & 1 ? v : u;
    }
    if (y[c] != y[c]) y[c] = w;
  }
}

// bf16: the rows that the joins listed, a CTA each: rows of blocks that are wide (ranges_kernel) with a
// value that fp16 cannot hold, hidden NaNs and infinities among them.  (In the
// joins themselves, as in fp32, this would take twice their registers, and they live from the warps
// under way.)
constexpr int kMendWarps = 16;

template <int D, bool GRAD>
__global__ void __launch_bounds__(32 * kMendWarps) mend_kernel(const __grid_constant__ SelArgs a) {
  __shared__ float s_x[kMendWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = __ldg(a.slow);
  for (int i = blockIdx.x; i < rows; i += gridDim.x) {
    const int row = __ldg(a.slow + 1 + i), t = row % a.n, hq = row / a.n % a.Hq, b = row / a.n / a.Hq;
    const float lse = a.lse[row];
    if (lse != lse) continue;  // a NaN that the row sees
    float x[8];
    sum_again<__nv_bfloat16, D, GRAD>(a, b * a.Hk + hq / a.group, t, hq % a.group, lse * kLog2e, GRAD ? a.delta[row] : 0.f, warp,
                                      kMendWarps, x);
    if (lane < D / 8) {
#pragma unroll
      for (int c = 0; c < 8; ++c) s_x[warp][lane * 8 + c] = x[c];
    }
    __syncthreads();
    if (threadIdx.x < D) {
      const int c = threadIdx.x;
      float y = 0.f;
#pragma unroll
      for (int w = 0; w < kMendWarps; ++w) y += s_x[w][c];
      __nv_bfloat16* o = row_ptr<__nv_bfloat16>(GRAD ? a.gq : a.o, b, hq, t) + c;
      if (__hisnan(*o)) {
        *o = __float2bfloat16_rn(y);
        if (!GRAD && a.rest != nullptr)
          a.rest[static_cast<size_t>(row) * D + c] = __float2bfloat16_rn(y - __bfloat162float(*o));
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------ forward

constexpr int kFwdThreads = 128, kFwdRows = 64;

template <int D, int B>
constexpr size_t fwd_smem() {
  return sizeof(float) * (kFwdRows * (D + 4) + 2 * B * (D + 4) + kFwdRows * (B + 4));
}

// One CTA per work unit: K and V once, then 64 query rows at a time.  Thread (rg, cg) holds
// rows 8 rg .. + 7 and keys cg + 16 i of S, then columns 4 cg + 64 i of O.
template <typename T, int D, int B>
__global__ void __launch_bounds__(kFwdThreads) forward_kernel(const SelArgs a, int first, int count) {
  extern __shared__ __align__(16) float smem[];
  const int ci = blockIdx.x % count, u = blockIdx.x / count, region = first + ci;
  const Unit un = a.units[static_cast<size_t>(region) * a.unit_cap + u];
  if (un.rows == 0) return;
  float *sq = smem, *sk = sq + kFwdRows * (D + 4), *sv = sk + B * (D + 4), *sp = sv + B * (D + 4);
  const int z = region / a.slices, b = z / a.Hk, kh = z % a.Hk;
  const int len = kv_len_of(a, b), j0 = un.g * B;
  const int qs = q_start_of(a, b);
  const size_t cap = static_cast<size_t>(a.slice) * a.top;
  const int* list = a.list + region * cap + un.off;
  const size_t out0 = (ci * cap + un.off) * a.group;  // partial row of the block's row 0
  load_block<T, D, B, kFwdThreads>(sk, a.k, b, kh, j0, len);
  load_block<T, D, B, kFwdThreads>(sv, a.v, b, kh, j0, len);
  const int rg = threadIdx.x / 16, cg = threadIdx.x % 16;
  const float scale2 = a.scale * kLog2e;
  for (int base = un.r0; base < un.r0 + un.rows; base += kFwdRows) {
    const int nrows = min(kFwdRows, un.r0 + un.rows - base);
    __syncthreads();
    for (int i = threadIdx.x; i < kFwdRows * (D / 4); i += kFwdThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nrows) {
        const int row = base + r;
        x = load4<T>(row_ptr<const T>(a.q, b, kh * a.group + row % a.group, list[row / a.group]) + c);
      }
      *reinterpret_cast<float4*>(sq + r * (D + 4) + c) = x;
    }
    __syncthreads();
    float s[8][B / 16];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < B / 16; ++j) s[i][j] = 0.f;
#pragma unroll 1
    for (int c = 0; c < D; c += 4) {
      float4 q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = *reinterpret_cast<const float4*>(sq + (rg * 8 + i) * (D + 4) + c);
#pragma unroll
      for (int j = 0; j < B / 16; ++j) {
        const float4 k = *reinterpret_cast<const float4*>(sk + (cg + 16 * j) * (D + 4) + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i][j] = dot4(q[i], k, s[i][j]);
      }
    }
    float2 stat[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = rg * 8 + i;
      int last = len - 1;  // last key the row may see
      if (a.causal && r < nrows) last = min(last, qs + list[(base + r) / a.group]);
      float m = -__builtin_huge_valf();
#pragma unroll
      for (int j = 0; j < B / 16; ++j) {
        s[i][j] = j0 + cg + 16 * j <= last ? s[i][j] * scale2 : -__builtin_huge_valf();
        m = fmaxf(m, s[i][j]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float ms = m == -__builtin_huge_valf() ? 0.f : m;
      float l = 0.f;
#pragma unroll
      for (int j = 0; j < B / 16; ++j) {
        const float p = exp2f(s[i][j] - ms);
        l += p;
        sp[r * (B + 4) + cg + 16 * j] = p;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      stat[i] = make_float2(m, l);
    }
    __syncwarp();
    float4 acc[8][D / 64];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int c = 0; c < D / 64; ++c) acc[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int j = 0; j < B; j += 4) {
      float4 p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = *reinterpret_cast<const float4*>(sp + (rg * 8 + i) * (B + 4) + j);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(sv + (j + jj) * (D + 4) + cg * 4 + 64 * c);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            axpy4(jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w, v, acc[i][c]);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = rg * 8 + i;
      if (r >= nrows) continue;
      const size_t row = out0 + base + r;
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        *reinterpret_cast<float4*>(a.part + row * D + cg * 4 + 64 * c) = acc[i][c];
      if (cg == 0) a.ml[row] = stat[i];
    }
  }
}

// One warp per query row: joins the row's parts.  Lane s holds slot s's statistics; then
// the lanes cover the row's columns and walk the parts.
template <typename T, int D>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ SelArgs a, int first, int count) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int per = a.slice * a.group;
  const int ci = static_cast<int>(w / per);
  if (ci >= count) return;
  const int region = first + ci, z = region / a.slices, s = region % a.slices;
  const int lr = static_cast<int>(w % per), t = s * a.slice + lr / a.group, h = lr % a.group;
  if (t >= a.n) return;
  const int b = z / a.Hk, kh = z % a.Hk;
  const int* inv = a.inv + (static_cast<size_t>(z) * a.n + t) * a.top;
  const size_t cap = static_cast<size_t>(a.slice) * a.top;
  float m = -__builtin_huge_valf();
  for (int j = lane; j < a.top; j += 32) {
    const int e = inv[j];
    if (e >= 0) m = fmaxf(m, a.ml[(ci * cap + e) * a.group + h].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ms = m == -__builtin_huge_valf() ? 0.f : m;
  float l = 0.f, acc[C] = {};
  for (int j0 = 0; j0 < a.top; j0 += 32) {
    const int e = j0 + lane < a.top ? inv[j0 + lane] : -1;
    float f = 0.f;
    long long row = 0;
    if (e >= 0) {
      row = (ci * cap + e) * a.group + h;
      const float2 st = a.ml[row];
      f = exp2f(st.x - ms);
      l = fmaf(f, st.y, l);
    }
    const int lim = min(32, a.top - j0);
    for (int j = 0; j < lim; ++j) {
      const float fj = __shfl_sync(0xffffffffu, f, j);
      const long long rj = __shfl_sync(0xffffffffu, row, j);
      const int ej = __shfl_sync(0xffffffffu, e, j);
      if (ej < 0) continue;
      const float* p = a.part + rj * D + lane * C;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = fmaf(fj, p[c], acc[c]);
    }
  }
  l = warp_sum(l);
  const float inv_l = l > 0.f ? 1.f / l : l == l ? 0.f : l;
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] *= inv_l;
  if (l == l) mend_row<D, false>(a, z, t, h, ms + log2f(l), 0.f, acc);
  T* o = row_ptr<T>(a.o, b, kh * a.group + h, t) + lane * C;
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = from_f32<T>(acc[c]);
  if (lane == 0)
    a.lse[(static_cast<size_t>(b) * a.Hq + kh * a.group + h) * a.n + t] =
        l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -__builtin_huge_valf();
}

// ------------------------------------------------------------------------------ backward

// delta_i = sum_c O_ic dO_ic: D / V lanes a row with 16-byte loads, four rows under way per lane.
// Its error is common to a row's dS, so it does not average out over the keys as the rounding of dS
// does: a bf16 O alone makes it the largest error of dQ (16 heads x 32,760 tokens, 8 blocks: 2.9e-3
// of dQ's norm, 1.7e-3 with REST, what O's rounding left off; dQ's own rounding is 1.7e-3).
template <typename T, int D, bool REST>
__global__ void __launch_bounds__(256) delta_kernel(const SelArgs a) {
  constexpr int V = 16 / sizeof(T), kPer = D / V, kRowsW = 32 / kPer, kBatch = 4;
  const int lane = threadIdx.x & 31, ch = lane % kPer;
  const long long rows = static_cast<long long>(a.Bt) * a.Hq * a.n;
  const long long w0 = (static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * kRowsW * kBatch + lane / kPer;
  uint4 o[kBatch], g[kBatch], r[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const long long w = min(w0 + i * kRowsW, rows - 1);
    const int t = static_cast<int>(w % a.n), h = static_cast<int>(w / a.n % a.Hq), b = static_cast<int>(w / a.n / a.Hq);
    o[i] = *reinterpret_cast<const uint4*>(row_ptr<const T>(a.o, b, h, t) + ch * V);
    g[i] = *reinterpret_cast<const uint4*>(row_ptr<const T>(a.go, b, h, t) + ch * V);
    if (REST) r[i] = *reinterpret_cast<const uint4*>(a.rest + static_cast<size_t>(w) * D + ch * V);
  }
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c)
      s = fmaf(to_f32<T>(reinterpret_cast<const T*>(&o[i])[c]), to_f32<T>(reinterpret_cast<const T*>(&g[i])[c]), s);
    if (REST) {
#pragma unroll
      for (int c = 0; c < V; ++c)
        s = fmaf(to_f32<T>(reinterpret_cast<const T*>(&r[i])[c]), to_f32<T>(reinterpret_cast<const T*>(&g[i])[c]), s);
    }
#pragma unroll
    for (int k = kPer / 2; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (ch == 0 && w0 + i * kRowsW < rows) a.delta[w0 + i * kRowsW] = s;
  }
}

// Four columns of a key's dK and dV: written, or added to the sums of the head's earlier slices.
template <typename T, int D>
__device__ __forceinline__ void store_gradients(const SelArgs& a, int b, int kh, int j, int col, float4 dk, float4 dv) {
  if (a.acc == nullptr) {
    store4<T>(row_ptr<T>(a.gk, b, kh, j) + col, dk);
    store4<T>(row_ptr<T>(a.gv, b, kh, j) + col, dv);
  } else {
    float* v = a.acc + static_cast<size_t>(j) * D + col;
    float* k = v + static_cast<size_t>(a.nk) * D;
    float4 x = *reinterpret_cast<const float4*>(k), y = *reinterpret_cast<const float4*>(v);
    axpy4(1.f, dk, x);
    axpy4(1.f, dv, y);
    *reinterpret_cast<float4*>(k) = x;
    *reinterpret_cast<float4*>(v) = y;
  }
}

// The sums over a head's slices, rounded once.  One thread for two columns of a key.
template <typename T>
__global__ void __launch_bounds__(256) slice_sums_kernel(const SelArgs a, int z) {
  const long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * 2;
  if (i >= static_cast<long long>(a.nk) * a.d) return;
  const int j = static_cast<int>(i / a.d), c = static_cast<int>(i % a.d), b = z / a.Hk, kh = z % a.Hk;
  const float2 dv = *reinterpret_cast<const float2*>(a.acc + i);
  const float2 dk = *reinterpret_cast<const float2*>(a.acc + static_cast<size_t>(a.nk) * a.d + i);
  T *v = row_ptr<T>(a.gv, b, kh, j) + c, *k = row_ptr<T>(a.gk, b, kh, j) + c;
  v[0] = from_f32<T>(dv.x), v[1] = from_f32<T>(dv.y);
  k[0] = from_f32<T>(dk.x), k[1] = from_f32<T>(dk.y);
}

constexpr int kBwdThreads = 256, kBwdRows = 32;

template <int D, int B>
constexpr size_t bwd_smem() {
  return sizeof(float) * (2 * B * (D + 4) + 2 * kBwdRows * (D + 4) + 2 * kBwdRows * (B + 4));
}

template <typename T, int D, int B>
__global__ void __launch_bounds__(kBwdThreads) backward_kernel(const SelArgs a, int first, int count) {
  extern __shared__ __align__(16) float smem[];
  const int ci = blockIdx.x % count, u = blockIdx.x / count, region = first + ci;
  const Unit un = a.units[static_cast<size_t>(region) * a.unit_cap + u];
  if (un.rows == 0) return;
  float *sk = smem, *sv = sk + B * (D + 4), *sq = sv + B * (D + 4), *sg = sq + kBwdRows * (D + 4),
        *sp = sg + kBwdRows * (D + 4), *sd = sp + kBwdRows * (B + 4);
  const int z = region / a.slices, b = z / a.Hk, kh = z % a.Hk;
  const int len = kv_len_of(a, b), j0 = un.g * B;
  const int qs = q_start_of(a, b);
  const size_t cap = static_cast<size_t>(a.slice) * a.top;
  const int* list = a.list + region * cap + un.off;
  const size_t out0 = (ci * cap + un.off) * a.group;
  load_block<T, D, B, kBwdThreads>(sk, a.k, b, kh, j0, len);
  load_block<T, D, B, kBwdThreads>(sv, a.v, b, kh, j0, len);
  const int rg = threadIdx.x / 16, cg = threadIdx.x % 16;
  const float scale2 = a.scale * kLog2e;
  // dK and dV of keys rg + 16 i, columns 4 cg + 64 c
  float4 gk[B / 16][D / 64], gv[B / 16][D / 64];
#pragma unroll
  for (int i = 0; i < B / 16; ++i)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) gk[i][c] = gv[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = un.r0; base < un.r0 + un.rows; base += kBwdRows) {
    const int nrows = min(kBwdRows, un.r0 + un.rows - base);
    __syncthreads();
    for (int i = threadIdx.x; i < kBwdRows * (D / 4); i += kBwdThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (r < nrows) {
        const int row = base + r, h = kh * a.group + row % a.group, t = list[row / a.group];
        x = load4<T>(row_ptr<const T>(a.q, b, h, t) + c);
        y = load4<T>(row_ptr<const T>(a.go, b, h, t) + c);
      }
      *reinterpret_cast<float4*>(sq + r * (D + 4) + c) = x;
      *reinterpret_cast<float4*>(sg + r * (D + 4) + c) = y;
    }
    __syncthreads();
    float s[2][B / 16], dp[2][B / 16];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < B / 16; ++j) s[i][j] = dp[i][j] = 0.f;
#pragma unroll 2
    for (int c = 0; c < D; c += 4) {
      float4 q[2], g[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        q[i] = *reinterpret_cast<const float4*>(sq + (rg * 2 + i) * (D + 4) + c);
        g[i] = *reinterpret_cast<const float4*>(sg + (rg * 2 + i) * (D + 4) + c);
      }
#pragma unroll
      for (int j = 0; j < B / 16; ++j) {
        const float4 k = *reinterpret_cast<const float4*>(sk + (cg + 16 * j) * (D + 4) + c);
        const float4 v = *reinterpret_cast<const float4*>(sv + (cg + 16 * j) * (D + 4) + c);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          s[i][j] = dot4(q[i], k, s[i][j]);
          dp[i][j] = dot4(g[i], v, dp[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = rg * 2 + i;
      int last = -1;
      float lse2 = 0.f, dl = 0.f;
      if (r < nrows) {
        const int row = base + r, h = kh * a.group + row % a.group, t = list[row / a.group];
        last = a.causal ? min(len - 1, qs + t) : len - 1;
        const size_t at = (static_cast<size_t>(b) * a.Hq + h) * a.n + t;
        lse2 = a.lse[at] * kLog2e;
        dl = a.delta[at];
        if (lse2 == -__builtin_huge_valf()) last = -1;  // a zero row of the forward pass
      }
#pragma unroll
      for (int j = 0; j < B / 16; ++j) {
        const bool live = j0 + cg + 16 * j <= last;
        const float p = live ? exp2f(fmaf(s[i][j], scale2, -lse2)) : 0.f;
        sp[r * (B + 4) + cg + 16 * j] = p;
        sd[r * (B + 4) + cg + 16 * j] = live ? p * (dp[i][j] - dl) * a.scale : 0.f;
      }
    }
    __syncthreads();
    // partial dQ: rows 2 rg + i, columns 4 cg + 64 c
    float4 gq[2][D / 64];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < D / 64; ++c) gq[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int j = 0; j < B; ++j) {
      const float d0 = sd[(rg * 2) * (B + 4) + j], d1 = sd[(rg * 2 + 1) * (B + 4) + j];
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const float4 k = *reinterpret_cast<const float4*>(sk + j * (D + 4) + cg * 4 + 64 * c);
        axpy4(d0, k, gq[0][c]);
        axpy4(d1, k, gq[1][c]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (rg * 2 + i < nrows) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          *reinterpret_cast<float4*>(a.part + (out0 + base + rg * 2 + i) * D + cg * 4 + 64 * c) = gq[i][c];
      }
    // dV += P^T dO, dK += dS^T Q
#pragma unroll 1
    for (int r = 0; r < nrows; ++r) {
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const float4 q = *reinterpret_cast<const float4*>(sq + r * (D + 4) + cg * 4 + 64 * c);
        const float4 g = *reinterpret_cast<const float4*>(sg + r * (D + 4) + cg * 4 + 64 * c);
#pragma unroll
        for (int i = 0; i < B / 16; ++i) {
          axpy4(sp[r * (B + 4) + rg + 16 * i], g, gv[i][c]);
          axpy4(sd[r * (B + 4) + rg + 16 * i], q, gk[i][c]);
        }
      }
    }
  }
  // a block with one unit writes its gradients; a split block's sums wait for their join
  const int4 bk = a.blk[static_cast<size_t>(region) * a.nb + un.g];
  const bool split = bk.x > 1;
  float* seg = a.seg + (static_cast<size_t>(ci) * a.seg_cap + bk.y + un.r0 / a.unit_rows) * 2 * B * D;
#pragma unroll
  for (int i = 0; i < B / 16; ++i)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const int j = rg + 16 * i, col = cg * 4 + 64 * c;
      if (split) {
        *reinterpret_cast<float4*>(seg + j * D + col) = gk[i][c];
        *reinterpret_cast<float4*>(seg + B * D + j * D + col) = gv[i][c];
      } else if (j0 + j < a.nk) {
        store_gradients<T, D>(a, b, kh, j0 + j, col, gk[i][c], gv[i][c]);
      }
    }
}

// dK and dV of split blocks (segment sums in order) and of blocks that no query selected.
template <typename T, int D>
__global__ void __launch_bounds__(256) join_kv_kernel(const SelArgs a, int first) {
  const int g = blockIdx.x, region = first + blockIdx.y, z = region / a.slices;
  const int b = z / a.Hk, kh = z % a.Hk;
  const int4 bk = a.blk[static_cast<size_t>(region) * a.nb + g];
  if (bk.x == 1 || (bk.x == 0 && a.acc != nullptr)) return;
  const size_t tile = static_cast<size_t>(a.block) * D;
  const float* seg = a.seg + (static_cast<size_t>(blockIdx.y) * a.seg_cap + bk.y) * 2 * tile;
  for (int i = threadIdx.x * 4; i < a.block * D; i += 1024) {
    const int j = g * a.block + i / D;
    if (j >= a.nk) break;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    for (int s = 0; s < bk.x; ++s) {
      axpy4(1.f, *reinterpret_cast<const float4*>(seg + s * 2 * tile + i), x);
      axpy4(1.f, *reinterpret_cast<const float4*>(seg + s * 2 * tile + tile + i), y);
    }
    store_gradients<T, D>(a, b, kh, j, i % D, x, y);
  }
}

// One warp per query row: dQ is the sum of the row's partial rows, slot by slot.
template <typename T, int D>
__global__ void __launch_bounds__(256) join_q_kernel(const __grid_constant__ SelArgs a, int first, int count) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int per = a.slice * a.group;
  const int ci = static_cast<int>(w / per);
  if (ci >= count) return;
  const int region = first + ci, z = region / a.slices, s = region % a.slices;
  const int lr = static_cast<int>(w % per), t = s * a.slice + lr / a.group, h = lr % a.group;
  if (t >= a.n) return;
  const int* inv = a.inv + (static_cast<size_t>(z) * a.n + t) * a.top;
  const size_t cap = static_cast<size_t>(a.slice) * a.top;
  float acc[C] = {};
  for (int j = 0; j < a.top; ++j) {
    const int e = inv[j];
    if (e < 0) continue;
    const float* p = a.part + ((ci * cap + e) * a.group + h) * D + lane * C;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] += p[c];
  }
  const size_t at = (static_cast<size_t>(z / a.Hk) * a.Hq + z % a.Hk * a.group + h) * a.n + t;
  if (a.lse[at] == a.lse[at]) mend_row<D, true>(a, z, t, h, a.lse[at] * kLog2e, a.delta[at], acc);
  T* o = row_ptr<T>(a.gq, z / a.Hk, z % a.Hk * a.group + h, t) + lane * C;
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = from_f32<T>(acc[c]);
}

template <typename T, int D, int B>
cudaError_t forward(const SelArgs& a, int first, int count, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(forward_kernel<T, D, B>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(fwd_smem<D, B>()));
  if (e != cudaSuccess) return e;
  forward_kernel<T, D, B><<<count * a.unit_cap, kFwdThreads, fwd_smem<D, B>(), st>>>(a, first, count);
  if ((e = counted(cudaGetLastError(), 1)) != cudaSuccess) return e;
  const long long rows = static_cast<long long>(count) * a.slice * a.group;
  join_kernel<T, D><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, st>>>(a, first, count);
  return counted(cudaGetLastError(), 1);
}

template <typename T, int D, int B>
cudaError_t backward(const SelArgs& a, int first, int count, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(backward_kernel<T, D, B>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(bwd_smem<D, B>()));
  if (e != cudaSuccess) return e;
  backward_kernel<T, D, B><<<count * a.unit_cap, kBwdThreads, bwd_smem<D, B>(), st>>>(a, first, count);
  if ((e = counted(cudaGetLastError(), 1)) != cudaSuccess) return e;
  join_kv_kernel<T, D><<<dim3(a.nb, count), 256, 0, st>>>(a, first);
  if ((e = counted(cudaGetLastError(), 1)) != cudaSuccess) return e;
  const long long rows = static_cast<long long>(count) * a.slice * a.group;
  join_q_kernel<T, D><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, st>>>(a, first, count);
  return counted(cudaGetLastError(), 1);
}

template <typename T, bool REST>
cudaError_t delta(const SelArgs& a, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.Bt) * a.Hq * a.n;
  const int per_cta = 8 * 4 * (32 / (a.d * static_cast<int>(sizeof(T)) / 16));
  const unsigned grid = static_cast<unsigned>((rows + per_cta - 1) / per_cta);
  if (a.d == 128)
    delta_kernel<T, 128, REST><<<grid, 256, 0, st>>>(a);
  else
    delta_kernel<T, 64, REST><<<grid, 256, 0, st>>>(a);
  return counted(cudaGetLastError(), 1);
}

}  // namespace

cudaError_t launch_selected_forward(const SelArgs& a, int first, int count, cudaStream_t st) {
  if (!a.f32) return launch_selected_forward_tc(a, first, count, st);
  if (a.d == 128)
    return a.block == 128 ? forward<float, 128, 128>(a, first, count, st) : forward<float, 128, 64>(a, first, count, st);
  return a.block == 128 ? forward<float, 64, 128>(a, first, count, st) : forward<float, 64, 64>(a, first, count, st);
}

cudaError_t launch_selected_backward(const SelArgs& a, int first, int count, cudaStream_t st) {
  if (!a.f32) return launch_selected_backward_tc(a, first, count, st);
  if (a.d == 128)
    return a.block == 128 ? backward<float, 128, 128>(a, first, count, st) : backward<float, 128, 64>(a, first, count, st);
  return a.block == 128 ? backward<float, 64, 128>(a, first, count, st) : backward<float, 64, 64>(a, first, count, st);
}

cudaError_t launch_slice_sums(const SelArgs& a, int z, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.nk) * a.d / 2 + 255) / 256);
  a.f32 ? slice_sums_kernel<float><<<grid, 256, 0, st>>>(a, z) : slice_sums_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a, z);
  return counted(cudaGetLastError(), 1);
}

cudaError_t launch_mend(const SelArgs& a, bool grad, cudaStream_t st) {
  if (a.d == 128)
    grad ? mend_kernel<128, true><<<2 * 148, 32 * kMendWarps, 0, st>>>(a) : mend_kernel<128, false><<<2 * 148, 32 * kMendWarps, 0, st>>>(a);
  else
    grad ? mend_kernel<64, true><<<2 * 148, 32 * kMendWarps, 0, st>>>(a) : mend_kernel<64, false><<<2 * 148, 32 * kMendWarps, 0, st>>>(a);
  return counted(cudaGetLastError(), 1);
}

cudaError_t launch_delta(const SelArgs& a, cudaStream_t st) {
  if (a.f32) return delta<float, false>(a, st);
  return a.rest != nullptr ? delta<__nv_bfloat16, true>(a, st) : delta<__nv_bfloat16, false>(a, st);
}

}  // namespace spr
