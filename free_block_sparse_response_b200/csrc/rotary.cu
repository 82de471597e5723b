// Rotary positions of query and key rows (sm_100a).
//
// A pair (a, b) of the rotated part of a head at position p becomes
//   f (a cos t - b sin t, b cos t + a sin t),   t = p * freq[pair],
// f the scaling's factor; the backward pass is the same map with -t.  Pairs are (2i, 2i+1)
// (interleaved) or (i, i + R/2) (half) of the R rotated dims; pair i takes its position from
// one of up to four position streams (a video grid has t, y and x).
//
// What bounds it: HBM, one read and one write of each row (~12 flops per 4 bytes).  Angles
// cost more than the rotation itself: p * freq needs 64 bits at far positions (131,072 x 1
// rad leaves 2^-7 rad in fp32), then a 32-bit sincos of the reduced angle.  So a thread
// owns one 16-byte piece of a token's row (two pieces in the half layout, the pairs' two
// sides), forms its angles once and applies them to that piece of up to 20 heads of q and k,
// four heads' loads in flight.  3.1 GB of q and k (80 heads x 75,600 tokens x 128) take 495 us among
// other calls, 6.3 TB/s: 97% of the rate of a plain copy.
#include <cuda_runtime.h>

#include "common.cuh"
#include "selected.cuh"

namespace spr {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Vec;  // 16 bytes of T as floats
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  __device__ static void unpack(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  __device__ static void store(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  __device__ static void unpack(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static void store(__nv_bfloat16* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// f cos t and f sin t of one pair at position p; the angle is reduced to one turn in 64
// bits, so its error stays near 2^-24 rad whatever the position.
__device__ __forceinline__ void turn(const RotaryArgs& a, const int* pos, int pair, float& c, float& s) {
  int axis = 0, first = 0;
  while (axis + 1 < a.axes && pair >= first + a.pairs[axis]) first += a.pairs[axis++];
  const double turns = static_cast<double>(pos[axis]) * a.freqs[pair] * 0.15915494309189535;
  sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
  c *= a.factor;
  s *= a.inverse ? -a.factor : a.factor;
}

// VEC: 16-byte pieces (rows on 16-byte boundaries, the rotated part and, in the half layout,
// each side of it a whole number of pieces); else one pair, or one plain dim, per thread.
template <typename T, bool HALF, bool VEC>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
  constexpr int V = VEC ? Vec<T>::kN : 1;
  constexpr int kPairs = VEC ? (HALF ? V : V / 2) : 1;
  const int half = a.rot / 2;
  const int rot_items = VEC ? (HALF ? half / V : a.rot / V) : half;
  const int items = rot_items + (a.copy_rest ? (a.d - a.rot) / V : 0);
  const long long idx = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (idx >= static_cast<long long>(a.Bt) * a.n * items) return;
  const int item = static_cast<int>(idx % items);
  const long long tok = idx / items;
  const int b = static_cast<int>(tok / a.n), t = static_cast<int>(tok % a.n);
  // dims of this thread: lo (and hi, the pairs' other side, in the half layout or scalar form)
  const bool rotated = item < rot_items;
  int lo, hi = 0;
  if (!rotated) {
    const int r = (item - rot_items) * V;  // dims outside [first, first + rot)
    lo = r < a.first ? r : r + a.rot;
  } else if (VEC) {
    lo = a.first + item * V;
    hi = lo + half;
  } else {
    lo = a.first + (HALF ? item : 2 * item);
    hi = HALF ? lo + half : lo + 1;
  }
  float c[kPairs], s[kPairs];
  if (rotated) {
    const int* pos = a.positions + b * a.pos_sb + t * a.pos_sn;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) turn(a, pos, item * kPairs + i, c[i], s[i]);
  }
  const int h0 = blockIdx.y * a.heads_per_thread, h1 = min(h0 + a.heads_per_thread, a.h[0] + a.h[1]);
  auto at = [&](const View* v, int h) -> T* {
    const int w = h >= a.h[0];
    return static_cast<T*>(v[w].p) + b * v[w].sb + (h - (w ? a.h[0] : 0)) * v[w].sh + t * v[w].sn;
  };
  if constexpr (VEC) {
    // kBatch heads' pieces are read before the first is written (in place, a thread writes only
    // what it has read itself)
    constexpr int kBatch = 4;
    for (int hb = h0; hb < h1; hb += kBatch) {
      uint4 u4[kBatch], w4[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (hb + k >= h1) break;
        const T* x = at(a.x, hb + k);
        u4[k] = __ldcs(reinterpret_cast<const uint4*>(x + lo));
        if (HALF && rotated) w4[k] = __ldcs(reinterpret_cast<const uint4*>(x + hi));
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (hb + k >= h1) break;
        T* y = at(a.y, hb + k);
        if (!rotated) {
          *reinterpret_cast<uint4*>(y + lo) = u4[k];
          continue;
        }
        float u[V], w[V];
        Vec<T>::unpack(u4[k], u);
        if (HALF) {
          Vec<T>::unpack(w4[k], w);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float p = u[i] * c[i % kPairs] - w[i] * s[i % kPairs];
            w[i] = w[i] * c[i % kPairs] + u[i] * s[i % kPairs];
            u[i] = p;
          }
          Vec<T>::store(y + lo, u);
          Vec<T>::store(y + hi, w);
        } else {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const float p = u[2 * i] * c[i] - u[2 * i + 1] * s[i];
            u[2 * i + 1] = u[2 * i + 1] * c[i] + u[2 * i] * s[i];
            u[2 * i] = p;
          }
          Vec<T>::store(y + lo, u);
        }
      }
    }
  } else {
    for (int h = h0; h < h1; ++h) {
      const T* x = at(a.x, h);
      T* y = at(a.y, h);
      const float p = to_f32<T>(x[lo]);
      if (!rotated) {
        y[lo] = x[lo];
      } else {
        const float q = to_f32<T>(x[hi]);
        y[lo] = from_f32<T>(p * c[0] - q * s[0]);
        y[hi] = from_f32<T>(q * c[0] + p * s[0]);
      }
    }
  }
}

template <typename T>
cudaError_t launch(RotaryArgs a, cudaStream_t st) {
  constexpr int V = Vec<T>::kN;
  bool vec = a.first % V == 0 && a.rot % V == 0 && (!a.half || (a.rot / 2) % V == 0);
  for (int w = 0; w < 2; ++w) {
    if (a.h[w] == 0) continue;
    for (const View* v : {&a.x[w], &a.y[w]}) {
      vec = vec && (reinterpret_cast<uintptr_t>(v->p) & 15u) == 0 && v->sb % V == 0 && v->sh % V == 0 && v->sn % V == 0;
    }
  }
  // dims outside the rotated part are copied unless every row is rotated in place
  a.copy_rest = false;
  for (int w = 0; w < 2; ++w) a.copy_rest = a.copy_rest || (a.h[w] > 0 && a.x[w].p != a.y[w].p);
  a.copy_rest = a.copy_rest && a.rot < a.d;
  const int v = vec ? V : 1;
  const int rot_items = vec ? (a.half ? a.rot / 2 / V : a.rot / V) : a.rot / 2;
  const long long items = static_cast<long long>(a.Bt) * a.n * (rot_items + (a.copy_rest ? (a.d - a.rot) / v : 0));
  const long long bx = (items + kThreads - 1) / kThreads;
  if (bx > 0x7fffffffLL) return cudaErrorInvalidValue;
  // Heads a thread applies its angles to, in equal shares of at most 20: the angles cost as much as
  // eight heads' pieces take from memory (80 heads x 75,600 tokens: 682 us at 4, 520 at 8, 478 at
  // 16, 489 at 40; 20 heads, token-major: 184, 153, 137 and at 20 124; 24 and 36
  // heads of one tensor, 0.77 GB, 126 to 133 us from 8 to 24 a thread and 144 at 4).  Few tokens spread their
  // heads over more blocks instead, until the grid covers the SMs twice.
  const int heads = a.h[0] + a.h[1];
  a.heads_per_thread = ceil_div(heads, ceil_div(heads, 20));
  while (a.heads_per_thread > 1 && bx * ceil_div(heads, a.heads_per_thread) < 2 * 148)
    a.heads_per_thread = (a.heads_per_thread + 1) / 2;
  const dim3 grid(static_cast<unsigned>(bx), ceil_div(heads, a.heads_per_thread));
  if (grid.y > 65535) return cudaErrorInvalidValue;
  if (a.half)
    vec ? rotary_kernel<T, true, true><<<grid, kThreads, 0, st>>>(a) : rotary_kernel<T, true, false><<<grid, kThreads, 0, st>>>(a);
  else
    vec ? rotary_kernel<T, false, true><<<grid, kThreads, 0, st>>>(a) : rotary_kernel<T, false, false><<<grid, kThreads, 0, st>>>(a);
  return counted(cudaGetLastError(), 1);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t st) {
  return a.f32 ? launch<float>(a, st) : launch<__nv_bfloat16>(a, st);
}

}  // namespace spr
