// Selected-block attention for few tokens: single tokens over a cache (bf16).
//
// Mathematics as in selected_attn.cu, without the detour over the blocks' lists: with a token
// or a few per key head there is nothing to share a key tile with but the token's own group.
// What bounds it: HBM, one read of the selected blocks' K and V; for a single sequence, latency.
// 32 sequences x 8 key heads, 32 blocks of 64 keys: 268 MB in 53 us, 5.1 TB/s; one sequence, 16
// blocks of 128: 10 us.
//
// One cluster per (batch, key head, token, 16 query heads of the group); the keys of the
// selected blocks are cut into pieces of 32, dealt to the cluster's warps.  A warp takes 16 keys
// at a time with mma.sync, the group's heads being the 16 rows: K and V go from global memory
// straight into operand registers, 16 bytes a lane, since the order of the head dims in a
// product is free (K: lane t of a quad has dims 32 s + 8 t .. + 7 of its key, two steps' worth;
// V: lane g has columns 8 g .. + 7 of each 64, one per column tile) and only pairs of keys have
// to be interleaved for V.  Each warp keeps a running maximum, sum and O; the warps' results
// are joined in shared memory, the CTAs' through the cluster.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "selected.cuh"
#include "selected_tc.cuh"
#include "warp_mma.cuh"

namespace cg = cooperative_groups;

namespace spr {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_huge_valf();
constexpr int kWarps = 4, kPiece = 32;

template <int D>
__global__ void __launch_bounds__(32 * kWarps, 2) decode_kernel(const SelArgs a, int splits) {
  constexpr int S = D / 32, H = D / 64;  // dim steps of a K load, column halves
  __shared__ float s_o[kWarps][16][D];
  __shared__ float2 s_ml[kWarps][16];
  __shared__ float s_co[16][D];          // this CTA's sums, read by the cluster
  __shared__ float2 s_cml[16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const int split = blockIdx.x % splits;
  long long unit = blockIdx.x / splits;
  const int row_groups = ceil_div(a.group, 16);
  const int h0 = static_cast<int>(unit % row_groups) * 16;
  unit /= row_groups;
  const int t = static_cast<int>(unit % a.n), z = static_cast<int>(unit / a.n), b = z / a.Hk, kh = z % a.Hk;
  const int heads = min(16, a.group - h0);
  const int len = kv_len_of(a, b);
  const int last = a.causal ? min(len - 1, q_start_of(a, b) + t) : len - 1;  // last visible key
  const int* row = a.sel + unit * a.top;

  // Q as the A operand: rows g and g + 8; step s: dims 32 s + 8 t4 + {0,1 | 2,3} then {4,5 | 6,7}
  uint32_t qa[2 * S][4];
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q.p) + b * a.q.sb + (kh * a.group + h0) * a.q.sh + t * a.q.sn;
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int h = g + 8 * half;
      const uint4 v = h < heads ? *reinterpret_cast<const uint4*>(q + h * a.q.sh + 32 * s + 8 * t4) : make_uint4(0, 0, 0, 0);
      qa[2 * s][half] = v.x, qa[2 * s][2 + half] = v.y;
      qa[2 * s + 1][half] = v.z, qa[2 * s + 1][2 + half] = v.w;
    }
  float acc[8 * H][4] = {}, m[2] = {-kInf, -kInf}, l[2] = {0.f, 0.f};
  const float scale2 = a.scale * kLog2e;
  const __nv_bfloat16* kbase = static_cast<const __nv_bfloat16*>(a.k.p) + b * a.k.sb + kh * a.k.sh + 8 * t4;
  const __nv_bfloat16* vbase = static_cast<const __nv_bfloat16*>(a.v.p) + b * a.v.sb + kh * a.v.sh + 8 * g;
  const int per = a.block / kPiece;  // pieces of a block
  const int stride = splits * kWarps;
  // The row's valid entries (ascending, in range, up to the first negative one), 32 slots at a
  // time by the lanes; their pieces go to the cluster's warps in turn.
  bool bad = false, ended = false;
  int above = -1, piece = split * kWarps + warp;
  for (int s0 = 0; s0 < a.top && !ended; s0 += 32) {
    const int blk = s0 + lane < a.top ? __ldg(row + s0 + lane) : -1;
    const unsigned neg = __ballot_sync(0xffffffffu, blk < 0);
    const bool past = (neg & ((2u << lane) - 1u)) != 0;
    const int v = past || blk >= a.nb ? -1 : blk;
    int mx = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, mx, o);
      if (lane >= o) mx = max(mx, y);
    }
    int prev = __shfl_up_sync(0xffffffffu, mx, 1);
    prev = max(above, lane > 0 ? prev : -1);
    if (!past && (blk >= a.nb || blk <= prev)) bad = true;
    const unsigned valid = __ballot_sync(0xffffffffu, v >= 0 && v > prev && v * a.block <= last);
    above = max(above, __shfl_sync(0xffffffffu, mx, 31));
    ended = neg != 0;
    const int n_pieces = __popc(valid) * per;
    // this warp's steps of 16 keys: two a piece; K of the next step is asked for once S is formed,
    // V once O is, so that loads are under way during the arithmetic
    const int steps = piece < n_pieces ? 2 * ((n_pieces - piece + stride - 1) / stride) : 0;
    auto key_of = [&](int k) {  // first key of step k
      const int p = piece + (k >> 1) * stride, at = static_cast<int>(__fns(valid, 0, p / per + 1));
      return __shfl_sync(0xffffffffu, blk, at) * a.block + p % per * kPiece + 16 * (k & 1);
    };
    uint4 kv[2][S], vv[4][H];
    auto load_k = [&](int j) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = j + 8 * i + g;
        const __nv_bfloat16* p = kbase + key * a.k.sn;
#pragma unroll
        for (int x = 0; x < S; ++x)
          kv[i][x] = key <= last ? __ldcs(reinterpret_cast<const uint4*>(p + 32 * x)) : make_uint4(0, 0, 0, 0);
      }
    };
    auto load_v = [&](int j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
        const int key = j + 2 * t4 + (i & 1) + 8 * (i >> 1);
        const __nv_bfloat16* p = vbase + key * a.v.sn;
#pragma unroll
        for (int h = 0; h < H; ++h)
          vv[i][h] = key <= last ? __ldcs(reinterpret_cast<const uint4*>(p + 64 * h)) : make_uint4(0, 0, 0, 0);
      }
    };
    int j = 0;
    if (steps > 0) {
      j = key_of(0);
      load_k(j);
      load_v(j);
    }
#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
      const int next = k + 1 < steps ? key_of(k + 1) : 0;
      float s[2][4] = {};
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 0; x < S; ++x) {
          const uint32_t b0[2] = {kv[i][x].x, kv[i][x].y}, b1[2] = {kv[i][x].z, kv[i][x].w};
          mma_bf16_16816(s[i], qa[2 * x], b0);
          mma_bf16_16816(s[i], qa[2 * x + 1], b1);
        }
      if (k + 1 < steps) load_k(next);
      float p[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {  // rows g and g + 8
        float mx = -kInf;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float& x = s[i][2 * r + c];
            x = j + 8 * i + 2 * t4 + c <= last ? x * scale2 : -kInf;
            mx = fmaxf(mx, x);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[r], mx), ms = mn == -kInf ? 0.f : mn;
        const float f = ex2(m[r] - ms);
        m[r] = mn;
        l[r] *= f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            p[i][2 * r + c] = ex2(s[i][2 * r + c] - ms);
            l[r] += p[i][2 * r + c];
          }
#pragma unroll
        for (int n = 0; n < 8 * H; ++n) acc[n][2 * r] *= f, acc[n][2 * r + 1] *= f;
      }
      const uint32_t pa[4] = {pack_bf16x2(p[0][0], p[0][1]), pack_bf16x2(p[0][2], p[0][3]), pack_bf16x2(p[1][0], p[1][1]),
                              pack_bf16x2(p[1][2], p[1][3])};
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t* x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = reinterpret_cast<const uint32_t*>(&vv[i][h]);
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {  // columns 64 h + 8 g + 2 w + odd
            const uint32_t sel = odd ? 0x7632 : 0x5410;
            const uint32_t bb[2] = {__byte_perm(x[0][w], x[1][w], sel), __byte_perm(x[2][w], x[3][w], sel)};
            mma_bf16_16816(acc[8 * h + 2 * w + odd], pa, bb);
          }
        }
      if (k + 1 < steps) load_v(next);
      j = next;
    }
    piece += steps / 2 * stride - n_pieces;
  }
  if (bad && split == 0 && warp == 0) record_error(a.status, kErrInvalidArg);
  // acc[8 h + n][2 r + c]: row g + 8 r, column 64 h + 8 (2 t4 + c) + n
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    if (t4 == 0) s_ml[warp][g + 8 * r] = make_float2(m[r], l[r]);
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int n = 0; n < 8; n += 4)
          *reinterpret_cast<float4*>(&s_o[warp][g + 8 * r][64 * h + 8 * (2 * t4 + c) + n]) =
              make_float4(acc[8 * h + n][2 * r + c], acc[8 * h + n + 1][2 * r + c], acc[8 * h + n + 2][2 * r + c],
                          acc[8 * h + n + 3][2 * r + c]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < heads * D; i += 32 * kWarps) {
    const int h = i / D, c = i % D;
    float mx = -kInf;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_ml[w][h].x);
    const float ms = mx == -kInf ? 0.f : mx;
    float sum = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(s_ml[w][h].x - ms);
      sum = fmaf(f, s_ml[w][h].y, sum);
      x = fmaf(f, s_o[w][h][c], x);
    }
    s_co[h][c] = x;
    if (c == 0) s_cml[h] = make_float2(mx, sum);
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (splits > 1)
    cluster.sync();
  else
    __syncthreads();
  // the cluster's CTAs take every splits-th head's columns
  for (int i = threadIdx.x + 32 * kWarps * split; i < heads * D; i += 32 * kWarps * splits) {
    const int h = i / D, c = i % D;
    float mx = -kInf;
    for (int w = 0; w < splits; ++w) mx = fmaxf(mx, (splits > 1 ? cluster.map_shared_rank(s_cml, w) : s_cml)[h].x);
    const float ms = mx == -kInf ? 0.f : mx;
    float sum = 0.f, x = 0.f;
    for (int w = 0; w < splits; ++w) {
      const float2 st = (splits > 1 ? cluster.map_shared_rank(s_cml, w) : s_cml)[h];
      const float f = ex2(st.x - ms);
      sum = fmaf(f, st.y, sum);
      x = fmaf(f, *((splits > 1 ? cluster.map_shared_rank(&s_co[0][0], w) : &s_co[0][0]) + i), x);
    }
    const int hq = kh * a.group + h0 + h;
    const float y = sum > 0.f ? x / sum : sum != sum ? sum : 0.f;
    const __nv_bfloat16 v = __float2bfloat16_rn(y);
    static_cast<__nv_bfloat16*>(a.o.p)[b * a.o.sb + hq * a.o.sh + t * a.o.sn + c] = v;
    if (a.rest != nullptr)
      a.rest[((static_cast<size_t>(b) * a.Hq + hq) * a.n + t) * D + c] = __float2bfloat16_rn(y - __bfloat162float(v));
    if (c == 0)
      a.lse[(static_cast<size_t>(b) * a.Hq + hq) * a.n + t] = sum > 0.f || sum != sum ? (mx + log2f(sum)) * kLn2 : -kInf;
  }
  if (splits > 1) cluster.sync();  // nobody leaves while its sums are read
}

template <int D>
cudaError_t decode(const SelArgs& a, cudaStream_t st) {
  const long long units = static_cast<long long>(a.Bt) * a.Hk * a.n * ceil_div(a.group, 16);
  // CTAs that the SMs hold at once: two an SM (three at d = 64).  The largest cluster that stays
  // within that, up to eight CTAs and to a warp for each piece: a second wave costs its start and
  // join again.  Measured, us at 1, 2, 4, 8 CTAs a cluster where tried (32 blocks of 64, 16 of 128,
  // 16 of 64 keys): 256 clusters of d 128 53, 59, 68, 91; 192 53, 58, 54, 69; 64 -, -, 18, 23;
  // 96 of d 64 -, 13.6, 10.8, 16.
  constexpr int kSlots = (D == 128 ? 2 : 3) * 148;
  const int pieces = std::min(a.top, a.nb) * (a.block / kPiece);
  int splits = 1;
  while (splits < 8 && 2 * units * splits <= kSlots && 2 * splits * kWarps <= pieces) splits *= 2;
  if (units * splits > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(units * splits));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return counted(cudaLaunchKernelEx(&cfg, decode_kernel<D>, a, splits), 1);
}

}  // namespace

// Few tokens read the selected blocks once each and straight; the lists share a block's tile
// between the tokens that selected it, at the price of five more launches and of tiles of 128 rows.
// Direct up to 12 tokens, and while a block has at most three tokens on average (n top / nb): where it won at
// every head count tried.  The rule does not look at how many CTAs a call fills, so that it gives away
// up to 1.6x where they are few (8 key heads, n = 16 .. 64 below); fp32 has no direct form.
// Measured, direct and lists in us (replayed graphs; batch x key heads x group):
//   1 x 8 x 4, d 128, 16 of 64 blocks of 128:  n = 1 9, 31;  8 15, 38;  16 24, 39;  32 39, 40
//   8 x 8 x 1, d 128, 16 of 64 blocks of 128:  n = 1 18, 70;  8 84, 117;  12 119, 122;  16 154, 125
//   1 x 8 x 8, d 128, 32 of 512 blocks of 64:  n = 1 10, 60;  32 47, 116;  64 87, 134;  128 163, 146
//   4 x 4 x 2, d 64, 16 of 256 blocks of 64:   n = 1 7, 42;  32 34, 74;  64 52, 82;  128 87, 91
bool use_decode(const SelArgs& a) {
  const long long n = static_cast<long long>(a.n) * ceil_div(a.group, 16);
  return !a.f32 && n <= std::max<long long>(12, 3ll * a.nb / a.top);
}

cudaError_t launch_decode(const SelArgs& a, cudaStream_t st) {
  return a.d == 128 ? decode<128>(a, st) : decode<64>(a, st);
}

}  // namespace spr
