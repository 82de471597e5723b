// Selected-block attention on the 5th-generation tensor cores (bf16).
//
// Mathematics as in selected_attn.cu: a work unit is one key block and up to unit_rows of the
// query rows that selected it.  K and V of the block stay in shared memory; 128 rows at a time
//   S = Q K^T (128 x B),  P = exp(S - row max),  O = P V (128 x D)
// need no running maximum, since one tile holds all the keys of the row's part.  The part goes
// out in fp16, with its log-sum-exp; join_half_kernel adds a row's parts.  So that O needs no
// scaling on its way out, P is formed as exp(S - row max) 2^-k: with |V| < 2^e over the keys that
// the row sees in the block, k = e + log2 B - 15 keeps |O| <= 2^15, inside fp16, and leaves its 11 bits
// to everything down to 2^-29 of that bound.  A part's rounding, 2^-12, is 16 times finer than the
// result's bf16; fp32 parts would double the traffic of the output and the join.  Below 2^-29 a
// part may lose 2^-40 of the bound (2^-33 of the largest |V|): blocks in which that could be much, or
// that hold what is not finite, are wide (ranges_kernel).  Their parts are watched on the way out
// (store_wide) and what does not fit is formed again from the inputs in fp32 (mend_kernel).  So nothing
// that a row does not see reaches it: k is its own, and a hidden NaN makes one that is formed again.
//
// Work of a tile (B = D = 128): 8.4 MFLOP, 16K exponentials, 32 KB of Q gathered, 32 KB written.
// A tile passes through five stages of 1 to 2 us (gather, S, softmax, O, output), so one persistent
// CTA per SM keeps five tiles in a ring of slots, each slot holding Q and then P of its tile, and
// gives each stage warps of its own; tiles alternate between two streams (S and O in TMEM each):
//   warps 0-7    softmax, one warpgroup a stream, one thread a row: maximum, then exponentials,
//                reading S twice (a second read costs ~100 cycles, 128 held values spill);
//   warps 8-11   output: O of each tile to memory;
//   warps 12-15  gather Q rows through the block's list (16-byte asynchronous copies, 16 lanes a
//                row, into the 128-byte swizzle), slots ahead of the products;
//   warps 16-17  issue the products of one stream each: S of the stream's next tile as soon as
//                the softmax has read the last one, O when P is written;
//   warp 18      TMA boxes of the units' K and V, and zeros over V rows at or past the length
//                (their P is 0, but 0 times what a cache holds there need not be).
// All waits are bounded; on a timeout every role leaves, products and copies in flight drained.
//
// Bound by the output warps, which drain every tile: 128 more instructions a tile there (a maximum and a
// scale for each row) took the kernel from 820 to 850 us (tensor pipe 31% active, HBM 53% of its nominal
// rate).  16 heads x 32,760 tokens, 16 of 256 blocks, D 128: this kernel 820 us, 1.85 us a tile (0.55
// TFLOP, 670 TFLOP/s; 2.1 GB of parts out), join_half_kernel 487 us (2.3 GB, 4.7 TB/s), the lists 140
// us, the ranges 31 us.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "selected.cuh"
#include "selected_tc.cuh"
#include "tcgen05.cuh"
#include "warp_mma.cuh"

namespace spr {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_huge_valf();

constexpr int kThreads = 640, kLoaders = 128;
constexpr int kRegSoftmax = 112, kRegOut = 136, kRegRest = 56;
constexpr int kOutWarp = 8, kLoadWarp = 12, kMmaWarp = 16, kKvWarp = 18;
// P takes this much of a k, so that its smallest and largest weights stay inside fp32; the output the rest
// (values above 2^68 or below 2^-93)
constexpr float kLeastK = -100.f, kMostK = 60.f;
__device__ __forceinline__ float p_share(float k) { return fminf(fmaxf(k, kLeastK), kMostK); }

template <int D, int B>
struct Fwd {
  static constexpr uint32_t kSlot = 128 * (D > B ? D : B) * 2, kKV = B * D * 2;
  static constexpr uint32_t kTail = 512;  // barriers
  static constexpr int kFit = (227 * 1024 - 2 * kKV - kTail) / kSlot;
  static constexpr int kSlots = kFit < 8 ? kFit : 8;
  static constexpr uint32_t kSmem = kSlots * kSlot + 2 * kKV + kTail;
};

// Per unit: K landed, V landed, V ready (zeros in place), K and V read by every product; per
// stream: S ready, P written (and S read), O ready, O read, drain; per slot: Q in place, free.
enum : int {
  kK = 0, kVLand, kV, kKFree, kVFree, kS, kP = kS + 2, kO = kP + 2, kOFree = kO + 2, kDrain = kOFree + 2,
  kQ = kDrain + 2, kFree = kQ + 8, kNumBars = kFree + 8
};
static_assert(8 * kNumBars + 32 <= 512, "barriers fit their room");

// Row maximum over 32 values, four chains of 3-input maxima; masking of columns from n on.
__device__ __forceinline__ void max_into(float (&mx)[4], const uint32_t (&s)[32]) {
#pragma unroll
  for (int c = 0; c < 32; c += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      mx[i] = fmax3(mx[i], __uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1]));
}
__device__ __forceinline__ void mask_from(uint32_t (&s)[32], int n) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (c >= n) s[c] = __float_as_uint(-kInf);
}

template <int D, int B>
__global__ void __launch_bounds__(kThreads, 1)
    selected_forward_tc_kernel(const __grid_constant__ BlockMap mk, const __grid_constant__ BlockMap mv, const SelArgs a,
                               int first, int count) {
  using F = Fwd<D, B>;
  constexpr int R = F::kSlots;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  uint8_t* const tail = dsmem + R * F::kSlot + 2 * F::kKV;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(tail);
  uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(bars + kNumBars);
  int& abort_flag = *reinterpret_cast<int*>(bars + kNumBars + 1);
  int* const s_first = reinterpret_cast<int*>(bars + kNumBars + 2);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sSlot = tc::saddr(dsmem), sK = sSlot + R * F::kSlot, sV = sK + F::kKV;
  if ((sSlot & 1023u) != 0) {  // the tiles' swizzle counts from 1024-byte lines
    if (tid == 0) record_error(a.status, kErrCuda);
    return;
  }
  auto bar = [&](int i) { return tc::saddr(&bars[i]); };
  if (tid == 0) {
    tc::mbar_init(bar(kK), 1);
    tc::mbar_init(bar(kVLand), 1);
    tc::mbar_init(bar(kV), 32);
    tc::mbar_init(bar(kKFree), 2);
    tc::mbar_init(bar(kVFree), 2);
    for (int x = 0; x < 2; ++x) {
      tc::mbar_init(bar(kS + x), 1);
      tc::mbar_init(bar(kP + x), 128);
      tc::mbar_init(bar(kO + x), 1);
      tc::mbar_init(bar(kOFree + x), 128);
      tc::mbar_init(bar(kDrain + x), 1);
    }
    for (int i = 0; i < 8; ++i) {
      tc::mbar_init(bar(kQ + i), kLoaders);
      tc::mbar_init(bar(kFree + i), 1);
    }
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tc::saddr(&tmem_slot), 512);
    tc::tmem_relinquish();
  }
  if (warp == kOutWarp) share_of_tiles(a, first, count, s_first);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = tmem_slot;  // S of stream x at 128 x, O at 256 + 128 x
  volatile int* abort_v = &abort_flag;
  const size_t cap = static_cast<size_t>(a.slice) * a.top;
  auto wait1 = [&](int i, int phase) { return wait_bar(bar(i), phase & 1, abort_v, a.status); };
  auto wait = [&](int i, int phase) { return __all_sync(0xffffffffu, wait1(i, phase)); };

  // registers: 96 a thread at launch, 480 x 128 in all; 2 x 112 + 136 + 2 x 56 of them are used
  if (warp < kOutWarp) {
    // ---------------------------------------------------------------- softmax
    tc::setmaxnreg_inc<kRegSoftmax>();
    const int x = warp >> 2, row = tid & 127;
    const uint32_t tS = tbase + 128 * x + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const float scale2 = a.scale * kLog2e;
    each_tile(a, first, s_first, x, 2, [&](const Unit& un, int ci, int t, int, bool, bool) {
        int nv = un.live;  // visible keys of this row in the block
        if (a.causal && row < un.rows)
          nv = min(nv, un.qs + __ldg(a.list + (first + ci) * cap + un.off + (un.r0 + row) / a.group) + 1);
        const int whole = min(B, un.live);
        float k = un.k;  // P is divided by 2^k; rows that see a part of the block go by that part
        if (__any_sync(0xffffffffu, nv < whole) || !(k < kInf))
          k = a.key_range[(static_cast<size_t>(un.b * a.Hk + un.kh) * a.nb + un.g) * B + max(min(nv, whole), 1) - 1];
        k = p_share(k);
        if (!wait(kS + x, t >> 1)) return false;
        tc::fence_after_sync();
        const bool cut = __any_sync(0xffffffffu, nv < B);
        float mx[4] = {-kInf, -kInf, -kInf, -kInf};
#pragma unroll 1
        for (int c0 = 0; c0 < B; c0 += 32) {
          uint32_t s[32];
          tc::tmem_ld32(tS + c0, s);
          tc::tmem_wait_ld();
          if (cut) mask_from(s, nv - c0);
          max_into(mx, s);
        }
        const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale2, shift = (m == -kInf ? 0.f : m) + k;
        const uint64_t sc2 = f32x2(scale2, scale2), nm2 = f32x2(-shift, -shift);
        uint64_t sum[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
        const uint32_t sP = sSlot + (t % R) * F::kSlot;  // over Q, which S has read
#pragma unroll 1
        for (int c0 = 0; c0 < B; c0 += 32) {
          uint32_t s[32], pk[16];
          tc::tmem_ld32(tS + c0, s);
          tc::tmem_wait_ld();
          if (cut) mask_from(s, nv - c0);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float y0, y1;
            f32x2_split(ffma2(f32x2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sc2, nm2), y0, y1);
            const float p0 = ex2(y0), p1 = ex2(y1);
            sum[i & 1] = fadd2(sum[i & 1], f32x2(p0, p1));
            pk[i] = pack_bf16x2(p0, p1);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c)
            st_shared_16(sP + tc::sw128_offset(row, c0 / 8 + c), pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        }
        tc::fence_proxy_async();
        tc::fence_before_sync();
        tc::mbar_arrive(bar(kP + x));
        float l0, l1, l2, l3;
        f32x2_split(sum[0], l0, l1);
        f32x2_split(sum[1], l2, l3);
        const float l = (l0 + l1) + (l2 + l3);  // not above 0: no visible key (or a NaN, which stays one)
        if (row < un.rows)
          a.ml[(ci * cap + un.off) * a.group + un.r0 + row] =
              l > 0.f || l != l ? make_float2(shift + __log2f(l), shift + (un.k < kInf ? un.k - p_share(un.k) : 0.f))
                                : make_float2(-kInf, -kInf);
        return true;
    });
  } else if (warp < kLoadWarp) {
    // ---------------------------------------------------------------- output
    tc::setmaxnreg_inc<kRegOut>();
    // A quad of lanes holds rows q and q + 8 of 16 TMEM lanes, lane i of it columns 8 j + 2 i
    // and + 1; each lane's 16 columns of a 64-column line go out as 32 contiguous bytes, a
    // row's quad as one 128-byte line (part_column() is the order inside the line).
    const int w4 = warp & 3, q = lane >> 2, i = lane & 3;
    uint8_t* const part = static_cast<uint8_t*>(static_cast<void*>(a.part));
    each_tile(a, first, s_first, 0, 1, [&](const Unit& un, int ci, int t, int, bool, bool) {
        const int x = t & 1;
        const long long out0 = static_cast<long long>((ci * cap + un.off) * a.group + un.r0);
        if (!wait(kO + x, t >> 1)) return false;
        tc::fence_after_sync();
        const uint32_t tO = tbase + 256 + 128 * x;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int lane0 = 32 * w4 + 16 * half;
          const uint32_t tRow = tO + (static_cast<uint32_t>(lane0) << 16);
          if (!(un.k < kInf)) {
            float up[2];
            store_wide<D, true>(tRow, un.k != un.k, lane0 + q, un.rows, part + 32 * i, out0, up);
          } else {
            uint32_t o[D / 2];
#pragma unroll
            for (int c = 0; c < D; c += 64) tmem_ld_16x64(tRow + c, *reinterpret_cast<uint32_t(*)[32]>(&o[c / 2]));
            tc::tmem_wait_ld();
            if (un.k != p_share(un.k)) {
              const float f = exp2f(p_share(un.k) - un.k);
#pragma unroll
              for (int c = 0; c < D / 2; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
            }
            store_part_as_is<D>(o, lane0 + q, un.rows, part + 32 * i, out0);
          }
        }
        tc::fence_before_sync();
        tc::mbar_arrive(bar(kOFree + x));
        return true;
    });
  } else if (warp < kMmaWarp) {
    // ---------------------------------------------------------------- Q rows, 32 a warp
    tc::setmaxnreg_dec<kRegRest>();
    constexpr int kPer = D / 8, kStep = 32 / kPer;  // lanes per row, rows per instruction
    const int lw = warp - kLoadWarp, ch = lane % kPer;
    // tile t - 1 has landed once at most one group of copies is in flight
    auto landed = [&](int tile) {
      tc::fence_proxy_async();
      tc::mbar_arrive(bar(kQ + tile % R));
    };
    // The copies of a tile are issued when the walk is at the next one, so that the list entry
    // read here has arrived.
    const __nv_bfloat16* q = nullptr;
    int entry = -1, h = 0;
    auto copy = [&](int t) {
      const long long off = entry < 0 ? -1 : entry * a.q.sn + h * a.q.sh;
      if (t >= R && !wait(kFree + t % R, t / R - 1)) return false;
      const uint32_t sQ = sSlot + (t % R) * F::kSlot;
#pragma unroll
      for (int s = 0; s < 32; s += kStep) {
        const int src = s + lane / kPer;
        const long long o = __shfl_sync(0xffffffffu, off, src);
        cp_async_16(sQ + tc::sw128_offset(32 * lw + src, ch), o < 0 ? q : q + o, o < 0 ? 0 : 16);
      }
      cp_async_commit();
      if (t > 0) {
        cp_async_wait<1>();
        landed(t - 1);
      }
      return true;
    };
    bool ok = each_tile(a, first, s_first, 0, 1, [&](const Unit& un, int ci, int t, int, bool, bool) {
      const int r = 32 * lw + lane, row = un.r0 + r, e = row / a.group;  // this lane's row of the tile
      const int next = r < un.rows ? __ldg(a.list + (first + ci) * cap + un.off + e) : -1;
      if (t > 0 && !copy(t - 1)) return false;
      q = static_cast<const __nv_bfloat16*>(a.q.p) + un.b * a.q.sb + un.kh * a.group * a.q.sh + ch * 8;
      entry = next, h = row - e * a.group;
      return true;
    });
    const int tiles = s_first[2];
    ok = ok && tiles > 0 && copy(tiles - 1);
    cp_async_wait<0>();
    if (ok) landed(tiles - 1);
  } else {
    tc::setmaxnreg_dec<kRegRest>();
  if (warp < kKvWarp) {
    // ---------------------------------------------------------------- products of one stream
    constexpr uint32_t kIdS = tc::idesc_bf16(128, B, false, false), kIdO = tc::idesc_bf16(128, D, false, true);
    const int x = warp - kMmaWarp;
    const uint32_t tS = tbase + 128 * x, tO = tbase + 256 + 128 * x;
    // the whole warp walks and waits, lane 0 issues
    int held = -1;           // tile whose O is still to be issued, of the unit held_u
    int held_u = 0;
    bool held_last = false;  // ... and the stream's last of that unit
    int of_unit = 0;         // the stream's tiles of the current unit
    auto issue_s = [&](int tile) {
      uint64_t dq = tc::sdesc_sw128(sSlot + (tile % R) * F::kSlot, 16, 1024), dk = tc::sdesc_sw128(sK, 16, 1024);
      keep_here(dq, dk);
      if (lane == 0) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_ss(tS, dq + ((kk >> 2) * (128 * 128) + (kk & 3) * 32) / 16,
                     dk + ((kk >> 2) * (B * 128) + (kk & 3) * 32) / 16, kIdS, kk > 0 ? 1u : 0u);
        tc::mma_commit(bar(kS + x));
      }
      __syncwarp();
    };
    auto issue_o = [&]() {  // of the held tile, whose P is written
      if (!wait(kV, held_u)) return false;
      if (held > 1 && !wait(kOFree + x, (held >> 1) - 1)) return false;
      tc::fence_after_sync();
      uint64_t dp = tc::sdesc_sw128(sSlot + (held % R) * F::kSlot, 16, 1024), dv = tc::sdesc_sw128(sV, B * 128, 1024);
      keep_here(dp, dv);
      if (lane == 0) {
#pragma unroll
        for (int kk = 0; kk < B / 16; ++kk)
          tc::mma_ss(tO, dp + ((kk >> 2) * (128 * 128) + (kk & 3) * 32) / 16, dv + kk * (2048 / 16), kIdO, kk > 0 ? 1u : 0u);
        tc::mma_commit(bar(kO + x));
        tc::mma_commit(bar(kFree + held % R));
        if (held_last) tc::mma_commit(bar(kVFree));
      }
      __syncwarp();
      held = -1;
      return true;
    };
    auto flush = [&]() { return held < 0 || (wait(kP + x, held >> 1) && issue_o()); };
    const bool ok = each_tile(a, first, s_first, 0, 1, [&](const Unit&, int, int t, int u, bool opens, bool closes) {
      if (opens) of_unit = 0;
      if ((t & 1) == x) {
        if (held >= 0) {
          if (!wait(kP + x, held >> 1)) return false;  // P written, S read
          tc::fence_after_sync();
          // S first where its operands are there, so that the softmax goes on at once
          const bool there = bar_done(bar(kK), u & 1) && bar_done(bar(kQ + t % R), (t / R) & 1);
          if (!__all_sync(0xffffffffu, there) && !issue_o()) return false;
        }
        if (!wait(kK, u) || !wait(kQ + t % R, t / R)) return false;
        tc::fence_after_sync();
        issue_s(t);
        if (held >= 0 && !issue_o()) return false;
        held = t, held_u = u, held_last = false;
        ++of_unit;
      }
      if (!closes) return true;
      // this stream's share of the unit's releases: K behind its last S, V behind its last O.
      // Without a tile in the unit, once the unit before is released (two arrivals of one
      // stream in a phase would stand for the other stream's).
      if (of_unit > 0) {
        if (lane == 0) tc::mma_commit(bar(kKFree));
        __syncwarp();
        held_last = true;
      } else {
        if (!flush() || !wait(kK, u) || !wait(kV, u)) return false;
        if (lane == 0) {
          tc::mbar_arrive(bar(kKFree));
          tc::mbar_arrive(bar(kVFree));
        }
        __syncwarp();
      }
      return true;
    });
    if (ok) flush();
    if (lane == 0) {
      tc::mma_commit(bar(kDrain + x));  // every product has finished before TMEM goes back
      tc::mbar_wait_quiet(bar(kDrain + x), 0);
    }
    __syncwarp();
  } else if (warp == kKvWarp) {
    // ---------------------------------------------------------------- K and V of each unit
    int issued = 0;
    const bool ok = each_tile(a, first, s_first, 0, 1, [&](const Unit& un, int, int, int u, bool opens, bool) {
      if (!opens) return true;
      if (u > 0 && !wait(kKFree, u - 1)) return false;
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(bar(kK), F::kKV);
#pragma unroll
        for (int c = 0; c < D; c += 64) load_box(sK + c * (B * 2), mk, c, un.g * B, un.kh, un.b, bar(kK));
      }
      issued = 2 * u + 1;
      if (u > 0 && !wait(kVFree, u - 1)) return false;
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(bar(kVLand), F::kKV);
#pragma unroll
        for (int c = 0; c < D; c += 64) load_box(sV + c * (B * 2), mv, c, un.g * B, un.kh, un.b, bar(kVLand));
      }
      __syncwarp();
      issued = 2 * u + 2;
      if (!wait(kVLand, u)) return false;
      for (int i = lane; i < (B - un.live) * (D / 8); i += 32)  // V rows of the block from the length on
        st_shared_zero(sV + sw128_rows<B>(un.live + i / (D / 8), i % (D / 8)));
      tc::fence_proxy_async();
      tc::mbar_arrive(bar(kV));
      return true;
    });
    // boxes still in flight after an abort land before the CTA exits
    if (!ok && lane == 0 && issued > 0) {
      tc::mbar_wait_quiet(bar(kK), (issued - 1) / 2 & 1);
      if (issued % 2 == 0) tc::mbar_wait_quiet(bar(kVLand), (issued / 2 - 1) & 1);
    }
    __syncwarp();
  }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, 512);
  }
}

// Joins a query row's parts (GRAD: adds the row's dQ parts, whose scales are in ml).  D / 8 lanes
// take a row, so that a warp has two or four rows under way; each lane looks up the slots of its
// number (entry, weight), then the lanes read eight parts at a time, 16 bytes each.  Bound by
// the parts' bytes, pieces of 256 in the tokens' order: 4.2 to 5.1 TB/s.  (Walking eight rows a
// group of lanes, with weights and entries asked for ahead, was slower: 186 against 175 us.)
template <int D, bool GRAD>
__global__ void __launch_bounds__(256, 6) join_half_kernel(const SelArgs a, int first, int count) {
  constexpr int kPer = D / 8, kRowsW = 32 / kPer;
  const int lane = threadIdx.x & 31, ch = lane % kPer;
  const long long w = (static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * kRowsW + lane / kPer;
  const int per = a.slice * a.group;
  const int ci = static_cast<int>(min(w / per, static_cast<long long>(count - 1)));
  const int region = first + ci, z = region / a.slices, s = region % a.slices;
  const int lr = static_cast<int>(w % per), t = s * a.slice + lr / a.group, h = lr % a.group;
  const bool live = w < static_cast<long long>(count) * per && t < a.n;  // the warp stays together
  const int b = z / a.Hk, kh = z % a.Hk;
  const int* inv = a.inv + (static_cast<size_t>(z) * a.n + (live ? t : 0)) * a.top;
  const size_t row0 = ci * static_cast<size_t>(a.slice) * a.top * a.group + h;
  // the lane's 16 bytes of a part
  const uint8_t* part = static_cast<const uint8_t*>(static_cast<const void*>(a.part)) + ch * 16;
  float m = -kInf, l = 0.f, acc[8] = {};
  for (int j0 = 0; j0 < a.top; j0 += kPer) {
    const int e = live && j0 + ch < a.top ? __ldg(inv + j0 + ch) : -1;
    const float2 st = e >= 0 ? __ldcs(a.ml + row0 + static_cast<size_t>(e) * a.group) : make_float2(-kInf, GRAD ? 0.f : -kInf);
    float f = st.y;
    if (!GRAD) {
      float mx = st.x;
#pragma unroll
      for (int o = kPer / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = fmaxf(m, mx);
      const float ms = mx == -kInf ? 0.f : mx, old = exp2f(m - ms), wt = exp2f(st.x - ms);
      m = mx;
      l = fmaf(l, old, wt);
      f = exp2f(st.y - ms);
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] *= old;
    }
    if (e < 0) f = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; j += 8) {
      if (j0 + j >= a.top) break;
      uint4 v[8];
      float fj[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int ej = __shfl_sync(0xffffffffu, e, j + i, kPer);
        fj[i] = __shfl_sync(0xffffffffu, f, j + i, kPer);
        v[i] = ej >= 0 ? __ldcs(reinterpret_cast<const uint4*>(part + (row0 + static_cast<size_t>(ej) * a.group) * (2 * D)))
                       : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x[c]));
          acc[2 * c] = fmaf(fj[i], y.x, acc[2 * c]);
          acc[2 * c + 1] = fmaf(fj[i], y.y, acc[2 * c + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int o = kPer / 2; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  // a part could not hold some of its row (a NaN): on the list for mend_kernel
  float any = 0.f;
#pragma unroll
  for (int c = 0; c < 8; ++c) any += acc[c];
  const unsigned open = __ballot_sync(0xffffffffu, live && any != any) >> (lane - ch);
  if (!live) return;
  if ((open & ((1u << kPer) - 1u)) != 0 && ch == 0) a.slow[1 + atomicAdd(a.slow, 1)] = (b * a.Hq + kh * a.group + h) * a.n + t;
  const float inv_l = GRAD ? 1.f : l > 0.f ? 1.f / l : l != l ? l : 0.f;
  const View& out = GRAD ? a.gq : a.o;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out.p) + b * out.sb + (kh * a.group + h) * out.sh + t * out.sn;
  __nv_bfloat16* rest = GRAD || a.rest == nullptr
                            ? nullptr
                            : a.rest + ((static_cast<size_t>(b) * a.Hq + kh * a.group + h) * a.n + t) * D;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float x = acc[2 * c] * inv_l, y = acc[2 * c + 1] * inv_l;
    const uint32_t v = pack_bf16x2(x, y);
    *reinterpret_cast<uint32_t*>(o + part_column(ch, c)) = v;
    if (rest != nullptr)
      *reinterpret_cast<uint32_t*>(rest + part_column(ch, c)) =
          pack_bf16x2(x - __uint_as_float(v << 16), y - __uint_as_float(v & 0xffff0000u));
  }
  if (!GRAD && ch == 0)
    a.lse[(static_cast<size_t>(b) * a.Hq + kh * a.group + h) * a.n + t] =
        l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -kInf;
}

// Larger magnitudes of pairs of bf16 values (signs of no meaning); a NaN is the largest.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A block's range, of its finite values.  Forward (V): k of the rows that see its keys up to each
// (SelArgs::key_range), that of the whole block, and whether it is wide: it holds a value that is not
// finite, or rows or columns (those of zeros aside) whose largest magnitudes' exponents are more than 20
// apart, so that the 2^-33 of the largest |V| that parts may lose can be more than 2^-12 of a row's or a
// column's largest (8 apart where the output takes a share of the block's k, the same for rows with smaller
// ones).  Backward (K): dQ's parts have scales of their own and lose 2^-39 of a row's largest; wide where
// columns are more than 24 apart or something is not finite.  One CTA a block, bound by the read of
// the tensor.
template <int D, bool BACKWARD>
__global__ void __launch_bounds__(256) ranges_kernel(const SelArgs a, const View x) {
  constexpr int L = D / 8, kRows = 256 / L, kPer = 128 / kRows;  // lanes a row, rows at a time, of a thread
  __shared__ uint4 s_mx[8][L];
  __shared__ int s_row[128];
  const int g = blockIdx.x, kh = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = min(a.block, kv_len_of(a, b) - g * a.block), ch = threadIdx.x % L, r0 = threadIdx.x / L;
  const size_t at = (static_cast<size_t>(b) * a.Hk + kh) * a.nb + g;
  const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(x.p) + b * x.sb + kh * x.sh +
                           static_cast<long long>(g) * a.block * x.sn + ch * 8;
  uint32_t mx[4];  // by column
  auto finite_only = [](uint32_t w) {
    return ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0xffffu) | ((w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0xffff0000u);
  };
  int pass = 0;  // a second one without what is not finite, where there is such
  for (;; ++pass) {
    uint4 v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      v[i] = r0 + i * kRows < rows ? *reinterpret_cast<const uint4*>(p + (r0 + i * kRows) * x.sn) : make_uint4(0, 0, 0, 0);
    uint32_t row[kPer];
#pragma unroll
    for (int w = 0; w < 4; ++w) mx[w] = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (pass > 0) u[w] = finite_only(u[w]);
        mx[w] = max_abs_bf16x2(mx[w], u[w]);
      }
      row[i] = max_abs_bf16x2(max_abs_bf16x2(u[0], u[1]), max_abs_bf16x2(u[2], u[3]));
    }
    if (!BACKWARD) {
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {  // two rows a word
        uint32_t m = max_abs_bf16x2(__byte_perm(row[i], row[i + 1], 0x5410), __byte_perm(row[i], row[i + 1], 0x7632));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = max_abs_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (ch == 0) s_row[r0 + i * kRows] = m & 0x7fffu, s_row[r0 + (i + 1) * kRows] = m >> 16 & 0x7fffu;
      }
    }
    bool finite = true;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
#pragma unroll
      for (int o = L; o < 32; o <<= 1) mx[w] = max_abs_bf16x2(mx[w], __shfl_xor_sync(0xffffffffu, mx[w], o));
      finite = finite && (mx[w] & 0x7f80u) != 0x7f80u && (mx[w] & 0x7f800000u) != 0x7f800000u;
    }
    if (lane < L) s_mx[warp][lane] = make_uint4(mx[0], mx[1], mx[2], mx[3]);
    if (__syncthreads_and(finite) || pass > 0) break;
  }
  if (warp > 0) return;
#pragma unroll
  for (int w = 1; w < 8; ++w) {
    const uint4 v = s_mx[w][ch];
    mx[0] = max_abs_bf16x2(mx[0], v.x), mx[1] = max_abs_bf16x2(mx[1], v.y);
    mx[2] = max_abs_bf16x2(mx[2], v.z), mx[3] = max_abs_bf16x2(mx[3], v.w);
  }
  int top = 0, low = 0x7fff;  // magnitudes' bits: ordered as integers
#pragma unroll
  for (int w = 0; w < 4; ++w)
#pragma unroll
    for (int i = 0; i < 32; i += 16) {
      const int m = static_cast<int>(mx[w] >> i & 0x7fffu);
      top = max(top, m);
      if (m != 0) low = min(low, m);
    }
  top = __reduce_max_sync(0xffffffffu, top);
  float k = 0.f;
  bool wide = pass > 0;
  if (!BACKWARD) {
    const int extra = (a.block == 128 ? 7 : 6) - 15;
    // |V| < 2^((bits >> 7) - 126); zeros take any k
    auto k_of = [&](int bits) { return bits == 0 ? 0 : max((bits >> 7) - 126 + extra, -120); };
    const int per = a.block / 32;  // a lane's rows
    int run = 0;                   // over the lanes before this one
    for (int i = 0; i < per; ++i) {
      const int r = lane * per + i, m = r < rows ? s_row[r] : 0;
      run = max(run, m);
      if (m != 0) low = min(low, m);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run = max(run, y);
    }
    run = __shfl_up_sync(0xffffffffu, run, 1);
    if (lane == 0) run = 0;
    for (int i = 0; i < per && lane * per + i < rows; ++i) {
      run = max(run, s_row[lane * per + i]);
      a.key_range[at * a.block + lane * per + i] = static_cast<signed char>(k_of(run));
    }
    k = static_cast<float>(k_of(top));
  }
  low = __reduce_min_sync(0xffffffffu, low);
  wide = wide || (top >> 7) > (low >> 7) + (BACKWARD ? 24 : k == p_share(k) ? 20 : 8);
  // (infinite: P is divided by so much that a value of O may have become 0 by it)
  if (lane == 0) a.range[at] = !wide ? k : k > 20.f ? kInf : __builtin_nanf("");
}

template <int D, int B>
cudaError_t forward(const SelArgs& a, int first, int count, cudaStream_t st) {
  BlockMap mk, mv;
  if (!block_map(&mk, a.k, a, B) || !block_map(&mv, a.v, a, B)) return cudaErrorInvalidValue;
  auto kern = selected_forward_tc_kernel<D, B>;
  constexpr int smem = static_cast<int>(Fwd<D, B>::kSmem);
  // the register split must fit in what a block is launched with, or its increase would wait for good
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (128 * (2 * kRegSoftmax + kRegOut + 2 * kRegRest) > fa.numRegs * kThreads) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<kShares, kThreads, smem, st>>>(mk, mv, a, first, count);
  if ((e = counted(cudaGetLastError(), 1)) != cudaSuccess) return e;
  return launch_join_half(a, first, count, false, st);
}

}  // namespace

cudaError_t launch_ranges(const SelArgs& a, bool backward, cudaStream_t st) {
  const dim3 grid(a.nb, a.Hk, a.Bt);
  if (a.d == 128)
    backward ? ranges_kernel<128, true><<<grid, 256, 0, st>>>(a, a.k) : ranges_kernel<128, false><<<grid, 256, 0, st>>>(a, a.v);
  else
    backward ? ranges_kernel<64, true><<<grid, 256, 0, st>>>(a, a.k) : ranges_kernel<64, false><<<grid, 256, 0, st>>>(a, a.v);
  return counted(cudaGetLastError(), 1);
}

cudaError_t launch_join_half(const SelArgs& a, int first, int count, bool grad, cudaStream_t st) {
  const long long rows = static_cast<long long>(count) * a.slice * a.group;
  const int per_cta = 8 * (32 / (a.d / 8));
  const unsigned grid = static_cast<unsigned>((rows + per_cta - 1) / per_cta);
  if (a.d == 128)
    grad ? join_half_kernel<128, true><<<grid, 256, 0, st>>>(a, first, count)
         : join_half_kernel<128, false><<<grid, 256, 0, st>>>(a, first, count);
  else
    grad ? join_half_kernel<64, true><<<grid, 256, 0, st>>>(a, first, count)
         : join_half_kernel<64, false><<<grid, 256, 0, st>>>(a, first, count);
  return counted(cudaGetLastError(), 1);
}

bool block_map(BlockMap* m, const View& v, const SelArgs& a, int rows) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess && q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
  }();
  if (fn == nullptr) return false;
  // a repeated (stride 0) dimension is one of size 1, always read at 0
  m->h = v.sh != 0 ? 1 : 0;
  m->b = v.sb != 0 ? 1 : 0;
  const long long row = static_cast<long long>(a.d) * 2;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.d), static_cast<cuuint64_t>(a.nk), static_cast<cuuint64_t>(m->h ? a.Hk : 1),
                        static_cast<cuuint64_t>(m->b ? a.Bt : 1)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(v.sn ? v.sn * 2 : row), static_cast<cuuint64_t>(v.sh ? v.sh * 2 : row),
                           static_cast<cuuint64_t>(v.sb ? v.sb * 2 : row)};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(&m->map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_selected_forward_tc(const SelArgs& a, int first, int count, cudaStream_t st) {
  if (a.d == 128) return a.block == 128 ? forward<128, 128>(a, first, count, st) : forward<128, 64>(a, first, count, st);
  return a.block == 128 ? forward<64, 128>(a, first, count, st) : forward<64, 64>(a, first, count, st);
}

}  // namespace spr
