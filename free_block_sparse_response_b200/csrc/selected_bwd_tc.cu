// Backward pass of selected-block attention on the 5th-generation tensor cores (bf16).
//
// Mathematics as in selected_attn.cu.  A tile is 128 of the query rows that selected a block;
// with Q and dO (128 x D) gathered and K and V (B x D) of the block in shared memory,
//   S = Q K^T, dP = dO V^T                        (128 x B, TMEM)
//   P = exp(S tau - lse), dS = P (dP - delta)     (bf16, shared memory; tau joins the outputs)
//   dQ part = dS K (128 x D),  dV^T += dO^T P,  dK^T += Q^T dS  (D x B, TMEM across the tiles)
// dV and dK are formed transposed, so that their M is D and both operands are read as they lie
// (rows of the contraction).  At D = 64 one product with M = 128 does both: [dO | Q]^T [P | dS],
// whose diagonal quarters are dV^T and dK^T.
//
// Every CTA takes an equal, contiguous share of the tiles in the order region, block, row.  A
// block inside one share is written directly; a block that a share's end cuts leaves one fp32
// sum per CTA (two slots each), added in order by join_kv_tc_kernel: the same in every run.
// dQ parts go out as in the forward pass (fp16 with a power of two per row, whole rows).
//
// Work of a tile (B = D = 128): 21 MFLOP, 16K exponentials, 64 KB gathered, 32 KB written.
// Shared memory (7 tiles of 32 KB) holds K, V, P, dS, one dO and two Q; TMEM is full (S, dP, dV^T,
// dK^T; dQ goes over dP).  So dO is gathered as soon as dV has read it, under the products of dK
// and dQ; Q a tile ahead; S of the next tile runs under dQ's way out.
//   warps 0-7    softmax: two threads a row, half the keys each; at a block's end dK and dV;
//   warps 8-11   dQ parts out of TMEM;
//   warps 12-15  gather Q and dO rows, their lse, delta and visible keys (three tiles deep: list
//                entry, numbers, rows);
//   warp 16      issues the products;  warp 17 TMA boxes of K and V, zeros from the length on.
//
// P and dS are rounded to bf16 as operands: 2^-8 of each at most, with signs of their own, so that
// dV and dK lose about as much again as their own rounding takes (2.3e-3 against 1.7e-3 in the norm).
// Bound by the chain of the products and the softmax of one tile at a time (tensor pipe 29%
// active): 16 heads x 32,760 tokens, 8 of 256 blocks, 1.24 ms, 550 TFLOP/s.
#include <cuda.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "selected.cuh"
#include "selected_tc.cuh"
#include "tcgen05.cuh"
#include "warp_mma.cuh"

namespace spr {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInf = __builtin_huge_valf();

constexpr int kThreads = 640, kWork = 256, kLoaders = 128;
constexpr int kOutWarp = 8, kLoadWarp = 12, kMmaWarp = 16, kKvWarp = 17;
constexpr int kRegSoftmax = 112, kRegOut = 104, kRegLoad = 88, kRegRest = 56;

template <int D, int B>
struct Bwd {
  static constexpr uint32_t kRowsD = 128 * D * 2, kRowsB = 128 * B * 2, kKV = B * D * 2;
  static constexpr uint32_t kNums = 128 * 9;  // lse, delta and visible keys (a byte) of a tile's rows
  static constexpr uint32_t kTail = 2 * kNums + 512;
  // dK and dV leave through 4 KB a warp: at B = 128 where the warp's own part of P lies
  static constexpr uint32_t kStage = B == 128 ? 0 : 8 * 4096;
  static constexpr uint32_t kSmem = 2 * kKV + 2 * kRowsB + 3 * kRowsD + kStage + kTail;
};
static_assert(Bwd<128, 128>::kSmem <= 227 * 1024, "the largest form fits an SM");

enum : int {
  kKvLand = 0, kKv, kKvFree, kS, kP, kDq, kDqFree, kAcc, kAccFree, kDrain, kG, kGFree, kQ, kQFree = kQ + 2,
  kNumBars = kQFree + 2
};

template <int D, int B>
__global__ void __launch_bounds__(kThreads, 1)
    selected_backward_tc_kernel(const __grid_constant__ BlockMap mk, const __grid_constant__ BlockMap mv, const SelArgs a,
                                int first, int count) {
  using F = Bwd<D, B>;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  uint8_t* const tail = dsmem + F::kSmem - F::kTail;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(tail);
  uint8_t* const s_num = tail + 512;  // [Q stage]: lse [128], delta [128], visible keys [128]
  uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(bars + kNumBars);
  int& abort_flag = *reinterpret_cast<int*>(bars + kNumBars + 1);
  int* const s_first = reinterpret_cast<int*>(bars + kNumBars + 2);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sK = tc::saddr(dsmem), sV = sK + F::kKV, sP = sV + F::kKV, sdS = sP + F::kRowsB, sRows = sdS + F::kRowsB;
  // dO, then the two Q tiles (at D = 64, dO and Q are one operand of 128 columns)
  const uint32_t sG = sRows;
  auto sQ = [&](int st) { return sRows + (1 + st) * F::kRowsD; };
  if ((sK & 1023u) != 0) {  // the tiles' swizzle counts from 1024-byte lines
    if (tid == 0) record_error(a.status, kErrCuda);
    return;
  }
  auto bar = [&](int i) { return tc::saddr(&bars[i]); };
  if (tid == 0) {
    tc::mbar_init(bar(kKvLand), 1);
    tc::mbar_init(bar(kKv), 32);
    tc::mbar_init(bar(kKvFree), 1);
    tc::mbar_init(bar(kS), 1);
    tc::mbar_init(bar(kP), kWork);
    tc::mbar_init(bar(kDq), 1);
    tc::mbar_init(bar(kDqFree), 128);
    tc::mbar_init(bar(kAcc), 1);
    tc::mbar_init(bar(kAccFree), kWork);
    tc::mbar_init(bar(kDrain), 1);
    tc::mbar_init(bar(kG), kLoaders);
    tc::mbar_init(bar(kGFree), 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(kQ + i), kLoaders);
      tc::mbar_init(bar(kQFree + i), 1);
    }
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tc::saddr(&tmem_slot), 512);
    tc::tmem_relinquish();
  }
  if (warp == 0) share_of_tiles(a, first, count, s_first);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tS = tmem_slot, tDp = tS + 128, tAcc = tS + 256;  // dQ over dP; dV^T, then dK^T from column B on
  volatile int* abort_v = &abort_flag;
  const size_t cap = static_cast<size_t>(a.slice) * a.top;
  auto wait1 = [&](int i, int phase) { return wait_bar(bar(i), phase & 1, abort_v, a.status); };
  auto wait = [&](int i, int phase) { return __all_sync(0xffffffffu, wait1(i, phase)); };

  // registers: 96 a thread at launch, 480 x 128 in all; 2 x 112 + 104 + 88 + 56 of them are used
  if (warp < kOutWarp) {
    // ---------------------------------------------------------------- softmax, dK and dV
    tc::setmaxnreg_inc<kRegSoftmax>();
    const int w4 = warp & 3, half = warp >> 2, row = 32 * w4 + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * w4) << 16;
    const float scale2 = a.scale * kLog2e;
    const uint32_t stage = B == 128 ? sP + half * (128 * 128) + w4 * 4096 : sRows + 3 * F::kRowsD + warp * 4096;
    bool cut_open = false;
    each_tile(a, first, s_first, 0, 1, [&](const Unit& un, int, int t, int u, bool opens, bool closes) {
      const int st = t & 1;
      if (!wait(kQ + st, t >> 1) || !wait(kS, t)) return false;  // the row's numbers; S and dP
      tc::fence_after_sync();
      const uint8_t* nums = s_num + st * F::kNums;
      const float lse2 = reinterpret_cast<const float*>(nums)[row], delta = reinterpret_cast<const float*>(nums)[128 + row];
      const int nv = nums[1024 + row];
#pragma unroll 1
      for (int c0 = half * (B / 2); c0 < (half + 1) * (B / 2); c0 += 32) {
        uint32_t s[32], dp[32];
        tc::tmem_ld32(tS + lanes + c0, s);
        tc::tmem_ld32(tDp + lanes + c0, dp);
        tc::tmem_wait_ld();
#pragma unroll
        for (int c8 = 0; c8 < 4; ++c8) {
          uint32_t p4[4], d4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = 8 * c8 + 2 * i;
            float p0 = ex2(fmaf(__uint_as_float(s[c]), scale2, -lse2)), p1 = ex2(fmaf(__uint_as_float(s[c + 1]), scale2, -lse2));
            float d0 = p0 * (__uint_as_float(dp[c]) - delta), d1 = p1 * (__uint_as_float(dp[c + 1]) - delta);
            if (c0 + c >= nv) p0 = d0 = 0.f;
            if (c0 + c + 1 >= nv) p1 = d1 = 0.f;
            p4[i] = pack_bf16x2(p0, p1);
            d4[i] = pack_bf16x2(d0, d1);
          }
          const uint32_t off = tc::sw128_offset(row, c0 / 8 + c8);
          st_shared_16(sP + off, p4[0], p4[1], p4[2], p4[3]);
          st_shared_16(sdS + off, d4[0], d4[1], d4[2], d4[3]);
        }
      }
      tc::fence_proxy_async();
      tc::fence_before_sync();
      tc::mbar_arrive(bar(kP));
      if (opens) cut_open = un.r0 > 0;  // the block's first tiles are another CTA's
      if (!closes) return true;
      // dK and dV: lane = head dim, columns = keys
      if (!wait(kAcc, u)) return false;
      tc::fence_after_sync();
      const bool cut = cut_open || un.r0 + un.rows < un.total;
      const int which = D == 128 ? half : w4 >> 1;  // 0: dV, 1: dK
      const int from = D == 128 ? 0 : half * (B / 2), to = D == 128 ? B : from + B / 2;
      const View& out = which ? a.gk : a.gv;
      const int d0 = D == 128 ? 32 * w4 : 32 * (w4 & 1);  // the warp's first head dim
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out.p) + un.b * out.sb + un.kh * out.sh +
                           static_cast<long long>(un.g) * B * out.sn + d0;
      float* seg = a.seg + (static_cast<size_t>(2 * blockIdx.x + (u > 0)) * 2 + which) * B * D + d0 + lane;
      const float f = which ? a.scale : 1.f;
      const int keys = min(B, a.nk - un.g * B);
#pragma unroll 1
      for (int c0 = from; c0 < to; c0 += 32) {
        uint32_t x[32];
        tc::tmem_ld32(tAcc + lanes + which * B + c0, x);
        tc::tmem_wait_ld();
        if (cut) {
#pragma unroll
          for (int c = 0; c < 32; ++c) seg[static_cast<size_t>(c0 + c) * D] = __uint_as_float(x[c]) * f;
          continue;
        }
        if (a.acc != nullptr) {
          float* acc = a.acc + (static_cast<size_t>(which) * a.nk + un.g * B) * D + d0 + lane;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c0 + c < keys) acc[static_cast<size_t>(c0 + c) * D] += __uint_as_float(x[c]) * f;
          continue;
        }
        // 32 keys x 32 dims turned in shared memory (rows of 80 bytes: no two keys
        // of a group in one bank), so that 4 lanes write 64 bytes of a key
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 32; ++c) st_shared_b16(stage + c * 80 + lane * 2, __float2bfloat16_rn(__uint_as_float(x[c]) * f));
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 32; c += 8) {
          const int key = c + (lane >> 2);
          const uint4 v = ld_shared_16(stage + key * 80 + (lane & 3) * 16);
          if (c0 + key < keys) *reinterpret_cast<uint4*>(dst + (c0 + key) * out.sn + (lane & 3) * 8) = v;
        }
      }
      tc::fence_before_sync();
      tc::mbar_arrive(bar(kAccFree));
      return true;
    });
  } else if (warp < kLoadWarp) {
    // ---------------------------------------------------------------- dQ parts
    tc::setmaxnreg_inc<kRegOut>();
    const int w4 = warp & 3, q = lane >> 2, i = lane & 3;
    uint8_t* const part = static_cast<uint8_t*>(static_cast<void*>(a.part));
    each_tile(a, first, s_first, 0, 1, [&](const Unit& un, int ci, int t, int, bool, bool) {
      const long long out0 = static_cast<long long>((ci * cap + un.off) * a.group + un.r0);
      if (!wait(kDq, t)) return false;
      tc::fence_after_sync();
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int lane0 = 32 * w4 + 16 * half;
        const uint32_t tRow = tDp + (static_cast<uint32_t>(lane0) << 16);
        float up[2];
        if (un.k != un.k) {
          store_wide<D, false>(tRow, true, lane0 + q, un.rows, part + 32 * i, out0, up);
          if (half == 1) {
            tc::fence_before_sync();
            tc::mbar_arrive(bar(kDqFree));
          }
        } else {
          uint32_t o[D / 2];
#pragma unroll
          for (int c = 0; c < D; c += 64) tmem_ld_16x64(tRow + c, *reinterpret_cast<uint32_t(*)[32]>(&o[c / 2]));
          tc::tmem_wait_ld();
          if (half == 1) {
            tc::fence_before_sync();
            tc::mbar_arrive(bar(kDqFree));
          }
          store_part<D>(o, lane0 + q, un.rows, part + 32 * i, out0, up);
        }
        if (i == 0) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (lane0 + q + 8 * k < un.rows) a.ml[out0 + lane0 + q + 8 * k] = make_float2(0.f, up[k] * a.scale);
        }
      }
      return true;
    });
  } else if (warp < kMmaWarp) {
    // ---------------------------------------------------------------- Q and dO rows, 32 a warp
    tc::setmaxnreg_dec<kRegLoad>();
    constexpr int kPer = D / 8, kStep = 32 / kPer;  // lanes per row, rows per instruction
    const int lw = warp - kLoadWarp, ch = lane % kPer, r = 32 * lw + lane;
    struct Row {  // this lane's row of a tile, and what its warp copies from
      const __nv_bfloat16 *q, *g;
      int tok, h, live, qs;
      float lse, delta;
      size_t base;  // row of lse and delta of token 0 of the group's first head
    };
    // The walk is two tiles ahead of the copies: list entry, then the row's numbers, then rows.
    Row fresh{}, known{};
    bool have_fresh = false, have_known = false;
    int t = 0;  // tile whose Q is copied next; dO follows one behind
    auto copy = [&](uint32_t tile, const __nv_bfloat16* from, const View& v, int tok, int h) {
#pragma unroll
      for (int s = 0; s < 32; s += kStep) {
        const int src = s + lane / kPer;
        const long long tk = __shfl_sync(0xffffffffu, tok, src);
        const int hh = __shfl_sync(0xffffffffu, h, src);
        cp_async_16(tile + tc::sw128_offset(32 * lw + src, ch), tk < 0 ? from : from + tk * v.sn + hh * v.sh, tk < 0 ? 0 : 16);
      }
      cp_async_commit();
    };
    Row held{};  // tile t - 1, whose dO is still to be copied
    // dO of tile t - 1 and Q of tile t (either may be none), in flight together
    auto load = [&](const Row* row) {
      if (t > 0) {
        if (t > 1 && !wait(kGFree, t - 2)) return false;
        copy(sG, held.g, a.go, held.tok, held.h);
      }
      if (row != nullptr) {
        const int st = t & 1;
        if (t >= 2 && !wait(kQFree + st, (t >> 1) - 1)) return false;
        uint8_t* nums = s_num + st * F::kNums;
        reinterpret_cast<float*>(nums)[r] = row->lse * kLog2e;
        reinterpret_cast<float*>(nums)[128 + r] = row->delta;
        // no row, or a zero row of the forward pass: nothing visible
        const int nv = min(a.causal ? min(row->live, row->qs + row->tok + 1) : row->live, B);
        nums[1024 + r] = static_cast<uint8_t>(row->tok < 0 || row->lse == -kInf ? 0 : max(nv, 0));
        copy(sQ(st), row->q, a.q, row->tok, row->h);
      }
      if (t > 0) {
        if (row != nullptr)
          cp_async_wait<1>();
        else
          cp_async_wait<0>();
        tc::fence_proxy_async();
        tc::mbar_arrive(bar(kG));
      }
      if (row != nullptr) {
        cp_async_wait<0>();
        tc::fence_proxy_async();
        tc::mbar_arrive(bar(kQ + (t & 1)));
        held = *row;
        ++t;
      }
      return true;
    };
    auto step = [&]() {  // numbers of the fresh row; copies of the known one
      Row next = fresh;
      const bool ok = !have_known || load(&known);
      if (have_fresh && next.tok >= 0) {
        const size_t at = next.base + static_cast<size_t>(next.h) * a.n + next.tok;
        next.lse = __ldg(a.lse + at);
        next.delta = a.delta[at];
      }
      known = next;
      have_known = have_fresh;
      return ok;
    };
    bool ok = each_tile(a, first, s_first, 0, 1, [&](const Unit& un, int ci, int, int, bool, bool) {
      if (!step()) return false;
      fresh = Row{};
      fresh.q = static_cast<const __nv_bfloat16*>(a.q.p) + un.b * a.q.sb + un.kh * a.group * a.q.sh + ch * 8;
      fresh.g = static_cast<const __nv_bfloat16*>(a.go.p) + un.b * a.go.sb + un.kh * a.group * a.go.sh + ch * 8;
      fresh.tok = -1, fresh.live = un.live, fresh.qs = un.qs;
      fresh.base = (static_cast<size_t>(un.b) * a.Hq + un.kh * a.group) * a.n;
      if (r < un.rows) {
        const int e = (un.r0 + r) / a.group;
        fresh.tok = __ldg(a.list + (first + ci) * cap + un.off + e);
        fresh.h = un.r0 + r - e * a.group;
      }
      have_fresh = true;
      return true;
    });
    if (ok && have_fresh) {
      ok = step();
      have_fresh = false;
      ok = ok && step() && load(nullptr);
    }
    cp_async_wait<0>();
  } else {
    tc::setmaxnreg_dec<kRegRest>();
  }
  if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- products
    constexpr uint32_t kIdS = tc::idesc_bf16(128, B, false, false), kIdQ = tc::idesc_bf16(128, D, false, true);
    constexpr uint32_t kIdAcc = tc::idesc_bf16(128, D == 128 ? B : 2 * B, true, true);
    // the whole warp walks and waits, lane 0 issues
    {
      const int tiles = s_first[2];
      auto issue_s = [&](int t) {  // once Q of the tile is there
        if (!wait(kQ + (t & 1), t >> 1)) return false;
        tc::fence_after_sync();
        uint64_t dq = tc::sdesc_sw128(sQ(t & 1), 16, 1024), dk = tc::sdesc_sw128(sK, 16, 1024);
        keep_here(dq, dk);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          if (lane == 0) tc::mma_ss(tS, dq + ((kk >> 2) * (128 * 128) + (kk & 3) * 32) / 16,
                     dk + ((kk >> 2) * (B * 128) + (kk & 3) * 32) / 16, kIdS, kk > 0 ? 1u : 0u);
        return true;
      };
      if (tiles > 0 && wait(kKv, 0) && issue_s(0))
        each_tile(a, first, s_first, 0, 1, [&](const Unit&, int, int t, int u, bool opens, bool closes) {
          const int st = t & 1;
          if (!wait(kG, t)) return false;
          if (t > 0 && !wait(kDqFree, t - 1)) return false;  // dQ, over dP, is read
          tc::fence_after_sync();
          uint64_t dg = tc::sdesc_sw128(sG, 16, 1024), dv = tc::sdesc_sw128(sV, 16, 1024);
          keep_here(dg, dv);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            if (lane == 0) tc::mma_ss(tDp, dg + ((kk >> 2) * (128 * 128) + (kk & 3) * 32) / 16,
                       dv + ((kk >> 2) * (B * 128) + (kk & 3) * 32) / 16, kIdS, kk > 0 ? 1u : 0u);
          if (lane == 0) tc::mma_commit(bar(kS));
          if (!wait(kP, t)) return false;
          if (opens && u > 0 && !wait(kAccFree, u - 1)) return false;
          tc::fence_after_sync();
          // dV first, so that the next dO can be gathered, then dQ, so that its way out runs under dK
          // and the next S.  Contraction over the 128 rows: both operands rows apart, 64-column blocks of P and dS
          // 16 KB apart, of dO (at D = 64: of dO and Q) as they lie
          uint64_t gt = tc::sdesc_sw128(sG, D == 128 ? 128 * 128 : sQ(st) - sG, 1024);
          uint64_t pt = tc::sdesc_sw128(sP, 128 * 128, 1024);
          keep_here(gt, pt);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            if (lane == 0) tc::mma_ss(tAcc, gt + kk * (2048 / 16), pt + kk * (2048 / 16), kIdAcc, !opens || kk > 0 ? 1u : 0u);
          if (lane == 0) tc::mma_commit(bar(kGFree));
          if (D == 64 && lane == 0) tc::mma_commit(bar(kQFree + st));
          uint64_t ds = tc::sdesc_sw128(sdS, 16, 1024), kt = tc::sdesc_sw128(sK, B * 128, 1024);
          keep_here(ds, kt);
#pragma unroll
          for (int kk = 0; kk < B / 16; ++kk)
            if (lane == 0) tc::mma_ss(tDp, ds + ((kk >> 2) * (128 * 128) + (kk & 3) * 32) / 16, kt + kk * (2048 / 16), kIdQ, kk > 0 ? 1u : 0u);
          if (lane == 0) tc::mma_commit(bar(kDq));
          if (D == 128) {
            uint64_t qt = tc::sdesc_sw128(sQ(st), 128 * 128, 1024), dt = tc::sdesc_sw128(sdS, 128 * 128, 1024);
            keep_here(qt, dt);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              if (lane == 0) tc::mma_ss(tAcc + B, qt + kk * (2048 / 16), dt + kk * (2048 / 16), kIdAcc, !opens || kk > 0 ? 1u : 0u);
            if (lane == 0) tc::mma_commit(bar(kQFree + st));
          }
          if (closes) {
            if (lane == 0) tc::mma_commit(bar(kAcc));
            if (lane == 0) tc::mma_commit(bar(kKvFree));
          }
          // S of the next tile: the softmax has read this one's
          if (t + 1 < tiles && ((closes && !wait(kKv, u + 1)) || !issue_s(t + 1))) return false;
          return true;
        });
      if (lane == 0) {
        tc::mma_commit(bar(kDrain));  // every product has finished before TMEM goes back
        tc::mbar_wait_quiet(bar(kDrain), 0);
      }
      __syncwarp();
    }
  } else if (warp == kKvWarp) {
    // ---------------------------------------------------------------- K and V of each block
    int issued = 0;
    const bool ok = each_tile(a, first, s_first, 0, 1, [&](const Unit& un, int, int, int u, bool opens, bool) {
      if (!opens) return true;
      if (u > 0 && !wait(kKvFree, u - 1)) return false;
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(bar(kKvLand), 2 * F::kKV);
#pragma unroll
        for (int c = 0; c < D; c += 64) {
          load_box(sK + c * (B * 2), mk, c, un.g * B, un.kh, un.b, bar(kKvLand));
          load_box(sV + c * (B * 2), mv, c, un.g * B, un.kh, un.b, bar(kKvLand));
        }
      }
      __syncwarp();
      issued = u + 1;
      if (!wait(kKvLand, u)) return false;
      for (int i = lane; i < (B - un.live) * (D / 8); i += 32) {  // rows of the block from the length on
        const uint32_t off = sw128_rows<B>(un.live + i / (D / 8), i % (D / 8));
        st_shared_zero(sK + off);
        st_shared_zero(sV + off);
      }
      tc::fence_proxy_async();
      tc::mbar_arrive(bar(kKv));
      return true;
    });
    // boxes still in flight after an abort land before the CTA exits
    if (!ok && lane == 0 && issued > 0) tc::mbar_wait_quiet(bar(kKvLand), (issued - 1) & 1);
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc::fence_after_sync();
    tc::tmem_dealloc(tS, 512);
  }
}

// dK and dV of the blocks that shares cut (their CTAs' sums, in order) and of blocks that no
// query selected (SLICES: sums added to a.acc); `shares` CTAs ran the backward kernel.  A CTA looks at eight blocks of a
// region, a warp each (most were written already), then works on those left, four loads a
// thread under way.
template <int D, bool SLICES>
__global__ void __launch_bounds__(256) join_kv_tc_kernel(const SelArgs a, int first, int count, int shares) {
  __shared__ int s_c0[8], s_c1[8], s_slot[8];  // shares of the block (c0 > c1: none, -1: nothing to do), slot of c0
  const int ci = blockIdx.y, region = first + ci, z = region / a.slices, b = z / a.Hk, kh = z % a.Hk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g0 = blockIdx.x * 8;
  int all = 0, before = 0;
  for (int i = lane; i < count; i += 32) {
    const int n = __ldg(a.n_units + first + i);
    all += n;
    if (i < ci) before += n;
  }
  const long long sum = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  // first tile of share c
  auto start = [&](int c) { return sum * c / shares; };
  if (lane == 0) {
    int c0 = -1, c1 = -1, slot = 0;
    if (g0 + warp < a.nb) {
      const int4 bk = a.blk[static_cast<size_t>(region) * a.nb + g0 + warp];  // tiles, -, first tile of its region
      if (bk.x == 0) {
        c0 = SLICES ? -1 : 0;  // zeros
      } else {
        const long long t0 = static_cast<long long>(before) + bk.z;
        auto share = [&](long long t) {
          int c = static_cast<int>(t * shares / sum);
          while (start(c + 1) <= t) ++c;
          while (start(c) > t) --c;
          return c;
        };
        c0 = share(t0), c1 = share(t0 + bk.x - 1);
        // the block is the first run of a share that starts at it or inside it, else the last
        slot = 2 * c0 + (start(c0) >= t0 ? 0 : 1);
        if (c0 == c1) c0 = c1 = -1;  // written by its one CTA
      }
    }
    s_c0[warp] = c0, s_c1[warp] = c1, s_slot[warp] = slot;
  }
  __syncthreads();
  const size_t tile = static_cast<size_t>(a.block) * D;
  constexpr int kBatch = 4;
  for (int w = 0; w < 8; ++w) {
    const int c0 = s_c0[w], c1 = s_c1[w], g = g0 + w;
    if (c0 < 0) continue;
    for (int i0 = threadIdx.x * 4; i0 < a.block * D; i0 += kBatch * 1024) {
      float4 x[kBatch], y[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) x[k] = y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c = c0; c <= c1; ++c) {
        if (start(c) == start(c + 1)) continue;  // an empty share
        const size_t slot = c == c0 ? s_slot[w] : 2 * c;
        float4 u[kBatch], v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (i0 + k * 1024 < a.block * D) {
            u[k] = *reinterpret_cast<const float4*>(a.seg + (2 * slot + 1) * tile + i0 + k * 1024);
            v[k] = *reinterpret_cast<const float4*>(a.seg + 2 * slot * tile + i0 + k * 1024);
          }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (i0 + k * 1024 < a.block * D) {
            x[k].x += u[k].x, x[k].y += u[k].y, x[k].z += u[k].z, x[k].w += u[k].w;
            y[k].x += v[k].x, y[k].y += v[k].y, y[k].z += v[k].z, y[k].w += v[k].w;
          }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * 1024, j = g * a.block + i / D;
        if (i >= a.block * D || j >= a.nk) continue;
        if (SLICES) {
          float4* v4 = reinterpret_cast<float4*>(a.acc + static_cast<size_t>(j) * D + i % D);
          float4* k4 = reinterpret_cast<float4*>(a.acc + (static_cast<size_t>(a.nk) + j) * D + i % D);
          const float4 v0 = *v4, k0 = *k4;
          *v4 = make_float4(v0.x + y[k].x, v0.y + y[k].y, v0.z + y[k].z, v0.w + y[k].w);
          *k4 = make_float4(k0.x + x[k].x, k0.y + x[k].y, k0.z + x[k].z, k0.w + x[k].w);
          continue;
        }
        __nv_bfloat16* dk = static_cast<__nv_bfloat16*>(a.gk.p) + b * a.gk.sb + kh * a.gk.sh + j * a.gk.sn + i % D;
        __nv_bfloat16* dv = static_cast<__nv_bfloat16*>(a.gv.p) + b * a.gv.sb + kh * a.gv.sh + j * a.gv.sn + i % D;
        *reinterpret_cast<uint2*>(dk) = make_uint2(pack_bf16x2(x[k].x, x[k].y), pack_bf16x2(x[k].z, x[k].w));
        *reinterpret_cast<uint2*>(dv) = make_uint2(pack_bf16x2(y[k].x, y[k].y), pack_bf16x2(y[k].z, y[k].w));
      }
    }
  }
}

template <int D, int B>
cudaError_t backward(const SelArgs& a, int first, int count, cudaStream_t st) {
  BlockMap mk, mv;
  if (!block_map(&mk, a.k, a, B) || !block_map(&mv, a.v, a, B)) return cudaErrorInvalidValue;
  auto kern = selected_backward_tc_kernel<D, B>;
  constexpr int smem = static_cast<int>(Bwd<D, B>::kSmem);
  // the register split must fit in what a block is launched with, or its increase would wait for good
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (128 * (2 * kRegSoftmax + kRegOut + kRegLoad + kRegRest) > fa.numRegs * kThreads) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<kShares, kThreads, smem, st>>>(mk, mv, a, first, count);
  if ((e = counted(cudaGetLastError(), 1)) != cudaSuccess) return e;
  const dim3 grid(ceil_div(a.nb, 8), count);
  a.acc == nullptr ? join_kv_tc_kernel<D, false><<<grid, 256, 0, st>>>(a, first, count, kShares)
                   : join_kv_tc_kernel<D, true><<<grid, 256, 0, st>>>(a, first, count, kShares);
  if ((e = counted(cudaGetLastError(), 1)) != cudaSuccess) return e;
  return launch_join_half(a, first, count, true, st);
}

}  // namespace

cudaError_t launch_selected_backward_tc(const SelArgs& a, int first, int count, cudaStream_t st) {
  if (a.d == 128) return a.block == 128 ? backward<128, 128>(a, first, count, st) : backward<128, 64>(a, first, count, st);
  return a.block == 128 ? backward<64, 128>(a, first, count, st) : backward<64, 64>(a, first, count, st);
}

}  // namespace spr
