// Device helpers shared by the tensor-core kernels of selected-block attention.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <algorithm>

#include "selected.cuh"
#include "tcgen05.cuh"

namespace spr {

// TMA map over a K or V view as (d, rows, heads, batch), boxes of 64 columns x one key block;
// h and b are 0 where the view repeats one head or batch element.
struct BlockMap {
  CUtensorMap map;
  int h, b;
};
bool block_map(BlockMap* m, const View& v, const SelArgs& a, int rows);

// The box at (column, row, head, batch) into `dst`; column is a multiple of 64 and rows past
// the tensor's end arrive as zeros.
__device__ __forceinline__ void load_box(uint32_t dst, const BlockMap& m, int col, int row, int h, int b, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(&m.map)), "r"(col), "r"(row), "r"(m.h ? h : 0), "r"(m.b ? b : 0), "r"(bar)
      : "memory");
}

// Byte offset of 16-byte chunk `ch` of row `r` in a 128-byte-swizzled tile of `ROWS` rows.
template <int ROWS>
__device__ __forceinline__ uint32_t sw128_rows(int r, int ch) {
  return static_cast<uint32_t>((ch >> 3) * (ROWS * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

// tc::mbar_wait with the bound counted in SM cycles (4e9: about two seconds) and looked at only
// every 64th try: a wait here is a microsecond in a chain of five per tile, and reading the
// global timer takes as long.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (tc::mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > 4000000000ll) {
      record_error(status, kErrTimeout);
      *abort_flag = 1;
      return false;
    }
  }
}

// Keeps what is computed from x and y inside the loop around it: a matrix descriptor of every
// step of a product, formed ahead of the loop, would hold registers until they spill.
__device__ __forceinline__ void keep_here(uint64_t& x, uint64_t& y) { asm volatile("" : "+l"(x), "+l"(y)); }

__device__ __forceinline__ void st_shared_zero(uint32_t addr) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

__device__ __forceinline__ void st_shared_16(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ void st_shared_b16(uint32_t addr, __nv_bfloat16 x) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(__bfloat16_as_ushort(x)) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// 32 bytes in one store: a whole sector per thread.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 16 TMEM lanes x 64 columns: lane 4 q + i of the warp gets row q (registers 4 j, 4 j + 1) and
// row q + 8 (4 j + 2, 4 j + 3) of columns 8 j + 2 i and 8 j + 2 i + 1, j < 8.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// The same for 8 columns.
__device__ __forceinline__ void tmem_ld_16x8(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}

// Partial rows of 2 D bytes, 128-byte lines of 64 columns.  First column of the c-th pair of
// 16-byte chunk `ch` of a row (8 chunks a line): the four lanes of a quad, which hold columns
// 2 i, 2 i + 1 of every eight, write 32 bytes each.
__device__ __forceinline__ int part_column(int ch, int c) {
  return (ch >> 3) * 64 + ((ch & 1) * 4 + c) * 8 + ((ch & 7) >> 1) * 2;
}

// Whether the phase with this parity has completed, without waiting.
__device__ __forceinline__ bool bar_done(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Powers of two with big * down in [2^14, 2^15), the upper end of fp16, and up * down = 1 (below
// 2^-112: as for 2^-112).
__device__ __forceinline__ void part_scale(float big, float& up, float& down) {
  const uint32_t e = max(__float_as_uint(big) >> 23, 15u);
  up = __uint_as_float((e - 14) << 23);
  down = __uint_as_float((268 - e) << 23);
}

// The tensor-core kernels run one CTA per SM; CTA c takes tiles [sum c / shares, sum (c + 1) /
// shares) of a chunk's `sum` tiles, in the order region, block, row.
constexpr int kShares = kTcShares;

// This CTA's share, by one warp: share[0], share[1] its first tile (region of the chunk, tile
// of the region), share[2] its number of tiles.
__device__ __forceinline__ void share_of_tiles(const SelArgs& a, int first, int count, int* share) {
  const int lane = threadIdx.x & 31;
  int sum = 0;
  for (int i = lane; i < count; i += 32) sum += __ldg(a.n_units + first + i);
  sum = __reduce_add_sync(0xffffffffu, sum);
  const int lo = static_cast<int>(static_cast<long long>(sum) * blockIdx.x / gridDim.x);
  const int hi = static_cast<int>(static_cast<long long>(sum) * (blockIdx.x + 1) / gridDim.x);
  if (lane == 0) {
    int ci = 0, before = 0, n = 0;
    while (ci < count && before + (n = __ldg(a.n_units + first + ci)) <= lo) before += n, ++ci;
    share[0] = ci, share[1] = lo - before, share[2] = hi - lo;
  }
}

// The tiles from, from + step, .. of a CTA's share, in order (a stream's warps take every second
// one); contiguous shares change K and V seldom.  Called by whole warps: the lanes read the records
// of the next 32 tiles at once and hand them out by shuffles.  (One record a tile read ahead in
// registers costs its full latency, ~700 cycles, at the move that carries it through the loop.)
// f(record, region of the chunk, tile, unit = run of tiles of one block, opens it, closes it);
// the last three hold at step 1.
template <typename F>
__device__ __forceinline__ bool each_tile(const SelArgs& a, int first, const int* share, int from, int step, F f) {
  const int lane = threadIdx.x & 31, tiles = share[2];
  int base_ci = share[0], base_idx = share[1], base_t = 0;  // a known place: tile base_t
  Unit rec{};
  int rec_ci = 0, u = 0;
  unsigned ends = 0;
  bool opens = true;
  for (int i = 0, t = from; t < tiles; ++i, t += step) {
    if ((i & 31) == 0) {
      const int mine = min(t + lane * step, tiles - 1);
      int ci = base_ci, idx = base_idx + mine - base_t, n;
      while (idx >= (n = __ldg(a.n_units + first + ci))) idx -= n, ++ci;
      const Unit* at = a.units + static_cast<size_t>(first + ci) * a.unit_cap + idx;
      rec = *at;
      rec_ci = ci;
      const bool end = mine + 1 == tiles || idx + 1 == n || at[1].g != rec.g;
      ends = __ballot_sync(0xffffffffu, end);
      base_ci = __shfl_sync(0xffffffffu, ci, 0), base_idx = __shfl_sync(0xffffffffu, idx, 0), base_t = t;
    }
    const int src = i & 31;
    auto get = [&](int x) { return __shfl_sync(0xffffffffu, x, src); };
    Unit un;
    un.g = get(rec.g), un.off = get(rec.off), un.r0 = get(rec.r0), un.rows = get(rec.rows), un.live = get(rec.live);
    un.qs = get(rec.qs), un.b = get(rec.b), un.kh = get(rec.kh), un.total = get(rec.total);
    un.k = __int_as_float(get(__float_as_int(rec.k)));
    const bool closes = (ends >> src) & 1u;
    if (!f(un, get(rec_ci), t, u, opens, closes)) return false;
    opens = closes;
    u += closes;
  }
  return true;
}

// Rows r and r + 8 of a tile, held by the quad's lanes as tmem_ld_16x64 leaves them (D / 2
// registers), to the partial rows out0 + r of a chunk: fp16, the row's largest magnitude scaled to
// [2^14, 2^15), so that 11 bits are left to everything down to 2^-29 of it and the rest is off by at
// most 2^-39 of it; up[k] is the power of two that undoes it.  The two rows go side by side, since
// this is bound by its latencies.  `part` is the lane's 32 bytes of row 0.  For blocks that are not
// wide (ranges_kernel).
template <int D>
__device__ __forceinline__ void store_part(const uint32_t (&o)[D / 2], int r, int rows, uint8_t* part, long long out0,
                                           float (&up)[2]) {
  float big[2][2] = {}, mx[2], g[2];
#pragma unroll
  for (int c = 0; c < D / 2; c += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      big[k & 1][k >> 1] = fmax3(big[k & 1][k >> 1], fabsf(__uint_as_float(o[c + 2 * k])), fabsf(__uint_as_float(o[c + 2 * k + 1])));
#pragma unroll
  for (int k = 0; k < 2; ++k) mx[k] = fmaxf(big[k][0], big[k][1]);
#pragma unroll
  for (int m = 1; m < 4; m <<= 1)
#pragma unroll
    for (int k = 0; k < 2; ++k) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], m));
#pragma unroll
  for (int k = 0; k < 2; ++k) part_scale(mx[k], up[k], g[k]);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (r + 8 * k >= rows) continue;
    const uint64_t g2 = f32x2(g[k], g[k]);
#pragma unroll
    for (int c = 0; c < D; c += 64) {
      uint32_t h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float x, y;
        f32x2_split(fmul2(f32x2(__uint_as_float(o[c / 2 + 4 * j + 2 * k]), __uint_as_float(o[c / 2 + 4 * j + 2 * k + 1])), g2), x, y);
        const __half2 v = __floats2half2_rn(x, y);
        h[j] = *reinterpret_cast<const uint32_t*>(&v);
      }
      st_global_32(part + (out0 + r + 8 * k) * (2 * D) + c * 2, h);
    }
  }
}

// The same without a scale: the values are inside fp16.
template <int D>
__device__ __forceinline__ void store_part_as_is(const uint32_t (&o)[D / 2], int r, int rows, uint8_t* part,
                                                 long long out0) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (r + 8 * k >= rows) continue;
#pragma unroll
    for (int c = 0; c < D; c += 64) {
      uint32_t h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __half2 v = __floats2half2_rn(__uint_as_float(o[c / 2 + 4 * j + 2 * k]), __uint_as_float(o[c / 2 + 4 * j + 2 * k + 1]));
        h[j] = *reinterpret_cast<const uint32_t*>(&v);
      }
      st_global_32(part + (out0 + r + 8 * k) * (2 * D) + c * 2, h);
    }
  }
}

// The parts of a wide block, straight from TMEM, without a scale (AS_IS) or with the rows' own.  A value
// that fp16 cannot hold goes out as a NaN: one below its normal range (but a 0 where `zeros` are to be
// trusted), above it, or a NaN, as 0 times a hidden NaN is.  The row's sum keeps it, and mend_kernel then forms
// it again from the inputs.  Eight columns at a time, twice with a scale: 5 and 10 us a tile, but small.
// Wider or unrolled code here, though never run, slowed the kernels by 3 to 30%.
template <int D, bool AS_IS>
__device__ __forceinline__ void store_wide(uint32_t taddr, bool zeros, int r, int rows, uint8_t* part, long long out0,
                                           float (&up)[2]) {
  float g[2] = {1.f, 1.f};
  uint32_t o[4];
  if (!AS_IS) {
    float mx[2] = {};
#pragma unroll 1
    for (int j = 0; j < D / 8; ++j) {
      tmem_ld_16x8(taddr + 8 * j, o);
      tc::tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float x = fabsf(__uint_as_float(o[c]));
        mx[c >> 1] = fmaxf(mx[c >> 1], x < __builtin_huge_valf() ? x : 0.f);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 1));
      mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 2));
      part_scale(mx[k], up[k], g[k]);
    }
  }
#pragma unroll 1
  for (int j = 0; j < D / 8; ++j) {
    tmem_ld_16x8(taddr + 8 * j, o);
    tc::tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float y[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float x = __uint_as_float(o[2 * k + c]);
        y[c] = AS_IS ? x : x * g[k];
        if (!(fabsf(y[c]) >= 0x1p-14f && fabsf(y[c]) <= 0x1p15f) && !(zeros && x == 0.f)) y[c] = __builtin_nanf("");
      }
      if (r + 8 * k < rows)
        *reinterpret_cast<__half2*>(part + (out0 + r + 8 * k) * (2 * D) + (j >> 3) * 128 + (j & 7) * 4) =
            __floats2half2_rn(y[0], y[1]);
    }
  }
}

cudaError_t launch_selected_forward_tc(const SelArgs& a, int first, int count, cudaStream_t st);
cudaError_t launch_selected_backward_tc(const SelArgs& a, int first, int count, cudaStream_t st);
// Joins the parts of a chunk's query rows into a.o and a.lse, or (grad) a.gq.
cudaError_t launch_join_half(const SelArgs& a, int first, int count, bool grad, cudaStream_t st);

}  // namespace spr
