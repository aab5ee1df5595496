// What the kernels of the gradient products share (gemm_grad.hip,
// dgrad_short.hip, wgrad_short.hip):
// their arguments, buffer descriptors, the transposing read and the stores of a
// wavefront's outputs.
#pragma once

#include <hip/hip_runtime.h>

#include "common.h"
#include "gemm_runs.h"

namespace moe {

struct GradArgs {
  const uint8_t* P;   // dC [M][N]
  const uint8_t* Q;   // dgrad: B [G][N][K]; wgrad: A [M][K]
  void* D;            // dgrad: dA [M][K]; wgrad: dB [G][N][K]
  const int32_t* m_indices;
  const int32_t* starts;
  const int32_t* counts;
  int64_t M;
  int N, K, G;
};

// wgrad_short.hip: dB of f32 or bf16, overwritten or (acc) added to.  Arguments are
// checked by the caller; there are fewer than 2^23 tiles of 128 x 128 over all experts.
int32_t launch_wgrad_short(const GradArgs& a, bool f32, bool acc, hipStream_t stream);

// dgrad_short.hip: arguments are checked by the caller; there are fewer than 2^23
// tiles of 128 x 128.
int32_t launch_dgrad_short(const GradArgs& a, hipStream_t stream);

namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) short s16x4;

constexpr int kStep = 64;   // of the reduction
constexpr int kGroupN = 8;  // wgrad: tiles along N of a block of the tile order

using runs::wait_vm;

__device__ __forceinline__ void fence() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}
// A barrier that nothing crosses.
__device__ __forceinline__ void barrier() {
  fence();
  __builtin_amdgcn_s_barrier();
  fence();
}
__device__ __forceinline__ void wait_lds() {
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
}

// No more than `bytes` from base: reads behind them give zeros, writes are dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, bytes > 0 ? bytes : 0, 0x00020000);
}

// Exchanges a of the lanes 16 .. 31 (48 .. 63) with b of the lanes 0 .. 15
// (32 .. 47), and c with d: (a, b, c, d) afterwards.
__device__ __forceinline__ f32x4 swap_rows(float a, float b, float c, float d) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  const auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(c), __float_as_uint(d), false, false);
  return f32x4{__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(q[0]), __uint_as_float(q[1])};
}

// The lanes 8 .. 15 of each 16 take b of the lanes 0 .. 7 for a, and these take
// a of the lanes 8 .. 15 for b.  Done twice, everything is where it was.
__device__ __forceinline__ void trade8(u32x4& a, u32x4& b) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t x = a[e], y = b[e];
    a[e] = __builtin_amdgcn_update_dpp(x, y, 0x128 /* row_ror:8 */, 0xf, 0xc, false);
    b[e] = __builtin_amdgcn_update_dpp(y, x, 0x128, 0xf, 0x3, false);
  }
}

// Stores a wavefront's 64 x 64 outputs (or adds them to what is there): acc[hq][i][j]
// holds, of the 16-column block 2 hq + j, four columns of row 16 i + (lane & 15).
// rd begins at the first one, line is a row's bytes.
//
// A store covers eight rows and a whole 128-byte line of each (16 rows of half a
// line take the texture unit longer), so lanes trade: bf16, first with the lane 16
// on (swap_rows: eight columns in a row, of block 0 in even lane groups and of
// block 1 in odd ones); then the lanes 0 .. 7 of each 16 give the second half of
// their line for the first half of the row eight on (trade8).  Always 8 stores
// (fp32 16), whatever lies outside rd.
template <bool F32, bool ACC>
__device__ __forceinline__ void store64(const f32x4 (&acc)[2][4][2], __amdgpu_buffer_rsrc_t rd, int line, int lane) {
  constexpr int ES = F32 ? 4 : 2;
  constexpr int NQ = F32 ? 2 : 1;  // lines of a row
  const int row = lane & 15, g = lane >> 4;
  const int col = F32 ? g * 4 + (row >> 3) * 16 : (g & 1) * 16 + (g >> 1) * 8 + (row >> 3) * 32;
  const uint32_t off = (row & 7) * line + col * ES;
  u32x4 old[4][NQ][2];
  if constexpr (ACC) {  // all in flight together
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          old[i][q][h] = __builtin_amdgcn_raw_buffer_load_b128(rd, off + (i * 16 + h * 8) * line + q * 128, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t at = off + i * 16 * line;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      u32x4 w[2];
      if constexpr (ACC) trade8(old[i][q][0], old[i][q][1]);
      if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          f32x4 v = acc[q][i][j];
          if constexpr (ACC) v += __builtin_bit_cast(f32x4, old[i][q][j]);
          w[j] = __builtin_bit_cast(u32x4, v);
        }
      } else {
#pragma unroll
        for (int hq = 0; hq < 2; ++hq) {
          const f32x4 v0 = acc[hq][i][0], v1 = acc[hq][i][1];
          if constexpr (ACC) {
            // added in fp32, so that the sum is rounded once
            const auto add = [&](uint32_t o, float lo, float hi) __attribute__((always_inline)) {
              return pack_bf16x2(lo + __uint_as_float(o << 16), hi + __uint_as_float(o & 0xffff0000u));
            };
            const f32x4 s0 = swap_rows(v0[0], v1[0], v0[1], v1[1]), s1 = swap_rows(v0[2], v1[2], v0[3], v1[3]);
            const u32x4 o = old[i][0][hq];
            w[hq] = u32x4{add(o[0], s0[0], s0[2]), add(o[1], s1[0], s1[2]), add(o[2], s0[1], s0[3]), add(o[3], s1[1], s1[3])};
          } else {
            const u32x4 o = __builtin_bit_cast(
                u32x4, swap_rows(__uint_as_float(pack_bf16x2(v0[0], v0[1])), __uint_as_float(pack_bf16x2(v1[0], v1[1])),
                                 __uint_as_float(pack_bf16x2(v0[2], v0[3])), __uint_as_float(pack_bf16x2(v1[2], v1[3]))));
            w[hq] = u32x4{o[0], o[2], o[1], o[3]};
          }
        }
      }
      trade8(w[0], w[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        __builtin_amdgcn_raw_buffer_store_b128(w[h], rd, at + h * 8 * line + q * 128, 0, 0);
    }
  }
}

// An int that this launch does not write, through the scalar cache.
__device__ __forceinline__ int scalar_load(const int32_t* p) {
  return *(const __attribute__((address_space(4))) int32_t*)(reinterpret_cast<uintptr_t>(p));
}

// 16 lanes read four rows of 16 values; each gets four values of one column.
__device__ __forceinline__ s16x4 read_tr(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)(p));
}

}  // namespace
}  // namespace moe
