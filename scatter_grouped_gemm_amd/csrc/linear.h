// What the kernels of the dense product with an epilogue share: arguments, and the
// epilogue of a lane's outputs.
#pragma once

#include "act.h"
#include "common.h"

namespace moe {

struct LinearArgs {
  const uint8_t* A;        // bf16, rows lda bytes apart
  const uint8_t* B;        // bf16 [G][N][K]
  const void* bias;        // [G][N], or null
  const void* residual;    // out's type, rows ldr elements apart, or null
  void* out;               // rows ldo elements apart
  uint16_t* pre;           // [M][N], or null
  const int32_t* m_indices;  // compact layout; null: one matrix
  int64_t M, lda, ldr, ldo;
  int N, K, G, cols;       // cols: of the output
  int bias32, out32;
  int vec;                 // groups of four columns are whole and aligned in every tensor of the epilogue
  int deep;                // compact layout: many rows an expert (linear_wide.hip)
  int vec8;                // groups of eight are, in the tensors of 16-bit values
  ActArgs act;
};

// The kernel that the sizes ask for; arguments are checked by the caller.
int32_t launch_linear(const LinearArgs& a, hipStream_t stream);

// CUs of the current device, rounded down to a multiple of 8; 0: an error.
int linear_cus();

// linear_wide.hip: whether it covers the call, and the launch.
bool linear_wide_covers(const LinearArgs& a);
int32_t launch_linear_wide(const LinearArgs& a, hipStream_t stream);

// linear_thin.hip: of one matrix and few rows.
int32_t launch_linear_thin(const LinearArgs& a, hipStream_t stream);

// Sets vec and vec8 from the other fields.
void linear_alignment(LinearArgs& a);

namespace {

typedef __attribute__((ext_vector_type(2))) uint32_t lin_u32x2;
typedef __attribute__((ext_vector_type(4))) float lin_f4;

__device__ __forceinline__ lin_f4 unpack_bf16x4(lin_u32x2 b) {
  return lin_f4{__uint_as_float(b[0] << 16), __uint_as_float(b[0] & 0xffff0000u),
                __uint_as_float(b[1] << 16), __uint_as_float(b[1] & 0xffff0000u)};
}

// A descriptor of up to 2^32 - 1 bytes: reads behind them give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_u(const uint8_t* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, static_cast<int>(bytes), 0x00020000);
}

// Four values from element `at` of an array of fp32 or bf16; of the columns n .. n + 3
// those below `end` are read, the others 0.
__device__ __forceinline__ lin_f4 load4(const void* p, int f32, int vec, int64_t at, int n, int end) {
  lin_f4 v = {0.f, 0.f, 0.f, 0.f};
  if (vec) {
    if (n < end)
      v = f32 ? *reinterpret_cast<const lin_f4*>(static_cast<const float*>(p) + at)
              : unpack_bf16x4(*reinterpret_cast<const lin_u32x2*>(static_cast<const uint16_t*>(p) + at));
    return v;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < end)
      v[e] = f32 ? static_cast<const float*>(p)[at + e] : bf16_to_f32(static_cast<const uint16_t*>(p)[at + e]);
  return v;
}
__device__ __forceinline__ void store4(void* p, int f32, int vec, int64_t at, int n, int end, lin_f4 v) {
  if (vec) {
    if (n >= end) return;
    if (f32)
      *reinterpret_cast<lin_f4*>(static_cast<float*>(p) + at) = v;
    else
      *reinterpret_cast<lin_u32x2*>(static_cast<uint16_t*>(p) + at) =
          lin_u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < end) {
      if (f32) static_cast<float*>(p)[at + e] = v[e];
      else static_cast<uint16_t*>(p)[at + e] = f32_to_bf16(v[e]);
    }
}

// The bias of columns n .. n + 3 of expert g.
__device__ __forceinline__ lin_f4 bias4(const LinearArgs& a, int g, int n, int end) {
  if (!a.bias) return lin_f4{0.f, 0.f, 0.f, 0.f};
  return load4(a.bias, a.bias32, a.vec, static_cast<int64_t>(g) * a.N + n, n, end);
}

// Row r's output columns n .. n + 3 from the products with bias: p alone, or the
// gate's (p) and the up part's (u).
template <bool GATED>
__device__ __forceinline__ void finish4(const LinearArgs& a, int64_t r, int n, lin_f4 p, lin_f4 u) {
  if (a.pre) {
    store4(a.pre, 0, a.vec, r * a.N + n, n, a.cols, p);
    if constexpr (GATED) store4(a.pre, 0, a.vec, r * a.N + a.cols + n, n, a.cols, u);
  }
  lin_f4 v = GATED ? act::gated4(a.act, p, u) : act::value4(a.act, p);
  if (a.residual) v += load4(a.residual, a.out32, a.vec, r * a.ldr + n, n, a.cols);
  store4(a.out, a.out32, a.vec, r * a.ldo + n, n, a.cols, v);
}

}  // namespace
}  // namespace moe
