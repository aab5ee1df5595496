// The two gradients of the compact grouped product C[r, :] = A[r, :] . B[g(r)]^T:
//   dA[r, :] = dC[r, :] . B[g(r)]          (grouped_gemm_contig_dgrad)
//   dB[g]    = sum over g's rows dC[r, :]^T A[r, :]   (grouped_gemm_contig_wgrad)
// BF16 operands, fp32 accumulation.
//
// First form: 128 x 128 tiles, four wavefronts of 64 x 64, 32 steps of the
// reduction at a time through LDS.
#include "common.h"

namespace moe {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;

constexpr int kBK = 32, kPad = 8;

struct GradArgs {
  const uint16_t* P;   // dC [M][N]
  const uint16_t* Q;   // dgrad: B [G][N][K]; wgrad: A [M][K]
  void* D;             // dgrad: dA [M][K]; wgrad: dB [G][N][K]
  const int32_t* m_indices;
  const int32_t* starts;
  const int32_t* counts;
  int64_t M;
  int N, K, G;
};

// LDS tiles hold [reduction][128 + pad]; a fragment is eight 2-byte reads.
__device__ __forceinline__ bf16x8 frag(const uint16_t* t, int col, int k0) {
  uint16_t v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = t[(k0 + j) * (128 + kPad) + col];
  return __builtin_bit_cast(bf16x8, v);
}

template <bool WGRAD, bool F32, bool ACC>
__global__ __launch_bounds__(256) void gemm_grad_kernel(const GradArgs a) {
  __shared__ uint16_t tp[kBK * (128 + kPad)], tq[kBK * (128 + kPad)];
  __shared__ int valid;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int fr = lane & 15, fg = lane >> 4;
  int64_t row0;  // first row of the tile (dgrad) or of the expert (wgrad)
  int rows, e;
  if constexpr (WGRAD) {
    e = blockIdx.z;
    int64_t s = a.starts[e], n = a.counts[e];
    if (s < 0 || s > a.M) s = 0, n = 0;
    if (n < 0) n = 0;
    if (n > a.M - s) n = a.M - s;
    row0 = s;
    rows = static_cast<int>(n);
  } else {
    row0 = static_cast<int64_t>(blockIdx.y) * 128;
    if (tid == 0) valid = 0;
    __syncthreads();
    e = a.m_indices[row0];
    if (e < 0 || e >= a.G) return;
    if (tid < 128 && row0 + tid < a.M && a.m_indices[row0 + tid] >= 0) atomicAdd(&valid, 1);
    __syncthreads();
    rows = valid;
  }
  const int c0 = blockIdx.x * 128;                       // output columns
  const int r0 = WGRAD ? static_cast<int>(blockIdx.y) * 128 : 0;  // output rows
  const int red = WGRAD ? rows : a.N;                    // length of the reduction
  const uint16_t* q = WGRAD ? a.Q + row0 * a.K : a.Q + static_cast<int64_t>(e) * a.N * a.K;
  const uint16_t* p = a.P + row0 * a.N;
  f32x4 acc[4][4] = {};
  for (int k0 = 0; k0 < red; k0 += kBK) {
    __syncthreads();
    for (int i = tid; i < kBK * 128; i += 256) {
      const int k = i >> 7, c = i & 127;
      const bool in = k0 + k < red;
      tq[k * (128 + kPad) + c] = in ? q[static_cast<int64_t>(k0 + k) * a.K + c0 + c] : 0;
      if constexpr (WGRAD)
        tp[k * (128 + kPad) + c] = in ? p[static_cast<int64_t>(k0 + k) * a.N + r0 + c] : 0;
    }
    if constexpr (!WGRAD)
      for (int i = tid; i < kBK * 128; i += 256) {
        const int r = i >> 5, k = i & 31;
        tp[k * (128 + kPad) + r] = r < rows ? p[static_cast<int64_t>(r) * a.N + k0 + k] : 0;
      }
    __syncthreads();
    bf16x8 fp[4], fq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fp[i] = frag(tp, (wave >> 1) * 64 + i * 16 + fr, fg * 8);
      fq[i] = frag(tq, (wave & 1) * 64 + i * 16 + fr, fg * 8);
    }
    // D^T: the lane ends with four consecutive columns of one output row
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[j], fp[i], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (wave >> 1) * 64 + i * 16 + fr;
    if (!WGRAD && r >= rows) continue;
    const int64_t orow = WGRAD ? static_cast<int64_t>(e) * a.N + r0 + r : row0 + r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t o = orow * a.K + c0 + (wave & 1) * 64 + j * 16 + fg * 4;
      f32x4 v = acc[i][j];
      if constexpr (F32) {
        f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(a.D) + o);
        if constexpr (ACC) v += *d;
        *d = v;
      } else {
        uint2* d = reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.D) + o);
        if constexpr (ACC) {
          const uint2 b = *d;
          v += f32x4{__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u),
                     __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u)};
        }
        *d = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
    }
  }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int32_t check_sizes(int64_t M, int32_t N, int32_t K, int32_t G) {
  if (M < 0 || N <= 0 || K <= 0 || G < 0) return MOE_EINVAL;
  if (N % 128 != 0 || K % 128 != 0) return MOE_EUNSUPPORTED;
  // a 64-row panel of an operand is addressed with 32-bit offsets
  if (N > (1 << 22) || K > (1 << 22)) return MOE_EUNSUPPORTED;
  if ((M + 127) / 128 > 8176 || G > 1024) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int32_t grouped_gemm_contig_dgrad(const void* dC, const void* B, void* dA,
                                             const int32_t* m_indices, int64_t M, int32_t N,
                                             int32_t K, int32_t G, void* stream) {
  const int32_t st = check_sizes(M, N, K, G);
  if (st != MOE_OK) return st;
  if (M == 0 || G == 0) return MOE_OK;
  if (!dC || !B || !dA || !m_indices) return MOE_EINVAL;
  if (!aligned16(dC) || !aligned16(B) || !aligned16(dA)) return MOE_EUNSUPPORTED;
  const GradArgs a{static_cast<const uint16_t*>(dC), static_cast<const uint16_t*>(B), dA, m_indices, nullptr,
                   nullptr, M, N, K, G};
  const dim3 grid(K / 128, static_cast<unsigned>((M + 127) / 128), 1);
  gemm_grad_kernel<false, false, false><<<grid, 256, 0, static_cast<hipStream_t>(stream)>>>(a);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" int32_t grouped_gemm_contig_wgrad(const void* dC, const void* A,
                                             const int32_t* expert_start_loc,
                                             const int32_t* num_valid, int32_t out_dtype,
                                             int32_t accumulate, void* dB, int64_t M, int32_t N,
                                             int32_t K, int32_t G, void* stream) {
  const int32_t st = check_sizes(M, N, K, G);
  if (st != MOE_OK) return st;
  if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_FP32) return MOE_EUNSUPPORTED;
  if (G == 0) return MOE_OK;
  if (!expert_start_loc || !num_valid || !dB || (M > 0 && (!dC || !A))) return MOE_EINVAL;
  if (!aligned16(dC) || !aligned16(A) || !aligned16(dB)) return MOE_EUNSUPPORTED;
  const GradArgs a{static_cast<const uint16_t*>(dC), static_cast<const uint16_t*>(A), dB, nullptr,
                   expert_start_loc, num_valid, M, N, K, G};
  const dim3 grid(K / 128, N / 128, G);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (out_dtype == MOE_DTYPE_FP32) {
    if (accumulate) gemm_grad_kernel<true, true, true><<<grid, 256, 0, s>>>(a);
    else gemm_grad_kernel<true, true, false><<<grid, 256, 0, s>>>(a);
  } else {
    if (accumulate) gemm_grad_kernel<true, false, true><<<grid, 256, 0, s>>>(a);
    else gemm_grad_kernel<true, false, false><<<grid, 256, 0, s>>>(a);
  }
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
