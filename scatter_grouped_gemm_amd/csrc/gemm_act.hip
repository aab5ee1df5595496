// Entry points of the grouped products with a bias and an activation in their
// epilogue (gemm_kernel.h: kEpiBias, kEpiAct*; compact BF16: linear.h).  FP8 weights in the
// compact layout too take the LDS-staged kernel: the register-streamed one, 10% faster
// without bias (256 experts of 256 rows, 4096 x 7168: us 2436 and 2696; slower with 40 rows
// an expert, 107 and 90), has no registers left for it.
#include "gemm_kernel.h"
#include "linear.h"

namespace moe {
namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// What both layouts check, and the launch arguments.  M is the rows of a group in
// the masked layout.
int32_t act_args(int32_t dtype, const void* A, const uint8_t* A_scale, const void* B, const uint8_t* B_scale,
                 const void* bias, int32_t bias_dtype, int32_t act, float alpha, float limit, int32_t out_dtype,
                 void* out, uint8_t* out_scale, void* pre, const int32_t* rowinfo, int64_t M, int32_t N, int32_t K,
                 int32_t G, GemmArgs& a) {
  if (M < 0 || N <= 0 || K <= 0 || G <= 0) return MOE_EINVAL;
  if (!make_act(act, alpha, limit, a.act)) return MOE_EINVAL;
  if (N % (a.act.gated ? 256 : 128) != 0) return MOE_EUNSUPPORTED;
  if (N > (1 << 30)) return MOE_EUNSUPPORTED;
  // per-lane 32-bit offsets reach the up rows, N / 2 weight rows in
  if (a.act.gated && (static_cast<int64_t>(N) / 2 + 256) * K * 2 >= (1ll << 32)) return MOE_EUNSUPPORTED;
  if (out_dtype != MOE_DTYPE_BF16 && !(out_dtype == MOE_DTYPE_FP8_E4M3_UE8M0 && a.act.gated)) return MOE_EUNSUPPORTED;
  if (bias && bias_dtype != MOE_DTYPE_BF16 && bias_dtype != MOE_DTYPE_FP32) return MOE_EUNSUPPORTED;
  if (pre && dtype != MOE_DTYPE_BF16) return MOE_EUNSUPPORTED;
  if (M == 0) {  // tensors without elements have no address
    A = B;
    out = const_cast<void*>(B);
    A_scale = B_scale;
  }
  const int32_t st = validate_gemm(dtype, A, A_scale, B, B_scale, out, N, K, G);
  if (st != MOE_OK || M == 0) return st;
  if (out == A || out == B || out == bias || (pre && (pre == A || pre == B || pre == out || pre == bias))) return MOE_EINVAL;
  if (!rowinfo || (out_dtype == MOE_DTYPE_FP8_E4M3_UE8M0 && !out_scale)) return MOE_EINVAL;
  if (!aligned16(A) || !aligned16(B) || !aligned16(bias) || !aligned16(out) || !aligned16(pre)) return MOE_EUNSUPPORTED;
  a.A = static_cast<const uint8_t*>(A);
  a.A_scale = A_scale;
  a.B = static_cast<const uint8_t*>(B);
  a.B_scale = B_scale;
  a.C = out;
  a.C_scale = out_scale;
  a.rowinfo = rowinfo;
  a.M = M;
  a.N = N;
  a.K = K;
  a.G = G;
  a.bias = bias;
  a.bias32 = bias_dtype == MOE_DTYPE_FP32;
  a.pre = static_cast<uint16_t*>(pre);
  return MOE_OK;
}

// Compact layout, quantised weights (BF16 ones take the kernels of linear.h).
template <int BN, int EPI>
int32_t launch_quantised(int32_t dtype, const GemmArgs& a, hipStream_t s) {
  switch (dtype) {
    case MOE_DTYPE_FP8_E4M3_UE8M0: return launch_gemm<128, BN, kWfFp8Block, false, EPI>(a, s);
    case MOE_DTYPE_FP8_E4M3_MXFP8: return launch_gemm<128, BN, kWfMxFp8, false, EPI>(a, s);
    case MOE_DTYPE_FP8_MXFP4: return launch_gemm<128, BN, kWfMxFp4, false, EPI>(a, s);
    default: return MOE_EUNSUPPORTED;
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int32_t grouped_gemm_contig_act(int32_t dtype, const void* A, const uint8_t* A_scale, const void* B,
                                           const uint8_t* B_scale, const void* bias, int32_t bias_dtype, int32_t act,
                                           float alpha, float limit, int32_t out_dtype, void* out, uint8_t* out_scale,
                                           void* pre, const int32_t* m_indices, int64_t M, int32_t N, int32_t K,
                                           int32_t G, void* stream) {
  GemmArgs a{};
  const int32_t st = act_args(dtype, A, A_scale, B, B_scale, bias, bias_dtype, act, alpha, limit, out_dtype, out,
                              out_scale, pre, m_indices, M, N, K, G, a);
  if (st != MOE_OK || M == 0) return st;
  if ((M + 127) / 128 > 8176) return MOE_EUNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (out_dtype == MOE_DTYPE_FP8_E4M3_UE8M0) return launch_dtype<128, 256, false, kEpiActFp8>(dtype, a, s);
  if (dtype == MOE_DTYPE_BF16) {
    LinearArgs l{};
    l.A = a.A;
    l.lda = static_cast<int64_t>(K) * 2;
    l.B = a.B;
    l.bias = bias;
    l.bias32 = a.bias32;
    l.out = out;
    l.cols = a.act.gated ? N / 2 : N;
    l.ldo = l.cols;
    l.pre = a.pre;
    l.m_indices = m_indices;
    l.M = M;
    l.N = N;
    l.K = K;
    l.G = G;
    l.act = a.act;
    l.deep = M >= 1024ll * G;
    linear_alignment(l);
    return launch_linear(l, s);
  }
  if (a.act.gated) return launch_quantised<256, kEpiActBf16>(dtype, a, s);
  if (N % 256 == 0) return launch_quantised<256, kEpiBias>(dtype, a, s);
  return launch_quantised<128, kEpiBias>(dtype, a, s);
}

extern "C" int32_t grouped_gemm_masked_act(int32_t dtype, const void* A, const uint8_t* A_scale, const void* B,
                                           const uint8_t* B_scale, const void* bias, int32_t bias_dtype, int32_t act,
                                           float alpha, float limit, int32_t out_dtype, void* out, uint8_t* out_scale,
                                           void* pre, const int32_t* masked_m, int32_t expected_m, int32_t max_m,
                                           int32_t N, int32_t K, int32_t G, void* stream) {
  if (max_m <= 0 || expected_m < 0) return MOE_EINVAL;
  if (G > kMaxMaskedGroups) return MOE_EUNSUPPORTED;
  GemmArgs a{};
  const int32_t st = act_args(dtype, A, A_scale, B, B_scale, bias, bias_dtype, act, alpha, limit, out_dtype, out,
                              out_scale, pre, masked_m, max_m, N, K, G, a);
  if (st != MOE_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool q8 = out_dtype == MOE_DTYPE_FP8_E4M3_UE8M0, gated = a.act.gated, n256 = N % 256 == 0;
  switch (masked_tile_rows(expected_m, N)) {
    case 16: return q8 ? launch_dtype<16, 256, true, kEpiActFp8>(dtype, a, s)
                  : gated ? launch_dtype<16, 256, true, kEpiActBf16>(dtype, a, s)
                          : launch_dtype<16, 256, true, kEpiBias>(dtype, a, s);
    case 32: return q8 ? launch_dtype<32, 256, true, kEpiActFp8>(dtype, a, s)
                  : gated ? launch_dtype<32, 256, true, kEpiActBf16>(dtype, a, s)
                          : launch_dtype<32, 256, true, kEpiBias>(dtype, a, s);
    case 64: return q8 ? launch_dtype<64, 256, true, kEpiActFp8>(dtype, a, s)
                  : gated ? launch_dtype<64, 256, true, kEpiActBf16>(dtype, a, s)
                  : n256 ? launch_dtype<64, 256, true, kEpiBias>(dtype, a, s)
                         : launch_dtype<64, 128, true, kEpiBias>(dtype, a, s);
    default: return q8 ? launch_dtype<128, 256, true, kEpiActFp8>(dtype, a, s)
                  : gated ? launch_dtype<128, 256, true, kEpiActBf16>(dtype, a, s)
                  : n256 ? launch_dtype<128, 256, true, kEpiBias>(dtype, a, s)
                         : launch_dtype<128, 128, true, kEpiBias>(dtype, a, s);
  }
}
