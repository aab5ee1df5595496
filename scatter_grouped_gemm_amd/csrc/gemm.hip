// Entry points of the grouped products (plain, and w13 with SiLU-and-mul): argument
// checks and the choice between the register-streamed kernel (gemm_wreg.hip: compact
// layout, BF16 or 128x128-block FP8 weights, N a multiple of 256) and the LDS-staged
// one (gemm_kernel.h).
#include "gemm_kernel.h"

using namespace moe;

extern "C" int32_t grouped_gemm_contig(int32_t dtype, const void* A, const uint8_t* A_scale,
                                       const void* B, const uint8_t* B_scale, void* C,
                                       const int32_t* m_indices, int64_t M, int32_t N, int32_t K,
                                       int32_t G, void* stream) {
  if (M < 0) return MOE_EINVAL;
  int32_t st = validate_gemm(dtype, A, A_scale, B, B_scale, C, N, K, G);
  if (st != MOE_OK) return st;
  if (M == 0) return MOE_OK;
  if (!m_indices) return MOE_EINVAL;
  GemmArgs a{};
  a.A = static_cast<const uint8_t*>(A);
  a.A_scale = A_scale;
  a.B = static_cast<const uint8_t*>(B);
  a.B_scale = B_scale;
  a.C = C;
  a.rowinfo = m_indices;
  a.M = M;
  a.N = N;
  a.K = K;
  a.G = G;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool fp8 = dtype == MOE_DTYPE_FP8_E4M3_UE8M0;
  if ((fp8 || dtype == MOE_DTYPE_BF16) && wreg_supported(M, N, K, G, fp8)) {
    WregArgs w{a.A, a.A_scale, a.B, a.B_scale, C, nullptr, m_indices, M, N, K, G};
    return launch_wreg(w, fp8, kWrEpiPlain, s);
  }
  if (N % 256 == 0) return launch_dtype<128, 256, false>(dtype, a, s);
  return launch_dtype<128, 128, false>(dtype, a, s);
}

extern "C" int64_t grouped_gemm_rows_executed(int32_t dtype, int32_t masked, const int32_t* counts,
                                              int32_t G, int32_t expected_m, int64_t M, int32_t N,
                                              int32_t K) {
  if (!counts || G <= 0 || N <= 0 || K <= 0 || M < 0 || expected_m < 0) return -1;
  int64_t rows = 0;
  if (masked) {
    const int64_t bm = masked_tile_rows(expected_m, N);
    for (int g = 0; g < G; ++g) {
      if (counts[g] < 0) return -1;
      rows += (counts[g] + bm - 1) / bm * bm;
    }
    return rows;
  }
  const bool fp8 = dtype == MOE_DTYPE_FP8_E4M3_UE8M0;
  const bool wreg = (fp8 || dtype == MOE_DTYPE_BF16) && wreg_supported(M, N, K, G, fp8);
  for (int g = 0; g < G; ++g) {
    const int64_t z = counts[g];
    if (z < 0) return -1;
    if (z == 0) continue;
    if (!wreg) {
      rows += (z + 127) / 128 * 128;
      continue;
    }
    // the register-streamed kernel: ceil(z / 256) tiles of equal height
    // rounded up to 16, each running its MFMAs on whole 16-row blocks
    const int64_t nt = (z + 255) / 256;
    const int64_t h = ((z + nt - 1) / nt + 15) / 16 * 16;
    for (int64_t t = 0; t < nt; ++t) {
      const int64_t r = z - t * h < h ? z - t * h : h;
      if (r > 0) rows += (r + 15) / 16 * 16;
    }
  }
  return rows;
}

extern "C" int32_t grouped_gemm_masked(int32_t dtype, const void* A, const uint8_t* A_scale,
                                       const void* B, const uint8_t* B_scale, void* C,
                                       const int32_t* masked_m, int32_t expected_m, int32_t max_m,
                                       int32_t N, int32_t K, int32_t G, void* stream) {
  if (max_m <= 0 || expected_m < 0) return MOE_EINVAL;
  int32_t st = validate_gemm(dtype, A, A_scale, B, B_scale, C, N, K, G);
  if (st != MOE_OK) return st;
  if (!masked_m) return MOE_EINVAL;
  if (G > kMaxMaskedGroups) return MOE_EUNSUPPORTED;
  GemmArgs a{};
  a.A = static_cast<const uint8_t*>(A);
  a.A_scale = A_scale;
  a.B = static_cast<const uint8_t*>(B);
  a.B_scale = B_scale;
  a.C = C;
  a.rowinfo = masked_m;
  a.M = max_m;
  a.N = N;
  a.K = K;
  a.G = G;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool n256 = N % 256 == 0;
  // tile height from the hint: small expected counts waste less work on 64 rows
  switch (masked_tile_rows(expected_m, N)) {
    case 16: return launch_dtype<16, 256, true>(dtype, a, s);
    case 32: return launch_dtype<32, 256, true>(dtype, a, s);
    case 64: return n256 ? launch_dtype<64, 256, true>(dtype, a, s) : launch_dtype<64, 128, true>(dtype, a, s);
    default: return n256 ? launch_dtype<128, 256, true>(dtype, a, s) : launch_dtype<128, 128, true>(dtype, a, s);
  }
}

// The w13 GEMM with SiLU-and-mul in its epilogue: B holds [G][2I][K] (gate
// rows then up rows); out receives the activation [rows][I].
static int32_t validate_silu(int32_t out_dtype, void* out, uint8_t* out_scale, int32_t I) {
  if (I <= 0 || !out) return MOE_EINVAL;
  if (I % 128 != 0) return MOE_EUNSUPPORTED;
  if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_FP8_E4M3_UE8M0) return MOE_EUNSUPPORTED;
  if (out_dtype == MOE_DTYPE_FP8_E4M3_UE8M0 && !out_scale) return MOE_EINVAL;
  return MOE_OK;
}

extern "C" int32_t grouped_gemm_contig_silu(int32_t dtype, const void* A, const uint8_t* A_scale,
                                            const void* B, const uint8_t* B_scale, int32_t out_dtype,
                                            void* out, uint8_t* out_scale, const int32_t* m_indices,
                                            int64_t M, int32_t I, int32_t K, int32_t G, void* stream) {
  if (M < 0) return MOE_EINVAL;
  int32_t st = validate_silu(out_dtype, out, out_scale, I);
  if (st != MOE_OK) return st;
  if (I > (1 << 29)) return MOE_EUNSUPPORTED;
  // per-lane 32-bit offsets reach the up rows, I weight rows in
  if (static_cast<int64_t>(I + 256) * K * 2 >= (1ll << 32)) return MOE_EUNSUPPORTED;
  st = validate_gemm(dtype, A, A_scale, B, B_scale, out, 2 * I, K, G);
  if (st != MOE_OK) return st;
  if (M == 0) return MOE_OK;
  if (!m_indices) return MOE_EINVAL;
  GemmArgs a{};
  a.A = static_cast<const uint8_t*>(A);
  a.A_scale = A_scale;
  a.B = static_cast<const uint8_t*>(B);
  a.B_scale = B_scale;
  a.C = out;
  a.C_scale = out_scale;
  a.rowinfo = m_indices;
  a.M = M;
  a.N = 2 * I;
  a.K = K;
  a.G = G;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool fp8 = dtype == MOE_DTYPE_FP8_E4M3_UE8M0;
  if ((fp8 || dtype == MOE_DTYPE_BF16) && wreg_supported(M, 2 * I, K, G, fp8)) {
    WregArgs w{a.A, a.A_scale, a.B, a.B_scale, out, out_scale, m_indices, M, 2 * I, K, G};
    return launch_wreg(w, fp8, out_dtype == MOE_DTYPE_FP8_E4M3_UE8M0 ? kWrEpiSiluFp8 : kWrEpiSiluBf16, s);
  }
  if (out_dtype == MOE_DTYPE_FP8_E4M3_UE8M0)
    return launch_dtype<128, 256, false, kEpiSiluFp8>(dtype, a, s);
  return launch_dtype<128, 256, false, kEpiSiluBf16>(dtype, a, s);
}

extern "C" int32_t grouped_gemm_masked_silu(int32_t dtype, const void* A, const uint8_t* A_scale,
                                            const void* B, const uint8_t* B_scale, int32_t out_dtype,
                                            void* out, uint8_t* out_scale, const int32_t* masked_m,
                                            int32_t expected_m, int32_t max_m, int32_t I, int32_t K,
                                            int32_t G, void* stream) {
  if (max_m <= 0 || expected_m < 0) return MOE_EINVAL;
  int32_t st = validate_silu(out_dtype, out, out_scale, I);
  if (st != MOE_OK) return st;
  if (I > (1 << 29)) return MOE_EUNSUPPORTED;
  if (static_cast<int64_t>(I + 256) * K * 2 >= (1ll << 32)) return MOE_EUNSUPPORTED;
  st = validate_gemm(dtype, A, A_scale, B, B_scale, out, 2 * I, K, G);
  if (st != MOE_OK) return st;
  if (!masked_m) return MOE_EINVAL;
  if (G > kMaxMaskedGroups) return MOE_EUNSUPPORTED;
  GemmArgs a{};
  a.A = static_cast<const uint8_t*>(A);
  a.A_scale = A_scale;
  a.B = static_cast<const uint8_t*>(B);
  a.B_scale = B_scale;
  a.C = out;
  a.C_scale = out_scale;
  a.rowinfo = masked_m;
  a.M = max_m;
  a.N = 2 * I;
  a.K = K;
  a.G = G;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool q8 = out_dtype == MOE_DTYPE_FP8_E4M3_UE8M0;
  switch (masked_tile_rows(expected_m, 2 * I)) {
    case 16: return q8 ? launch_dtype<16, 256, true, kEpiSiluFp8>(dtype, a, s)
                       : launch_dtype<16, 256, true, kEpiSiluBf16>(dtype, a, s);
    case 32: return q8 ? launch_dtype<32, 256, true, kEpiSiluFp8>(dtype, a, s)
                       : launch_dtype<32, 256, true, kEpiSiluBf16>(dtype, a, s);
    case 64: return q8 ? launch_dtype<64, 256, true, kEpiSiluFp8>(dtype, a, s)
                       : launch_dtype<64, 256, true, kEpiSiluBf16>(dtype, a, s);
    default: return q8 ? launch_dtype<128, 256, true, kEpiSiluFp8>(dtype, a, s)
                       : launch_dtype<128, 256, true, kEpiSiluBf16>(dtype, a, s);
  }
}
