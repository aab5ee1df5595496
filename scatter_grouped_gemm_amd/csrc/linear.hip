// Dense product with bias, activation and residual in its epilogue (moe_linear):
// tiles of BM rows by BN columns of B, four wavefronts of BM/2 by BN/2.
//
// The sum of an output runs through v_mfma_f32_16x16x32_bf16 over ascending k; a
// step of 64 takes the 16-byte chunks 0, 2, 4, 6 of a row's 128 bytes in its first
// instruction and the odd ones in its second, as the grouped products do, so an
// output has the same bits from every kernel.
//   - Loads go straight to LDS (16 bytes a lane), a stage holds a step's rows of A
//     and B; chunks are permuted within a row so that the 16 lanes of a fragment
//     read hit different banks.  Three stages, two steps in flight.
//   - Whatever lies outside (rows behind the last, k behind K) is read as 0 through
//     the bounds of the buffer descriptor: a lane's offset is moved out of it.
//   - Gated: a wavefront holds BN/4 gate columns and the same channels of the up
//     half, so that both are in one lane's registers.
#include "grad_tile.h"
#include "linear.h"

namespace moe {
namespace {

constexpr uint32_t kOutside = 0xfffffff0u;  // beyond any descriptor here

template <int BM, int BN, bool GATED>
__global__ __launch_bounds__(256, 2) void linear_tile_kernel(const LinearArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int WM = BM / 2, WN = BN / 2, TM = WM / 16, TN = WN / 16;
  constexpr int LA = BM / 32, LB = BN / 32;  // 1 KB loads of a wavefront and step
  constexpr int NC = GATED ? BN / 2 : BN;    // output columns of a tile
  __shared__ __attribute__((aligned(1024))) uint8_t s0[(BM + BN) * 128], s1[(BM + BN) * 128], s2[(BM + BN) * 128];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int fr = lane & 15, fg = lane >> 4;
  const int nct = (a.cols + NC - 1) / NC;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / nct) * BM;
  const int col0 = static_cast<int>(blockIdx.x % nct) * NC;
  int e = 0, rows = a.M - row0 < BM ? static_cast<int>(a.M - row0) : BM;
  if (a.m_indices) {  // a block of 128 rows has one expert, and its valid rows come first
    e = __builtin_amdgcn_readfirstlane(a.m_indices[row0]);
    if (e < 0 || e >= a.G) return;
    int valid = 0;
#pragma unroll
    for (int h = 0; h < BM; h += 64) valid += static_cast<int>(__popcll(__ballot(h + lane < rows && a.m_indices[row0 + h + lane] >= 0)));
    rows = valid;
  }
  const int64_t ldb = static_cast<int64_t>(a.K) * 2;

  // Offsets of this lane's 16 bytes from the tile's first row of A and of B (below 2^32
  // by the limits of the call).
  uint32_t va[LA], vb[LB];
  const int chunk = (lane & 7) ^ (lane >> 3);  // of the row's 128 bytes: a load covers 8 rows
#pragma unroll
  for (int j = 0; j < LA; ++j) {
    const int r = (wave * LA + j) * 8 + (lane >> 3);
    va[j] = r < rows ? static_cast<uint32_t>(r * a.lda) + chunk * 16 : kOutside;
  }
#pragma unroll
  for (int j = 0; j < LB; ++j) {
    const int r = (wave * LB + j) * 8 + (lane >> 3);
    int n;
    bool in;
    if constexpr (GATED) {
      const int c = col0 + (r / WN) * (WN / 2) + r % (WN / 2);
      in = c < a.cols;
      n = c - col0 + ((r % WN) / (WN / 2)) * a.cols;
    } else {
      n = r;
      in = col0 + r < a.N;
    }
    vb[j] = in ? static_cast<uint32_t>(n * ldb) + chunk * 16 : kOutside;
  }
  const uint8_t* pa = a.A + row0 * a.lda;
  const uint8_t* pb = a.B + (static_cast<int64_t>(e) * a.N + col0) * ldb;
  const int na = rows * static_cast<int>(a.lda);       // bytes of the tile's rows
  int nr = GATED ? a.cols + NC : BN;                    // B rows that the tile's offsets reach
  nr = nr < a.N - col0 ? nr : a.N - col0;
  const uint32_t nb = static_cast<uint32_t>(nr * ldb);
  const int steps = (a.K + kStep - 1) / kStep;
  int loaded = 0;
  auto load = [&](uint8_t* s) __attribute__((always_inline)) {
    // behind the last step nothing is read, but the same number of loads is issued
    const int left = a.K - loaded * kStep;
    const bool in = chunk * 8 < left;
    const auto ra = buffer(pa, left > 0 ? na - loaded * (kStep * 2) : 0), rb = buffer_u(pb, left > 0 ? nb - loaded * (kStep * 2) : 0);
#pragma unroll
    for (int j = 0; j < LA; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (__attribute__((address_space(3))) void*)(s + (wave * LA + j) * 1024), 16,
                                               in ? va[j] : kOutside, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < LB; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (__attribute__((address_space(3))) void*)(s + BM * 128 + (wave * LB + j) * 1024), 16,
                                               in ? vb[j] : kOutside, 0, 0, 0);
    pa += kStep * 2;
    pb += kStep * 2;
    ++loaded;
  };
  uint32_t oa[2], ob[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = ((2 * fg + k) ^ (fr & 7)) << 4;
    oa[k] = (wm * WM + fr) * 128 + c;
    ob[k] = (BM + wn * WN + fr) * 128 + c;
  }
  f32x4 acc[TN][TM] = {};
  auto step = [&](uint8_t* s, uint8_t* next) __attribute__((always_inline)) {
    fence();
    wait_vm<LA + LB>();  // this step's loads, of two steps'
    barrier();           // everyone's, and everyone has read the step before
    load(next);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      bf16x8 fa[TM], fb[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[i] = *reinterpret_cast<const bf16x8*>(s + oa[k] + i * 2048);
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[j] = *reinterpret_cast<const bf16x8*>(s + ob[k] + j * 2048);
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i) acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[j][i], 0, 0, 0);
    }
    wait_lds();
  };
  load(s0);
  load(s1);
  for (int t = 0;;) {
    step(s0, s2);
    if (++t >= steps) break;
    step(s1, s0);
    if (++t >= steps) break;
    step(s2, s1);
    if (++t >= steps) break;
  }
  fence();
  wait_vm<0>();  // the loads behind the last step write LDS too

  constexpr int TH = GATED ? TN / 2 : TN;
  const int cw = col0 + wn * (GATED ? WN / 2 : WN) + fg * 4;
#pragma unroll
  for (int j = 0; j < TH; ++j) {
    const int n = cw + j * 16;
    const f32x4 bg = bias4(a, e, n, a.cols);
    f32x4 bu{};
    if constexpr (GATED)
      if (a.bias) bu = load4(a.bias, a.bias32, a.vec, static_cast<int64_t>(e) * a.N + a.cols + n, n, a.cols);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = wm * WM + i * 16 + fr;
      if (r < rows) finish4<GATED>(a, row0 + r, n, acc[j][i] + bg, GATED ? acc[(j + TH) % TN][i] + bu : bg);
    }
  }
#endif
}

template <int BM, int BN>
int32_t launch(const LinearArgs& a, hipStream_t s) {
  const int nc = a.act.gated ? BN / 2 : BN;
  const int64_t tiles = (a.M + BM - 1) / BM * ((a.cols + nc - 1) / nc);
  if (tiles >= (1 << 24)) return MOE_EUNSUPPORTED;  // threads of a launch
  if (a.act.gated)
    linear_tile_kernel<BM, BN, true><<<static_cast<unsigned>(tiles), 256, 0, s>>>(a);
  else
    linear_tile_kernel<BM, BN, false><<<static_cast<unsigned>(tiles), 256, 0, s>>>(a);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

inline bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

}  // namespace

void linear_alignment(LinearArgs& a) {
  const int os = a.out32 ? 4 : 2;
  a.vec = a.cols % 4 == 0 && a.ldo % 4 == 0 && aligned(a.out, 4 * os) &&
          (!a.residual || (a.ldr % 4 == 0 && aligned(a.residual, 4 * os))) && (!a.pre || aligned(a.pre, 8)) &&
          (!a.bias || aligned(a.bias, a.bias32 ? 16 : 8));
  a.vec8 = a.vec && a.cols % 8 == 0 && a.ldo % 8 == 0 && aligned(a.out, 16) &&
           (!a.residual || (a.ldr % 8 == 0 && aligned(a.residual, 16))) && (!a.pre || aligned(a.pre, 16));
}

int32_t launch_linear(const LinearArgs& a, hipStream_t s) {
  const int64_t n = a.N;
  if (linear_wide_covers(a) && (a.M + 255) / 256 * ((n + 255) / 256) >= 200) return launch_linear_wide(a, s);
  // tiles of 128 x 128 where they fill the card
  return (a.M + 127) / 128 * ((n + 127) / 128) >= 256 ? launch<128, 128>(a, s) : launch<64, 64>(a, s);
}

}  // namespace moe

using namespace moe;

extern "C" int32_t moe_linear(const void* A, int64_t lda, const void* B, const void* bias, int32_t bias_dtype,
                              int32_t act, float alpha, float limit, const void* residual, int64_t ld_residual,
                              int32_t out_dtype, void* out, int64_t ld_out, void* pre, int64_t M, int32_t N,
                              int32_t K, void* stream) {
  LinearArgs a{};
  if (M < 0 || N <= 0 || K <= 0) return MOE_EINVAL;
  if (!make_act(act, alpha, limit, a.act)) return MOE_EINVAL;
  if (a.act.gated && N % 2 != 0) return MOE_EINVAL;
  a.cols = a.act.gated ? N / 2 : N;
  if (lda < K || ld_out < a.cols || (residual && ld_residual < a.cols)) return MOE_EINVAL;
  if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_FP32) return MOE_EUNSUPPORTED;
  if (bias && bias_dtype != MOE_DTYPE_BF16 && bias_dtype != MOE_DTYPE_FP32) return MOE_EUNSUPPORTED;
  if (K % 8 != 0 || lda % 8 != 0) return MOE_EUNSUPPORTED;
  // offsets within a tile's rows are 32-bit; a gated tile's reach the up rows
  if (lda >= (1 << 22) || (a.act.gated && (static_cast<int64_t>(N) / 2 + 256) * K * 2 >= (1ll << 32))) return MOE_EUNSUPPORTED;
  if (M >= (1ll << 31) || (M + 127) / 128 * ((static_cast<int64_t>(N) + 127) / 128) >= (1 << 24)) return MOE_EUNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!A || !B || !out) return MOE_EINVAL;
  if (!aligned(A, 16) || !aligned(B, 16)) return MOE_EUNSUPPORTED;
  a.out32 = out_dtype == MOE_DTYPE_FP32;
  a.bias32 = bias_dtype == MOE_DTYPE_FP32;
  const int os = a.out32 ? 4 : 2;
  if (!aligned(out, os) || !aligned(residual, os) || !aligned(pre, 2) || (bias && !aligned(bias, a.bias32 ? 4 : 2)))
    return MOE_EUNSUPPORTED;
  a.A = static_cast<const uint8_t*>(A);
  a.lda = lda * 2;
  a.B = static_cast<const uint8_t*>(B);
  a.bias = bias;
  a.residual = residual;
  a.ldr = ld_residual;
  a.out = out;
  a.ldo = ld_out;
  a.pre = static_cast<uint16_t*>(pre);
  a.M = M;
  a.N = N;
  a.K = K;
  a.G = 1;
  linear_alignment(a);
  return launch_linear(a, static_cast<hipStream_t>(stream));
}
