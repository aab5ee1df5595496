// Products with bias, activation and residual in their epilogue: tiles of BM rows by BN
// rows of B, four wavefronts of BM/2 by BN/2, for the dense product (moe_linear) and the
// compact grouped one, where it is too small for linear_wide.hip or has a form that that
// kernel does not (columns or rows that are not whole aligned groups; a residual with
// a gated activation, a kept product or fp32 output).
//
// The sum of an output runs through v_mfma_f32_16x16x32_bf16 over ascending k; a
// step of 64 takes the 16-byte chunks 0, 2, 4, 6 of a row's 128 bytes in its first
// instruction and the odd ones in its second, as the grouped products do, so an
// output has the same bits from every kernel.
//   - Loads go straight to LDS (16 bytes a lane), a stage holds a step's rows of A
//     and B; chunks are permuted within a row so that the 16 lanes of a fragment
//     read hit different banks.  The next step's fragments are read while a step's MFMAs
//     run.  What bounds a tile by itself is LDS: a 64 x 64 step (0.29 us) reads 32 KB
//     from it and writes 16.
//   - The order of the tiles keeps those that share rows on one XCD: 8192 rows, K 7168, N
//     256 46 us, dealt over all of them 68 (each L2 then reads A).
//   - Whatever lies outside (rows behind the last, k behind K) is read as 0 through
//     the bounds of the buffer descriptor: a lane's offset is moved out of it.
//   - Gated: a wavefront holds BN/4 gate columns and the same channels of the up
//     half, so that both are in one lane's registers.
#include "gemm_runs.h"
#include "grad_tile.h"
#include "linear.h"

namespace moe {
namespace {

constexpr uint32_t kOutside = 0xfffffff0u;  // beyond any descriptor here

template <int BM, int BN, int S, bool GATED>
__global__ __launch_bounds__(256, S > 4 ? 1 : 2) void linear_tile_kernel(const LinearArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int WM = BM / 2, WN = BN / 2, TM = WM / 16, TN = WN / 16;
  constexpr int LA = BM / 32, LB = BN / 32;  // 1 KB loads of a wavefront and step
  constexpr int NC = GATED ? BN / 2 : BN;    // output columns of a tile
  constexpr int STAGE = (BM + BN) * 128;
  static_assert(LA % 2 == 0 && LB % 2 == 0, "whole pairs of loads");
  static_assert((S == 2 || S == 4 || S == 6) && (LA + LB) * (S - 2) < 64, "loads in flight");
  // Arrays of their own: the compiler then knows which loads to LDS a read can depend on.
  __shared__ __attribute__((aligned(1024))) uint8_t s0[STAGE], s1[STAGE], s2[S > 2 ? STAGE : 1], s3[S > 2 ? STAGE : 1],
      s4[S > 4 ? STAGE : 1], s5[S > 4 ? STAGE : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int fr = lane & 15, fg = lane >> 4;
  // Workgroup ids are dealt round-robin over the XCDs, each with its own L2: an XCD takes
  // a contiguous eighth of the order, in which eight tile columns go down the rows
  // together, so that what runs at the same time shares rows of both operands.
  const int nct = (a.cols + NC - 1) / NC, nrt = static_cast<int>((a.M + BM - 1) / BM);
  const int tile = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  if (tile >= nrt * nct) return;
  const int cg = tile / (8 * nrt) * 8, in_group = tile - cg * nrt;
  const int cw = nct - cg < 8 ? nct - cg : 8;
  const int64_t row0 = static_cast<int64_t>(in_group / cw) * BM;
  const int col0 = (cg + in_group % cw) * NC;
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
  // 16-byte chunk of the row's 128: a load covers 8 rows, an even one those with (row & 8) == 0
  const int chunk[2] = {(lane & 7) ^ (lane >> 3), (lane & 7) ^ (lane >> 3) ^ 1};
#pragma unroll
  for (int j = 0; j < LA; ++j) {
    const int r = (wave * LA + j) * 8 + (lane >> 3);
    va[j] = r < rows ? static_cast<uint32_t>(r * a.lda) + chunk[j & 1] * 16 : kOutside;
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
    vb[j] = in ? static_cast<uint32_t>(n * ldb) + chunk[j & 1] * 16 : kOutside;
  }
  int nr = GATED ? a.cols + NC : BN;  // B rows that the tile's offsets reach
  nr = nr < a.N - col0 ? nr : a.N - col0;
  const auto ra = buffer(a.A + row0 * a.lda, rows * static_cast<int>(a.lda));
  const auto rb = buffer_u(a.B + (static_cast<int64_t>(e) * a.N + col0) * ldb, static_cast<uint32_t>(nr * ldb));
  auto to_lds = [&](__amdgpu_buffer_rsrc_t rs, uint8_t* dst, uint32_t off, int more) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16, off, more, 0, 0);
  };
  const int steps = (a.K + kStep - 1) / kStep, whole = a.K / kStep;
  int next = 0;  // step to be loaded
  // The same number of loads in every step; of what lies behind K nothing is read.
  auto load = [&](uint8_t* s) __attribute__((always_inline)) {
    const int at = next * (kStep * 2);
    if (next < whole) {
#pragma unroll
      for (int j = 0; j < LA; ++j) to_lds(ra, s + (wave * LA + j) * 1024, va[j], at);
#pragma unroll
      for (int j = 0; j < LB; ++j) to_lds(rb, s + BM * 128 + (wave * LB + j) * 1024, vb[j], at);
    } else {
      const int left = a.K - next * kStep;
      const bool in[2] = {chunk[0] * 8 < left, chunk[1] * 8 < left};
#pragma unroll
      for (int j = 0; j < LA; ++j) to_lds(ra, s + (wave * LA + j) * 1024, in[j & 1] && va[j] != kOutside ? va[j] + at : kOutside, 0);
#pragma unroll
      for (int j = 0; j < LB; ++j)
        to_lds(rb, s + BM * 128 + (wave * LB + j) * 1024, in[j & 1] && vb[j] != kOutside ? vb[j] + at : kOutside, 0);
    }
    ++next;
  };
  uint32_t oa[2], ob[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = ((2 * fg + k) ^ (fr & 7) ^ (fr >> 3)) << 4;
    oa[k] = (wm * WM + fr) * 128 + c;
    ob[k] = (BM + wn * WN + fr) * 128 + c;
  }
  struct Frags {
    bf16x8 a[2][TM], b[2][TN];
  } f0, f1;
  auto read = [&](Frags& f, const uint8_t* s) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int i = 0; i < TM; ++i) f.a[k][i] = *reinterpret_cast<const bf16x8*>(s + oa[k] + i * 2048);
#pragma unroll
      for (int j = 0; j < TN; ++j) f.b[k][j] = *reinterpret_cast<const bf16x8*>(s + ob[k] + j * 2048);
    }
  };
  f32x4 acc[TN][TM] = {};
  // A step whose fragments are in f: the next step's are read into g while its MFMAs
  // run, and its stage is filled again.
  auto step = [&](Frags& f, Frags& g, uint8_t* stage, const uint8_t* following) __attribute__((always_inline)) {
    wait_lds();
    fence();
    wait_vm<(LA + LB) * (S - 2)>();  // the next step's loads
    barrier();                       // everyone's, and everyone has read this stage
    read(g, following);
    load(stage);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i)
          acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[k][j], f.a[k][i], acc[j][i], 0, 0, 0);
  };
  load(s0);
  load(s1);
  if constexpr (S > 2) {
    load(s2);
    load(s3);
  }
  if constexpr (S > 4) {
    load(s4);
    load(s5);
  }
  fence();
  wait_vm<(LA + LB) * (S - 1)>();
  barrier();
  read(f0, s0);
  for (int t = 0;;) {
    step(f0, f1, s0, s1);
    if (++t >= steps) break;
    step(f1, f0, s1, S > 2 ? s2 : s0);
    if (++t >= steps) break;
    if constexpr (S > 2) {
      step(f0, f1, s2, s3);
      if (++t >= steps) break;
      step(f1, f0, s3, S > 4 ? s4 : s0);
      if (++t >= steps) break;
    }
    if constexpr (S > 4) {
      step(f0, f1, s4, s5);
      if (++t >= steps) break;
      step(f1, f0, s5, s0);
      if (++t >= steps) break;
    }
  }
  fence();
  wait_vm<0>();  // the loads behind the last step write LDS too

  constexpr int TH = GATED ? TN / 2 : TN;
  const int c0 = col0 + wn * (GATED ? WN / 2 : WN) + fg * 4;
#pragma unroll
  for (int j = 0; j < TH; ++j) {
    const int n = c0 + j * 16;
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

template <int BM, int BN, int S, bool GATED>
int32_t launch(const LinearArgs& a, hipStream_t s) {
  constexpr int nc = GATED ? BN / 2 : BN;
  const int64_t tiles = (a.M + BM - 1) / BM * ((a.cols + nc - 1) / nc);
  if (tiles >= (1 << 24)) return MOE_EUNSUPPORTED;  // threads of a launch
  linear_tile_kernel<BM, BN, S, GATED><<<static_cast<unsigned>((tiles + 7) / 8 * 8), 256, 0, s>>>(a);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
template <int BM, int BN, int S>
int32_t launch(const LinearArgs& a, hipStream_t s) {
  return a.act.gated ? launch<BM, BN, S, true>(a, s) : launch<BM, BN, S, false>(a, s);
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

// Which kernel takes a call, by the tiles that each would have (in the compact layout by
// the buffers' height: the rows in them are on the device); the bits are the same.
// us, one matrix, K 4096 (7168 where marked):
//   up to 32 rows, the thin kernel: 1 row, N 4096* 12 (64 x 64 tiles 32), N 16384* 35 (40);
//     with wider N the 64 x 64 tiles' reads are as good, and they read A less often (32
//     rows, N 28672 43 / 35)
//   256 x 256 tiles for more than half of the CUs: 128 tiles 76 (128 x 128 ones 74), 160
//     78 (108), 256 96 (123)
//   128 x 128 for three tiles for two CUs and up, two workgroups a CU: 448 tiles 62 (128 x
//     64 92, 64 x 64 87)
//   64 x 64 up to two tiles a CU: 64 tiles* 33 (128 x 64 49, 128 x 128 73), 512 tiles* (N
//     256) 46 (53, 78); with one tile a CU in six stages, for operands that come from HBM:
//     256 tiles* 45 (four stages 48), 512 tiles* 88 (70)
//   128 x 64 between them: 512 tiles* 75 (128 x 128 76, 64 x 64 88)
int32_t launch_linear(const LinearArgs& a, hipStream_t s) {
  const int64_t cus = linear_cus(), n = a.N;
  if (cus == 0) return MOE_EDEVICE;
  if (!a.m_indices && a.M <= 32 && n <= 16384) return launch_linear_thin(a, s);
  if (linear_wide_covers(a) && 2 * ((a.M + 255) / 256 * ((n + 255) / 256)) > cus) return launch_linear_wide(a, s);
  if (2 * ((a.M + 127) / 128 * ((n + 127) / 128)) >= 3 * cus) return launch<128, 128, 2>(a, s);
  const int64_t small = (a.M + 63) / 64 * ((n + 63) / 64);
  if (small <= cus) return launch<64, 64, 6>(a, s);
  if (small <= 2 * cus) return launch<64, 64, 4>(a, s);
  return launch<128, 64, 2>(a, s);
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
  if (out == A || out == B || out == bias || (pre && (pre == A || pre == B || pre == out || pre == bias || pre == residual)))
    return MOE_EINVAL;
  if (residual == out && ld_residual != ld_out && M > 1) return MOE_EINVAL;
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
