// Products with an epilogue of few rows: one wavefront a workgroup, 16 NB rows of B and
// up to 32 rows of A.
//
// With few rows the product is one pass over B, and what counts is how many CUs read it
// and how much each has in flight; a row's sum has to run over ascending k in one chain
// (the other kernels' bits), so the reduction is not shared out.  A wavefront of its own
// needs no barrier: it keeps as many loads on their way to its LDS as the counter of
// outstanding loads holds, and two of them fit on a CU.
//
// Gated: the 16 rows are 8 of the gate and the same 8 of the up half; the lanes that
// hold the up parts hand them over at the end.
//
// us (N 4096, K 7168, gated; in brackets 64 x 64 tiles): 1 row 11.8 (36), 16 rows 13.7 (37),
// 32 rows 18 (37); 7 rows, N 256 11 (24).  The first reads its 59 MB at 5 TB/s, the last
// is bound by the one chain of steps.
#include "gemm_runs.h"
#include "grad_tile.h"
#include "linear.h"

namespace moe {
namespace {

constexpr uint32_t kOutside = 0xfffffff0u;  // beyond any descriptor here

// A step takes L = AL + 2 NB loads of 1 KB (AL of A, 8 rows each).  A group of U steps is
// waited for, read and multiplied together: one wavefront issues everything, and step by
// step its waits, reads and two MFMAs follow each other.
template <int AL, int NB>
constexpr int thin_group() { return AL + 2 * NB == 3 ? 4 : 2; }
// Groups in LDS, one of them being read: as many as the counter of loads in flight holds.
template <int AL, int NB>
constexpr int thin_groups() { return 63 / ((AL + 2 * NB) * thin_group<AL, NB>()) + 1; }

template <int AL, int NB, bool GATED>
__global__ __launch_bounds__(64) void linear_thin_kernel(const LinearArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  static_assert((AL == 1 || AL == 2 || AL == 4) && (NB == 1 || NB == 2), "the reads below");
  constexpr int L = AL + 2 * NB, U = thin_group<AL, NB>(), S = thin_groups<AL, NB>(), STAGE = L * 1024;
  constexpr int RB = (AL + 1) / 2;             // blocks of 16 rows
  constexpr int NC = GATED ? NB * 8 : NB * 16;  // output columns
  static_assert(S >= 3 && L * U * (S - 1) < 64 && S * U * STAGE <= 80 * 1024, "two workgroups on a CU");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * U * STAGE];
  const int lane = threadIdx.x;
  const int fr = lane & 15, fg = lane >> 4;
  const int nct = (a.cols + NC - 1) / NC;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / nct) * (AL * 8);
  const int col0 = static_cast<int>(blockIdx.x % nct) * NC;
  const int rows = a.M - row0 < AL * 8 ? static_cast<int>(a.M - row0) : AL * 8;
  const int64_t ldb = static_cast<int64_t>(a.K) * 2;

  uint32_t va[AL], vb[2 * NB], chunk[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) chunk[j] = (lane & 7) ^ (lane >> 3) ^ j;
#pragma unroll
  for (int j = 0; j < AL; ++j) {
    const int r = j * 8 + (lane >> 3);
    va[j] = r < rows ? static_cast<uint32_t>(r * a.lda) + chunk[j & 1] * 16 : kOutside;
  }
#pragma unroll
  for (int j = 0; j < 2 * NB; ++j) {
    // gated: a load of 8 rows is of the gate or of the up half
    const int r = GATED ? (j >> 1) * 8 + (lane >> 3) : j * 8 + (lane >> 3);
    vb[j] = col0 + r < a.cols ? static_cast<uint32_t>((r + (GATED ? (j & 1) * a.cols : 0)) * ldb) + chunk[j & 1] * 16 : kOutside;
  }
  const int na = rows * static_cast<int>(a.lda);
  int nr = GATED ? a.cols + NC : NC;
  nr = nr < a.N - col0 ? nr : a.N - col0;
  const auto ra = buffer(a.A + row0 * a.lda, na);
  const auto rb = buffer_u(a.B + col0 * ldb, static_cast<uint32_t>(nr * ldb));
  auto to_lds = [&](__amdgpu_buffer_rsrc_t rs, uint8_t* dst, uint32_t off, int more) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16, off, more, 0, 0);
  };
  const int steps = (a.K + kStep - 1) / kStep;
  const int whole = a.K / (kStep * U) * U;  // steps in groups that end before K
  int next = 0;                             // step to be loaded
  // The same number of loads in every group; of what lies behind K nothing is read.
  auto load = [&](uint8_t* s) __attribute__((always_inline)) {
    if (next < whole) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = (next + u) * (kStep * 2);
#pragma unroll
        for (int j = 0; j < AL; ++j) to_lds(ra, s + u * STAGE + j * 1024, va[j], at);
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j) to_lds(rb, s + u * STAGE + (AL + j) * 1024, vb[j], at);
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = (next + u) * (kStep * 2), left = a.K - (next + u) * kStep;
        const bool in[2] = {static_cast<int>(chunk[0]) * 8 < left, static_cast<int>(chunk[1]) * 8 < left};
#pragma unroll
        for (int j = 0; j < AL; ++j)
          to_lds(ra, s + u * STAGE + j * 1024, in[j & 1] && va[j] != kOutside ? va[j] + at : kOutside, 0);
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j)
          to_lds(rb, s + u * STAGE + (AL + j) * 1024, in[j & 1] && vb[j] != kOutside ? vb[j] + at : kOutside, 0);
      }
    }
    next += U;
  };
  // with 8 rows of A the lanes 8 .. 15 of each 16 read them again (and hold nothing)
  const int ar = AL == 1 ? fr & 7 : fr;
  const uint32_t base = runs::lds_off(smem);
  uint32_t oa[2], ob[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    oa[k] = base + ar * 128 + (((2 * fg + k) ^ (ar & 7) ^ (ar >> 3)) << 4);
    ob[k] = base + AL * 1024 + fr * 128 + (((2 * fg + k) ^ (fr & 7) ^ (fr >> 3)) << 4);
  }
  f32x4 acc[NB][RB] = {};
  for (int i = 0; i < S - 1; ++i) load(smem + i * U * STAGE);
  int at = 0, to = (S - 1) * U * STAGE;
  for (int t = 0; t < steps; t += U) {
    fence();
    wait_vm<L * U * (S - 2)>();  // this group's loads
    fence();
    load(smem + to);             // where the group before was
    bf16x8 fa[U][2][RB], fb[U][2][NB];
    // Reads and wait in one statement: the compiler would otherwise wait for the loads in
    // flight, which go to other groups.
    if constexpr (AL == 1 && NB == 1)
      asm volatile(
          "ds_read_b128 %0, %16\n\t"
          "ds_read_b128 %1, %18\n\t"
          "ds_read_b128 %2, %17\n\t"
          "ds_read_b128 %3, %19\n\t"
          "ds_read_b128 %4, %16 offset:3072\n\t"
          "ds_read_b128 %5, %18 offset:3072\n\t"
          "ds_read_b128 %6, %17 offset:3072\n\t"
          "ds_read_b128 %7, %19 offset:3072\n\t"
          "ds_read_b128 %8, %16 offset:6144\n\t"
          "ds_read_b128 %9, %18 offset:6144\n\t"
          "ds_read_b128 %10, %17 offset:6144\n\t"
          "ds_read_b128 %11, %19 offset:6144\n\t"
          "ds_read_b128 %12, %16 offset:9216\n\t"
          "ds_read_b128 %13, %18 offset:9216\n\t"
          "ds_read_b128 %14, %17 offset:9216\n\t"
          "ds_read_b128 %15, %19 offset:9216\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(fa[0][0][0]), "=&v"(fb[0][0][0]), "=&v"(fa[0][1][0]), "=&v"(fb[0][1][0]),
            "=&v"(fa[1][0][0]), "=&v"(fb[1][0][0]), "=&v"(fa[1][1][0]), "=&v"(fb[1][1][0]),
            "=&v"(fa[2][0][0]), "=&v"(fb[2][0][0]), "=&v"(fa[2][1][0]), "=&v"(fb[2][1][0]),
            "=&v"(fa[3][0][0]), "=&v"(fb[3][0][0]), "=&v"(fa[3][1][0]), "=&v"(fb[3][1][0])
          : "v"(oa[0] + at), "v"(oa[1] + at), "v"(ob[0] + at), "v"(ob[1] + at)
          : "memory");
    else if constexpr (AL == 2 && NB == 1)
      asm volatile(
          "ds_read_b128 %0, %8\n\t"
          "ds_read_b128 %1, %10\n\t"
          "ds_read_b128 %2, %9\n\t"
          "ds_read_b128 %3, %11\n\t"
          "ds_read_b128 %4, %8 offset:4096\n\t"
          "ds_read_b128 %5, %10 offset:4096\n\t"
          "ds_read_b128 %6, %9 offset:4096\n\t"
          "ds_read_b128 %7, %11 offset:4096\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(fa[0][0][0]), "=&v"(fb[0][0][0]), "=&v"(fa[0][1][0]), "=&v"(fb[0][1][0]),
            "=&v"(fa[1][0][0]), "=&v"(fb[1][0][0]), "=&v"(fa[1][1][0]), "=&v"(fb[1][1][0])
          : "v"(oa[0] + at), "v"(oa[1] + at), "v"(ob[0] + at), "v"(ob[1] + at)
          : "memory");
    else if constexpr (AL == 4 && NB == 1)
      asm volatile(
          "ds_read_b128 %0, %12\n\t"
          "ds_read_b128 %1, %12 offset:2048\n\t"
          "ds_read_b128 %2, %14\n\t"
          "ds_read_b128 %3, %13\n\t"
          "ds_read_b128 %4, %13 offset:2048\n\t"
          "ds_read_b128 %5, %15\n\t"
          "ds_read_b128 %6, %12 offset:6144\n\t"
          "ds_read_b128 %7, %12 offset:8192\n\t"
          "ds_read_b128 %8, %14 offset:6144\n\t"
          "ds_read_b128 %9, %13 offset:6144\n\t"
          "ds_read_b128 %10, %13 offset:8192\n\t"
          "ds_read_b128 %11, %15 offset:6144\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(fa[0][0][0]), "=&v"(fa[0][0][1]), "=&v"(fb[0][0][0]), "=&v"(fa[0][1][0]),
            "=&v"(fa[0][1][1]), "=&v"(fb[0][1][0]), "=&v"(fa[1][0][0]), "=&v"(fa[1][0][1]),
            "=&v"(fb[1][0][0]), "=&v"(fa[1][1][0]), "=&v"(fa[1][1][1]), "=&v"(fb[1][1][0])
          : "v"(oa[0] + at), "v"(oa[1] + at), "v"(ob[0] + at), "v"(ob[1] + at)
          : "memory");
    else if constexpr (AL == 1 && NB == 2)
      asm volatile(
          "ds_read_b128 %0, %12\n\t"
          "ds_read_b128 %1, %14\n\t"
          "ds_read_b128 %2, %14 offset:2048\n\t"
          "ds_read_b128 %3, %13\n\t"
          "ds_read_b128 %4, %15\n\t"
          "ds_read_b128 %5, %15 offset:2048\n\t"
          "ds_read_b128 %6, %12 offset:5120\n\t"
          "ds_read_b128 %7, %14 offset:5120\n\t"
          "ds_read_b128 %8, %14 offset:7168\n\t"
          "ds_read_b128 %9, %13 offset:5120\n\t"
          "ds_read_b128 %10, %15 offset:5120\n\t"
          "ds_read_b128 %11, %15 offset:7168\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(fa[0][0][0]), "=&v"(fb[0][0][0]), "=&v"(fb[0][0][1]), "=&v"(fa[0][1][0]),
            "=&v"(fb[0][1][0]), "=&v"(fb[0][1][1]), "=&v"(fa[1][0][0]), "=&v"(fb[1][0][0]),
            "=&v"(fb[1][0][1]), "=&v"(fa[1][1][0]), "=&v"(fb[1][1][0]), "=&v"(fb[1][1][1])
          : "v"(oa[0] + at), "v"(oa[1] + at), "v"(ob[0] + at), "v"(ob[1] + at)
          : "memory");
    else if constexpr (AL == 2 && NB == 2)
      asm volatile(
          "ds_read_b128 %0, %12\n\t"
          "ds_read_b128 %1, %14\n\t"
          "ds_read_b128 %2, %14 offset:2048\n\t"
          "ds_read_b128 %3, %13\n\t"
          "ds_read_b128 %4, %15\n\t"
          "ds_read_b128 %5, %15 offset:2048\n\t"
          "ds_read_b128 %6, %12 offset:6144\n\t"
          "ds_read_b128 %7, %14 offset:6144\n\t"
          "ds_read_b128 %8, %14 offset:8192\n\t"
          "ds_read_b128 %9, %13 offset:6144\n\t"
          "ds_read_b128 %10, %15 offset:6144\n\t"
          "ds_read_b128 %11, %15 offset:8192\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(fa[0][0][0]), "=&v"(fb[0][0][0]), "=&v"(fb[0][0][1]), "=&v"(fa[0][1][0]),
            "=&v"(fb[0][1][0]), "=&v"(fb[0][1][1]), "=&v"(fa[1][0][0]), "=&v"(fb[1][0][0]),
            "=&v"(fb[1][0][1]), "=&v"(fa[1][1][0]), "=&v"(fb[1][1][0]), "=&v"(fb[1][1][1])
          : "v"(oa[0] + at), "v"(oa[1] + at), "v"(ob[0] + at), "v"(ob[1] + at)
          : "memory");
    else if constexpr (AL == 4 && NB == 2)
      asm volatile(
          "ds_read_b128 %0, %16\n\t"
          "ds_read_b128 %1, %16 offset:2048\n\t"
          "ds_read_b128 %2, %18\n\t"
          "ds_read_b128 %3, %18 offset:2048\n\t"
          "ds_read_b128 %4, %17\n\t"
          "ds_read_b128 %5, %17 offset:2048\n\t"
          "ds_read_b128 %6, %19\n\t"
          "ds_read_b128 %7, %19 offset:2048\n\t"
          "ds_read_b128 %8, %16 offset:8192\n\t"
          "ds_read_b128 %9, %16 offset:10240\n\t"
          "ds_read_b128 %10, %18 offset:8192\n\t"
          "ds_read_b128 %11, %18 offset:10240\n\t"
          "ds_read_b128 %12, %17 offset:8192\n\t"
          "ds_read_b128 %13, %17 offset:10240\n\t"
          "ds_read_b128 %14, %19 offset:8192\n\t"
          "ds_read_b128 %15, %19 offset:10240\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(fa[0][0][0]), "=&v"(fa[0][0][1]), "=&v"(fb[0][0][0]), "=&v"(fb[0][0][1]),
            "=&v"(fa[0][1][0]), "=&v"(fa[0][1][1]), "=&v"(fb[0][1][0]), "=&v"(fb[0][1][1]),
            "=&v"(fa[1][0][0]), "=&v"(fa[1][0][1]), "=&v"(fb[1][0][0]), "=&v"(fb[1][0][1]),
            "=&v"(fa[1][1][0]), "=&v"(fa[1][1][1]), "=&v"(fb[1][1][0]), "=&v"(fb[1][1][1])
          : "v"(oa[0] + at), "v"(oa[1] + at), "v"(ob[0] + at), "v"(ob[1] + at)
          : "memory");
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int i = 0; i < RB; ++i)
            acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[u][k][j], fa[u][k][i], acc[j][i], 0, 0, 0);
    at = at + U * STAGE == S * U * STAGE ? 0 : at + U * STAGE;
    to = to + U * STAGE == S * U * STAGE ? 0 : to + U * STAGE;
  }
  fence();
  wait_vm<0>();  // the loads behind the last step write LDS too

#pragma unroll
  for (int j = 0; j < NB; ++j) {
    // gated: lanes 0 .. 31 have the gate's four channels, lanes 32 .. 63 the up part's
    const int n = GATED ? col0 + j * 8 + (fg & 1) * 4 : col0 + j * 16 + fg * 4;
    const f32x4 bg = bias4(a, 0, n, a.cols);
    f32x4 bu{};
    if constexpr (GATED)
      if (a.bias) bu = load4(a.bias, a.bias32, a.vec, a.cols + n, n, a.cols);
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      f32x4 v = acc[j][i], u{};
      if constexpr (GATED) {
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = __shfl_xor(v[e], 32, 64);
      }
      if (i * 16 + fr < rows && (!GATED || fg < 2)) finish4<GATED>(a, row0 + i * 16 + fr, n, v + bg, u + bu);
    }
  }
#endif
}

template <int AL, int NB>
int32_t launch(const LinearArgs& a, hipStream_t s) {
  const int nc = a.act.gated ? NB * 8 : NB * 16;
  const int64_t blocks = (a.M + AL * 8 - 1) / (AL * 8) * ((a.cols + nc - 1) / nc);
  if (blocks >= (1 << 26)) return MOE_EUNSUPPORTED;  // threads of a launch
  if (a.act.gated)
    linear_thin_kernel<AL, NB, true><<<static_cast<unsigned>(blocks), 64, 0, s>>>(a);
  else
    linear_thin_kernel<AL, NB, false><<<static_cast<unsigned>(blocks), 64, 0, s>>>(a);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

}  // namespace

int32_t launch_linear_thin(const LinearArgs& a, hipStream_t s) {
  const bool wide = a.N > 16 * 512;  // more than two wavefronts a CU: twice the columns each
  if (a.M <= 8) return wide ? launch<1, 2>(a, s) : launch<1, 1>(a, s);
  if (a.M <= 16) return wide ? launch<2, 2>(a, s) : launch<2, 1>(a, s);
  return wide ? launch<4, 2>(a, s) : launch<4, 1>(a, s);
}

}  // namespace moe
