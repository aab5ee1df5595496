// grouped_gemm_contig_dgrad of few tiles: 128 rows by 128 columns a workgroup of
// four wavefronts of 64 x 64, two workgroups on a CU.
//
// Where 256 x 256 tiles do not fill the card, four times as many do.  Two stages of
// 32 KB in LDS, loaded again as soon as everyone has read them.  The sums run
// through the same MFMAs in the same order as in the other kernels of this product
// (gemm_grad.hip), so a row comes out the same from each.
//
// What bounds it, with one workgroup on a CU: a step's loads from LDS, its MFMAs and
// its two barriers follow each other (0.58 us a step of 64).  Four stages, reads of
// the next half step between the MFMAs of this one and one barrier a step took 38 us
// to 33 at N 4096 and nothing at N 1024, and with two workgroups' worth of tiles
// were slower (69 us to 76), so it is left at two.  The kernels' times are beside
// the rule that chooses, in gemm_grad.hip.
#include "grad_tile.h"

namespace moe {
namespace {

__global__ __launch_bounds__(256, 2) void dgrad_short_kernel(const GradArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) uint8_t p0[16384], p1[16384], q0[16384], q1[16384];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int fr = lane & 15, fg = lane >> 4;
  const int64_t ldp = static_cast<int64_t>(a.N) * 2, ldq = static_cast<int64_t>(a.K) * 2;
  // consecutive workgroups go to different XCDs: a tile column stays on few of them
  const int ntk = a.K / 128;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / ntk) * 128;
  const int qt = static_cast<int>(blockIdx.x % ntk);
  // valid rows come first in a block of 128, which has one expert
  const int e = __builtin_amdgcn_readfirstlane(a.m_indices[row0]);
  if (e < 0 || e >= a.G) return;
  int rows = 0;
#pragma unroll
  for (int h = 0; h < 128; h += 64) {
    const bool valid = row0 + h + lane < a.M && a.m_indices[row0 + h + lane] >= 0;
    rows += static_cast<int>(__popcll(__ballot(valid)));
  }

  uint32_t vp[4], vq[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = (wave * 4 + j) * 8 + (lane >> 3);
    vp[j] = static_cast<uint32_t>(r * ldp) + (((lane & 7) ^ (lane >> 3)) << 4);
    const int n = wave * 16 + j * 4 + (lane >> 4);
    const int f = (n & 3) | (((n >> 3) & 1) << 2);
    vq[j] = static_cast<uint32_t>(n * ldq) + ((((lane & 15) >> 1) ^ f) << 5) + ((lane & 1) << 4);
  }
  const uint8_t* bp = a.P + row0 * ldp;
  const uint8_t* bq = a.Q + static_cast<int64_t>(e) * a.N * ldq + qt * 256;
  const int np = rows * static_cast<int>(ldp), nq = kStep * static_cast<int>(ldq) - qt * 256;
  int left = a.N / kStep;
  // the next step; behind the last one nothing is read
  auto load = [&](uint8_t* dp, uint8_t* dq) __attribute__((always_inline)) {
    const auto rp = buffer(bp, left > 0 ? np : 0), rq = buffer(bq, left > 0 ? nq : 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, (__attribute__((address_space(3))) void*)(dp + (wave * 4 + j) * 1024), 16,
                                               vp[j], 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (__attribute__((address_space(3))) void*)(dq + (wave * 4 + j) * 1024), 16,
                                               vq[j], 0, 0, 0);
    }
    bp += kStep * 2;
    bq += kStep * ldq;
    --left;
  };
  const int tr_row = fg * 8 + (fr >> 2);
  const int tr_f = (tr_row & 3) | (((tr_row >> 3) & 1) << 2);
  uint32_t op[2], oq[4];
#pragma unroll
  for (int k = 0; k < 2; ++k) op[k] = (wm * 64 + fr) * 128 + (((k * 4 + fg) ^ (fr & 7)) << 4);
#pragma unroll
  for (int b = 0; b < 4; ++b) oq[b] = tr_row * 256 + (((wn * 4 + b) ^ tr_f) << 5) + (fr & 3) * 8;
  f32x4 acc[2][4][2] = {};
  auto pair = [](s16x4 lo, s16x4 hi) __attribute__((always_inline)) {
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto step = [&](uint8_t* p, uint8_t* q) __attribute__((always_inline)) {
    fence();
    wait_vm<8>();  // this stage's loads, of two stages'
    barrier();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      bf16x8 fp[4], fq[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        fp[b] = *reinterpret_cast<const bf16x8*>(p + op[k] + b * 2048);
        fq[b] = pair(read_tr(q + oq[b] + k * 8192), read_tr(q + oq[b] + k * 8192 + 1024));
      }
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          acc[c >> 1][b][c & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[c], fp[b], acc[c >> 1][b][c & 1], 0, 0, 0);
    }
    wait_lds();
    barrier();  // everyone has read the stage
    load(p, q);
  };
  load(p0, q0);
  load(p1, q1);
  for (int t = 0; t < a.N; t += 2 * kStep) {  // N is a multiple of 128
    step(p0, q0);
    step(p1, q1);
  }
  fence();
  wait_vm<0>();  // the loads behind the last step write LDS too
  const int line = a.K * 2, r0 = wm * 64, col0 = qt * 128 + wn * 64;
  const int n = rows - r0 < 64 ? rows - r0 : 64;
  uint8_t* d = static_cast<uint8_t*>(a.D) + (row0 + r0) * line + col0 * 2;
  store64<false, false>(acc, buffer(d, n > 0 ? n * line - col0 * 2 : 0), line, lane);
#endif
}

}  // namespace

int32_t launch_dgrad_short(const GradArgs& a, hipStream_t s) {
  const int64_t blocks = (a.M + 127) / 128 * (a.K / 128);
  dgrad_short_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(a);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

}  // namespace moe
