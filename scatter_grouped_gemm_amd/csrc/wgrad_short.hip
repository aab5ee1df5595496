// grouped_gemm_contig_wgrad of few tiles or few rows: 128 x 128 tiles, one a
// workgroup of four wavefronts of 64 x 64, two workgroups on a CU.
//
// Where 256 x 256 tiles do not fill the card, four times as many do; and with a
// handful of steps a tile's time is its stores and what it holds already: the
// wide kernel (gemm_grad.hip) waits for them with the whole CU, here the CU's
// other workgroup works meanwhile.  Two stages of 32 KB in LDS, loaded again as
// soon as everyone has read them.  The sums run through the same MFMAs in the same
// order as in the wide kernel, so both give the same bits.
//
// What bounds it: every value is loaded and goes through LDS twice as often as in
// the wide kernel.  16384 rows: 1230 TFLOP/s with 512 tiles (two a
// CU, all at once), 900 with 1024, 730 with 2048, the wide kernel 860, 1270, 1350.
// With few rows it runs at the copy's rate (8 experts of 64 rows, 28672 x 4096,
// added to fp32: 5.5 TB/s).
// Both kernels' times are beside the rule that chooses, in gemm_grad.hip.
#include "grad_tile.h"

namespace moe {
namespace {

template <bool F32, bool ACC>
__global__ __launch_bounds__(256, 2) void wgrad_short_kernel(const GradArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) uint8_t p0[16384], p1[16384], q0[16384], q1[16384];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int fr = lane & 15, fg = lane >> 4;
  const int64_t ldp = static_cast<int64_t>(a.N) * 2, ldq = static_cast<int64_t>(a.K) * 2;
  // an eighth of every expert's tiles to each XCD, in its order of workgroups
  const int ntn = a.N / 128, ntk = a.K / 128, per = (ntn * ntk + 7) / 8;
  const int turn = static_cast<int>(blockIdx.x >> 3), e = turn / per;
  const int i = static_cast<int>((blockIdx.x + e) & 7) * per + (turn - e * per);
  if (i >= ntn * ntk) return;
  int64_t s = scalar_load(a.starts + e), n = scalar_load(a.counts + e);
  if (s < 0 || s > a.M || n < 0) s = 0, n = 0;
  n = n < a.M - s ? n : a.M - s;
  if (ACC && n == 0) return;  // what the expert holds stays
  const int grp = i / (kGroupN * ntk), g0 = grp * kGroupN;
  const int gs = ntn - g0 < kGroupN ? ntn - g0 : kGroupN;
  const int rest = i - g0 * ntk;
  const int qt = rest / gs, pt = g0 + rest - qt * gs;

  uint32_t vp[4], vq[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = wave * 16 + j * 4 + (lane >> 4);
    const int f = (r & 3) | (((r >> 3) & 1) << 2);
    const uint32_t piece = ((((lane & 15) >> 1) ^ f) << 5) + ((lane & 1) << 4);
    vp[j] = static_cast<uint32_t>(r * ldp) + piece;
    vq[j] = static_cast<uint32_t>(r * ldq) + piece;
  }
  const uint8_t* bp = a.P + s * ldp + pt * 256;
  const uint8_t* bq = a.Q + s * ldq + qt * 256;
  int left = static_cast<int>(n);
  // the next step; behind the last one nothing is read
  auto load = [&](uint8_t* dp, uint8_t* dq) __attribute__((always_inline)) {
    const int v = left < kStep ? left : kStep;
    const auto rp = buffer(bp, v > 0 ? v * static_cast<int>(ldp) - pt * 256 : 0);
    const auto rq = buffer(bq, v > 0 ? v * static_cast<int>(ldq) - qt * 256 : 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, (__attribute__((address_space(3))) void*)(dp + (wave * 4 + j) * 1024), 16,
                                               vp[j], 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (__attribute__((address_space(3))) void*)(dq + (wave * 4 + j) * 1024), 16,
                                               vq[j], 0, 0, 0);
    }
    bp += kStep * ldp;
    bq += kStep * ldq;
    left -= kStep;
  };
  const int tr_row = fg * 8 + (fr >> 2);
  const int tr_f = (tr_row & 3) | (((tr_row >> 3) & 1) << 2);
  uint32_t op[4], oq[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    op[b] = tr_row * 256 + (((wm * 4 + b) ^ tr_f) << 5) + (fr & 3) * 8;
    oq[b] = tr_row * 256 + (((wn * 4 + b) ^ tr_f) << 5) + (fr & 3) * 8;
  }
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
        fp[b] = pair(read_tr(p + op[b] + k * 8192), read_tr(p + op[b] + k * 8192 + 1024));
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
  const int steps = static_cast<int>((n + kStep - 1) / kStep);
  load(p0, q0);
  load(p1, q1);
  for (int t = 0; t < steps; t += 2) {  // a step behind the last adds zeros
    step(p0, q0);
    step(p1, q1);
  }
  fence();
  wait_vm<0>();  // the loads behind the last step write LDS too
  constexpr int ES = F32 ? 4 : 2;
  const int line = a.K * ES, row0 = pt * 128 + wm * 64, col0 = qt * 128 + wn * 64;
  uint8_t* d = static_cast<uint8_t*>(a.D) + (static_cast<int64_t>(e) * a.N + row0) * line + col0 * ES;
  store64<F32, ACC>(acc, buffer(d, 64 * line - col0 * ES), line, lane);
#endif
}

template <bool F32, bool ACC>
void run(const GradArgs& a, unsigned blocks, hipStream_t s) {
  wgrad_short_kernel<F32, ACC><<<blocks, 256, 0, s>>>(a);
}

}  // namespace

int32_t launch_wgrad_short(const GradArgs& a, bool f32, bool acc, hipStream_t s) {
  // every expert's tiles in eight equal parts, the last ones filled up
  const int64_t per = (static_cast<int64_t>(a.N / 128) * (a.K / 128) + 7) / 8;
  const unsigned n = static_cast<unsigned>(8 * per * a.G);
  if (f32)
    acc ? run<true, true>(a, n, s) : run<true, false>(a, n, s);
  else
    acc ? run<false, true>(a, n, s) : run<false, false>(a, n, s);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

}  // namespace moe
