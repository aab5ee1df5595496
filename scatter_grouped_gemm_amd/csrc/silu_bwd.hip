// Gradient of SiLU-and-mul: act = silu(g) u with s = sigma(g), given da:
//   dg = da u s (1 + g (1 - s)),   du = da g s,
// and, where asked for, act again for the weight gradient of w2 (the forward
// need not keep it).  Elementwise: bound by memory, 6 bytes read and 4 (6 with
// act) written per channel and row (8192 rows, I 14336, with act: 298-313 us,
// 4.5-4.7 TB/s; in place without act 230 us).
#include "common.h"

namespace moe {
namespace {

typedef __attribute__((ext_vector_type(4))) unsigned int u32x4;

// A wavefront takes kPass * 512 channels of one row, 8 a lane and pass, and
// issues all its loads (three a pass) before any arithmetic.  Long rows are
// shared by several wavefronts: few rows fill the device too.
constexpr int kPass = 2;

// No __restrict__ on gateup and dgateup: they may be one buffer.  Every
// channel is read before it is written, by the lane that writes it.
__global__ __launch_bounds__(256) void silu_bwd_kernel(const uint16_t* gateup,
                                                       const uint16_t* __restrict__ dact, int64_t M,
                                                       int I, const int32_t* __restrict__ m_indices,
                                                       const int32_t* __restrict__ masked_m,
                                                       int max_m, uint16_t* dgateup,
                                                       uint16_t* __restrict__ act) {
  const int lane = threadIdx.x & 63;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (r >= M) return;
  if (m_indices && m_indices[r] < 0) return;
  if (masked_m) {
    const int64_t g = r / max_m;
    if (r - g * max_m >= masked_m[g]) return;
  }
  const int64_t two = r * 2 * static_cast<int64_t>(I), one = r * static_cast<int64_t>(I);
  const int c0 = blockIdx.y * (kPass * 512) + lane * 8;
  u32x4 gv[kPass], uv[kPass], dv[kPass];
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const int c = c0 + p * 512;
    if (c >= I) break;
    gv[p] = *reinterpret_cast<const u32x4*>(gateup + two + c);
    uv[p] = *reinterpret_cast<const u32x4*>(gateup + two + I + c);
    dv[p] = *reinterpret_cast<const u32x4*>(dact + one + c);
  }
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const int c = c0 + p * 512;
    if (c >= I) break;
    u32x4 og, ou, oa;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float dg[2], du[2], a[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const auto part = [h](uint32_t v) {
          return h ? __uint_as_float(v & 0xffff0000u) : __uint_as_float(v << 16);
        };
        const float g = part(gv[p][i]), u = part(uv[p][i]), d = part(dv[p][i]);
        const float e = __builtin_amdgcn_exp2f(-g * 1.4426950408889634f);
        const float s = __builtin_amdgcn_rcpf(1.0f + e);
        // 1 - s is 0 where g is large; a finite g there keeps the product 0
        const float gf = fminf(fmaxf(g, -3e38f), 3e38f);
        dg[h] = d * u * (s * (1.0f + gf * (1.0f - s)));
        du[h] = d * (g * s);
        a[h] = silu_f32(g) * u;  // rounded as the forward's, bit for bit
      }
      og[i] = pack_bf16x2(dg[0], dg[1]);
      ou[i] = pack_bf16x2(du[0], du[1]);
      oa[i] = pack_bf16x2(a[0], a[1]);
    }
    *reinterpret_cast<u32x4*>(dgateup + two + c) = og;
    *reinterpret_cast<u32x4*>(dgateup + two + I + c) = ou;
    if (act) *reinterpret_cast<u32x4*>(act + one + c) = oa;
  }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int32_t silu_and_mul_bwd(const void* gateup, const void* dact, int64_t M, int32_t I,
                                    const int32_t* m_indices, const int32_t* masked_m,
                                    int32_t max_m, void* dgateup, void* act, void* stream) {
  if (M < 0 || I <= 0) return MOE_EINVAL;
  if (I % 128 != 0) return MOE_EUNSUPPORTED;
  if (masked_m && m_indices) return MOE_EINVAL;
  if (masked_m && (max_m <= 0 || M % max_m != 0)) return MOE_EINVAL;
  if (M == 0) return MOE_OK;
  if (!gateup || !dact || !dgateup) return MOE_EINVAL;
  if (!aligned16(gateup) || !aligned16(dact) || !aligned16(dgateup) || !aligned16(act))
    return MOE_EUNSUPPORTED;
  const int64_t nb = (M + 3) / 4, cols = (static_cast<int64_t>(I) + kPass * 512 - 1) / (kPass * 512);
  if (nb >= (1 << 24) || cols > 65535) return MOE_EUNSUPPORTED;  // threads of a launch, its grid
  silu_bwd_kernel<<<dim3(static_cast<unsigned>(nb), static_cast<unsigned>(cols)), 256, 0,
                    static_cast<hipStream_t>(stream)>>>(
      static_cast<const uint16_t*>(gateup), static_cast<const uint16_t*>(dact), M, I, m_indices,
      masked_m, max_m, static_cast<uint16_t*>(dgateup), static_cast<uint16_t*>(act));
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
