// Gradient of a product's epilogue: dpre = dout act'(pre), and for each expert the sum
// of its rows of dpre (before it is rounded), the bias gradient.
//
// Bound by memory: a gated element pair reads 6 bytes and writes 4.  The sums ride
// along: a workgroup takes a block of rows (whole in one expert) by some columns,
// keeps its columns' sums in registers over the rows, joins its threads' through LDS
// and writes one line of partial sums for the block; a second launch adds each
// expert's lines in their order.  So no sum depends on who finishes first, and the
// partial sums are 1 / (10 .. 80) of the traffic.
#include "act.h"
#include "common.h"

namespace moe {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

struct ActBwdArgs {
  const uint16_t* pre;
  const uint16_t* dout;
  uint16_t* dpre;
  float* part;              // [blocks][N], or null
  const int32_t* m_indices;
  const int32_t* masked_m;
  const int32_t* starts;
  const int32_t* counts;
  int64_t M;
  int N, cols, max_m;       // cols: of dout
  int R, nb;                // rows of a block; masked: blocks of a group
  int lanes;                // threads of a row, 8 columns each
  ActArgs act;
};

__device__ __forceinline__ float half_of(uint32_t v, int h) {
  return h ? __uint_as_float(v & 0xffff0000u) : __uint_as_float(v << 16);
}

template <bool GATED>
__global__ __launch_bounds__(256) void act_bwd_kernel(const ActBwdArgs a) {
  constexpr int H = GATED ? 2 : 1;
  __shared__ float sums[256 * 8 * H];
  const int tid = threadIdx.x;
  const int sub = tid / a.lanes, col = tid % a.lanes, rows_at_once = 256 / a.lanes;
  const int64_t block = blockIdx.x;
  int64_t row0, end;  // of the block; rows with an assignment come first in it
  if (a.masked_m) {
    const int64_t g = block / a.nb;
    const int first = static_cast<int>(block - g * a.nb) * a.R;
    const int valid = a.masked_m[g];
    int last = first + a.R;
    last = last < a.max_m ? last : a.max_m;
    last = last < valid ? last : valid;
    row0 = g * a.max_m + first;
    end = g * a.max_m + last;
  } else {
    row0 = block * a.R;
    end = row0 + a.R < a.M ? row0 + a.R : a.M;
    if (a.m_indices && a.m_indices[row0] < 0) return;
  }
  if (row0 >= end) return;
  const int c = (blockIdx.y * a.lanes + col) * 8;
  float sg[8] = {}, su[8] = {};
  if (c < a.cols) {
    for (int64_t r = row0 + sub; r < end; r += rows_at_once) {
      if (a.m_indices && a.m_indices[r] < 0) break;
      const int64_t wide = r * a.N + c;
      const u32x4 d = *reinterpret_cast<const u32x4*>(a.dout + r * a.cols + c);
      u32x4 g{}, u{}, og, ou;
      if (a.pre) {
        g = *reinterpret_cast<const u32x4*>(a.pre + wide);
        if constexpr (GATED) u = *reinterpret_cast<const u32x4*>(a.pre + wide + a.cols);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float dg[2], du[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float da = half_of(d[i], h), x = half_of(g[i], h);
          float v, s;
          if constexpr (GATED) {
            const float y = half_of(u[i], h);
            act::slope(a.act, act::cut_gate(a.act, x), v, s);
            dg[h] = x > a.act.limit ? 0.0f : da * (act::cut_up(a.act, y) + a.act.offset) * s;
            du[h] = y > a.act.limit || y < -a.act.limit ? 0.0f : da * v;
            su[2 * i + h] += du[h];
          } else {
            act::slope(a.act, x, v, s);
            dg[h] = a.act.kind == kActNone ? da : da * s;
          }
          sg[2 * i + h] += dg[h];
        }
        og[i] = pack_bf16x2(dg[0], dg[1]);
        if constexpr (GATED) ou[i] = pack_bf16x2(du[0], du[1]);
      }
      if (a.dpre) {
        *reinterpret_cast<u32x4*>(a.dpre + wide) = og;
        if constexpr (GATED) *reinterpret_cast<u32x4*>(a.dpre + wide + a.cols) = ou;
      }
    }
  }
  if (!a.part) return;
  // sums[half][e][sub][col]
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    sums[e * 256 + tid] = sg[e];
    if constexpr (GATED) sums[(8 + e) * 256 + tid] = su[e];
  }
  __syncthreads();
  // element e of column group q, for each half
  const int n = a.lanes * 8;  // columns of this workgroup
  for (int i = tid; i < n * H; i += 256) {
    const int h = i / n, x = i - h * n, q = x >> 3, e = x & 7;
    const int at = blockIdx.y * n + x;
    if (at >= a.cols) continue;
    float t = 0.0f;
    for (int k = 0; k < rows_at_once; ++k) t += sums[(h * 8 + e) * 256 + k * a.lanes + q];
    a.part[block * a.N + h * a.cols + at] = t;
  }
}

// dbias[g][n] from the partial sums of g's blocks.  64 columns and one expert a
// workgroup, a quarter of the blocks each wavefront.
__global__ __launch_bounds__(256) void bias_grad_kernel(const ActBwdArgs a, void* dbias, int f32, int acc) {
  __shared__ float sums[256];
  const int g = blockIdx.y, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int n = blockIdx.x * 64 + lane;
  int64_t b0, b1;
  if (a.masked_m) {
    int valid = a.masked_m[g];
    valid = valid < a.max_m ? valid : a.max_m;
    b0 = static_cast<int64_t>(g) * a.nb;
    b1 = b0 + (valid > 0 ? (valid + a.R - 1) / a.R : 0);
  } else if (a.starts) {
    int64_t s = a.starts[g], e = s + a.counts[g];
    e = e < a.M ? e : a.M;
    s = s > 0 ? s : 0;
    b0 = s / a.R;
    b1 = e > s ? (e + a.R - 1) / a.R : b0;
  } else {
    b0 = 0;
    b1 = (a.M + a.R - 1) / a.R;
  }
  const int64_t each = (b1 - b0 + 3) / 4;
  int64_t lo = b0 + w * each, hi = lo + each;
  hi = hi < b1 ? hi : b1;
  float t = 0.0f;
  if (n < a.N)
#pragma unroll 8
    for (int64_t b = lo; b < hi; ++b) t += a.part[b * a.N + n];
  sums[threadIdx.x] = t;
  __syncthreads();
  if (w != 0 || n >= a.N) return;
  t = ((sums[lane] + sums[64 + lane]) + sums[128 + lane]) + sums[192 + lane];
  const int64_t at = static_cast<int64_t>(g) * a.N + n;
  if (f32) {
    float* const p = static_cast<float*>(dbias) + at;
    *p = acc ? *p + t : t;
  } else {
    uint16_t* const p = static_cast<uint16_t*>(dbias) + at;
    *p = f32_to_bf16(acc ? bf16_to_f32(*p) + t : t);
  }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Rows of a block: few enough that the blocks fill the card, a divisor of the 128 to
// which the compact layout pads.
int block_rows(int64_t M, int N) {
  int R = 128;
  while (R > 16 && (M + R - 1) / R * ((N + 1023) / 1024) < 2048) R /= 2;
  return R;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_act_bwd_ws_bytes(int64_t M, int32_t N, int32_t G) {
  if (M <= 0 || N <= 0 || G <= 0) return 0;
  // a masked group's last block may be cut: at most one block more a group
  return (static_cast<size_t>((M + 15) / 16) + G) * N * sizeof(float);
}

extern "C" int32_t moe_act_bwd(const void* pre, const void* dout, int64_t M, int32_t N, int32_t act, float alpha,
                               float limit, const int32_t* m_indices, const int32_t* masked_m, int32_t max_m,
                               const int32_t* expert_start_loc, const int32_t* num_valid, int32_t G, void* dpre,
                               int32_t dbias_dtype, int32_t accumulate, void* dbias, void* ws, size_t ws_bytes,
                               void* stream) {
  ActBwdArgs a{};
  if (M < 0 || N <= 0 || G <= 0) return MOE_EINVAL;
  if (!make_act(act, alpha, limit, a.act)) return MOE_EINVAL;
  if (N % (a.act.gated ? 16 : 8) != 0) return MOE_EUNSUPPORTED;
  if (N > (1 << 27) || M >= (1 << 26) || G > 65535) return MOE_EUNSUPPORTED;
  if (masked_m && m_indices) return MOE_EINVAL;
  if (masked_m && (max_m <= 0 || M % max_m != 0 || (dbias && M / max_m != G))) return MOE_EINVAL;
  if (!masked_m && !m_indices && G != 1) return MOE_EINVAL;
  if (dbias && dbias_dtype != MOE_DTYPE_BF16 && dbias_dtype != MOE_DTYPE_FP32) return MOE_EUNSUPPORTED;
  if (dbias && m_indices && (!expert_start_loc || !num_valid)) return MOE_EINVAL;
  if (a.act.kind != kActNone && !dpre) return MOE_EINVAL;
  if (!dpre && !dbias) return MOE_EINVAL;
  if (M > 0 && (!dout || (a.act.kind != kActNone && !pre))) return MOE_EINVAL;
  if (dbias && ws_bytes < moe_act_bwd_ws_bytes(M, N, G)) return MOE_ECAPACITY;
  if (dbias && M > 0 && !ws) return MOE_EINVAL;
  if (!aligned16(pre) || !aligned16(dout) || !aligned16(dpre) || !aligned16(dbias) || !aligned16(ws)) return MOE_EUNSUPPORTED;
  if (M == 0 && (!dbias || accumulate)) return MOE_OK;
  a.pre = a.act.kind == kActNone ? nullptr : static_cast<const uint16_t*>(pre);
  a.dout = static_cast<const uint16_t*>(dout);
  a.dpre = static_cast<uint16_t*>(dpre);
  a.part = dbias ? static_cast<float*>(ws) : nullptr;
  a.m_indices = m_indices;
  a.masked_m = masked_m;
  a.starts = m_indices ? expert_start_loc : nullptr;
  a.counts = num_valid;
  a.M = M;
  a.N = N;
  a.cols = a.act.gated ? N / 2 : N;
  a.max_m = max_m;
  a.R = block_rows(M, N);
  a.nb = masked_m ? (max_m + a.R - 1) / a.R : 0;
  const int groups = a.cols / 8;
  a.lanes = groups > 32 ? 64 : groups > 16 ? 32 : 16;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (M > 0) {
    const int64_t blocks = masked_m ? M / max_m * a.nb : (M + a.R - 1) / a.R;
    const int64_t cy = (groups + a.lanes - 1) / a.lanes;
    if (blocks >= (1 << 24) || cy > 65535) return MOE_EUNSUPPORTED;  // a launch's threads and grid
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(cy));
    if (a.act.gated) act_bwd_kernel<true><<<grid, 256, 0, s>>>(a);
    else act_bwd_kernel<false><<<grid, 256, 0, s>>>(a);
    MOE_CHECK_LAUNCH();
  }
  if (dbias) {
    const dim3 grid(static_cast<unsigned>((N + 63) / 64), static_cast<unsigned>(G));
    bias_grad_kernel<<<grid, 256, 0, s>>>(a, dbias, dbias_dtype == MOE_DTYPE_FP32, accumulate != 0);
    MOE_CHECK_LAUNCH();
  }
  return MOE_OK;
}
