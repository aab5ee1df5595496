// Gradient of a product's epilogue: dpre = dout act'(pre), and for each expert the sum
// of its rows of dpre (before it is rounded), the bias gradient.
//
// Bound by memory: a gated element pair reads 6 bytes and writes 4 (us: 8192 rows of 8
// experts, N 28672 253, 4.6 TB/s; 8191 rows, N 4096, not gated 48, 4.2 TB/s).  The sums ride
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
  const void* dout;         // bf16, or (dout32) fp32
  int dout32;
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
  void* dbias;              // [G][N]
  int f32, acc;             // fp32, and added to
  ActArgs act;
};

__device__ __forceinline__ float half_of(uint32_t v, int h) {
  return h ? __uint_as_float(v & 0xffff0000u) : __uint_as_float(v << 16);
}

// Eight columns of row r, if it holds an assignment.  (Several rows at a time to have more
// loads in flight are slower: two rows of a dense N 4096, 8191 rows, us 51.5 for 50.4.)
template <bool GATED>
__device__ __forceinline__ void one_row(const ActBwdArgs& a, int64_t r, int c, float (&sg)[8], float (&su)[8]) {
  const int64_t wide = r * a.N + c;
  // in flight together: whether the row counts is seen when they are there
  const int tag = a.m_indices ? a.m_indices[r] : 0;
  u32x4 d, d1{};
  if (a.dout32) {
    const u32x4* const q = reinterpret_cast<const u32x4*>(static_cast<const float*>(a.dout) + r * a.cols + c);
    d = q[0];
    d1 = q[1];
  } else {
    d = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.dout) + r * a.cols + c);
  }
  u32x4 g{}, u{}, og, ou;
  if (a.pre) {
    g = *reinterpret_cast<const u32x4*>(a.pre + wide);
    if constexpr (GATED) u = *reinterpret_cast<const u32x4*>(a.pre + wide + a.cols);
  }
  if (tag < 0) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float dg[2], du[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float da = a.dout32 ? __uint_as_float(i < 2 ? d[2 * i + h] : d1[2 * i + h - 4]) : half_of(d[i], h), x = half_of(g[i], h);
      float v, s;
      if constexpr (GATED) {
        const float y = half_of(u[i], h);
        act::slope(a.act, act::cut_gate(a.act, x), v, s);
        dg[h] = x > a.act.limit ? 0.0f : da * (act::cut_up(a.act, y) + a.act.offset) * s;
        du[h] = y > a.act.limit || y < -a.act.limit ? 0.0f : da * v;
        su[2 * i + h] += du[h];
      } else if (a.act.kind == kActNone) {
        dg[h] = da;
      } else {
        act::slope(a.act, x, v, s);
        dg[h] = da * s;
      }
      sg[2 * i + h] += dg[h];
    }
    og[i] = pack_bf16x2(dg[0], dg[1]);
    if constexpr (GATED) ou[i] = pack_bf16x2(du[0], du[1]);
  }
  if (!a.dpre) return;
  *reinterpret_cast<u32x4*>(a.dpre + wide) = og;
  if constexpr (GATED) *reinterpret_cast<u32x4*>(a.dpre + wide + a.cols) = ou;
}

__device__ __forceinline__ void put_bias_grad(void* dbias, int f32, int acc, int64_t at, float t) {
  if (f32) {
    float* const p = static_cast<float*>(dbias) + at;
    *p = acc ? *p + t : t;
  } else {
    uint16_t* const p = static_cast<uint16_t*>(dbias) + at;
    *p = f32_to_bf16(acc ? bf16_to_f32(*p) + t : t);
  }
}

// Rows of expert g: [first, second).
__device__ __forceinline__ void rows_of(const ActBwdArgs& a, int g, int64_t& first, int64_t& second) {
  if (a.masked_m) {
    int n = a.masked_m[g];
    n = n < a.max_m ? n : a.max_m;
    first = static_cast<int64_t>(g) * a.max_m;
    second = first + (n > 0 ? n : 0);
  } else if (a.starts) {
    const int64_t at = a.starts[g], end = at + a.counts[g];
    first = at > 0 ? at : 0;
    second = end < a.M ? end : a.M;
  } else {
    first = 0;
    second = a.M;
  }
}

// WHOLE: a workgroup takes all rows of expert blockIdx.x and writes its columns' bias
// gradients itself; else a block of R rows, and their sums go to part.
template <bool GATED, bool WHOLE>
__global__ __launch_bounds__(256) void act_bwd_kernel(const ActBwdArgs a) {
  constexpr int H = GATED ? 2 : 1;
  __shared__ float sums[256 * 8 * H];
  const int tid = threadIdx.x;
  const int sub = tid / a.lanes, col = tid % a.lanes, rows_at_once = 256 / a.lanes;
  const int64_t block = blockIdx.x;
  const int chunk = blockIdx.z * gridDim.y + blockIdx.y;  // of the columns; of the last ones some may be behind them
  int64_t row0, end;
  if constexpr (WHOLE) {
    rows_of(a, static_cast<int>(block), row0, end);
  } else {
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
  }
  const int c = (chunk * a.lanes + col) * 8;
  float sg[8] = {}, su[8] = {};
  if (c < a.cols)
    for (int64_t r = row0 + sub; r < end; r += rows_at_once) one_row<GATED>(a, r, c, sg, su);
  if (!WHOLE && !a.part) return;
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
    const int at = chunk * n + x;
    if (at >= a.cols) continue;
    float t = 0.0f;
    for (int k = 0; k < rows_at_once; ++k) t += sums[(h * 8 + e) * 256 + k * a.lanes + q];
    if constexpr (WHOLE) put_bias_grad(a.dbias, a.f32, a.acc, block * a.N + h * a.cols + at, t);
    else a.part[block * a.N + h * a.cols + at] = t;
  }
}

// dbias[g][n] from the partial sums of g's blocks: COLS columns and one expert a
// workgroup, 256 / COLS stretches of the blocks.  16 columns where that makes few
// workgroups (one matrix of N 4096, 8191 rows: us 4.7 for 8.0), 64 where it makes many (64
// experts of N 4096, both launches 110 for 118).
template <int COLS>
__global__ __launch_bounds__(256) void bias_grad_kernel(const ActBwdArgs a) {
  constexpr int PARTS = 256 / COLS;
  __shared__ float sums[256];
  const int g = blockIdx.y, col = threadIdx.x % COLS, w = threadIdx.x / COLS;
  const int n = blockIdx.x * COLS + col;
  int64_t first, second;
  rows_of(a, g, first, second);
  const int64_t b0 = a.masked_m ? static_cast<int64_t>(g) * a.nb : first / a.R;
  const int64_t blocks = second > first ? (second - first + a.R - 1) / a.R : 0;
  const int64_t each = (blocks + PARTS - 1) / PARTS;
  const int64_t lo = w * each, hi = lo + each < blocks ? lo + each : blocks;
  float t = 0.0f;
  if (n < a.N)
#pragma unroll 4
    for (int64_t b = lo; b < hi; ++b) t += a.part[(b0 + b) * a.N + n];
  sums[threadIdx.x] = t;
  __syncthreads();
  if (w != 0 || n >= a.N) return;
#pragma unroll
  for (int k = 1; k < PARTS; ++k) t += sums[k * COLS + col];
  put_bias_grad(a.dbias, a.f32, a.acc, static_cast<int64_t>(g) * a.N + n, t);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Rows of a block: few enough that the blocks fill the card, a divisor of the 128 to
// which the compact layout pads.
int block_rows(int64_t M, int64_t chunks) {
  int R = 128;
  while (R > 16 && (M + R - 1) / R * chunks < 2048) R /= 2;
  return R;
}

// Few rows an expert: one launch, in which each workgroup takes all rows of an expert by
// 128 columns, 16 rows at a time.  us (N 1024, gated): 8 experts of 8 rows 9.5 (with a
// second launch for the sums 13.9).
bool few_rows(int64_t M, int G) { return M <= 128ll * G && M <= 1024; }

// rows: workgroups in the first dimension.  The chunks of a row's columns are more than the
// second one holds (65535) from 8 M columns on.
template <bool WHOLE>
void launch(const ActBwdArgs& a, int64_t rows, hipStream_t s) {
  const int chunks = (a.cols / 8 + a.lanes - 1) / a.lanes, y = chunks < 65535 ? chunks : 65535;
  const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(y), static_cast<unsigned>((chunks + y - 1) / y));
  if (a.act.gated) act_bwd_kernel<true, WHOLE><<<grid, 256, 0, s>>>(a);
  else act_bwd_kernel<false, WHOLE><<<grid, 256, 0, s>>>(a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_act_bwd_ws_bytes(int64_t M, int32_t N, int32_t G) {
  if (M <= 0 || N <= 0 || G <= 0 || few_rows(M, G)) return 0;
  // a masked group's last block may be cut: at most one block more a group
  return (static_cast<size_t>((M + 15) / 16) + G) * N * sizeof(float);
}

extern "C" int32_t moe_act_bwd(const void* pre, int32_t dout_dtype, const void* dout, int64_t M, int32_t N, int32_t act,
                               float alpha, float limit, const int32_t* m_indices, const int32_t* masked_m, int32_t max_m,
                               const int32_t* expert_start_loc, const int32_t* num_valid, int32_t G, void* dpre,
                               int32_t dbias_dtype, int32_t accumulate, void* dbias, void* ws, size_t ws_bytes,
                               void* stream) {
  ActBwdArgs a{};
  if (M < 0 || N <= 0 || G <= 0) return MOE_EINVAL;
  if (!make_act(act, alpha, limit, a.act)) return MOE_EINVAL;
  if (N % (a.act.gated ? 16 : 8) != 0) return MOE_EUNSUPPORTED;
  if (N > (1 << 27) || M >= (1 << 26) || G > 65535) return MOE_EUNSUPPORTED;
  if (dout_dtype != MOE_DTYPE_BF16 && dout_dtype != MOE_DTYPE_FP32) return MOE_EUNSUPPORTED;
  if (masked_m && m_indices) return MOE_EINVAL;
  if (masked_m && (max_m <= 0 || M % max_m != 0 || (dbias && M / max_m != G))) return MOE_EINVAL;
  if (M > 0 && !masked_m && !m_indices && G != 1) return MOE_EINVAL;  // tensors without elements have no address
  if (dbias && dbias_dtype != MOE_DTYPE_BF16 && dbias_dtype != MOE_DTYPE_FP32) return MOE_EUNSUPPORTED;
  if (dbias && m_indices && (!expert_start_loc || !num_valid)) return MOE_EINVAL;
  if (M > 0 && !dpre && (a.act.kind != kActNone || !dbias)) return MOE_EINVAL;
  if (M > 0 && (!dout || (a.act.kind != kActNone && !pre))) return MOE_EINVAL;
  if (dbias && ws_bytes < moe_act_bwd_ws_bytes(M, N, G)) return MOE_ECAPACITY;
  if (dbias && !ws && moe_act_bwd_ws_bytes(M, N, G) > 0) return MOE_EINVAL;
  if (!aligned16(pre) || !aligned16(dout) || !aligned16(dpre) || !aligned16(dbias) || !aligned16(ws)) return MOE_EUNSUPPORTED;
  if (M == 0 && (!dbias || accumulate)) return MOE_OK;
  if (M > 0 && dpre == dout && (a.act.gated || dout_dtype == MOE_DTYPE_FP32)) return MOE_EINVAL;  // other places for the same element
  if (M > 0 && dbias && (dbias == dpre || dbias == dout || (a.act.kind != kActNone && dbias == pre))) return MOE_EINVAL;
  a.pre = a.act.kind == kActNone ? nullptr : static_cast<const uint16_t*>(pre);
  a.dout = dout;
  a.dout32 = dout_dtype == MOE_DTYPE_FP32;
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
  a.dbias = dbias;
  a.f32 = dbias_dtype == MOE_DTYPE_FP32;
  a.acc = accumulate != 0;
  const int groups = a.cols / 8;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dbias && few_rows(M, G)) {
    a.lanes = 16;
    launch<true>(a, G, s);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
  }
  a.lanes = groups > 32 ? 64 : groups > 16 ? 32 : 16;
  a.R = block_rows(M, (groups + a.lanes - 1) / a.lanes);
  a.nb = masked_m ? (max_m + a.R - 1) / a.R : 0;
  if (M > 0) {
    const int64_t blocks = masked_m ? M / max_m * a.nb : (M + a.R - 1) / a.R;
    if (blocks >= (1 << 24)) return MOE_EUNSUPPORTED;  // threads of a launch
    launch<false>(a, blocks, s);
    MOE_CHECK_LAUNCH();
  }
  if (dbias) {
    const bool many = static_cast<int64_t>(N) * G > 16 * 4096;
    const dim3 grid(static_cast<unsigned>(many ? (N + 63) / 64 : (N + 15) / 16), static_cast<unsigned>(G));
    if (many) bias_grad_kernel<64><<<grid, 256, 0, s>>>(a);
    else bias_grad_kernel<16><<<grid, 256, 0, s>>>(a);
    MOE_CHECK_LAUNCH();
  }
  return MOE_OK;
}
