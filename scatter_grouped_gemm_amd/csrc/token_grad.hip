// Gradients of the weighted combine and of the top-k routing weights.
//
// With out[t] = sum_j w[t][j] Y[r(t,j)] and the gradient dout of out:
//   dY[r(t,j)] = w[t][j] dout[t],   dw[t][j] = <dout[t], Y[r(t,j)]>.
// One pass reads dout once and every expert-output row once and writes every
// gradient row once, so the kernel is bound by memory: 2 T H + 4 A H bytes for
// A held assignments (8192 tokens, H 7168, top-8 with the routing gradient: 400
// us, 5.0 TB/s, what a plain copy reaches; 4096 tokens, top-16 382 us, 5.1 TB/s, top-32
// 764 us, 5.0 TB/s: dout is read again for every eight slots, from the caches).
#include "common.h"

namespace moe {
namespace {

typedef __attribute__((ext_vector_type(4))) unsigned int u32x4;

__device__ __forceinline__ float lo16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi16(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Sums of eight values over the 64 lanes: three exchange steps halve the
// number of values a lane carries (lane bits 5, 4, 3 select which), three more
// finish the one that is left; `slot` is the value whose sum a lane ends with.  Ten
// shuffles in place of forty-eight, and always the same order of additions.
__device__ __forceinline__ float reduce8(float (&v)[8], int lane, int& slot) {
  float a[4], b[2], c;
  const bool h5 = lane & 32, h4 = lane & 16, h3 = lane & 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = (h5 ? v[i + 4] : v[i]) + __shfl_xor(h5 ? v[i] : v[i + 4], 32, 64);
#pragma unroll
  for (int i = 0; i < 2; ++i) b[i] = (h4 ? a[i + 2] : a[i]) + __shfl_xor(h4 ? a[i] : a[i + 2], 16, 64);
  c = (h3 ? b[1] : b[0]) + __shfl_xor(h3 ? b[0] : b[1], 8, 64);
  c += __shfl_xor(c, 4, 64);
  c += __shfl_xor(c, 2, 64);
  c += __shfl_xor(c, 1, 64);
  slot = (h5 ? 4 : 0) + (h4 ? 2 : 0) + (h3 ? 1 : 0);
  return c;
}

// One workgroup per token, each thread 8 consecutive channels at a time, the
// workgroup as wide as the row or half of it.  Slots go
// in groups of eight: a group's Y rows are loaded together (independent
// 16-byte loads in flight), multiplied into eight dot products held in fp32,
// and the gradient rows written.  The partial sums of a token are added in an
// order that depends on H alone.
template <int SLOTS>
__global__ __launch_bounds__(1024) void combine_bwd_kernel(
    const uint16_t* __restrict__ dout, const uint16_t* __restrict__ Y, int64_t num_rows,
    const int32_t* __restrict__ src2dst, const float* __restrict__ w, int k, int H,
    uint16_t* __restrict__ dY, float* __restrict__ dw) {
  __shared__ float part[16][8];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const uint16_t* const g = dout + t * H;
  for (int j0 = 0; j0 < k; j0 += SLOTS) {
    int64_t row[SLOTS];
    float wt[SLOTS], dot[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dot[j] = 0.0f;
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      row[j] = -1;
      wt[j] = 0.0f;
      if (j0 + j < k) {
        const int64_t r = src2dst[t * k + j0 + j];
        row[j] = r < num_rows ? r : -1;
        wt[j] = w[t * k + j0 + j];
      }
    }
    for (int col = threadIdx.x * 8; col < H; col += blockDim.x * 8) {
      const u32x4 gv = *reinterpret_cast<const u32x4*>(g + col);
      u32x4 y[SLOTS];
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) {
        y[j] = u32x4{0u, 0u, 0u, 0u};
        if (row[j] >= 0)  // read once here: past the caches
          y[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(Y + row[j] * H + col));
      }
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) {
        if (row[j] < 0) continue;
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = lo16(gv[i]), b = hi16(gv[i]);
          dot[j] = __builtin_fmaf(a, lo16(y[j][i]), dot[j]);
          dot[j] = __builtin_fmaf(b, hi16(y[j][i]), dot[j]);
          o[i] = pack_bf16x2(wt[j] * a, wt[j] * b);
        }
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(dY + row[j] * H + col));
      }
    }
    int slot;
    const float s = reduce8(dot, lane, slot);
    if (j0) __syncthreads();  // the group before has been read
    if ((lane & 7) == 0) part[wave][slot] = s;
    __syncthreads();
    if (threadIdx.x < SLOTS && j0 + threadIdx.x < k) {
      float sum = 0.0f;
      for (int q = 0; q < waves; ++q) sum += part[q][threadIdx.x];
      dw[t * k + j0 + threadIdx.x] = sum;  // a slot held elsewhere has no products: 0
    }
  }
}

// Router gradient: the weights are the softmax of the k kept logits, so
// dL[id_j] = w_j (dw_j - sum_i w_i dw_i) and 0 for the others.  One wavefront
// per token; a lane holds the logits lane + 64 i and adds the slots that name
// them in slot order (an id named twice gets both terms; ids outside [0, E)
// are skipped).
template <int PER_LANE>
__global__ __launch_bounds__(256) void route_topk_bwd_kernel(const int32_t* __restrict__ ids,
                                                             const float* __restrict__ w,
                                                             const float* __restrict__ dw, int T,
                                                             int E, int k, float* __restrict__ dl) {
  const int lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  int id = -1;
  float wj = 0.0f, g = 0.0f;
  if (lane < k) {
    id = ids[t * k + lane];
    wj = w[t * k + lane];
    g = dw[t * k + lane];
  }
  float sum = 0.0f;
  for (int j = 0; j < k; ++j) sum += __shfl(wj * g, j, 64);
  const float term = wj * (g - sum);
  float acc[PER_LANE];
#pragma unroll
  for (int i = 0; i < PER_LANE; ++i) acc[i] = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int e = __shfl(id, j, 64);
    const float v = __shfl(term, j, 64);
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) acc[i] += lane + 64 * i == e ? v : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < PER_LANE; ++i)
    if (lane + 64 * i < E) dl[t * E + lane + 64 * i] = acc[i];
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int32_t moe_combine_bwd(const void* dout, const void* Y, int64_t num_rows,
                                   const int32_t* src2dst, const float* topk_weights, int32_t T,
                                   int32_t k, int32_t H, void* dY, float* dtopk_weights,
                                   void* stream) {
  if (T < 0 || k < 1 || k > 32 || H <= 0 || num_rows < 0) return MOE_EINVAL;
  if (H % 8 != 0 || H > (1 << 30)) return MOE_EUNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!dout || !src2dst || !topk_weights || !dtopk_weights) return MOE_EINVAL;
  if (num_rows > 0 && (!Y || !dY)) return MOE_EINVAL;
  if (!aligned16(dout) || !aligned16(Y) || !aligned16(dY)) return MOE_EUNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  // Rows of more than 512 threads in two passes of half as many: more workgroups on
  // a CU, so more loads in flight where most slots are held elsewhere (1021 tokens,
  // H 7168, an eighth of their 8 slots held: 11.6 us, 16.0 in one pass; all held
  // 47.4, 48.6; 256 tokens 6.0, 5.6; 8192 tokens 377.7, 376.0).
  const int need = (H / 8 + 63) / 64 * 64;
  const int half = (need / 2 + 63) / 64 * 64;
  const int nt = need <= 512 ? need : half < 1024 ? half : 1024;
  if (static_cast<int64_t>(T) * (need < 1024 ? need : 1024) >= (1ll << 32)) return MOE_EUNSUPPORTED;  // threads of a launch
  const uint16_t *g = static_cast<const uint16_t*>(dout), *y = static_cast<const uint16_t*>(Y);
  uint16_t* d = static_cast<uint16_t*>(dY);
  if (k <= 2)
    combine_bwd_kernel<2><<<T, nt, 0, s>>>(g, y, num_rows, src2dst, topk_weights, k, H, d, dtopk_weights);
  else if (k <= 4)
    combine_bwd_kernel<4><<<T, nt, 0, s>>>(g, y, num_rows, src2dst, topk_weights, k, H, d, dtopk_weights);
  else
    combine_bwd_kernel<8><<<T, nt, 0, s>>>(g, y, num_rows, src2dst, topk_weights, k, H, d, dtopk_weights);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" int32_t moe_route_topk_bwd(const int32_t* topk_ids, const float* topk_weights,
                                      const float* dtopk_weights, int32_t T, int32_t E, int32_t k,
                                      float* dlogits, void* stream) {
  if (T < 0 || E < 1 || E > 1024 || k < 1 || k > E || k > 32) return MOE_EINVAL;
  if (T >= (1 << 26)) return MOE_EUNSUPPORTED;  // threads of a launch
  if (T == 0) return MOE_OK;
  if (!topk_ids || !topk_weights || !dtopk_weights || !dlogits) return MOE_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(T) + 3) / 4)), block(256);
  const int per = (E + 63) / 64;
  if (per <= 1)
    route_topk_bwd_kernel<1><<<grid, block, 0, s>>>(topk_ids, topk_weights, dtopk_weights, T, E, k, dlogits);
  else if (per <= 2)
    route_topk_bwd_kernel<2><<<grid, block, 0, s>>>(topk_ids, topk_weights, dtopk_weights, T, E, k, dlogits);
  else if (per <= 4)
    route_topk_bwd_kernel<4><<<grid, block, 0, s>>>(topk_ids, topk_weights, dtopk_weights, T, E, k, dlogits);
  else if (per <= 8)
    route_topk_bwd_kernel<8><<<grid, block, 0, s>>>(topk_ids, topk_weights, dtopk_weights, T, E, k, dlogits);
  else
    route_topk_bwd_kernel<16><<<grid, block, 0, s>>>(topk_ids, topk_weights, dtopk_weights, T, E, k, dlogits);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
