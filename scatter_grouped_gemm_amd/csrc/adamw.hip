// One AdamW step over many tensors, states in fp32 or in 8 bits.
//
// With t the number of this step and g the (scaled) gradient, all in fp32:
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps).
//
// 8-bit states: groups of 128 elements share one UE8M0 scale (2^e, e the smallest
// with amax <= 448 * 2^e, as everywhere in this library; what differs here is the
// reciprocal that a value is multiplied by, see the kernel).  m is kept as e4m3,
// v as the e4m3 of its root: the root needs half the octaves, so a group may
// mix gradients 2^17 apart before the small ones reach the last code, and a
// positive root keeps at least that code (a root of zero would turn the next
// small m into a step of m / eps).  Both are rounded up with the probability
// of the remainder: a step moves v by a factor of at most 1 - b2 (0.1% at b2 =
// 0.999), far less than the 6-12% between codes, so rounding to nearest would
// leave v where it is for good.  This way the expectation of m and of the root
// is what the formula gives.  That of v, the root's square, is higher by the
// root's variance f (1 - f) u^2 (f the remainder in units u of the last place),
// and the next step goes on from there: with normally distributed gradients v
// settles 2% above its mean at b2 = 0.95 and 4% at 0.999 (3% and 7% where nine
// in ten gradients are zero; never by more than an eighth of the mean of
// |g^2 - v|), and the steps come out half as much short.
// The random bits are a hash of (seed, step, tensor, element), so a step is
// reproducible and needs no generator state.
//
// Bound by memory: per element 28 bytes (32-bit states, bf16 weight and
// gradient with an fp32 master; 268M elements 1520 us, 4.9 TB/s) or 16 (8-bit states).  One launch for all
// tensors: the plan lists the chunks of 2048 elements, and each workgroup takes
// every gridDim-th one.
#include <float.h>
#include <string.h>

#include "common.h"

namespace moe {
namespace {

typedef __attribute__((ext_vector_type(4))) unsigned int u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned int u32x2;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) float f32x2;

constexpr int kChunk = 2048;  // elements: 256 threads of 8
constexpr uint64_t kMagic = 0x6d6f656164616d77ull;

// The plan: this header, the tensors, then an int2 (tensor, chunk) per chunk.
struct Header {
  uint64_t magic;
  int32_t tensors, chunks;
};
static_assert(sizeof(Header) == 16 && sizeof(moe_adamw_tensor) == 80, "plan layout");

// A 32-bit hash of shifts and products.  The factors are the first two 32-bit primes
// of the xxHash specification (the first is 2^32 over the golden ratio, nearly).
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B1u;
  x ^= x >> 15;
  x *= 0x85EBCA77u;
  return x ^ (x >> 16);
}

// b^t by squaring, in double (t >= 1)
__device__ __forceinline__ double power(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

struct Coeff {
  float b1, a1, b2, a2, keep, rate, root, eps, gscale;
};

// Codes of eight values (in units of the group's scale, whose reciprocal is
// given; at most 448 then) rounded up where the remainder plus 16 random bits
// carries.
template <bool KEEP>
__device__ __forceinline__ u32x2 encode8(const float (&x)[8], float inverse, const uint32_t (&bits)[8]) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]) * inverse;
    // last place of a's code: 2^(E - 3), E its exponent, not below 2^-9
    const int top = max(static_cast<int>(__float_as_uint(a) >> 23), 127 - 6);
    float n = floorf(__builtin_fmaf(static_cast<float>(bits[i]), 0x1p-16f, __builtin_amdgcn_ldexpf(a, 130 - top)));
    if (KEEP) n = fmaxf(n, a > 0.0f ? 1.0f : 0.0f);
    q[i] = copysignf(__builtin_amdgcn_ldexpf(n, top - 130), x[i]);
  }
  u32x2 c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // exact: every value is a code's
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
    c[h] = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], lo, true);
  }
  return c;
}

__device__ __forceinline__ void decode8(u32x2 c, int e, float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(c[h], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(c[h], true);
    x[4 * h] = __builtin_amdgcn_ldexpf(a[0], e);
    x[4 * h + 1] = __builtin_amdgcn_ldexpf(a[1], e);
    x[4 * h + 2] = __builtin_amdgcn_ldexpf(b[0], e);
    x[4 * h + 3] = __builtin_amdgcn_ldexpf(b[1], e);
  }
}

// Eight elements at i of a 16- or 32-bit tensor, n of them inside it.
__device__ __forceinline__ void load8(const void* p, bool half, int64_t i, int n, float (&x)[8]) {
  if (half) {
    const uint16_t* s = static_cast<const uint16_t*>(p) + i;
    if (n == 8) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(s);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(v[j] << 16);
        x[2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = j < n ? bf16_to_f32(s[j]) : 0.0f;
    }
  } else {
    const float* s = static_cast<const float*>(p) + i;
    if (n == 8) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(s), b = *reinterpret_cast<const f32x4*>(s + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = a[j];
        x[4 + j] = b[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = j < n ? s[j] : 0.0f;
    }
  }
}

__device__ __forceinline__ void store8(void* p, bool half, int64_t i, int n, const float (&x)[8]) {
  if (half) {
    uint16_t* d = static_cast<uint16_t*>(p) + i;
    if (n == 8) {
      *reinterpret_cast<u32x4*>(d) = u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                           pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) d[j] = f32_to_bf16(x[j]);
    }
  } else {
    float* d = static_cast<float*>(p) + i;
    if (n == 8) {
      *reinterpret_cast<f32x4*>(d) = f32x4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4*>(d + 4) = f32x4{x[4], x[5], x[6], x[7]};
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) d[j] = x[j];
    }
  }
}

// 64 registers, so that eight workgroups fit a CU: in 8 bits the arithmetic of an
// element (two hashes, two roundings, a root) takes about as long as its 16 bytes
// (268M elements: 913 us, 4.7 TB/s; 84 registers 5% slower).
//
// The quotient of the update is a product with the hardware's reciprocal, within two
// fp32 places.  That of a subnormal denominator may be infinite, and a weight that no
// gradient has reached would get 0 * inf: DIVIDE, for a subnormal eps, divides (8 bits,
// 268M elements 923 us, 913 with the reciprocal; in 32 bits 1520 us either way).
template <bool DIVIDE>
__global__ __launch_bounds__(256, 8) void adamw_kernel(const uint8_t* __restrict__ plan, size_t plan_bytes,
                                                    const float* __restrict__ lr,
                                                    const float* __restrict__ grad_scale,
                                                    int64_t* counter, double beta1, double beta2,
                                                    float eps, uint32_t seed) {
  // The reciprocal of each scale, taken as powf(2, -e): within 2^-24 of 2^-e (one place
  // off for 41 of the 254 exponents), and what a torch program that scales by a power
  // multiplies by on this card, so that such a program gets the same codes bit for bit.
  // The exact power gives another code where the remainder and the random bits add up
  // to 1 but for that place (one in half a million), and takes as long.
  __shared__ float inverse[256];
  float two = 2.0f;
  asm volatile("" : "+v"(two));  // as a constant it becomes exp2f, which is another function
  inverse[threadIdx.x] = powf(two, static_cast<float>(127 - static_cast<int>(threadIdx.x)));
  __syncthreads();
  const Header* const h = reinterpret_cast<const Header*>(plan);
  const moe_adamw_tensor* const tensors = reinterpret_cast<const moe_adamw_tensor*>(plan + sizeof(Header));
  const int2* const chunks = reinterpret_cast<const int2*>(tensors + h->tensors);
  // a plan cut short lists nothing, and its call is no step
  const bool whole = h->magic == kMagic && sizeof(Header) + h->tensors * sizeof(moe_adamw_tensor) +
                                                   h->chunks * sizeof(int2) <= plan_bytes;
  const int nchunk = whole ? h->chunks : 0;
  const int64_t step = counter[0] + 1;
  const float rate0 = lr[0];
  const float gscale = grad_scale ? grad_scale[0] : 1.0f;
  const float rate = static_cast<float>(rate0 / (1.0 - power(beta1, step)));
  const float root = static_cast<float>(1.0 / sqrt(1.0 - power(beta2, step)));
  const float b1 = static_cast<float>(beta1), a1 = static_cast<float>(1.0 - beta1);
  const float b2 = static_cast<float>(beta2), a2 = static_cast<float>(1.0 - beta2);

  for (int c = blockIdx.x; c < nchunk; c += gridDim.x) {
    const int2 at = chunks[c];
    const moe_adamw_tensor d = tensors[at.x];
    const int64_t i = static_cast<int64_t>(at.y) * kChunk + threadIdx.x * 8;
    const int64_t left = d.numel - i;
    const int n = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
    const bool pbf = d.param_dtype == MOE_DTYPE_BF16, gbf = d.grad_dtype == MOE_DTYPE_BF16;
    const int64_t grp = i >> 7;
    float p[8], g[8], m[8], v[8];
    // lanes behind the tensor's end stay (zeros) for the group maxima below
    load8(pbf ? d.master : d.param, false, i, n, p);
    load8(d.grad, gbf, i, n, g);
    if (d.state_bits == 8) {
      int em = 0, ev = 0;
      u32x2 cm{0u, 0u}, cv{0u, 0u};
      if (n > 0) {  // the 8-bit states hold whole groups
        em = d.m_scale[grp] - 127;
        ev = d.v_scale[grp] - 127;
        cm = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(d.m) + i);
        cv = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(d.v) + i);
      }
      decode8(cm, em, m);
      decode8(cv, ev, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < n ? v[j] * v[j] : 0.0f;
    } else {
      load8(d.m, false, i, n, m);
      load8(d.v, false, i, n, v);
    }
    const float keep = 1.0f - rate0 * d.weight_decay;
    float r[8], mmax = 0.0f, rmax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = g[j] * gscale;
      m[j] = j < n ? b1 * m[j] + a1 * x : 0.0f;
      v[j] = b2 * v[j] + a2 * x * x;
      // correctly rounded, as the sums above: the codes that the random bits
      // choose then follow from the definition in fp32 alone
      r[j] = sqrtf(v[j]);
      const float den = r[j] * root + eps;
      p[j] = p[j] * keep - (DIVIDE ? rate * m[j] / den : rate * m[j] * __builtin_amdgcn_rcpf(den));
      mmax = fmaxf(mmax, fabsf(m[j]));
      rmax = fmaxf(rmax, r[j]);
    }
    if (d.state_bits == 8) {
      // 16 lanes hold a group
      const int em = ue8m0_exponent(group_max<16>(mmax)), ev = ue8m0_exponent(group_max<16>(rmax));
      if (n > 0) {
        const uint32_t key = mix(mix(seed + 0x9E3779B9u * static_cast<uint32_t>(at.x + 1)) + static_cast<uint32_t>(step)) ^
                             static_cast<uint32_t>(i >> 32);
        uint32_t lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t b = mix(mix(static_cast<uint32_t>(i) + j) ^ key);
          lo[j] = b & 0xffffu;
          hi[j] = b >> 16;
        }
        *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(d.m) + i) = encode8<false>(m, inverse[em + 127], lo);
        *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(d.v) + i) = encode8<true>(r, inverse[ev + 127], hi);
        if ((threadIdx.x & 15) == 0) {
          d.m_scale[grp] = static_cast<uint8_t>(em + 127);
          d.v_scale[grp] = static_cast<uint8_t>(ev + 127);
        }
      }
    } else if (n > 0) {
      store8(d.m, false, i, n, m);
      store8(d.v, false, i, n, v);
    }
    if (n > 0) {
      if (pbf) store8(d.master, false, i, n, p);
      store8(d.param, pbf, i, n, p);
    }
  }
  // The last workgroup to finish moves the step counter on: every other one
  // has read it before it took its ticket.
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned long long ticket = atomicAdd(reinterpret_cast<unsigned long long*>(counter + 1), 1ull);
    if (ticket == gridDim.x - 1) {
      if (whole) counter[0] = step;
      counter[1] = 0;
    }
  }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// MOE_OK and the chunk count of valid tensors, else the status.
int32_t check(const moe_adamw_tensor* t, int32_t n, int64_t* chunks) {
  if (n < 0 || (n > 0 && !t)) return MOE_EINVAL;
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    const moe_adamw_tensor& d = t[i];
    if (d.numel < 0) return MOE_EINVAL;
    if (d.param_dtype != MOE_DTYPE_BF16 && d.param_dtype != MOE_DTYPE_FP32) return MOE_EUNSUPPORTED;
    if (d.grad_dtype != MOE_DTYPE_BF16 && d.grad_dtype != MOE_DTYPE_FP32) return MOE_EUNSUPPORTED;
    if (d.state_bits != 8 && d.state_bits != 32) return MOE_EUNSUPPORTED;
    if (d.numel == 0) continue;
    if (!d.param || !d.grad || !d.m || !d.v) return MOE_EINVAL;
    if (d.param_dtype == MOE_DTYPE_BF16 && !d.master) return MOE_EINVAL;
    if (d.state_bits == 8 && (!d.m_scale || !d.v_scale)) return MOE_EINVAL;
    if (!aligned16(d.param) || !aligned16(d.grad) || !aligned16(d.m) || !aligned16(d.v)) return MOE_EUNSUPPORTED;
    if (d.param_dtype == MOE_DTYPE_BF16 && !aligned16(d.master)) return MOE_EUNSUPPORTED;
    // compared before it is added: neither sum passes 64 bits
    if (d.numel > static_cast<int64_t>(INT32_MAX) * kChunk) return MOE_EUNSUPPORTED;
    total += (d.numel + kChunk - 1) / kChunk;
    if (total > INT32_MAX) return MOE_EUNSUPPORTED;
  }
  *chunks = total;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_adamw_plan_bytes(const moe_adamw_tensor* tensors, int32_t n) {
  int64_t chunks = 0;
  if (check(tensors, n, &chunks) != MOE_OK) return 0;
  return sizeof(Header) + static_cast<size_t>(n) * sizeof(moe_adamw_tensor) + static_cast<size_t>(chunks) * sizeof(int2);
}

extern "C" int32_t moe_adamw_plan(const moe_adamw_tensor* tensors, int32_t n, void* host_plan,
                                  size_t plan_bytes) {
  int64_t chunks = 0;
  const int32_t st = check(tensors, n, &chunks);
  if (st != MOE_OK) return st;
  if (!host_plan) return MOE_EINVAL;
  if (plan_bytes < moe_adamw_plan_bytes(tensors, n)) return MOE_ECAPACITY;
  uint8_t* out = static_cast<uint8_t*>(host_plan);
  const Header h{kMagic, n, static_cast<int32_t>(chunks)};
  memcpy(out, &h, sizeof h);
  out += sizeof h;
  if (n > 0) memcpy(out, tensors, n * sizeof(moe_adamw_tensor));
  out += n * sizeof(moe_adamw_tensor);
  for (int32_t i = 0; i < n; ++i)
    for (int64_t c = 0; c * kChunk < tensors[i].numel; ++c) {
      const int2 at = make_int2(i, static_cast<int>(c));
      memcpy(out, &at, sizeof at);
      out += sizeof at;
    }
  return MOE_OK;
}

extern "C" int32_t moe_adamw_step(const void* plan, size_t plan_bytes, const float* lr,
                                  const float* grad_scale, int64_t* counter, double beta1,
                                  double beta2, float eps, uint32_t seed, void* stream) {
  if (!plan || !lr || !counter || plan_bytes < sizeof(Header)) return MOE_EINVAL;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps > 0.0f)) return MOE_EINVAL;
  if (!aligned16(plan) || (reinterpret_cast<uintptr_t>(counter) & 7)) return MOE_EUNSUPPORTED;
  // no more workgroups than the plan can hold chunks; than are resident
  // together (more would each work out the table of scales again: 8192, 4% slower)
  const size_t most = (plan_bytes - sizeof(Header)) / sizeof(int2);
  const unsigned grid = most < 1 ? 1u : most < 2048 ? static_cast<unsigned>(most) : 2048u;
  // a normal eps keeps the denominator normal
  const auto kernel = eps < FLT_MIN ? adamw_kernel<true> : adamw_kernel<false>;
  kernel<<<grid, 256, 0, static_cast<hipStream_t>(stream)>>>(
      static_cast<const uint8_t*>(plan), plan_bytes, lr, grad_scale, counter, beta1, beta2, eps, seed);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
