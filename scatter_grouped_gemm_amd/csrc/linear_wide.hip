// Products with bias, activation and residual in their epilogue, BF16, in tiles of 256
// rows by 256 rows of B: the dense one (moe_linear) and the compact grouped one
// (grouped_gemm_contig_act).
//
//   - Workgroup = 8 wavefronts in two groups of four, one wavefront of each group on
//     every SIMD.  A wavefront owns 64 + 64 rows by 64 columns of the tile in four
//     quadrants.  A step of 64 of the reduction is four phases, a phase is a load part
//     (LDS reads, global loads) and an MFMA part (16 instructions of one quadrant),
//     each ended by a barrier; the second group runs half a phase behind the first, so
//     on every SIMD one wavefront feeds the matrix core while the other one reads.
//   - Global loads go straight to LDS.  Two stages; each piece of a stage (A's two
//     halves, B) is loaded again as soon as both groups have read it.  16-byte chunks
//     are permuted within their 128-byte row (at the source, since a load fills LDS in
//     lane order), so that fragment reads hit different banks.
//   - The loop is one stream of steps over all of a workgroup's tiles: the loads cross
//     into the next tile while the current one is finished.  Tiles in the order of
//     gemm_runs.h; one matrix is one run.
//   - A tile of up to 128 rows leaves out the MFMAs and reads of its lower half.  An
//     expert's rows are cut 256 at a time where they are many (deep: 1024 an expert, by
//     the buffers' height), and the XCDs' shares made equal with the last tile counted
//     for what it takes; where they are few into tiles of equal height, which read a
//     weight panel side by side and come out of the L2 together.  us, cut by 256 / equal
//     heights: 8 experts of 1024 rows (28672 x 4096) 1610 / 1750, 128 ragged ones of 1024
//     (4096 x 1536) 1525 / 1635; 256 of 256 rows (4096 x 7168) 4860 / 4460, 64 of 128
//     (4096 x 2048) 268 / 248.
//   - Gated: the tile's B rows are 128 of the gate and the same 128 of the up half,
//     laid out so that a wavefront's two column halves are 32 channels' gate and up
//     parts: both are in one lane's registers.
//   - The bias of a wavefront's 64 columns goes to LDS behind the stores of the tile
//     before, a load that the waits count like those stores.
//
// Measured (us; in brackets TFLOP/s; one matrix, torch's bf16 library product in turn, which
// has no epilogue):
//   4096 x 4096 x 28672 650 (1480), gated with pre 690; library 624 (1541).  8192 cubed 716
//   (1534); 666 (1651).  16384 x 1536 x 4096 154 (1340), residual 178; 150 (1377).  8191 x
//   2048 x 7168 188 (1278), residual 208, fp32 out 200; 174 (1385).  8000 x 4104 x 8200 469
//   (1148; K and N with part steps and columns), fp32 out 535 (128 x 128 tiles 657)
//   8 experts of 1024 rows, 28672 x 4096 gated with pre 1580 (1220); 128 ragged ones, 4096
//   x 1536, 131072 rows 1540 (1070)
// What bounds it: within a tile the card's power (matrix cores busy 80% of the cycles at
// 1.64 GHz; 1.33 us a step, 1620 TFLOP/s); between tiles 6 to 8 us, of which 2 to 5 are all
// CUs' stores at the same time and 3 the arithmetic of the epilogue.  No LDS bank conflicts.
//
// Sums run through v_mfma_f32_16x16x32_bf16 in the order of the other kernels of these
// products (linear.hip, gemm_kernel.h), so a row has the same bits from each.
#include <mutex>
#include <type_traits>

#include "gemm_runs.h"
#include "grad_tile.h"
#include "linear.h"

namespace moe {
namespace {

constexpr int kThreads = 512;

struct Tile {
  int64_t row;
  int rows, id, nt;
};

// A copy that the compiler takes for a new value: what is worked out from it once in a
// tile is not kept in registers over the whole loop.
__device__ __forceinline__ int fresh_copy(int x) {
  asm volatile("" : "+s"(x));
  return x;
}

// Eight columns of a row as a lane holds them after swap_rows of two 16-column blocks'
// values v0, v1 (four columns of each before): block 0 in even lane groups, 1 in odd ones.
__device__ __forceinline__ u32x4 pack8(f32x4 v0, f32x4 v1) {
  const u32x4 o = __builtin_bit_cast(
      u32x4, swap_rows(__uint_as_float(pack_bf16x2(v0[0], v0[1])), __uint_as_float(pack_bf16x2(v1[0], v1[1])),
                       __uint_as_float(pack_bf16x2(v0[2], v0[3])), __uint_as_float(pack_bf16x2(v1[2], v1[3]))));
  return u32x4{o[0], o[2], o[1], o[3]};
}
// The same with the bf16 values of r added in fp32.
__device__ __forceinline__ u32x4 pack8_add(f32x4 v0, f32x4 v1, u32x4 r) {
  const auto add = [&](uint32_t o, float lo, float hi) __attribute__((always_inline)) {
    return pack_bf16x2(lo + __uint_as_float(o << 16), hi + __uint_as_float(o & 0xffff0000u));
  };
  const f32x4 s0 = swap_rows(v0[0], v1[0], v0[1], v1[1]), s1 = swap_rows(v0[2], v1[2], v0[3], v1[3]);
  return u32x4{add(r[0], s0[0], s0[2]), add(r[1], s1[0], s1[2]), add(r[2], s0[1], s0[3]), add(r[3], s1[1], s1[3])};
}

// GROUPED: the compact layout; else one matrix, whose tiles are whole but for one row of
// them, so that leaving out a half would cost more (a branch a phase, 1%) than it gains.
// TAIL: K is no multiple of 64.  What a row's last step holds behind K is read as 0 by
// both operands: the lanes that carry it get an offset outside the buffer.
template <bool GROUPED, bool GATED, bool PRE, bool RES, bool F32, bool TAIL>
__global__ __launch_bounds__(kThreads, 2) void linear_wide_kernel(const LinearArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  static_assert(!RES || !(GROUPED || GATED || PRE || F32), "no store for gated ones; too many registers with pre or fp32");
  static_assert(!F32 || !(GROUPED || PRE), "the grouped products have no fp32 output");
  // A half h of stage s, B of stage s.  Arrays of their own: the compiler then knows
  // which loads to LDS a read can depend on.
  __shared__ __attribute__((aligned(1024))) uint8_t p00[16384], p01[16384], p10[16384], p11[16384];
  __shared__ __attribute__((aligned(1024))) uint8_t q0[32768], q1[32768];
  __shared__ __attribute__((aligned(16))) uint8_t sbias[8 * 256];
  __shared__ int4 table[GROUPED ? runs::kTable : 1];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int fr = lane & 15, fg = lane >> 4;
  constexpr int kCols = GATED ? 128 : 256;  // output columns of a tile
  const int64_t ldb = static_cast<int64_t>(a.K) * 2;
  const int ntn = (a.cols + kCols - 1) / kCols;

  // ======== the tiles of this workgroup ========
  int pos, pos_end, stride, NR, cur = 0;
  if constexpr (GROUPED) {
    runs::Share sh;
    static_assert(runs::kMaxBlocks * 4 <= 32768, "the set-up arrays fit in the stages");
    if (!runs::build_share<8, true, true>(a.m_indices, a.M, a.G, ntn, reinterpret_cast<int*>(q0),
                                    reinterpret_cast<int*>(q1), reinterpret_cast<int*>(p00), table, sh, a.deep != 0))
      return;
    NR = __builtin_amdgcn_readfirstlane(sh.NR);
    pos = __builtin_amdgcn_readfirstlane(sh.lo) + static_cast<int>(blockIdx.x >> 3);
    pos_end = __builtin_amdgcn_readfirstlane(sh.hi);
    stride = sh.per_xcd;
  } else {
    const int M = static_cast<int>(a.M);
    if (threadIdx.x == 0) table[0] = make_int4(0, 0, M, 0);
    __syncthreads();
    NR = 1;
    const int64_t U = static_cast<int64_t>(runs::tiles_of(M)) * ntn;
    const int xcd = blockIdx.x & 7;
    pos = static_cast<int>((U * xcd) >> 3) + static_cast<int>(blockIdx.x >> 3);
    pos_end = static_cast<int>((U * (xcd + 1)) >> 3);
    stride = gridDim.x >> 3;
  }
  const int quantum = GROUPED && !a.deep ? 16 : runs::kTileRows;  // of a tile's rows
  // The workgroup's next tile; false: none left.
  auto fetch = [&](Tile& t) __attribute__((always_inline)) -> bool {
    int at = pos, c = cur;
    runs::Tile r;
    r.rows = 0;
    for (; at < pos_end && r.rows <= 0; at += stride) r = runs::decode<16>(table, NR, c, at, fresh_copy(ntn), quantum);
    if (r.rows <= 0) return false;
    pos = at;
    cur = c;
    t.row = r.row;
    t.rows = r.rows;
    t.id = r.id;
    t.nt = r.nt;
    return true;
  };
  const int real = TAIL ? (a.K + kStep - 1) / kStep : a.K / kStep;  // steps that hold something
  const int steps = (real + 1) / 2 * 2;    // a tile is a whole number of pairs of steps
  Tile lt;  // load side
  if (!fetch(lt)) return;
  // Compute side: it is two steps behind the load side, a tile has at least two, so its
  // next tile is the load side's or the one before that.
  Tile ct = lt, before = lt;
  int ahead = 0;  // tiles between the two

  // ======== load side ========
  // A load fills 1 KB: eight rows of 128 bytes, an even load (row & 8) == 0.
  const uint32_t chunk[2] = {static_cast<uint32_t>(((lane & 7) ^ (lane >> 3)) << 4),
                             static_cast<uint32_t>(((lane & 7) ^ (lane >> 3) ^ 1) << 4)};
  uint32_t vp[2], vq[4];
#pragma unroll
  for (int j = 0; j < 2; ++j) vp[j] = static_cast<uint32_t>(((wave * 2 + j) * 8 + (lane >> 3)) * a.lda) + chunk[j & 1];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    int r = (wave * 4 + j) * 8 + (lane >> 3);
    // gated: 32 gate rows, then the up rows of the same channels, for each column wavefront
    if constexpr (GATED) r = (r >> 6) * 32 + (r & 31) + ((r >> 5) & 1) * a.cols;
    vq[j] = static_cast<uint32_t>(r * ldb) + chunk[j & 1];
  }
  // lanes whose 16 bytes are in the step, of even and of odd loads
  [[maybe_unused]] uint64_t keep[2] = {~0ull, ~0ull};
  [[maybe_unused]] uint64_t last[2];
  if constexpr (TAIL)
#pragma unroll
    for (int j = 0; j < 2; ++j) last[j] = __ballot(static_cast<int>(chunk[j]) < (a.K - (real - 1) * kStep) * 2);
  const uint8_t *bp, *bq;  // this step's operands
  int np, np1;             // bytes within bounds of A's halves
  uint32_t nq;
  int lk = 0;
  auto lset = [&]() __attribute__((always_inline)) {
    const int64_t lq = fresh_copy(a.K) * 2ll;
    const int N = fresh_copy(a.N), n0 = lt.nt * kCols;
    bp = a.A + lt.row * a.lda;
    bq = a.B + (static_cast<int64_t>(lt.id) * N + n0) * lq;
    np = (lt.rows < 128 ? lt.rows : 128) * static_cast<int>(a.lda);
    np1 = (lt.rows - 128) * static_cast<int>(a.lda);
    int nr = GATED ? a.cols + kCols : kCols;  // B rows that the tile's offsets reach
    nr = nr < N - n0 ? nr : N - n0;
    nq = static_cast<uint32_t>(nr * lq);
    if constexpr (TAIL) keep[0] = keep[1] = ~0ull;  // a tile has two steps at least
  };
  lset();
  // No immediate offset in these loads: the instruction adds it to the LDS address too.
  auto to_lds = [&](__amdgpu_buffer_rsrc_t rs, uint8_t* dst, uint32_t off) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16, off, 0, 0, 0);
  };
  auto kept = [&](uint32_t off, int j) __attribute__((always_inline)) -> uint32_t {
    if constexpr (TAIL) return __builtin_amdgcn_inverse_ballot_w64(keep[j & 1]) ? off : 0xfffffff0u;
    return off;
  };
  auto load_p = [&](uint8_t* dst, int half) __attribute__((always_inline)) {
    const auto rs = !half ? buffer(bp, np) : buffer(bp + 128 * a.lda, np1);
#pragma unroll
    for (int j = 0; j < 2; ++j) to_lds(rs, dst + (wave * 2 + j) * 1024, kept(vp[j], j));
  };
  auto load_q = [&](uint8_t* dst) __attribute__((always_inline)) {
    const auto rs = buffer_u(bq, nq);
#pragma unroll
    for (int j = 0; j < 4; ++j) to_lds(rs, dst + (wave * 4 + j) * 1024, kept(vq[j], j));
  };
  // on to the next step; behind the last tile its last step is read again (and never
  // used), so that every step issues the same loads.  The step that makes an odd
  // number even holds zeros.
  auto advance = [&]() __attribute__((always_inline)) {
    if (++lk == steps) {
      Tile t = lt;
      if (fetch(t)) {
        before = lt;
        lt = t;
        ++ahead;
        lk = 0;
        lset();
      } else {
        lk = steps - 1;
      }
    } else if (lk == real) {
      np = np1 = 0;
      nq = 0;
    } else {
      bp += kStep * 2;
      bq += kStep * 2;
      if constexpr (TAIL)
        if (lk == real - 1) {
          keep[0] = last[0];
          keep[1] = last[1];
        }
    }
  };

  // ======== compute side ========
  uint32_t op[2], oq[2];  // LDS offsets of this lane's part of a fragment
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t c = ((2 * fg + k) ^ (fr & 7) ^ (fr >> 3)) << 4;
    op[k] = (wm * 64 + fr) * 128 + c;
    oq[k] = (wn * 64 + fr) * 128 + c;
  }
  // Keeps the compiler from working out the address in every array before the loop.
  auto hold = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      asm volatile("" : "+v"(op[k]));
      asm volatile("" : "+v"(oq[k]));
    }
  };
  bf16x8 fp[2][4];     // A half in use: [k half][16-row block]
  bf16x8 fq[2][2][2];  // B half: [half][k half][16-column block]
  f32x4 acc[2][2][4][2];
  auto read_p = [&](const uint8_t* s) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) fp[k][i] = *reinterpret_cast<const bf16x8*>(s + op[k] + i * 2048);
  };
  auto read_q = [&](const uint8_t* s, int h) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) fq[h][k][j] = *reinterpret_cast<const bf16x8*>(s + oq[k] + h * 4096 + j * 2048);
  };
  // D^T: a lane ends with four consecutive columns of one row
  // (a tile's first products start from zero, which saves clearing the accumulators)
  auto mma = [&](int hp, int hq, auto fresh) __attribute__((always_inline)) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[hp][hq][i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              fq[hq][k][j], fp[k][i], decltype(fresh)::value && k == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[hp][hq][i][j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
  };

  // ======== bias: of this wavefront's 64 columns of the compute side's tile ========
  // fp32: a dword a column; bf16: a dword two columns, in the first 32 lanes.  Without
  // a bias, and for columns outside, the load writes zeros.
  uint8_t* const bias_lds = sbias + wave * 256;
  auto load_bias = [&]() __attribute__((always_inline)) {
    int l = lane;
    asm volatile("" : "+v"(l));
    const int es = a.bias32 ? 4 : 2, N = fresh_copy(a.N);
    int c = a.bias32 ? l : 2 * l;           // of the 64
    const bool in = c < 64;
    const int c0 = ct.nt * kCols + wn * (GATED ? 32 : 64);
    if constexpr (GATED) c = (c & 31) + ((c >> 5) & 1) * a.cols;
    const auto rs = buffer(static_cast<const uint8_t*>(a.bias) + (static_cast<int64_t>(ct.id) * N + c0) * es,
                           a.bias ? (N - c0) * es : 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)bias_lds, 4,
                                             in ? static_cast<uint32_t>(c * es) : 0x7ffffff0u, 0, 0, 0);
  };

  // Outputs of the finished tile.  Every wavefront issues the
  // same number of stores whatever its tile holds (rows and columns outside fall
  // outside the buffer and are dropped), so that the waits of the next two steps can
  // count them.
  auto epilogue = [&]() __attribute__((always_inline)) {
    // the lane's place, worked out here: kept over the loop it would cost the registers
    // that the fragments need
    int l = lane;
    asm volatile("" : "+v"(l));
    const int row = l & 15, g = l >> 4;
    if (a.bias) {
      f32x4 bias[2][2];
      // read by hand: the compiler would wait for all loads in flight.  This one was
      // issued before the tile's first step.
      const uint32_t at = runs::lds_off(bias_lds) + g * (a.bias32 ? 16 : 8);
      if (a.bias32) {
        asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:64\n\tds_read_b128 %2, %4 offset:128\n\t"
                     "ds_read_b128 %3, %4 offset:192\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(bias[0][0]), "=&v"(bias[0][1]), "=&v"(bias[1][0]), "=&v"(bias[1][1]) : "v"(at) : "memory");
      } else {
        lin_u32x2 b[4];
        asm volatile("ds_read_b64 %0, %4\n\tds_read_b64 %1, %4 offset:32\n\tds_read_b64 %2, %4 offset:64\n\t"
                     "ds_read_b64 %3, %4 offset:96\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(b[0]), "=&v"(b[1]), "=&v"(b[2]), "=&v"(b[3]) : "v"(at) : "memory");
#pragma unroll
        for (int q = 0; q < 4; ++q) bias[q >> 1][q & 1] = unpack_bf16x4(b[q]);
      }
#pragma unroll
      for (int hp = 0; hp < 2; ++hp)
#pragma unroll
        for (int hq = 0; hq < 2; ++hq)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[hp][hq][i][j] += bias[hq][j];
    }
    const int c0 = ct.nt * kCols + wn * (GATED ? 32 : 64);
    const int cols = fresh_copy(a.cols), N = fresh_copy(a.N);
    const int oline = static_cast<int>(a.ldo) * (F32 ? 4 : 2), pline = N * 2;
    // of a lane's 16 bytes in a half's 64: a store covers 16 rows.  (Whole lines of eight
    // rows take an exchange between lanes, which costs more than the stores gain: 4096 x
    // 1536, 16384 rows, us 162 and 160, with GELU 202 and 198.)
    const int lc = (g & 1) * 16 + (g >> 1) * 8;
    // columns behind the last one: outside every buffer here (below 2^31 bytes)
    const uint32_t o32[2] = {c0 + lc < cols ? lc * 2u : 0x80000000u, c0 + lc + 32 < cols ? lc * 2u + 64 : 0x80000000u};
    // fp32: a lane's four columns of a block
    const auto of = [&](int hq, int j) __attribute__((always_inline)) -> uint32_t {
      const int c = hq * 32 + j * 16 + g * 4;
      return c0 + c < cols ? c * 4u : 0x80000000u;
    };
    // the lines of the quadrants' 64 rows from column col on
    const auto part = [&](const void* p, int64_t line, int hp, int col, int es = 2) __attribute__((always_inline)) {
      const int r0 = hp * 128 + wm * 64;
      int rows = ct.rows - r0;
      rows = rows < 64 ? rows : 64;
      if (c0 >= cols) rows = 0;
      return buffer(static_cast<const uint8_t*>(p) + (ct.row + r0) * line + static_cast<int64_t>(col) * es,
                    rows > 0 ? rows * static_cast<int>(line) - col * es : 0);
    };
    u32x4 old[2][4][2];
    if constexpr (RES) {  // all in flight together
      const int rline = static_cast<int>(a.ldr) * 2;
#pragma unroll
      for (int hp = 0; hp < 2; ++hp) {
        const auto rr = part(a.residual, rline, hp, c0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            old[hp][i][h] = __builtin_amdgcn_raw_buffer_load_b128(rr, (i * 16 + row) * rline + o32[h], 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int hp = 0; hp < 2; ++hp) {
      if constexpr (GATED) {
        if constexpr (PRE) {
          const auto rg = part(a.pre, pline, hp, c0), ru = part(a.pre, pline, hp, c0 + cols);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t off = (i * 16 + row) * pline + o32[0];
            __builtin_amdgcn_raw_buffer_store_b128(pack8(acc[hp][0][i][0], acc[hp][0][i][1]), rg, off, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b128(pack8(acc[hp][1][i][0], acc[hp][1][i][1]), ru, off, 0, 0);
          }
        }
        const auto rd = part(a.out, oline, hp, c0, F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f32x4 v[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) v[j] = act::gated4(a.act, acc[hp][0][i][j], acc[hp][1][i][j]);
          if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v[j]), rd, (i * 16 + row) * oline + of(0, j), 0, 0);
            continue;
          }
          __builtin_amdgcn_raw_buffer_store_b128(pack8(v[0], v[1]), rd, (i * 16 + row) * oline + o32[0], 0, 0);
        }
      } else {
        if constexpr (PRE) {
          const auto rd = part(a.pre, pline, hp, c0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u32x4 w[2];
#pragma unroll
            for (int hq = 0; hq < 2; ++hq) w[hq] = pack8(acc[hp][hq][i][0], acc[hp][hq][i][1]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              __builtin_amdgcn_raw_buffer_store_b128(w[h], rd, (i * 16 + row) * pline + o32[h], 0, 0);
          }
        }
        const auto rd = part(a.out, oline, hp, c0, F32 ? 4 : 2);
        if constexpr (F32) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              f32x4 v = act::value4(a.act, acc[hp][q >> 1][i][q & 1]);
              asm volatile("" : "+v"(v));  // one store, not one behind each activation
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rd, (i * 16 + row) * oline + of(q >> 1, q & 1), 0, 0);
            }
          continue;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u32x4 w[2];
#pragma unroll
          for (int hq = 0; hq < 2; ++hq) {
            const f32x4 v0 = act::value4(a.act, acc[hp][hq][i][0]), v1 = act::value4(a.act, acc[hp][hq][i][1]);
            w[hq] = RES ? pack8_add(v0, v1, old[hp][i][hq]) : pack8(v0, v1);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
            __builtin_amdgcn_raw_buffer_store_b128(w[h], rd, (i * 16 + row) * oline + o32[h], 0, 0);
        }
      }
    }
  };

  // ======== the stream ========
  // Vector memory instructions complete in the order of issue, so a wait for loads
  // counts what was issued behind them; in the two steps behind an epilogue its stores
  // and the bias too (63 is the counter's limit).  Each wait is for loads whose data is
  // read one phase later: the barrier behind it makes them visible to both groups
  // before the first one reads.
  constexpr int kStores = (GATED ? 8 : 16) * (F32 ? 2 : 1) + (PRE ? 16 : 0) + 1;
  constexpr int kW1 = 10 + kStores < 63 ? 10 + kStores : 63, kW2 = 8 + kStores < 63 ? 8 + kStores : 63;
  bool half = false;  // the tile has no rows in its lower half
  // One step from stage S, starting with B's half S.
  auto step = [&](uint8_t* ps0, uint8_t* ps1, uint8_t* qs, uint8_t* qn, auto S_, auto first_) __attribute__((always_inline)) {
    constexpr int S = decltype(S_)::value;
    constexpr bool first = decltype(first_)::value;
    constexpr std::integral_constant<bool, first && S == 0> fresh{};
    // phase 0
    hold();
    read_p(ps0);
    wait_lds();
    barrier();
    mma(0, S, fresh);
    barrier();
    // phase 1: A half 0 of this stage is free
    read_q(qs, 1 - S);
    load_p(ps0, 0);
    wait_lds();
    fence();
    wait_vm<first ? kW1 : 10>();  // A half 1 of this step
    barrier();
    mma(0, 1 - S, fresh);
    barrier();
    // phase 2: so is B
    if (!GROUPED || !half) read_p(ps1);
    load_q(qs);
    wait_lds();
    fence();
    wait_vm<first && S == 0 ? kW2 : 8>();  // B and A half 0 of the next step
    barrier();
    if (!GROUPED || !half) mma(1, 1 - S, fresh);
    barrier();
    // phase 3
    read_q(qn, 1 - S);
    load_p(ps1, 1);
    advance();
    wait_lds();
    barrier();
    if (!GROUPED || !half) mma(1, S, fresh);
    barrier();
  };
  using std::integral_constant;
  auto pair = [&](auto first) __attribute__((always_inline)) {
    step(p00, p10, q0, q1, integral_constant<int, 0>(), first);
    step(p01, p11, q1, q0, integral_constant<int, 1>(), first);
  };

  load_bias();
  load_p(p00, 0);
  load_q(q0);
  load_p(p10, 1);
  advance();
  load_p(p01, 0);
  load_q(q1);
  load_p(p11, 1);
  advance();
  fence();
  wait_vm<0>();  // both steps: the first tile has no stores before it to count
  barrier();
  read_q(q0, 0);
  wait_lds();
  barrier();
  if (wm == 1) __builtin_amdgcn_s_barrier();  // half a phase behind
  for (;;) {
    half = ct.rows <= 128;
    pair(integral_constant<bool, true>());
    for (int s = 2; s < steps; s += 2) pair(integral_constant<bool, false>());
    fence();
    epilogue();
    fence();
    if (ahead == 0) break;
    ct = --ahead == 0 ? lt : before;
    load_bias();
    fence();
  }
  if (wm == 0) __builtin_amdgcn_s_barrier();
  wait_vm<0>();  // the loads behind the last step
#endif
}

template <bool GROUPED, bool GATED, bool PRE, bool RES = false, bool F32 = false>
int32_t launch(const LinearArgs& a, hipStream_t s) {
  const int grid = linear_cus();  // one workgroup per CU
  if (grid == 0) return MOE_EDEVICE;
  if constexpr (GROUPED)
    linear_wide_kernel<GROUPED, GATED, PRE, RES, F32, false><<<grid, kThreads, 0, s>>>(a);
  else if (a.K % kStep == 0)
    linear_wide_kernel<GROUPED, GATED, PRE, RES, F32, false><<<grid, kThreads, 0, s>>>(a);
  else
    linear_wide_kernel<GROUPED, GATED, PRE, RES, F32, true><<<grid, kThreads, 0, s>>>(a);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

}  // namespace

// CUs of the current device, a multiple of 8 (one share of the tiles per XCD).
int linear_cus() {
  static int grid[64] = {0};
  static std::once_flag once[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
  std::call_once(once[dev], [dev]() {
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess)
      grid[dev] = cus < 8 ? 8 : cus / 8 * 8;
  });
  return grid[dev];
}

bool linear_wide_covers(const LinearArgs& a) {
  const int64_t ldb = static_cast<int64_t>(a.K) * 2;
  return (a.out32 ? a.vec && !a.residual && !a.pre && !a.m_indices
                  : a.vec8 && !(a.residual && (a.m_indices || a.act.gated || a.pre))) && (!a.m_indices || a.K % kStep == 0) && a.K > kStep &&
         // 32-bit offsets: 256 rows of A, out and pre, of B 256 rows or (gated) half of all
         a.lda <= (1 << 22) && a.ldo <= (1 << (a.out32 ? 20 : 21)) && a.ldr <= (1 << 21) && a.N <= (1 << 21) &&
         (a.act.gated ? (static_cast<int64_t>(a.cols) + 256) * ldb < (1ll << 32) : a.K <= (1 << 21)) &&
         // run table and tile positions
         (a.m_indices ? (a.M + 127) / 128 <= runs::kMaxBlocks && a.G <= 1024 : true) &&
         ((a.M + 127) / 128) * ((a.cols + 127) / 128) < (1 << 30);
}

int32_t launch_linear_wide(const LinearArgs& a, hipStream_t s) {
  if (a.m_indices) {
    if (a.act.gated) return a.pre ? launch<true, true, true>(a, s) : launch<true, true, false>(a, s);
    return a.pre ? launch<true, false, true>(a, s) : launch<true, false, false>(a, s);
  }
  if (a.out32)
    return a.act.gated ? launch<false, true, false, false, true>(a, s) : launch<false, false, false, false, true>(a, s);
  if (a.act.gated) return a.pre ? launch<false, true, true>(a, s) : launch<false, true, false>(a, s);
  if (a.residual) return launch<false, false, false, true>(a, s);
  return a.pre ? launch<false, false, true>(a, s) : launch<false, false, false>(a, s);
}

}  // namespace moe
