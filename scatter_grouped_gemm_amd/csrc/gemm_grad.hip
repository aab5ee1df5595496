// The two gradients of the compact grouped product C[r, :] = A[r, :] . B[g(r)]^T:
//   dA[r, :] = dC[r, :] . B[g(r)]                     (grouped_gemm_contig_dgrad)
//   dB[g]    = sum over g's rows of dC[r, :]^T A[r, :]   (grouped_gemm_contig_wgrad)
// BF16 operands, fp32 accumulation.
//
// Both are tiles D[i, j] = sum_k P[i, k] Q[k, j] of 256 x 256 outputs.  Q is
// stored with its reduction outermost in both (B [N][K] and A [rows][K]), P
// along its reduction in dgrad (dC rows) and with it outermost in wgrad.
//   - Operands with the reduction outermost go to LDS as they lie in memory and
//     are transposed on the way out (ds_read_b64_tr_b16: 16 lanes read four rows
//     of 16 values, each lane gets four values of one column).
//   - Workgroup = 8 wavefronts in two groups of four, one wavefront of each
//     group on every SIMD.  A wavefront owns 64 + 64 rows by 64 columns of the
//     tile in four quadrants.  A step of 64 of the reduction is four phases, a
//     phase is a load part (LDS reads, global loads) and an MFMA part (16
//     instructions of one quadrant), each ended by a barrier; the second group
//     runs half a phase behind the first, so on every SIMD one wavefront feeds
//     the matrix core while the other one reads.
//   - Global loads go straight to LDS.  Two stages; each piece of a stage (P's
//     two halves, Q) is loaded again as soon as both groups have read it, which
//     gives a load 1.25 to 1.75 steps (about 1 us) to arrive.
//   - The phases of a step use the quadrants in the order P0 Q0, P0 Q1, P1 Q1,
//     P1 Q0, and the next step starts with Q1: so the reads of a step spread
//     over the phases as 8, 4, 8, 4 KB a wavefront and Q's registers need no copy.
//   - The loop is one stream of steps over all of a workgroup's tiles: the loads
//     cross into the next tile while the current one is finished.
//   - Tiles: dgrad in the order of gemm_runs.h, wgrad as grad_schedule.h deals them.
//
// Where 256 x 256 tiles do not fill the card, or hold a few steps only, smaller
// ones take the call: dgrad_thin_kernel below, dgrad_short.hip, wgrad_short.hip.
//
// Measured (us; in brackets TFLOP/s; of one matrix also torch's library product of
// the same sizes and layout, in turn):
//   dgrad  4096 rows, N 8192, K 4096 185 (1488), library 198 (1390); 8192 rows 360
//          (1528), 393 (1398); 8192 rows, N 28672 1266 (1520), 1382 (1392)
//   wgrad  16384 rows, 4096 x 4096 403 (1365), 468 (1175); 8192 rows, 4096 x 8192 387
//          (1422), 455 (1208); 1024 rows, 28672 x 4096 211 (1139), 247 (974)
//   8 experts, N 28672, K 4096: of 1024 rows dgrad 1290-1490 (1290-1490), wgrad
//          1650-1750 (1100-1160); of 964 to 1084 rows dgrad 1720-1740 (1110): 560 to 592
//          tiles take three rounds of 256 workgroups, where 1024 rows take two
//   64 ragged experts (N 2816, K 2048, 4662 rows) dgrad 138: B is read at 5.5 TB/s
// What bounds them: dgrad the card's power (matrix cores busy 81% of the cycles at
// 1.55 GHz); wgrad the load parts (busy 57-67% at 1.8 GHz: its P takes twice the
// LDS instructions) and, with short reductions, the stores (without them the 8
// experts above take 12% less).  No LDS bank conflicts.  Tried without gain: the
// reads spread evenly over the phases, 32x32x16 instructions, leaving out the
// MFMAs of a short tile's empty rows, both groups storing at once, a staggered
// start, non-temporal stores, other tile orders.
#include <mutex>
#include <type_traits>

#include "common.h"
#include "gemm_runs.h"
#include "grad_schedule.h"
#include "grad_tile.h"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kTileN = 256;
using sched::kMaxG;

// A tile as both sides of the stream see it.
struct Tile {
  int64_t row;  // dgrad: first row; wgrad: first row of the expert
  int rows;     // dgrad: rows of the tile; wgrad: rows of the expert
  int id, pt, qt;
  int steps;    // of 64 of the reduction, an even number
};

// A copy that the compiler takes for a new value.  What is worked out from it
// once in a tile would otherwise be kept in registers over the whole loop, and
// there are more such values than registers.
__device__ __forceinline__ int fresh_copy(int x) {
  asm volatile("" : "+s"(x));
  return x;
}

template <bool WGRAD, bool F32, bool ACC>
__global__ __launch_bounds__(kThreads, 2) void gemm_grad_kernel(const GradArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  // P half h of stage s, Q of stage s.  Arrays of their own: the compiler then
  // knows which loads to LDS a read can depend on.
  __shared__ __attribute__((aligned(1024))) uint8_t p00[16384], p01[16384], p10[16384], p11[16384];
  __shared__ __attribute__((aligned(1024))) uint8_t q0[32768], q1[32768];
  __shared__ int4 table[WGRAD ? 1 : runs::kTable];
  __shared__ typename std::conditional<WGRAD, sched::Lds, int>::type dealt;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int fr = lane & 15, fg = lane >> 4;
  const int64_t ldp = static_cast<int64_t>(a.N) * 2, ldq = static_cast<int64_t>(a.K) * 2;  // bytes
  const int ntk = (a.K + kTileN - 1) / kTileN;

  // ======== the tiles of this workgroup ========
  int pos = 0, pos_end = 0, stride = 0, NR = 0, cur = 0;
  [[maybe_unused]] sched::Dealer dealer;
  // of a tile's start and stores, in steps of the reduction
  constexpr int kTileCost = (F32 ? 8 : 4) * (ACC ? 2 : 1);
  const int ntn = (a.N + kTileN - 1) / kTileN;
  if constexpr (WGRAD) {
    sched::deal<8>(dealer, &dealt, reinterpret_cast<int2*>(q0), a.starts, a.counts, a.M, a.G, ntn * ntk, kStep, kTileCost, ACC);
  } else {
    runs::Share sh;
    static_assert(runs::kMaxBlocks * 4 <= 32768, "the set-up arrays fit in the stages");
    if (!runs::build_share<8, true>(a.m_indices, a.M, a.G, ntk, reinterpret_cast<int*>(q0),
                                    reinterpret_cast<int*>(q1), reinterpret_cast<int*>(p00), table, sh))
      return;
    NR = sched::uniform(sh.NR);
    pos = sched::uniform(sh.lo) + static_cast<int>(blockIdx.x >> 3);
    pos_end = sched::uniform(sh.hi);
    stride = sh.per_xcd;
  }
  // The workgroup's next tile; false: none left.
  auto fetch = [&](Tile& t) __attribute__((always_inline)) -> bool {
    if constexpr (WGRAD) {
      int s, i;
      if (!sched::next(dealer, s, i)) return false;
      const int ntk_ = fresh_copy(ntk), ntn_ = fresh_copy(ntn);
      const int2 range = sched::lds_int2(&dealt.range[s]);
      const int grp = i / (kGroupN * ntk_), p0 = grp * kGroupN;
      const int gs = ntn_ - p0 < kGroupN ? ntn_ - p0 : kGroupN;
      const int r = i - p0 * ntk_;
      t.row = sched::uniform(range.x);
      t.rows = sched::uniform(range.y);
      t.id = sched::uniform(sched::lds_int(&dealt.id[s]));
      t.qt = r / gs;
      t.pt = p0 + r - t.qt * gs;
      t.steps = sched::tile_steps(t.rows, kStep);
      return true;
    } else {
      int at = pos, c = cur;
      runs::Tile r;
      r.rows = 0;
      for (; at < pos_end && r.rows <= 0; at += stride) r = runs::decode<16>(table, NR, c, at, fresh_copy(ntk));
      if (r.rows <= 0) return false;
      pos = at;
      cur = c;
      t.row = r.row;
      t.rows = r.rows;
      t.id = r.id;
      t.pt = 0;
      t.qt = r.nt;
      t.steps = a.N / kStep;
      return true;
    }
  };
  Tile lt;  // load side
  if (!fetch(lt)) return;
  // Compute side: it is two steps behind the load side, a tile has at least two,
  // so its next tile is the load side's or the one before that.
  Tile ct = lt, before = lt;
  int ahead = 0;  // tiles between the two

  // ======== load side ========
  // offsets of this lane's 16 bytes within a step of the operand; a load fills
  // 1 KB of LDS in lane order, so the order of the 32-byte pieces (16-byte
  // pieces in dgrad's P) is permuted here, at the source
  uint32_t vp[2], vq[4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (WGRAD) {
      const int r = wave * 8 + j * 4 + (lane >> 4);
      const int f = (r & 3) | (((r >> 3) & 1) << 2);
      vp[j] = static_cast<uint32_t>(r * ldp) + ((((lane & 15) >> 1) ^ f) << 5) + ((lane & 1) << 4);
    } else {
      const int r = (wave * 2 + j) * 8 + (lane >> 3);
      vp[j] = static_cast<uint32_t>(r * ldp) + (((lane & 7) ^ (lane >> 3)) << 4);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = wave * 8 + j * 2 + (lane >> 5);
    const int f = (r & 3) | (((r >> 3) & 1) << 2);
    vq[j] = static_cast<uint32_t>(r * ldq) + ((((lane & 31) >> 1) ^ f) << 5) + ((lane & 1) << 4);
  }
  const uint8_t *bp, *bq;  // this step's operands
  int np, nq;              // and the bytes within bounds (dgrad: of P's first half)
  int np1 = 0;             // dgrad: of P's second half
  int left;                // wgrad: rows from here on
  int lk = 0;
  // 64 rows of an operand are below 2^30 bytes, 128 below 2^31
  auto lbound = [&]() __attribute__((always_inline)) {
    const int v = left < kStep ? left : kStep;
    np = v * static_cast<int>(ldp) - lt.pt * (kTileN * 2);
    nq = v * static_cast<int>(ldq) - lt.qt * (kTileN * 2);
  };
  auto lset = [&]() __attribute__((always_inline)) {
    const int64_t lp = fresh_copy(a.N) * 2ll, lq = fresh_copy(a.K) * 2ll;
    if constexpr (WGRAD) {
      bp = a.P + lt.row * lp + lt.pt * (kTileN * 2);
      bq = a.Q + lt.row * lq + lt.qt * (kTileN * 2);
      left = lt.rows;
      lbound();
    } else {
      bp = a.P + lt.row * lp;
      bq = a.Q + static_cast<int64_t>(lt.id) * a.N * lq + lt.qt * (kTileN * 2);
      np = (lt.rows < 128 ? lt.rows : 128) * static_cast<int>(lp);
      np1 = (lt.rows - 128) * static_cast<int>(lp);
      nq = kStep * static_cast<int>(lq) - lt.qt * (kTileN * 2);
    }
  };
  lset();
  // No immediate offset in these loads: the instruction adds it to the LDS
  // address too.
  auto to_lds = [&](__amdgpu_buffer_rsrc_t rs, uint8_t* dst, uint32_t off) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16, off, 0, 0, 0);
  };
  auto load_p = [&](uint8_t* dst, int half) __attribute__((always_inline)) {
    const auto rs = !half ? buffer(bp, np) : WGRAD ? buffer(bp + 256, np - 256) : buffer(bp + 128 * ldp, np1);
#pragma unroll
    for (int j = 0; j < 2; ++j) to_lds(rs, dst + (wave * 2 + j) * 1024, vp[j]);
  };
  auto load_q = [&](uint8_t* dst) __attribute__((always_inline)) {
    const auto rs = buffer(bq, nq);
#pragma unroll
    for (int j = 0; j < 4; ++j) to_lds(rs, dst + (wave * 4 + j) * 1024, vq[j]);
  };
  // on to the next step; behind the last tile its last step is read again (and
  // never used), so that every step issues the same loads
  auto advance = [&]() __attribute__((always_inline)) {
    if (++lk == lt.steps) {
      Tile t = lt;
      if (fetch(t)) {
        before = lt;
        lt = t;
        ++ahead;
        lk = 0;
        lset();
      } else {
        lk = lt.steps - 1;
      }
    } else {
      bq += kStep * ldq;
      if constexpr (WGRAD) {
        bp += kStep * ldp;
        left -= kStep;
        lbound();
      } else {
        bp += kStep * 2;
      }
    }
  };

  // ======== compute side ========
  // LDS offsets of this lane's part of a fragment.  tr: rows 8 fg + fr / 4 (and
  // + 4) of the 32 of an MFMA, four values of column group fr & 3.
  const int tr_row = fg * 8 + (fr >> 2);
  const int tr_f = (tr_row & 3) | (((tr_row >> 3) & 1) << 2);
  uint32_t op[4], oq[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // dgrad: one piece of 16 bytes for each half of the step, blocks 2 KB apart
    if constexpr (WGRAD)
      op[i] = tr_row * 256 + (((wm * 4 + i) ^ tr_f) << 5) + (fr & 3) * 8;
    else
      op[i] = (wm * 64 + fr) * 128 + ((((i & 1) * 4 + fg) ^ (fr & 7)) << 4);
    oq[i] = tr_row * 512 + (((wn * 4 + i) ^ tr_f) << 5) + (fr & 3) * 8;
  }
  // Keeps the compiler from working out the address in every array before the
  // loop (and spilling them): from here on it has to add the array's place in
  // the instruction's offset.
  auto hold = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < (WGRAD ? 4 : 2); ++i) asm volatile("" : "+v"(op[i]));
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(oq[i]));
  };

  bf16x8 fp[2][4];     // P half in use: [k half][16-row block]
  bf16x8 fq[2][2][2];  // Q half: [half][k half][16-column block]
  f32x4 acc[2][2][4][2] = {};
  auto pair = [](s16x4 lo, s16x4 hi) __attribute__((always_inline)) {
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto read_p = [&](const uint8_t* s) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (WGRAD)
          fp[k][i] = pair(read_tr(s + op[i] + k * 8192), read_tr(s + op[i] + k * 8192 + 1024));
        else
          fp[k][i] = *reinterpret_cast<const bf16x8*>(s + op[k] + i * 2048);
      }
  };
  auto read_q = [&](const uint8_t* s, int h) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        fq[h][k][j] = pair(read_tr(s + oq[h * 2 + j] + k * 16384), read_tr(s + oq[h * 2 + j] + k * 16384 + 2048));
  };
  // D^T: a lane ends with four consecutive columns of one row
  auto mma = [&](int hp, int hq) __attribute__((always_inline)) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[hp][hq][i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[hq][k][j], fp[k][i], acc[hp][hq][i][j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
  };

  // Stores of the finished tile, then zero accumulators.  Every wavefront
  // issues the same number of them whatever its tile holds (rows and columns
  // outside fall outside the buffer and are dropped), so that the waits of the
  // next two steps can count them.
  auto epilogue = [&]() __attribute__((always_inline)) {
    constexpr int ES = F32 ? 4 : 2;
    const int K = fresh_copy(a.K), N = fresh_copy(a.N);
    const int col0 = ct.qt * kTileN + wn * 64;
    // the lane's place, worked out here: kept over the loop it would cost the
    // registers that the fragments need
    int l = lane;
    asm volatile("" : "+v"(l));
    const int line = K * ES;  // 64 rows of it are at most 2^30 bytes
#pragma unroll
    for (int hp = 0; hp < 2; ++hp) {
      const int r0 = hp * 128 + wm * 64;  // of the tile
      const int64_t first = WGRAD ? static_cast<int64_t>(ct.id) * N + ct.pt * kTileN + r0 : ct.row + r0;
      int rows = WGRAD ? N - ct.pt * kTileN - r0 : ct.rows - r0;
      rows = rows < 64 ? rows : 64;
      const int bytes = col0 < K && rows > 0 ? rows * line - col0 * ES : 0;
      store64<F32, ACC>(acc[hp], buffer(static_cast<uint8_t*>(a.D) + first * line + col0 * ES, bytes), line, l);
    }
    float zero = 0.0f;  // in a vector register: as constants, 128 scalar ones are taken for it
    asm volatile("" : "+v"(zero));
#pragma unroll
    for (int hp = 0; hp < 2; ++hp)
#pragma unroll
      for (int hq = 0; hq < 2; ++hq)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[hp][hq][i][j] = f32x4{zero, zero, zero, zero};
  };

  // ======== the stream ========
  // Vector memory instructions complete in the order of issue, so a wait for
  // loads counts what was issued behind them; in the two steps behind an
  // epilogue its stores too (63 is the counter's limit).  Each wait is for loads
  // whose data is read one phase later: the barrier behind it makes them
  // visible to both groups before the first one reads.
  constexpr int kStores = F32 ? 32 : 16;
  constexpr int kW1 = 10 + kStores < 63 ? 10 + kStores : 63, kW2 = 8 + kStores < 63 ? 8 + kStores : 63;
  // One step from stage S, starting with Q's half S.
  auto step = [&](uint8_t* ps0, uint8_t* ps1, uint8_t* qs, uint8_t* qn, auto S_, auto first_) __attribute__((always_inline)) {
    constexpr int S = decltype(S_)::value;
    constexpr bool first = decltype(first_)::value;
    // phase 0
    hold();
    read_p(ps0);
    wait_lds();
    barrier();
    mma(0, S);
    barrier();
    // phase 1: P half 0 of this stage is free
    read_q(qs, 1 - S);
    load_p(ps0, 0);
    wait_lds();
    fence();
    wait_vm<first ? kW1 : 10>();  // P half 1 of this step
    barrier();
    mma(0, 1 - S);
    barrier();
    // phase 2: so is Q
    read_p(ps1);
    load_q(qs);
    wait_lds();
    fence();
    wait_vm<first && S == 0 ? kW2 : 8>();  // Q and P half 0 of the next step
    barrier();
    mma(1, 1 - S);
    barrier();
    // phase 3
    read_q(qn, 1 - S);
    load_p(ps1, 1);
    advance();
    wait_lds();
    barrier();
    mma(1, S);
    barrier();
  };
  using std::integral_constant;
  // A tile is a whole number of pairs of steps, one from each stage.
  auto steps = [&](auto first) __attribute__((always_inline)) {
    step(p00, p10, q0, q1, integral_constant<int, 0>(), first);
    step(p01, p11, q1, q0, integral_constant<int, 1>(), first);
  };

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
    steps(integral_constant<bool, true>());
    for (int s = 2; s < ct.steps; s += 2) steps(integral_constant<bool, false>());
    // Accumulating, both groups do this at the same time to have twice the loads
    // in flight: the first one waits for the second one's MFMAs, the second one
    // falls back by half a phase again behind it.
    if (ACC && wm == 0) barrier();
    fence();
    epilogue();
    fence();
    if (ACC && wm == 1) barrier();
    if (ahead == 0) break;
    ct = --ahead == 0 ? lt : before;
  }
  if (wm == 0) __builtin_amdgcn_s_barrier();
  wait_vm<0>();  // the loads behind the last step
#endif
}

// dgrad with few tiles: 64 rows by 64 columns a workgroup.
//
// With few rows the product is one pass over B, and what counts is how many CUs
// read it and how much each has in flight.  A 256-column tile of a B [8192][2048]
// leaves 8 workgroups an expert, each reading 4 MB a step at a time: 133 us for
// one token and two experts, where the bytes take 14 (44 here: its 64 workgroups are
// a quarter of the CUs).  Here four wavefronts of 16
// columns each keep seven steps of 64 (56 KB of B) in flight in eight LDS stages
// of 16 KB.  The sum of an output runs through the same MFMAs in the same order
// as in the large kernel, so a row comes out the same from either.
constexpr int kThinStages = 8;
constexpr int kThinStage = 16384;  // P [64 rows][64], then Q [64][64 columns]

__global__ __launch_bounds__(256, 1) void dgrad_thin_kernel(const GradArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fg = lane >> 4;
  const int64_t ldp = static_cast<int64_t>(a.N) * 2, ldq = static_cast<int64_t>(a.K) * 2;
  const int cols = a.K / 64;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / cols) * 64;
  const int col0 = static_cast<int>(blockIdx.x % cols) * 64;
  // valid rows come first in a block of 128, which has one expert
  const int e = __builtin_amdgcn_readfirstlane(a.m_indices[row0]);
  if (e < 0 || e >= a.G) return;
  const bool valid = row0 + lane < a.M && a.m_indices[row0 + lane] >= 0;
  const int rows = static_cast<int>(__popcll(__ballot(valid)));
  const int steps = a.N / kStep;

  uint32_t vp[2], vq[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = (wave * 2 + j) * 8 + (lane >> 3);
    vp[j] = static_cast<uint32_t>(r * ldp) + (((lane & 7) ^ (lane >> 3)) << 4);
    vq[j] = static_cast<uint32_t>(r * ldq) + ((((lane & 7) >> 1) ^ (r & 3)) << 5) + ((lane & 1) << 4);
  }
  const uint8_t* bp = a.P + row0 * ldp;
  const uint8_t* bq = a.Q + static_cast<int64_t>(e) * a.N * ldq + col0 * 2;
  const int np = rows * static_cast<int>(ldp), nq = kStep * static_cast<int>(ldq) - col0 * 2;
  int loaded = 0;
  // The next step into its stage; behind the last one nothing is read, but the
  // same number of loads is issued.
  auto load = [&]() __attribute__((always_inline)) {
    uint8_t* const st = smem + (loaded % kThinStages) * kThinStage;
    const bool in = loaded < steps;
    const auto rp = buffer(bp, in ? np : 0), rq = buffer(bq, in ? nq : 0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, (__attribute__((address_space(3))) void*)(st + (wave * 2 + j) * 1024),
                                               16, vp[j], 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rq, (__attribute__((address_space(3))) void*)(st + 8192 + (wave * 2 + j) * 1024), 16, vq[j], 0, 0, 0);
    }
    bp += kStep * 2;
    bq += kStep * ldq;
    ++loaded;
  };
  for (int i = 0; i < kThinStages - 1; ++i) load();
  const int tr_row = fg * 8 + (fr >> 2);
  const uint32_t base = runs::lds_off(smem);
  const uint32_t op0 = base + fr * 128 + ((fg ^ (fr & 7)) << 4), op1 = base + fr * 128 + (((4 + fg) ^ (fr & 7)) << 4);
  const uint32_t oq = base + 8192 + tr_row * 128 + ((wave ^ (tr_row & 3)) << 5) + (fr & 3) * 8;
  f32x4 acc[4] = {};
  for (int t = 0; t < steps; ++t) {
    fence();
    wait_vm<4 * (kThinStages - 2)>();  // this step's loads, of seven steps' in flight
    barrier();                         // all wavefronts', and all have read the step before
    load();
    const uint32_t at = (t % kThinStages) * kThinStage;
    bf16x8 fp[2][4];
    s16x4 q[4];
    // Reads and wait in one statement: the compiler would otherwise wait for the
    // loads in flight, which go to other stages.
    asm volatile(
        "ds_read_b64_tr_b16 %8, %14\n\t"
        "ds_read_b64_tr_b16 %9, %14 offset:512\n\t"
        "ds_read_b128 %0, %12\n\t"
        "ds_read_b128 %1, %12 offset:2048\n\t"
        "ds_read_b128 %2, %12 offset:4096\n\t"
        "ds_read_b128 %3, %12 offset:6144\n\t"
        "ds_read_b64_tr_b16 %10, %14 offset:4096\n\t"
        "ds_read_b64_tr_b16 %11, %14 offset:4608\n\t"
        "ds_read_b128 %4, %13\n\t"
        "ds_read_b128 %5, %13 offset:2048\n\t"
        "ds_read_b128 %6, %13 offset:4096\n\t"
        "ds_read_b128 %7, %13 offset:6144\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(fp[0][0]), "=&v"(fp[0][1]), "=&v"(fp[0][2]), "=&v"(fp[0][3]), "=&v"(fp[1][0]), "=&v"(fp[1][1]),
          "=&v"(fp[1][2]), "=&v"(fp[1][3]), "=&v"(q[0]), "=&v"(q[1]), "=&v"(q[2]), "=&v"(q[3])
        : "v"(op0 + at), "v"(op1 + at), "v"(oq + at)
        : "memory");
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bf16x8 fq = __builtin_bit_cast(bf16x8, __builtin_shufflevector(q[2 * k], q[2 * k + 1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq, fp[k][i], acc[i], 0, 0, 0);
    }
  }
  fence();
  wait_vm<0>();
  const int line = a.K * 2;
  const auto rd = buffer(static_cast<uint8_t*>(a.D) + row0 * line + col0 * 2, rows * line - col0 * 2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
    const u32x2 w{pack_bf16x2(acc[i][0], acc[i][1]), pack_bf16x2(acc[i][2], acc[i][3])};
    __builtin_amdgcn_raw_buffer_store_b64(w, rd, (i * 16 + fr) * line + wave * 32 + fg * 8, 0, 0);
  }
#endif
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int32_t check_sizes(int64_t M, int32_t N, int32_t K, int32_t G) {
  if (M < 0 || N <= 0 || K <= 0 || G < 0) return MOE_EINVAL;
  if (N % 128 != 0 || K % 128 != 0) return MOE_EUNSUPPORTED;
  // 256 rows of an operand are addressed with 32-bit offsets
  if (N > (1 << 22) || K > (1 << 22)) return MOE_EUNSUPPORTED;
  if ((M + 127) / 128 > runs::kMaxBlocks || G > kMaxG) return MOE_EUNSUPPORTED;
  // tile positions
  if (((static_cast<int64_t>(N) + 255) / 256) * ((K + 255) / 256) / 8 * G >= (1 << 30)) return MOE_EUNSUPPORTED;
  if ((static_cast<int64_t>(K) + 255) / 256 * ((M + 127) / 128) >= (1 << 30)) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// One workgroup per CU, a multiple of 8 (one share of the tiles per XCD).
int grid_size() {
  static int grid[64] = {0};
  static std::once_flag once[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
  std::call_once(once[dev], [dev]() {
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess)
      grid[dev] = cus < 8 ? 8 : cus / 8 > sched::kMaxP ? 8 * sched::kMaxP : cus / 8 * 8;
  });
  return grid[dev];
}

template <bool WGRAD, bool F32, bool ACC>
int32_t launch(const GradArgs& a, void* stream) {
  const int grid = grid_size();
  if (grid == 0) return MOE_EDEVICE;
  gemm_grad_kernel<WGRAD, F32, ACC><<<grid, kThreads, 0, static_cast<hipStream_t>(stream)>>>(a);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

// Which kernel takes a wgrad.  us, wide / 128 x 128 tiles (bf16; fp32 added):
//   up to two small tiles a CU, always the small ones.  256 tiles of 256 rows 18 / 8;
//     28 / 11, of 4096 rows 91 / 45; 101 / 48; 512 tiles of 16384 rows 350 / 264;
//     325 / 227.  (896 tiles: 4096 rows 112 / 115; 117 / 118, 16384 rows 399 / 441;
//     406 / 585.)
//   up to six a CU, with few rows an expert.  1024 tiles: 64 rows 26 / 15; 38 / 29,
//     1024 rows 46 / 36; 57 / 51, 4096 rows 117 / 118; 123 / 126; 1536 tiles: 512
//     rows 42 / 33; 64 / 53.  (2048 tiles, 32 experts of 512 rows 56 / 55; 81 / 85.)
//   added to fp32, with fewer yet, however many.  8 experts, 4096 x 4096: 64 rows
//     276 / 211, 256 rows 277 / 241, 384 rows 279 / 284; 64 experts, 2048 x 1408: 64
//     rows 316 / 294, 256 rows 342 / 333, 384 rows 369 / 378; 8 experts, 28672 x 4096:
//     64 rows 1618 / 1366 (5.5 TB/s), 512 rows 1779 / 1902.  (Not so in bf16: 8
//     experts, 4096 x 4096, 64 rows 78 / 86, added 119 / 131.)
// Rows are M over G, which the host knows; rows dealt unevenly change little (64
// experts, 2048 x 1408, fp32 added, 8192 rows in one and two in each other 401 / 363).
// M is the buffers' height and not the rows held: in buffers that hold few, the wide
// tiles take the call (2 of 64 experts with 32 rows each, 4096 x 2048, bf16: 14 us in
// buffers of 256 rows, 22 in buffers of 2176).
template <bool F32, bool ACC>
int32_t launch_wgrad(const GradArgs& a, void* stream) {
  const int64_t tiles = static_cast<int64_t>(a.N / 128) * (a.K / 128) * a.G;
  const int64_t cus = grid_size(), G = a.G;
  if (cus == 0) return MOE_EDEVICE;
  if (tiles <= 2 * cus || (tiles <= 6 * cus && a.M <= 1024 * G) ||
      (F32 && ACC && a.M <= 256 * G && tiles < (1 << 23)))
    return launch_wgrad_short(a, F32, ACC, static_cast<hipStream_t>(stream));
  return launch<true, F32, ACC>(a, stream);
}

int32_t launch_thin(const GradArgs& a, void* stream) {
  constexpr int lds = kThinStages * kThinStage;
  static std::once_flag once[64];
  static bool ok[64] = {};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return MOE_EDEVICE;
  std::call_once(once[dev], [&]() {
    ok[dev] = hipFuncSetAttribute(reinterpret_cast<const void*>(dgrad_thin_kernel),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, lds) == hipSuccess;
  });
  if (!ok[dev]) return MOE_EDEVICE;
  const int64_t grid = (a.M + 63) / 64 * (a.K / 64);
  dgrad_thin_kernel<<<static_cast<unsigned>(grid), 256, lds, static_cast<hipStream_t>(stream)>>>(a);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int32_t grouped_gemm_contig_dgrad(const void* dC, const void* B, void* dA,
                                             const int32_t* m_indices, int64_t M, int32_t N,
                                             int32_t K, int32_t G, void* stream) {
  const int32_t st = check_sizes(M, N, K, G);
  if (st != MOE_OK) return st;
  if (M == 0 || G == 0) return MOE_OK;
  if (!dC || !B || !dA || !m_indices) return MOE_EINVAL;
  if (!aligned16(dC) || !aligned16(B) || !aligned16(dA)) return MOE_EUNSUPPORTED;
  const GradArgs a{static_cast<const uint8_t*>(dC), static_cast<const uint8_t*>(B), dA, m_indices, nullptr,
                   nullptr, M, N, K, G};
  // 64 x 64 tiles (thin) as long as each has a CU, 128 x 128 ones up to three for
  // two CUs.  us, thin / 128 x 128 / 256 x 256:
  //   256 of 64 x 64:  N 4096, 1024 rows, K 1024 26 / 38 / 74; N 14336, 512 rows,
  //     K 2048 81 / 123 / 229
  //   512 of 64 x 64:  N 4096, 2048 rows, K 1024 49 / 39 / 76; N 14336, 1024 rows,
  //     K 2048 155 / 127 / 229 (but 8 experts of 17 rows, N 4096, K 2048: half of
  //     the 64 x 64 tiles are empty, which M does not show, and thin is ahead)
  //   256 of 128 x 128:  N 4096, 1024 rows, K 4096 96 / 43 / 77; 8 experts of 256
  //     rows, N 14336, K 2048 320 / 179 / 261
  //   384 of 128 x 128:  8 experts of 300 rows, K 2048, N 2816 86 / 46 / 59, N 14336
  //     395 / 259 / 266
  //   512 of 128 x 128:  N 4096, 2048 rows, K 4096 185 / 69 / 84; 64 experts of 73
  //     rows, K 1024 204 / 126 / 105
  // M is the buffers' height, and the rows held may be far fewer: 4 of 64 experts with
  // 64 rows each, N 4096, K 2048 25 us in buffers of 512 rows, 71 in buffers of 4480
  // (which could take all assignments of 512 tokens).
  const int64_t cus = grid_size();
  if (cus == 0) return MOE_EDEVICE;
  if ((M + 63) / 64 * (K / 64) <= cus) return launch_thin(a, stream);
  if (2 * ((M + 127) / 128 * (K / 128)) <= 3 * cus) return launch_dgrad_short(a, static_cast<hipStream_t>(stream));
  return launch<false, false, false>(a, stream);
}

extern "C" int32_t grouped_gemm_contig_wgrad(const void* dC, const void* A,
                                             const int32_t* expert_start_loc,
                                             const int32_t* num_valid, int32_t out_dtype,
                                             int32_t accumulate, void* dB, int64_t M, int32_t N,
                                             int32_t K, int32_t G, void* stream) {
  const int32_t st = check_sizes(M, N, K, G);
  if (st != MOE_OK) return st;
  if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_FP32) return MOE_EUNSUPPORTED;
  if (G == 0) return MOE_OK;
  if (!expert_start_loc || !num_valid || !dB || (M > 0 && (!dC || !A))) return MOE_EINVAL;
  if (!aligned16(dC) || !aligned16(A) || !aligned16(dB)) return MOE_EUNSUPPORTED;
  const GradArgs a{static_cast<const uint8_t*>(dC), static_cast<const uint8_t*>(A), dB, nullptr,
                   expert_start_loc, num_valid, M, N, K, G};
  if (out_dtype == MOE_DTYPE_FP32)
    return accumulate ? launch_wgrad<true, true>(a, stream) : launch_wgrad<true, false>(a, stream);
  return accumulate ? launch_wgrad<false, true>(a, stream) : launch_wgrad<false, false>(a, stream);
}
