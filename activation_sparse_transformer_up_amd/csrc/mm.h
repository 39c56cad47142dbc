// Matrix products on gfx950 matrix cores with either operand stored along k or across it.
//
//   D[m][n] = sum_k A(m, k) B(n, k),   bf16 operands, fp32 accumulators
//
// An operand "along k" has rows of consecutive k (A[m][k]); one "across k" has rows of
// consecutive m (A[k][m]), as the gradients' products need it, and is turned on the way from
// LDS to registers (ds_read_b64_tr_b16), so that no transposed copy is ever made.
//
// A workgroup computes BM x BN, a wave WM x WN of 16 x 16 blocks (v_mfma_f32_16x16x32_bf16).
// Every stage of the LDS ring holds 32 k of both operands, moved straight from HBM by loads that
// write LDS (lane l of a wave fills bytes [16 l, 16 l + 16) of a 1 KB block); NS - 1 stages are
// in flight while one is multiplied. Where the stage lies in LDS:
//   along k:   row r at 64 r, its 16-byte chunk c at c ^ ((r >> 1) & 3)
//   across k:  1 KB block q (512 / BX k rows) at MmTr::BLK q, in it the 64-byte chunk c of k row j
//              at c ^ MmTr::swz(j)
// Both keep the lanes that LDS serves together on different banks (SQ_LDS_BANK_CONFLICT = 0).
// Along k a 16-byte read serves lanes 0-3, 12-15 and 20-27 of a half-wave in one turn and the
// others in the next: their 16 rows are r = 0 .. 15 once each, with two different c, and (r & 3,
// c ^ ((r >> 1) & 3)) takes 16 values (with (r >> 2) in its place, 8: twice the time). Across k
// the 8 k rows that a half-wave reads (its lane i brings 8 bytes of k row 8 (i / 16) + i % 16 / 4)
// land in 8 different 32-byte groups.
// Elements outside the operands read as zeros (a byte offset beyond the buffer's range), so
// ragged sizes need no branches.
//
// fp32 operands come as three bf16 planes (hi + mid + lo, 24 bits, exact) and the loop runs over
// the six products of planes that reach 2^-24 of the largest, smallest first: fp32 accuracy at a
// sixth of the bf16 rate, which is above the rate of the fp32 matrix instructions (1/16).
#pragma once
#include "common.h"
#include "stage.h"

namespace tw {

// An operand across k in the stage, BX columns.
template <int BX> struct MmTr {
  static_assert(BX == 64 || BX == 256, "columns");
  static constexpr int RPB = 512 / BX;                    // k rows of a block
  static constexpr int BLK = 1056;                        // bytes from block to block
  // from k row j (j % 8 < 4) to j + 4, whose exchange is the same
  static constexpr int DOWN4 = BX == 64 ? 512 : 2 * BLK;
  static TW_DEV int swz(int j) { return BX == 256 ? j & 1 : (j >> 1) & 1; }
};

template <int BM_, int BN_, int WM_, int WN_, int NS_, bool ATR_, bool BTR_> struct MM {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr bool ATR = ATR_, BTR = BTR_;
  static constexpr int NWM = BM / WM, NWN = BN / WN, NW = NWM * NWN, NT = NW * 64;
  static constexpr int FM = WM / 16, FN = WN / 16;
  static constexpr int KS = 32;                           // k per stage
  static constexpr int A_BLK = BM * KS * 2 / 1024, B_BLK = BN * KS * 2 / 1024;      // 1 KB blocks of a stage
  static constexpr int LPW = (A_BLK + B_BLK) / NW;        // 1 KB wave-loads per wave and stage
  static constexpr int A_STEP = ATR ? MmTr<BM>::BLK : 1024, B_STEP = BTR ? MmTr<BN>::BLK : 1024;
  static constexpr int A_BYTES = A_BLK * A_STEP;
  static constexpr int STAGE = A_BYTES + B_BLK * B_STEP, SMEM = NS * STAGE;
  static_assert((A_BLK + B_BLK) % NW == 0 && NS >= 3, "tile");
  static_assert((!ATR || WM % 64 == 0) && (!BTR || WN % 64 == 0), "across k");
};

// p: element (first row of the tile, k = 0) for an operand along k, (k = 0, first column of the
// tile) for one across k; ld: elements between rows; n: rows (columns) of the tile that exist (a
// multiple of 8 across k); plane: elements between the bf16 planes of an fp32 operand; rows (B of
// mm_loop64 only): where the tile's rows are not consecutive, their numbers (n of them, in LDS, may
// lie in smem).
struct MmOperand {
  const uint16_t *p;
  int64_t ld, plane;
  int n;
  const int *rows = nullptr;
};

// The six products of planes, smallest first: (lo, hi) (hi, lo) (mid, mid) (mid, hi) (hi, mid)
// (hi, hi), as planes 0 = hi, 1 = mid, 2 = lo.
TW_DEV int mm_plane_a(int term) { return term == 0 ? 2 : term == 2 || term == 3 ? 1 : 0; }
TW_DEV int mm_plane_b(int term) { return term == 1 ? 2 : term == 2 || term == 4 ? 1 : 0; }

typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;

// One turning read. The pointer is __restrict__ for the alias scope that this gives the builtin's
// memory operand: without one the compiler takes the read for a user of every load into LDS that is
// in flight and waits for all of them (vmcnt(0)), which stops the ring (dw at T = 8192, d = 4096, V =
// 128000: 10.9 ms). mm_loop's own waits order the reads behind the loads of their stage.
TW_DEV i16x4_t mm_read_tr(const lds_i16x4_t *__restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)p);
}

// Fragment i of a wave (16 rows from w0 + 16 i) of a staged operand of BX rows: lane l gets row
// l % 16, k = 8 (l / 16) .. + 7. Across k, w0 is a multiple of 64: the exchange of chunks stays in i.
template <int BX, bool TR> TW_DEV u32x4_t mm_frag(const char *st, int w0, int i, int lane) {
  if constexpr (!TR) {
    const int r = w0 + (lane & 15);
    return *(const u32x4_t *)(st + r * 64 + (((lane >> 4) ^ ((r >> 1) & 3)) << 4) + i * 1024);
  } else {
    typedef MmTr<BX> L;
    const int j = 8 * (lane >> 4) + ((lane & 15) >> 2), sw = L::swz(j);
    const char *a = st + j / L::RPB * L::BLK + j % L::RPB * (2 * BX) + w0 * 2 + (((i >> 1) ^ sw) << 6) + ((i & 1) << 5) +
                    ((lane & 3) << 3);
    const i16x4_t lo = mm_read_tr((const lds_i16x4_t *)a);
    const i16x4_t hi = mm_read_tr((const lds_i16x4_t *)(a + L::DOWN4));
    u32x4_t v;
    __builtin_memcpy(&v, &lo, 8);
    __builtin_memcpy((char *)&v + 8, &hi, 8);
    return v;
  }
}

// acc += A B^T over k in [0, K) (NP = 1: bf16 operands; NP = 6: three planes each). smem: G::SMEM
// bytes; every wave of the workgroup calls it, and no wave may touch smem afterwards before a
// barrier. One barrier per stage:
//   wait for stage kt + 1's loads, barrier
//   products of stage kt's fragments, between them the reads of stage kt + 1's fragments (into the
//   other set) and the loads of stage kt + NS - 1
// The stage overwritten by those loads, (kt - 1) mod NS, was read during step kt - 2, and the
// barrier that follows a wave's reads waits for them (lgkmcnt).
template <class G, int NP>
TW_DEV void mm_loop(const MmOperand &A, const MmOperand &B, int K, f32x4_t (&acc)[G::FM][G::FN], char *smem) {
  constexpr int NM = G::FM * G::FN, NR = G::FM + G::FN;
  constexpr int RI = NM / NR >= 2 ? NM / NR : 1;          // a fragment read after every RI products
  constexpr int DI = NM / G::LPW >= 1 ? NM / G::LPW : 1;  // a stage load after every DI products
  constexpr uint32_t OOB = 0x80000000u;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / G::NWN, wn = wave % G::NWN;

  uint32_t voff[G::LPW];                                  // this lane's byte offset in each load
  int kof[G::LPW];                                        // the k (row) it starts at
  int dst[G::LPW];                                        // and the load's place in the stage
  bool isA[G::LPW];
#pragma unroll
  for (int i = 0; i < G::LPW; ++i) {
    const int q = wave + G::NW * i;                       // 1 KB block of the stage
    isA[i] = G::A_BLK % G::NW == 0 ? i * G::NW < G::A_BLK : q < G::A_BLK;
    auto place = [&](const MmOperand &o, int blk, auto tr, auto bx) {
      if constexpr (!decltype(tr)::value) {
        const int r = blk * 16 + (lane >> 2), c = (lane & 3) ^ ((r >> 1) & 3);
        kof[i] = c * 8;
        voff[i] = r < o.n ? (uint32_t)(r * o.ld + c * 8) * 2 : OOB;
      } else {
        constexpr int BX = decltype(bx)::value, LR = BX / 8;          // lanes per k row
        const int j = blk * MmTr<BX>::RPB + lane / LR;
        const int col = (((lane % LR) >> 2) ^ MmTr<BX>::swz(j)) * 32 + (lane & 3) * 8;
        kof[i] = j;
        voff[i] = col < o.n ? (uint32_t)(j * o.ld + col) * 2 : OOB;
      }
    };
    const int qb = q - G::A_BLK;
    dst[i] = isA[i] ? q * G::A_STEP : G::A_BYTES + qb * G::B_STEP;
    if (isA[i]) place(A, q, std::integral_constant<bool, G::ATR>(), std::integral_constant<int, G::BM>());
    else place(B, qb, std::integral_constant<bool, G::BTR>(), std::integral_constant<int, G::BN>());
  }
  const int nk1 = (K + G::KS - 1) / G::KS;                // stages of one product of planes
  const int nk = nk1 * NP;
  if (nk == 0) return;

  int lt = 0, lk = 0;                                     // term and k of the next stage to load
  auto issue1 = [&](int kt, int i) {
    char *at = smem + (kt % G::NS) * G::STAGE + dst[i];
    const uint32_t vo = lk + kof[i] < K ? voff[i] : OOB;
    const uint16_t *base;
    if (isA[i]) base = A.p + (NP > 1 ? mm_plane_a(lt) * A.plane : 0) + (G::ATR ? lk * A.ld : lk);
    else base = B.p + (NP > 1 ? mm_plane_b(lt) * B.plane : 0) + (G::BTR ? lk * B.ld : lk);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rows_rsrc(base), (lds_void_t *)at, 16, vo, 0, 0, 0);
  };
  auto issued = [&]() {
    lk += G::KS;
    if (NP > 1 && lk >= K) {
      lk = 0;
      ++lt;
    }
  };
  typedef u32x4_t FA[G::FM];
  typedef u32x4_t FB[G::FN];
  auto read1 = [&](int kt, int j, FA &a, FB &b) {
    const char *st = smem + (kt % G::NS) * G::STAGE;
    if (j < G::FM) a[j] = mm_frag<G::BM, G::ATR>(st, wm * G::WM, j, lane);
    else b[j - G::FM] = mm_frag<G::BN, G::BTR>(st + G::A_BYTES, wn * G::WN, j - G::FM, lane);
  };
  auto mma = [&](int i, const FA &a, const FB &b) {
    acc[i / G::FN][i % G::FN] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(bf16x8_t, a[i / G::FN]), __builtin_bit_cast(bf16x8_t, b[i % G::FN]),
        acc[i / G::FN][i % G::FN], 0, 0, 0);
  };
  for (int st = 0; st < G::NS - 1 && st < nk; ++st) {
#pragma unroll
    for (int i = 0; i < G::LPW; ++i) issue1(st, i);
    issued();
  }
  if (nk >= G::NS - 1) wait_vmcnt<(G::NS - 2) * G::LPW>();
  else wait_vmcnt<0>();
  block_barrier();
  FA a0, a1;
  FB b0, b1;
#pragma unroll
  for (int j = 0; j < NR; ++j) read1(0, j, a0, b0);
  // step kt < nk - 1; LOAD: stage kt + NS - 1 exists and is loaded in this step
  auto step = [&](int kt, const FA &ac, const FB &bc, FA &an, FB &bn, auto load_tag) {
    constexpr bool LOAD = decltype(load_tag)::value;
    if (LOAD) wait_vmcnt<(G::NS - 3) * G::LPW>();         // stage kt + 1 has landed
    else wait_vmcnt<0>();
    block_barrier_lds();
    __builtin_amdgcn_sched_barrier(0);
    static_for<NM>([&](auto I) {
      constexpr int i = decltype(I)::value;
      mma(i, ac, bc);
      if constexpr (i % RI == 0 && i / RI < NR) read1(kt + 1, i / RI, an, bn);
      if constexpr (LOAD && i % DI == DI - 1 && i / DI < G::LPW) issue1(kt + G::NS - 1, i / DI);
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr ((NM + RI - 1) / RI < NR)
#pragma unroll
      for (int j = (NM + RI - 1) / RI; j < NR; ++j) read1(kt + 1, j, an, bn);
    if constexpr (LOAD && NM / DI < G::LPW)
#pragma unroll
      for (int i = NM / DI; i < G::LPW; ++i) issue1(kt + G::NS - 1, i);
    if (LOAD) issued();
    __builtin_amdgcn_sched_barrier(0);
  };
  const std::integral_constant<bool, true> ld;
  const std::integral_constant<bool, false> nold;
  auto settle = [&]() {                                   // next fragment set -> current (tail only)
#pragma unroll
    for (int j = 0; j < G::FM; ++j) a0[j] = a1[j];
#pragma unroll
    for (int j = 0; j < G::FN; ++j) b0[j] = b1[j];
  };
  const int nl = nk >= G::NS ? nk - G::NS + 1 : 0;        // steps that load
  int kt = 0;
  for (; kt + 1 < nl; kt += 2) {
    step(kt, a0, b0, a1, b1, ld);
    step(kt + 1, a1, b1, a0, b0, ld);
  }
  if (kt < nl) {
    step(kt, a0, b0, a1, b1, ld);
    settle();
    ++kt;
  }
  for (; kt + 1 < nk; ++kt) {
    step(kt, a0, b0, a1, b1, nold);
    settle();
  }
#pragma unroll
  for (int i = 0; i < NM; ++i) mma(i, a0, b0);
}

// The same for two operands along k, in stages of 64 k: a row's 128 bytes of a stage are one cache
// line. (With 32 k the two halves of a line are fetched by different stages, and the L2 serves half
// lines at the price of whole ones: 13 TB/s at most, which bound the logits' 128 x 128 tiles: 10.0 ms
// at T = 8192, d = 4096, V = 128000, with whole lines 7.4.) A's ring has NSA stages, B's NSB = NSA or NSA
// - 1: what LDS has left goes to A, which comes from HBM. In LDS row r lies at 128 r, its 16-byte
// chunk c at c ^ ((r >> 1) & 7), again without bank conflicts. A stage is multiplied in two halves,
// with one barrier:
//   products of (kt, first half), between them the reads of the second half's fragments
//   wait for stage kt + 1's loads, barrier (all waves have read stage kt)
//   products of (kt, second half), between them the reads of (kt + 1, first half) and the loads of
//   stages kt + NSB of B and kt + NSA of A into the places of stage kt
// The order of the loads (B's before A's in every step) makes the wait a fixed count.
template <int BM_, int BN_, int WM_, int WN_, int NSA_, int NSB_> struct MM64 {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NSA = NSA_, NSB = NSB_;
  static constexpr int NWM = BM / WM, NWN = BN / WN, NW = NWM * NWN, NT = NW * 64;
  static constexpr int FM = WM / 16, FN = WN / 16;
  static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;            // 1 KB wave-loads per wave and stage
  static constexpr int A_STAGE = BM * 128, B_STAGE = BN * 128, SMEM = NSA * A_STAGE + NSB * B_STAGE;
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && NSB >= 2 && (NSA == NSB || NSA == NSB + 1), "tile");
};

template <class G, int NP>
TW_DEV void mm_loop64(const MmOperand &A, const MmOperand &B, int K, f32x4_t (&acc)[G::FM][G::FN], char *smem) {
  constexpr int NM = G::FM * G::FN, NR = G::FM + G::FN, NL = G::LA + G::LB;
  constexpr int RI = NM / NR >= 2 ? NM / NR : 1;          // a fragment read after every RI products
  constexpr int DI = NM / NL >= 1 ? NM / NL : 1;          // a stage load after every DI products
  constexpr uint32_t OOB = 0x80000000u;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / G::NWN, wn = wave % G::NWN;

  // B's loads, then A's: this lane's byte offset in each and the k it starts at. A load is a block of 8
  // rows; its row of this lane is 8 blk + lane / 8.
  uint32_t voff[NL];
  int kof[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const MmOperand &o = i < G::LB ? B : A;
    const int blk = wave + G::NW * (i < G::LB ? i : i - G::LB), r = blk * 8 + (lane >> 3);
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    kof[i] = c * 8;
    voff[i] = r < o.n ? (uint32_t)((o.rows ? o.rows[r] : r) * o.ld + c * 8) * 2 : OOB;
  }
  const int nk = (K + 63) / 64 * NP;
  if (nk == 0) return;
  if (B.rows) __syncthreads();                            // the numbers lie where the loads go

  // term, k and place of the next stage to load, of B and of A. Loads past the last stage fill a free
  // place with zeros: the count of the waits stays the same.
  int lt[2] = {0, 0}, lk[2] = {0, 0}, lp[2] = {0, 0};
  auto issue1 = [&](int i) {
    const bool isB = i < G::LB;
    const int o = isB ? 0 : 1, blk = wave + G::NW * (isB ? i : i - G::LB);
    char *at = smem + (isB ? G::NSA * G::A_STAGE + lp[0] * G::B_STAGE : lp[1] * G::A_STAGE) + blk * 1024;
    const uint32_t vo = lk[o] + kof[i] < K && (NP == 1 || lt[o] < NP) ? voff[i] : OOB;
    const int64_t pb = NP > 1 ? mm_plane_b(lt[0]) * B.plane : 0, pa = NP > 1 ? mm_plane_a(lt[1]) * A.plane : 0;
    const uint16_t *base = isB ? B.p + pb : A.p + pa;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rows_rsrc(base + lk[o]), (lds_void_t *)at, 16, vo, 0, 0, 0);
    if (i != G::LB - 1 && i != NL - 1) return;            // the operand's last load of the stage
    lk[o] += 64;
    if (NP > 1 && lk[o] >= K) {
      lk[o] = 0;
      ++lt[o];
    }
    lp[o] = lp[o] + 1 == (isB ? G::NSB : G::NSA) ? 0 : lp[o] + 1;
  };
  typedef u32x4_t FA[G::FM];
  typedef u32x4_t FB[G::FN];
  const int r0 = lane & 15;
  const int at0 = r0 * 128 + (((lane >> 4) ^ (r0 >> 1)) << 4);        // second half: chunk + 4
  int pa = 0, pb = 0;                                     // places of the stage to read next
  auto read1 = [&](int h, int j, FA &a, FB &b) {
    const char *sa = smem + pa * G::A_STAGE, *sb = smem + G::NSA * G::A_STAGE + pb * G::B_STAGE;
    const int at = at0 ^ (h << 6);
    if (j < G::FM) a[j] = *(const u32x4_t *)(sa + (wm * G::WM + j * 16) * 128 + at);
    else b[j - G::FM] = *(const u32x4_t *)(sb + (wn * G::WN + (j - G::FM) * 16) * 128 + at);
  };
  auto next = [&]() {
    pa = pa + 1 == G::NSA ? 0 : pa + 1;
    pb = pb + 1 == G::NSB ? 0 : pb + 1;
  };
  auto mma = [&](int i, const FA &a, const FB &b) {
    acc[i / G::FN][i % G::FN] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(bf16x8_t, a[i / G::FN]), __builtin_bit_cast(bf16x8_t, b[i % G::FN]),
        acc[i / G::FN][i % G::FN], 0, 0, 0);
  };
  // the order that the steady state has: A's extra stage first, then B and A of a stage in turn
  if (G::NSA > G::NSB)
#pragma unroll
    for (int i = G::LB; i < NL; ++i) issue1(i);
#pragma unroll
  for (int st = 0; st < G::NSB; ++st)
#pragma unroll
    for (int i = 0; i < NL; ++i) issue1(i);
  // loads issued after those of the stage waited for
  constexpr int AFTER = (G::NSA > G::NSB ? G::LA : 0);
  wait_vmcnt<AFTER + (G::NSB - 1) * NL>();
  block_barrier();
  FA a0, a1;
  FB b0, b1;
#pragma unroll
  for (int j = 0; j < NR; ++j) read1(0, j, a0, b0);
  auto first = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    static_for<NM>([&](auto I) {
      constexpr int i = decltype(I)::value;
      mma(i, a0, b0);
      if constexpr (i % RI == 0 && i / RI < NR) read1(1, i / RI, a1, b1);
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr ((NM + RI - 1) / RI < NR)
#pragma unroll
      for (int j = (NM + RI - 1) / RI; j < NR; ++j) read1(1, j, a1, b1);
  };
  auto second = [&]() {
    wait_vmcnt<AFTER + (G::NSB - 2) * NL>();              // stage kt + 1 has landed
    block_barrier_lds();
    next();
    __builtin_amdgcn_sched_barrier(0);
    static_for<NM>([&](auto I) {
      constexpr int i = decltype(I)::value;
      mma(i, a1, b1);
      if constexpr (i % RI == 0 && i / RI < NR) read1(0, i / RI, a0, b0);
      if constexpr (i % DI == DI - 1 && i / DI < NL) issue1(i / DI);
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr ((NM + RI - 1) / RI < NR)
#pragma unroll
      for (int j = (NM + RI - 1) / RI; j < NR; ++j) read1(0, j, a0, b0);
    if constexpr (NM / DI < NL)
#pragma unroll
      for (int i = NM / DI; i < NL; ++i) issue1(i);
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int kt = 0; kt + 1 < nk; ++kt) {
    first();
    second();
  }
  first();
  wait_vmcnt<0>();                                        // no load into LDS outlives the loop
#pragma unroll
  for (int i = 0; i < NM; ++i) mma(i, a1, b1);
}

// fp32 operands as they lie, on v_mfma_f32_16x16x4_f32 (157 TFLOP/s, below six bf16 products, but each
// element is read once, as 4 bytes, where the planes take 10 to be made and 12 to be read): for few
// rows and small products. A workgroup of four waves computes BM x BN (64 where an operand lies across
// k), a wave 32 x 32, of which 16-column parts of B that do not exist are left out; a stage holds 32 k,
// four stages in a ring. The k of the four lane groups g of an instruction may be any four, the same
// for both operands: instruction j of half h takes k = 16 h + 4 g + j, so that along k a lane reads its
// four j in one load. In LDS, without bank conflicts:
//   along k:   row r at 128 r, its 16-byte chunk c at c ^ ((r >> 1) & 7), as in mm_loop64
//   across k:  k row j at 256 j, its 64-byte chunk c at c ^ ((j >> 2) & 3)
template <int BM_, int BN_, bool ATR_, bool BTR_> struct MMF {
  static constexpr int BM = BM_, BN = BN_, WM = 32, WN = 32, NS = 4;
  static constexpr bool ATR = ATR_, BTR = BTR_;
  static constexpr int NWM = BM / WM, NWN = BN / WN, NW = 4, NT = 256, FM = 2, FN = 2;
  static constexpr int LA = BM / 32, LB = BN / 32, NL = LA + LB;      // 1 KB wave-loads per wave and stage
  static constexpr int A_BYTES = BM * 128, STAGE = A_BYTES + BN * 128, SMEM = NS * STAGE;
  static_assert(NWM * NWN == NW && (!ATR || BM == 64) && (!BTR || BN == 64), "tile");
};
struct MmfOperand {                                       // as MmOperand; n a multiple of 4 across k
  const float *p;
  int64_t ld;
  int n;
};

// Fragment at row r0 of a staged operand, half h: element j of lane l is row r0 + l % 16, k = 16 h + 4 (l
// / 16) + j.
template <bool TR> TW_DEV f32x4_t mmf_frag(const char *st, int r0, int h, int lane) {
  const int g = lane >> 4;
  if constexpr (!TR) {
    const int r = r0 + (lane & 15);
    return *(const f32x4_t *)(st + r * 128 + (((4 * h + g) ^ ((r >> 1) & 7)) << 4));
  } else {
    const float *p = (const float *)(st + (16 * h + 4 * g) * 256 + (((r0 >> 4) ^ g) << 6)) + (lane & 15);
    return f32x4_t{p[0], p[64], p[128], p[192]};
  }
}

// acc += A B^T over k in [0, K), as mm_loop. A step waits for its stage, loads the one that is three
// ahead into the place of the last step's, and multiplies.
template <class G> TW_DEV void mmf_loop(const MmfOperand &A, const MmfOperand &B, int K, f32x4_t (&acc)[2][2], char *smem) {
  constexpr uint32_t OOB = 0x80000000u;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / G::NWN, wn = wave % G::NWN;
  const bool half = B.n - wn * 32 <= 16, none = B.n <= wn * 32;       // columns of this wave that exist
  uint32_t voff[G::NL];                                   // A's 1 KB blocks of this wave, then B's
  int kof[G::NL];
#pragma unroll
  for (int i = 0; i < G::NL; ++i) {
    const MmfOperand &o = i < G::LA ? A : B;
    const int blk = wave + 4 * (i < G::LA ? i : i - G::LA);
    if (i < G::LA ? G::ATR : G::BTR) {                     // 4 k rows
      const int col = (((lane >> 2 & 3) ^ (blk & 3)) << 4) + (lane & 3) * 4;
      kof[i] = blk * 4 + (lane >> 4);
      voff[i] = col < o.n ? (uint32_t)(kof[i] * o.ld + col) * 4 : OOB;
    } else {                                              // 8 rows
      const int r = blk * 8 + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
      kof[i] = c * 4;
      voff[i] = r < o.n ? (uint32_t)(r * o.ld + c * 4) * 4 : OOB;
    }
  }
  const int nk = (K + 31) / 32;
  if (nk == 0) return;
  auto issue = [&](int kt) {                              // zeros past the last stage
    const int lk = kt * 32;
#pragma unroll
    for (int i = 0; i < G::NL; ++i) {
      const bool isA = i < G::LA;
      char *at = smem + kt % G::NS * G::STAGE + (isA ? 0 : G::A_BYTES) + (wave + 4 * (isA ? i : i - G::LA)) * 1024;
      const float *base = isA ? A.p + (G::ATR ? lk * A.ld : lk) : B.p + (G::BTR ? lk * B.ld : lk);
      const uint32_t vo = lk + kof[i] < K ? voff[i] : OOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rows_rsrc(base), (lds_void_t *)at, 16, vo, 0, 0, 0);
    }
  };
  for (int st = 0; st < G::NS - 1; ++st) issue(st);
  for (int kt = 0; kt < nk; ++kt) {
    wait_vmcnt<(G::NS - 2) * G::NL>();                    // stage kt has landed
    block_barrier_lds();                                  // for all waves, which have read stage kt - 1
    issue(kt + G::NS - 1);
    const char *st = smem + kt % G::NS * G::STAGE;
    if (none) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4_t a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = mmf_frag<G::ATR>(st, wm * 32 + i * 16, h, lane);
        b[i] = mmf_frag<G::BTR>(st + G::A_BYTES, wn * 32 + i * 16, h, lane);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if (n == 1 && half) break;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int m = 0; m < 2; ++m)
            acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[m][j], b[n][j], acc[m][n], 0, 0, 0);
      }
    }
  }
  wait_vmcnt<0>();                                        // no load into LDS outlives the loop
}

// Workgroup b of `total` tiles -> tile. The XCDs take workgroups in turn (b % 8), each its own
// L2: every XCD gets a contiguous run of tiles, so that neighbours share operand rows there. A
// launch has 8 ceil(total / 8) workgroups; those past the end get -1.
TW_DEV int mm_xcd_tile(int b, int total) {
  const int per = (total + 7) / 8, t = (b & 7) * per + (b >> 3);
  return (b >> 3) < per && t < total ? t : -1;
}
// Tile -> (m, n) in groups of GM m tiles: within a group all n of the m's before the next, so
// that the 32 tiles in flight on an XCD form a block of about GM x 32 / GM.
template <int GM> TW_DEV void mm_tile_mn(int t, int mt, int nt, int &m, int &n) {
  const int g = t / (GM * nt), m0 = g * GM, gm = mt - m0 < GM ? mt - m0 : GM, r = t - m0 * nt;
  m = m0 + r % gm;
  n = r / gm;
}

}  // namespace tw
