// The dense layers on gfx950 matrix cores: a linear layer with bias, activation and residual in its
// epilogue, the gated feed-forward block, and the backward passes of both.
//
//   linear   z = x w^T + b (or x w + b);  y = act(z) + residual
//            dz = dy act'(z);  dx = dz w;  dw = dz^T x;  db = sum_t dz
//   gated    g = x Wg^T + bg;  u = x Wu^T + bu;  h = act(g) u;  y = h W2 + residual
//            dh = dy W2^T;  dg = dh u act'(g);  du = dh act(g)
//            dx = dg Wg + du Wu;  dWg = dg^T x;  dWu = du^T x;  dW2 = h^T dy
//
// Every product is out[n][m] = sum_k A(m, k) B(n, k) with m along the output's rows, on the loops of
// mm.h; three kinds occur: both operands along k (forward, dh), A across k (dx, products with a [k][m]
// weight) and both across k (the weights' gradients). No transposed copy is made. A lane of the result
// holds 4 neighbouring columns of a row, which the epilogue turns into outputs where they are:
//   - the gated forward stages 16 rows of Wg and 16 of Wu in turn, so that a wave holds g and u of the
//     same columns and h leaves the kernel instead of them (they are written too where a backward follows);
//   - dh is never written: the epilogue reads g and u and leaves dg, du and h, the next products' operands;
//   - column sums (db) are taken from the fp32 values, per wave and then over the waves in a fixed order.
// h, dg, du (and dz where there is an activation) are rounded to the operands' type once, as operands of
// the next product; sums, biases, activations and residuals are fp32. In bf16 that rounding and the result's make
// the error 0.0023 of the result in the root mean square where the result's alone makes 0.0017 (gated backward of
// 16384 x 4096 x 14336 against 64 bits; 0.0019 behind a residual); parts of h that kept its digits would double the
// products that read it.
//
// Products with fewer tiles than the CUs can hold split k; the fp32 partial sums are added in a fixed
// order by k_dense_rows, which runs the same epilogue. (Splits that meet in the product's kernel, the last to
// arrive adding the others' tiles, save that launch but wait three times for memory behind the stream of
// weights: 1 x 14336 by 4096 across k in 4 splits 25 us so, 30 met.)
//
// fp32 operands of large products are split into three bf16 planes first (six products, 24 bits); the
// others run on the fp32 matrix instructions.
#include "act.h"
#include "dense_plan.h"
#include "launch.h"
#include "mm.h"
#include "row8.h"

namespace tw {
namespace {

typedef uint16_t bf16_t;

TW_DEV void store4(float *p, f32x4_t v) { *(f32x4_t *)p = v; }

// 8 neighbouring elements; plain stores, for what the next product reads.
TW_DEV void keep8(float *p, const float (&v)[8]) {
  *(f32x4_t *)p = f32x4_t{v[0], v[1], v[2], v[3]};
  *(f32x4_t *)(p + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
}
TW_DEV void keep8(bf16_t *p, const float (&v)[8]) {
  *(uint4 *)p = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
TW_DEV void opt8(const float *p, int c, float (&o)[8]) {
  if (p) {
    load8(p + c, o);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 0.f;
  }
}

// --------------------------------------------------------------------------------- epilogues
// shift(r, c) moves the pointers to a tile's first row and column, from which offsets fit 32 bits. Of 8
// columns c .. c + 7 of row r: col(c) is loaded once per column, Row::load(e, r, c) ahead of put(), which
// writes the outputs and adds to the NSUM column sums that the backward needs. v: the product (the first
// of a dual one), w: the second. ACTS: by activation.

// y = act(v + bias) + residual; pre = v + bias. RES: with a residual, of y's type YT. The activation's short forms
// are for a y that is rounded to bf16; an fp32 y of bf16 operands takes the same forms as that of fp32 ones (4096 x
// 2048 by 8192 into fp32, gelu 145 us, silu 129; with the short forms 155 and 157, the stores of y closer together).
template <typename T, typename YT, bool ACTS_, bool RES> struct EpiLinear {
  static constexpr bool DUAL = false, ACTS = ACTS_;
  static constexpr bool FAST = std::is_same<T, bf16_t>::value && std::is_same<YT, bf16_t>::value;
  static constexpr int NSUM = 0;
  const float *bias;
  const YT *res;
  int64_t ldr, ldy;
  YT *y, *y1, *y2;                          // y1, y2: of the second and third batch
  T *pre;
  int act;
  float *sums;
  struct Col { float bias[8]; };
  struct Row {
    Raw8<YT> res;
    TW_DEV void load(const EpiLinear &e, int r, int c) {
      if constexpr (RES) res.load(e.res + (uint32_t)(r * (int)e.ldr + c));
    }
  };
  TW_DEV void shift(int b, int64_t r, int c) {
    YT *const y0 = y, *const o = b == 1 ? y1 + 0 : y2 + 0;  // (values: a choice of members would lie in scratch)
    y = (ACTS || b == 0 ? y0 : o) + r * ldy + c;
    if (pre) pre += r * ldy + c;
    if (bias) bias += c;
    if constexpr (RES) res += r * ldr + c;
  }
  TW_DEV void col(int c, Col &k) const {
    if constexpr (ACTS) opt8(bias, c, k.bias);
  }
  template <int ACT>
  TW_DEV void put(int r, int c, const Col &k, const Row &q, float (&v)[8], float (&)[8], float (*)[8]) const {
    const uint32_t at = r * (int)ldy + c;
    if constexpr (ACTS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += k.bias[i];
      if (pre) store8(pre + at, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_of<ACT, FAST>(v[i]);
    }
    if constexpr (RES) {
      float u[8];
      q.res.to(u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += u[i];
    }
    store8(y + at, v);
  }
};

// h = act(v + bg) (w + bu), and both factors where a backward follows.
template <typename T> struct EpiGlu {
  static constexpr bool DUAL = true, ACTS = true;
  static constexpr int NSUM = 0;
  const float *bg, *bu;
  T *h, *g, *u;
  int64_t ldy;
  int act;
  float *sums;
  struct Col { float bg[8], bu[8]; };
  struct Row {
    TW_DEV void load(const EpiGlu &, int, int) {}
  };
  TW_DEV void shift(int, int64_t r, int c) {
    h += r * ldy + c;
    if (g) {
      g += r * ldy + c;
      u += r * ldy + c;
    }
    if (bg) bg += c;
    if (bu) bu += c;
  }
  TW_DEV void col(int c, Col &k) const {
    opt8(bg, c, k.bg);
    opt8(bu, c, k.bu);
  }
  template <int ACT>
  TW_DEV void put(int r, int c, const Col &k, const Row &, float (&v)[8], float (&w)[8], float (*)[8]) const {
    const uint32_t at = r * (int)ldy + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] += k.bg[i];
      w[i] += k.bu[i];
    }
    if (g) {
      store8(g + at, v);
      store8(u + at, w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_of<ACT, std::is_same<T, bf16_t>::value>(v[i]) * w[i];
    keep8(h + at, v);
  }
};

// dg = v u act'(g), du = v act(g), h = act(g) u for v = dh. SUMS: with the sums of dg and du.
template <typename T, bool SUMS> struct EpiGluBack {
  static constexpr bool DUAL = false, ACTS = true;
  static constexpr int NSUM = SUMS ? 2 : 0;
  const T *g, *u;
  T *dg, *du, *h;
  int64_t ldy;
  int act;
  float *sums, *out[2];                     // out: the sums themselves, from a single strip
  struct Col {};
  struct Row {
    Raw8<T> g, u;
    TW_DEV void load(const EpiGluBack &e, int r, int c) {
      const uint32_t at = r * (int)e.ldy + c;
      g.load(e.g + at);
      u.load(e.u + at);
    }
  };
  TW_DEV void shift(int, int64_t r, int c) {
    const int64_t at = r * ldy + c;
    g += at;
    u += at;
    dg += at;
    du += at;
    h += at;
  }
  TW_DEV void col(int, Col &) const {}
  template <int ACT>
  TW_DEV void put(int r, int c, const Col &, const Row &q, float (&v)[8], float (&)[8], float (*sum)[8]) const {
    const uint32_t at = r * (int)ldy + c;
    float g[8], u[8], hv[8];
    q.g.to(g);
    q.u.to(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float d;
      const float a = act_grad<ACT, std::is_same<T, bf16_t>::value>(g[i], d);
      hv[i] = a * u[i];
      g[i] = v[i] * u[i] * d;
      u[i] = v[i] * a;
      if constexpr (SUMS) {
        sum[0][i] += g[i];
        sum[1][i] += u[i];
      }
      if (i % 2) __builtin_amdgcn_sched_barrier(0);       // the registers of two elements at a time
    }
    keep8(dg + at, g);
    keep8(du + at, u);
    keep8(h + at, hv);
  }
};

// dz = v act'(pre) for v = dy (dz == NULL: the column sums only).
template <typename T> struct EpiDz {
  static constexpr bool DUAL = false, ACTS = true;
  static constexpr int NSUM = 1;
  const T *pre;
  T *dz;
  int64_t ldy;
  int act;
  float *sums, *out[2];                     // out: the sums themselves, from a single strip
  struct Col {};
  struct Row {
    Raw8<T> z;
    TW_DEV void load(const EpiDz &e, int r, int c) {
      if (e.pre) z.load(e.pre + (uint32_t)(r * (int)e.ldy + c));
    }
  };
  TW_DEV void shift(int, int64_t r, int c) {
    if (pre) pre += r * ldy + c;
    if (dz) dz += r * ldy + c;
  }
  TW_DEV void col(int, Col &) const {}
  template <int ACT>
  TW_DEV void put(int r, int c, const Col &, const Row &q, float (&v)[8], float (&)[8], float (*sum)[8]) const {
    if constexpr (ACT != kActNone) {
      float z[8];
      q.z.to(z);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float d;
        act_grad<ACT, std::is_same<T, bf16_t>::value>(z[i], d);
        v[i] *= d;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[0][i] += v[i];
    if (dz) keep8(dz + (uint32_t)(r * (int)ldy + c), v);
  }
};

template <class E, typename F> TW_DEV void epi_act(const E &e, F &&f) {
  if constexpr (E::ACTS) with_act(e.act, f);
  else f(std::integral_constant<int, kActNone>());
}

// ---------------------------------------------------------------------------------- products

// `batch` products of one shape, each summed over `segs` pairs of operands (A[b], B[b] for batches, A[s],
// B[s] for segments; one of batch and segs is 1), k split S times in ranges of ks of the segs * K.
struct Prod {
  const void *A[3], *B[3], *A2;             // A2: the second matrix of a dual A
  int64_t lda[3], ldb, planeA, planeB;      // elements between the planes of split fp32 operands
  int M, N, K, batch, segs, S, ks;
  float *part;                              // [S][batch][N][M], dual [..][2 M] (S > 1)
};

// Entry b of three (a register array indexed by b would lie in scratch).
template <typename P> TW_DEV P pick(const P (&p)[3], int b) { return b == 0 ? p[0] : b == 1 ? p[1] : p[2]; }

template <class G, class OP, typename T>
TW_DEV void operands(const Prod &a, int b, int m0, int n0, int k0, OP &A, OP &B) {
  constexpr bool along = !G::ATR;
  const int dual = G::DUAL ? 2 : 1;
  A = {};
  B = {};
  const int64_t lda = pick(a.lda, b), ao = along ? m0 * lda + k0 : k0 * lda + m0;
  const int64_t bo = !G::BTR ? (int64_t)n0 * a.ldb + k0 : (int64_t)k0 * a.ldb + n0;
  A.p = (const T *)pick(a.A, b) + ao;
  A.ld = lda;
  A.n = min(a.M - m0, G::BM / dual);
  if (G::DUAL) A.p2 = (const T *)a.A2 + ao;
  if constexpr (std::is_same<T, bf16_t>::value) {
    A.plane = a.planeA;
    B.plane = a.planeB;
  }
  B.p = (const T *)pick(a.B, b) + bo;
  B.ld = a.ldb;
  B.n = min(a.N - n0, G::BN);
}

// What mm.h's three tile types have in common, by loop; NP: products of planes.
template <class G, int NP = 1> struct AsMM : G {
  static constexpr bool DUAL = false;
  template <typename ACC> static TW_DEV void mul(const Prod &a, int b, int m0, int n0, int k0, int K, ACC &acc, char *smem) {
    MmOperand A, B;
    operands<AsMM, MmOperand, bf16_t>(a, b, m0, n0, k0, A, B);
    mm_loop<G, NP>(A, B, K, acc, smem);
  }
};
template <class G, int NP = 1> struct AsMM64 : G {
  static constexpr bool ATR = false, BTR = false;
  template <typename ACC> static TW_DEV void mul(const Prod &a, int b, int m0, int n0, int k0, int K, ACC &acc, char *smem) {
    MmOperand A, B;
    operands<AsMM64, MmOperand, bf16_t>(a, b, m0, n0, k0, A, B);
    mm_loop64<G, NP>(A, B, K, acc, smem);
  }
};
template <class G> struct AsMMF : G {
  template <typename ACC> static TW_DEV void mul(const Prod &a, int b, int m0, int n0, int k0, int K, ACC &acc, char *smem) {
    MmfOperand A, B;
    operands<AsMMF, MmfOperand, float>(a, b, m0, n0, k0, A, B);
    mmf_loop<G>(A, B, K, acc, smem);
  }
};

// The epilogue turns each wave's tile through LDS, which the loop no longer needs, 32 rows at a time: a lane of
// the accumulators holds 4 columns of one row (32-byte pieces of 16 rows per access), turned it holds 8, and a
// wave reads and writes whole 128-byte lines. What an epilogue reads (a residual, g and u) is loaded 32 rows ahead.
// T = 4096, N = 8192, two rounds of tiles: K = 64 36 -> 21 us, with a residual 69 -> 27; the gated backward of
// T = 16384, d = 4096, f = 14336 10.2 -> 9.0 ms, of which dh's epilogue moves 2.3 GB.
// The wave's column sums go to sums[block][NSUM][M], block = the number of its rows' tile.
template <class G, class E, int GM> __global__ __launch_bounds__(G::NT) void k_dense(Prod a, E e) {
  constexpr int DU = E::DUAL ? 2 : 1, BU = G::BM / DU, WU = G::WM / DU;       // columns of a tile, of a wave
  constexpr int LD = G::WM + 4;                           // floats from row to row in LDS
  __shared__ __attribute__((aligned(16))) char smem[G::SMEM];
  const int mt = (a.M + BU - 1) / BU, nt = (a.N + G::BN - 1) / G::BN;
  const int t = mm_xcd_tile(blockIdx.x, mt * nt * a.S * a.batch);
  if (t < 0) return;
  int m, n;
  const int sp = t / (mt * nt), b = sp / a.S, s = sp % a.S;
  mm_tile_mn<GM>(t % (mt * nt), mt, nt, m, n);
  const int m0 = m * BU, n0 = n * G::BN;
  f32x4_t acc[G::FM][G::FN];
#pragma unroll
  for (int i = 0; i < G::FM; ++i)
#pragma unroll
    for (int j = 0; j < G::FN; ++j) acc[i][j] = f32x4_t{};
  const int k0 = s * a.ks, k1 = min(a.segs * a.K, k0 + a.ks);
  bool again = false;
  for (int g = 0; g < a.segs; ++g) {
    const int from = max(k0 - g * a.K, 0), to = min(k1 - g * a.K, a.K);
    if (from >= to) continue;
    if (again) __syncthreads();
    again = true;
    G::mul(a, b + g, m0, n0, from, to - from, acc, smem);
  }

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, grp = lane >> 4;
  const int wm = wave / G::NWN, wn = wave % G::NWN;
  if (a.S > 1) {
    const int c0 = m0 + wm * WU + grp * 4, r0 = n0 + wn * G::WN + (lane & 15);
    float *p = a.part + ((int64_t)s * a.batch + b) * a.N * a.M * DU;
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm) {
      const int c = c0 + fm / DU * 16;
      if (c >= a.M) continue;                             // M is a multiple of 8
#pragma unroll
      for (int fn = 0; fn < G::FN; ++fn) {
        const int r = r0 + fn * 16;
        if (r < a.N) store4(p + (int64_t)r * a.M * DU + fm % DU * a.M + c, acc[fm][fn]);
      }
    }
    return;
  }
  // rows of a pass, lanes per row, rows per access, accesses; 16 rows where the inputs of 32 would not stay in
  // registers beside the accumulators
  constexpr int PR = G::WN == 16 || (WU == 128 && sizeof(typename E::Row) > 16) ? 16 : 32;
  constexpr int LPR = WU / 8, RPI = 64 / LPR < PR ? 64 / LPR : PR, NI = PR / RPI;
  static_assert(LPR <= 64 && NI * RPI == PR && G::WN % PR == 0 && G::NW * PR * LD * 4 <= G::SMEM, "turning");
  e.shift(b, n0, m0);
  const int c = wm * WU + lane % LPR * 8, r0 = wn * G::WN + lane / LPR, rows = a.N - n0;      // of the tile
  float *own = (float *)smem + wave * PR * LD;            // this wave's rows
  const bool ok = c < a.M - m0 && lane < LPR * RPI;
  typename E::Col k;
  typename E::Row q[NI];
  if (ok) {
    e.col(c, k);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (r0 + i * RPI < rows) q[i].load(e, r0 + i * RPI, c);
  }
  __syncthreads();                                        // the other waves have read the last stage
  epi_act(e, [&](auto ACT) __attribute__((always_inline)) {
    float sum[2][8] = {};
#pragma unroll
    for (int h = 0; h < G::WN / PR; ++h) {
      wave_lds_order();
#pragma unroll
      for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
        for (int j = 0; j < PR / 16; ++j)
          *(f32x4_t *)(own + (j * 16 + (lane & 15)) * LD + fm % DU * WU + fm / DU * 16 + grp * 4) = acc[fm][h * PR / 16 + j];
      wave_lds_order();
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = r0 + h * PR + i * RPI;
        if (ok && r < rows) {
          float v[8], w[8];
          const float *at = own + (i * RPI + lane / LPR) * LD + lane % LPR * 8;
          load8(at, v);
          if constexpr (DU == 2) load8(at + WU, w);
          e.template put<decltype(ACT)::value>(r, c, k, q[i], v, w, sum);
          if (h + 1 < G::WN / PR && r + PR < rows) q[i].load(e, r + PR, c);
        }
        __builtin_amdgcn_sched_barrier(0);                // one access's registers at a time
      }
    }
    if constexpr (E::NSUM > 0) {
      if (e.sums) {
#pragma unroll
        for (int j = 0; j < E::NSUM; ++j) {
#pragma unroll
          for (int o = LPR; o < LPR * RPI; o <<= 1)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[j][i] += __shfl_xor(sum[j][i], o, 64);
          if (ok && lane < LPR) keep8(e.sums + ((int64_t)(n * G::NWN + wn) * E::NSUM + j) * a.M + m0 + c, sum[j]);
        }
      }
    }
  });
}

// The epilogue over rows of partial sums, or of a matrix v (EpiDz): a workgroup takes 8 CG columns of a strip of
// `strip` rows, thread t the 8 columns 8 (t % CG) of every RG-th row, RG = 256 / CG. Its sums go to sums[4 strip's
// number + t / 64], the rows of a wave added; a single strip's sums are the result (one launch less), for which 64
// columns a workgroup (CG = 8) leave a thread a quarter of the rows that 256 do.
template <int CG, typename T, class E>
__global__ __launch_bounds__(256) void k_dense_rows(const float *__restrict__ part, int S, int batch, const T *__restrict__ v,
                                                    int64_t ldv, int N, int M, int strip, E e) {
  constexpr int DU = E::DUAL ? 2 : 1, UR = 4;             // rows in flight
  constexpr int RG = 256 / CG;
  __shared__ __attribute__((aligned(16))) float red[E::NSUM > 0 ? 4 : 1][CG * 8];
  const int m0 = blockIdx.x * (CG * 8), n0 = blockIdx.y * strip, b = blockIdx.z, c = threadIdx.x % CG * 8;
  const bool ok = c < M - m0;
  const int end = ok ? min(N - n0, strip) : 0;
  const int64_t plane = (int64_t)batch * N * M * DU;
  e.shift(b, n0, m0);
  if (part) part += ((int64_t)b * N + n0) * M * DU + m0;
  else v += n0 * ldv + m0;
  epi_act(e, [&](auto ACT) __attribute__((always_inline)) {
    typename E::Col k;
    if (ok) e.col(c, k);
    float sum[2][8] = {};
    int r = threadIdx.x / CG;
    if (part) {
      for (; r < end; r += RG) {
        typename E::Row q;
        q.load(e, r, c);
        float x[8] = {}, x2[8] = {};
        const float *p = part + (int64_t)r * M * DU + c;
#pragma unroll 4
        for (int s = 0; s < S; ++s) {
          float u[8];
          load8(p + s * plane, u);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] += u[i];
          if constexpr (DU == 2) {
            load8(p + s * plane + M, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) x2[i] += u[i];
          }
        }
        e.template put<decltype(ACT)::value>(r, c, k, q, x, x2, sum);
      }
    } else {
      for (; r < end; r += RG * UR) {
        typename E::Row q[UR];
        Raw8<T> raw[UR];
#pragma unroll
        for (int i = 0; i < UR; ++i)
          if (r + RG * i < end) {
            raw[i].load(v + (r + RG * i) * ldv + c);
            q[i].load(e, r + RG * i, c);
          }
#pragma unroll
        for (int i = 0; i < UR; ++i)
          if (r + RG * i < end) {
            float x[8];
            raw[i].to(x);
            e.template put<decltype(ACT)::value>(r + RG * i, c, k, q[i], x, x, sum);
          }
      }
    }
    if constexpr (E::NSUM > 0) {
      if (!e.sums) return;
#pragma unroll
      for (int j = 0; j < E::NSUM; ++j) {
#pragma unroll
        for (int o = CG; o < 64; o <<= 1)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[j][i] += __shfl_xor(sum[j][i], o, 64);
        const bool mine = (threadIdx.x & 63) < CG;
        if (gridDim.y > 1) {
          if (ok && mine) keep8(e.sums + ((int64_t)(blockIdx.y * 4 + (threadIdx.x >> 6)) * E::NSUM + j) * M + m0 + c, sum[j]);
        } else {
          if (mine) keep8(&red[threadIdx.x >> 6][c], sum[j]);
          __syncthreads();
          const int t = threadIdx.x;
          if (e.out[j] && t < CG * 8 && t < M - m0) e.out[j][m0 + t] = (red[0][t] + red[1][t]) + (red[2][t] + red[3][t]);
          __syncthreads();
        }
      }
    }
  });
}

// out_j[c] = sum over blocks of sums[block][j][c]: a workgroup takes 64 columns, thread t the 4 columns 4 (t % 16)
// of every sixteenth block.
__global__ __launch_bounds__(256) void k_dense_sums(const float *__restrict__ sums, int blocks, int M, int nsum,
                                                    float *__restrict__ out0, float *__restrict__ out1) {
  __shared__ float red[16][64];
  const int c = (threadIdx.x & 15) * 4, at = blockIdx.x * 64 + c, w = threadIdx.x >> 4, j = blockIdx.y;
  f32x4_t v = {};
  if (at < M)                                             // M is a multiple of 8
#pragma unroll 8
    for (int i = w; i < blocks; i += 16) v += *(const f32x4_t *)(sums + ((int64_t)i * nsum + j) * M + at);
  *(f32x4_t *)&red[w][c] = v;
  __syncthreads();
  float *out = j ? out1 : out0;
  const int t = threadIdx.x, o = blockIdx.x * 64 + t;
  if (t < 64 && o < M && out) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += red[i][t];
    out[o] = s;
  }
}

__global__ __launch_bounds__(256) void k_dense_zero(uint4 *__restrict__ p, size_t n) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) p[i] = make_uint4(0, 0, 0, 0);
}

// The three planes of a [rows][cols] fp32 operand (cols a multiple of 8), each [rows][cols].
__global__ __launch_bounds__(256) void k_dense_split(const float *__restrict__ x, int64_t ld, int rows, int cols,
                                                     bf16_t *__restrict__ to, int64_t plane) {
  const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= cols) return;
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    float v[8];
    load8(x + r * ld + c, v);
    split8(v, to + (int64_t)r * cols + c, plane);
  }
}

// ------------------------------------------------------------------------------------- tiles

// The kernels of the plan's kinds and classes.
template <int KIND, int C, bool DUAL, int NP = 1> struct Shape;
template <bool D> struct Shape<kAlong, kSmall, D> { typedef AsMM64<MM64<64, 64, 32, 32, 4, 4, D>> G; };
template <bool D, int NP> struct Shape<kAlong, kMid, D, NP> { typedef AsMM64<MM64<128, 128, 64, 64, 3, 2, D>, NP> G; };
template <bool D, int NP> struct Shape<kAlong, kLarge, D, NP> { typedef AsMM64<MM64<256, 256, 128, 64, 3, 2, D>, NP> G; };
template <> struct Shape<kAlong, kNarrow, false> { typedef AsMM64<MM64<32, 32, 16, 16, 8, 8>> G; };
template <> struct Shape<kAlong, kNarrow, true> { typedef AsMM64<MM64<64, 32, 32, 16, 6, 6, true>> G; };
template <> struct Shape<kAcross, kSmall, false> { typedef AsMM<MM<256, 64, 64, 64, 3, true, false>> G; };
template <int NP> struct Shape<kAcross, kMid, false, NP> { typedef AsMM<MM<256, 128, 64, 64, 6, true, false>, NP> G; };
template <int NP> struct Shape<kAcross, kLarge, false, NP> { typedef AsMM<MM<256, 256, 64, 128, 4, true, false>, NP> G; };
template <> struct Shape<kAcross, kNarrow, false> { typedef AsMM<MM<64, 64, 64, 16, 8, true, false>> G; };
template <> struct Shape<kAcross, kDeep, false> { typedef AsMM<MM<256, 64, 64, 64, 6, true, false>> G; };
template <> struct Shape<kBoth, kSmall, false> { typedef AsMM<MM<256, 64, 64, 64, 3, true, true>> G; };
template <int NP> struct Shape<kBoth, kLarge, false, NP> { typedef AsMM<MM<256, 256, 64, 128, 4, true, true>, NP> G; };
template <int KIND, bool DUAL> struct ShapeF {            // fp32 as it is
  typedef AsMMF<MMF<64, 64, KIND != kAlong, KIND == kBoth, DUAL, 3>> G;
};
template <bool DUAL> struct ShapeFew { typedef AsMMF<MMF<128, 32, false, false, DUAL>> G; };

int grid8(int64_t tiles) { return (int)((tiles + 7) / 8 * 8); }

template <typename T, class E>
hipError_t launch_rows(const Prod &a, const T *v, int64_t ldv, const E &e, hipStream_t s) {
  const bool sums = E::NSUM > 0 && e.sums;
  auto go = [&](auto cg) {
    constexpr int CG = decltype(cg)::value;
    const dim3 grid((unsigned)ceil_div(a.M, CG * 8), row_strips(a.N, sums, !v), a.batch);
    k_dense_rows<CG, T, E><<<grid, 256, 0, s>>>(v ? nullptr : a.part, a.S, a.batch, v, ldv, a.N, a.M, strip_of(a.N, sums, !v), e);
    return hipGetLastError();
  };
  if constexpr (E::NSUM > 0)
    if (sums && narrow_strip(a.N, a.M, !v)) return go(std::integral_constant<int, 8>());
  return go(std::integral_constant<int, 32>());
}

// One product (a's shape and operands set) by plan p; ws: room for p.ws bytes.
template <typename T, int KIND, class E>
hipError_t product(Prod a, const Split &p, void *ws, const E &e, hipStream_t s) {
  a.S = p.S;
  a.ks = p.ks;
  a.part = (float *)ws;
  auto go = [&](auto X) {
    typedef typename decltype(X)::G G;
    constexpr int BU = G::BM / (E::DUAL ? 2 : 1);
    const int64_t tiles = ceil_div(a.M, BU) * ceil_div(a.N, G::BN) * a.S * a.batch;
    k_dense<G, E, KIND == kAlong ? 4 : 8><<<grid8(tiles), G::NT, 0, s>>>(a, e);
    return hipGetLastError();
  };
  constexpr bool D = E::DUAL;
  if constexpr (std::is_same<T, float>::value) {
    if (p.planes) {
      // every operand once: [3][rows][columns], 256-byte aligned
      bf16_t *at = (bf16_t *)((char *)ws + p.part);
      const int n = a.batch * a.segs;                     // operands on each side
      const void *from[7];
      int64_t stride[7];
      bf16_t *to[7];
      int made = 0;
      auto planes = [&](const void *src, int rows, int cols, int64_t ld) -> const void * {
        for (int i = 0; i < made; ++i)
          if (from[i] == src && stride[i] == ld) return to[i];
        from[made] = src;
        stride[made] = ld;
        to[made] = at;
        k_dense_split<<<dim3((unsigned)ceil_div(cols, 2048), (unsigned)(rows < 4096 ? rows : 4096)), 256, 0, s>>>(
            (const float *)src, ld, rows, cols, at, (int64_t)rows * cols);
        at += align256((size_t)rows * cols * 6) / 2;
        return to[made++];
      };
      constexpr bool AT = KIND != kAlong, BT = KIND == kBoth;
      for (int i = 0; i < n; ++i) a.A[i] = planes(a.A[i], AT ? a.K : a.M, AT ? a.M : a.K, a.lda[i]);
      if (D) a.A2 = planes(a.A2, a.M, a.K, a.lda[0]);
      made = 0;                                           // B's may be A's, in another shape
      for (int i = 0; i < n; ++i) a.B[i] = planes(a.B[i], BT ? a.K : a.N, BT ? a.N : a.K, a.ldb);
      TW_TRY_HIP(hipGetLastError());
      a.lda[0] = a.lda[1] = a.lda[2] = AT ? a.M : a.K;
      a.ldb = BT ? a.N : a.K;
      a.planeA = (int64_t)a.M * a.K;
      a.planeB = (int64_t)a.N * a.K;
      if (p.cls == kLarge) TW_TRY_HIP(go(Shape<KIND, kLarge, D, 6>()));
      else if constexpr (KIND != kBoth) TW_TRY_HIP(go(Shape<KIND, kMid, D, 6>()));
    } else if constexpr (KIND == kAlong) {
      if (p.cls == kNarrow) TW_TRY_HIP(go(ShapeFew<D>()));
      else TW_TRY_HIP(go(ShapeF<KIND, D>()));
    } else {
      TW_TRY_HIP(go(ShapeF<KIND, D>()));
    }
  } else if constexpr (KIND == kAlong) {
    switch (p.cls) {
      case kSmall: TW_TRY_HIP(go(Shape<KIND, kSmall, D>())); break;
      case kMid: TW_TRY_HIP(go(Shape<KIND, kMid, D>())); break;
      case kLarge: TW_TRY_HIP(go(Shape<KIND, kLarge, D>())); break;
      default: TW_TRY_HIP(go(Shape<KIND, kNarrow, D>())); break;
    }
  } else {
    if (p.cls == kSmall) TW_TRY_HIP(go(Shape<KIND, kSmall, D>()));
    else if (p.cls == kLarge) TW_TRY_HIP(go(Shape<KIND, kLarge, D>()));
    if constexpr (KIND == kAcross) {
      if (p.cls == kNarrow) TW_TRY_HIP(go(Shape<KIND, kNarrow, D>()));
      else if (p.cls == kDeep) TW_TRY_HIP(go(Shape<KIND, kDeep, D>()));
      else if (p.cls == kMid) TW_TRY_HIP(go(Shape<KIND, kMid, D>()));
    }
  }
  return p.S > 1 ? launch_rows<T, E>(a, nullptr, 0, e, s) : hipSuccess;
}

Prod prod_of(int M, int N, int K) {
  Prod a = {};
  a.M = M; a.N = N; a.K = K;
  a.batch = a.segs = 1;
  return a;
}

hipError_t zero(void *p, size_t bytes, hipStream_t s) {
  const size_t n = bytes / 16, wg = (n + 255) / 256;
  if (n) k_dense_zero<<<(unsigned)(wg < 4096 ? wg : 4096), 256, 0, s>>>((uint4 *)p, n);
  return hipGetLastError();
}

hipError_t add_sums(const float *sums, int blocks, int M, int nsum, float *o0, float *o1, hipStream_t s) {
  k_dense_sums<<<dim3((unsigned)ceil_div(M, 64), nsum), 256, 0, s>>>(sums, blocks, M, nsum, o0, o1);
  return hipGetLastError();
}

template <typename T> EpiLinear<T, T, false, false> store_epi(void *y, int64_t ldy) {
  EpiLinear<T, T, false, false> e = {};
  e.y = (T *)y;
  e.ldy = ldy;
  return e;
}

// f(epilogue) for y in its type, with or without a residual
template <typename T, typename F>
hipError_t with_linear(const float *bias, const void *res, int64_t ldr, void *y, int64_t ldy, int y_bf16, void *pre, int act, F &&f) {
  auto go = [&](auto yt, auto with_res) {
    typedef decltype(yt) YT;
    EpiLinear<T, YT, true, decltype(with_res)::value> e = {};
    e.bias = bias;
    e.res = (const YT *)res; e.ldr = ldr;
    e.y = (YT *)y; e.ldy = ldy;
    e.pre = (T *)pre; e.act = act;
    return f(e);
  };
  const std::true_type yes;
  const std::false_type no;
  if (y_bf16) return res ? go(bf16_t(), yes) : go(bf16_t(), no);
  return res ? go(float(), yes) : go(float(), no);
}

// Offsets of a workspace, in order.
struct Take {
  size_t at = 0;
  size_t operator()(size_t n) {
    const size_t o = at;
    at += align256(n);
    return o;
  }
};

// ------------------------------------------------------------------------------------ linear

struct LinearBackPlan {
  Split dx, dw;
  size_t dz, sums, part, bytes;
};
LinearBackPlan linear_back_plan(int T, int K, int N, bool bf16, bool kn, int act, bool want_dx, bool want_dw, bool want_db) {
  LinearBackPlan p = {};
  Take take;
  if (act != kActNone && (want_dx || want_dw)) p.dz = take((size_t)T * N * (bf16 ? 2 : 4));
  if (want_db) p.sums = take((size_t)4 * row_strips(T, true, false) * N * 4);
  size_t part = 0;
  if (want_dx) {
    p.dx = split_of(bf16, kn ? kAlong : kAcross, false, K, T, N, 1);
    part = p.dx.ws;
  }
  if (want_dw) {
    p.dw = kn ? split_of(bf16, kBoth, false, N, K, T, 1) : split_of(bf16, kBoth, false, K, N, T, 1);
    part = p.dw.ws > part ? p.dw.ws : part;
  }
  p.part = take(part);
  p.bytes = take.at;
  return p;
}

template <typename T> hipError_t linear_fwd_run(const LinearArgs &a, hipStream_t s) {
  const Split p = split_of(!std::is_same<T, float>::value, a.kn ? kAcross : kAlong, false, a.N, a.T, a.K, 1);
  Prod q = prod_of(a.N, a.T, a.K);
  q.A[0] = a.w; q.lda[0] = a.kn ? a.N : a.K;
  q.B[0] = a.x; q.ldb = a.ldx;
  return with_linear<T>(a.bias, a.res, a.ldr, a.y, a.N, a.y_bf16, a.pre, a.act, [&](const auto &e) {
    return a.kn ? product<T, kAcross>(q, p, a.ws, e, s) : product<T, kAlong>(q, p, a.ws, e, s);
  });
}

template <typename T> hipError_t linear_bwd_run(const LinearBackArgs &a, hipStream_t s) {
  const LinearBackPlan p = linear_back_plan(a.T, a.K, a.N, !std::is_same<T, float>::value, a.kn, a.act, a.dx != nullptr,
                                            a.dw != nullptr, a.db != nullptr);
  char *ws = (char *)a.ws;
  const T *dz = (const T *)a.dy;
  int64_t lddz = a.lddy;
  if (a.act != kActNone || a.db) {
    EpiDz<T> e = {};
    e.act = a.act;
    e.ldy = a.N;
    if (a.act != kActNone) e.pre = (const T *)a.pre;
    if (a.act != kActNone && (a.dx || a.dw)) {
      e.dz = (T *)(ws + p.dz);
      dz = e.dz;
      lddz = a.N;
    }
    if (a.db) e.sums = (float *)(ws + p.sums);
    e.out[0] = a.db;
    TW_TRY_HIP(launch_rows(prod_of(a.N, a.T, 0), (const T *)a.dy, a.lddy, e, s));
    if (a.db && row_strips(a.T, true, false) > 1) TW_TRY_HIP(add_sums(e.sums, 4 * row_strips(a.T, true, false), a.N, 1, a.db, nullptr, s));
  }
  if (a.dx) {
    Prod q = prod_of(a.K, a.T, a.N);
    q.A[0] = a.w; q.lda[0] = a.kn ? a.N : a.K;
    q.B[0] = dz; q.ldb = lddz;
    const auto e = store_epi<T>(a.dx, a.K);
    if (a.kn) TW_TRY_HIP((product<T, kAlong>(q, p.dx, ws + p.part, e, s)));
    else TW_TRY_HIP((product<T, kAcross>(q, p.dx, ws + p.part, e, s)));
  }
  if (a.dw) {
    Prod q = a.kn ? prod_of(a.N, a.K, a.T) : prod_of(a.K, a.N, a.T);
    const void *x = a.x;
    q.A[0] = a.kn ? dz : x; q.lda[0] = a.kn ? lddz : a.ldx;
    q.B[0] = a.kn ? x : dz; q.ldb = a.kn ? a.ldx : lddz;
    TW_TRY_HIP((product<T, kBoth>(q, p.dw, ws + p.part, store_epi<T>(a.dw, q.M), s)));
  }
  return hipSuccess;
}

// ------------------------------------------------------------------------------------- gated

struct GatedPlan {
  Split up, down;
  size_t h, part, bytes;
};
GatedPlan gated_plan(int T, int d, int f, bool bf16) {
  GatedPlan p = {};
  Take take;
  p.h = take((size_t)T * f * (bf16 ? 2 : 4));
  p.up = split_of(bf16, kAlong, true, f, T, d, 1);
  p.down = split_of(bf16, kAcross, false, d, T, f, 1);
  p.part = take(p.up.ws > p.down.ws ? p.up.ws : p.down.ws);
  p.bytes = take.at;
  return p;
}

struct GatedBackPlan {
  Split dh, dx, dw;
  size_t dg, du, h, sums, part, bytes;
};
GatedBackPlan gated_back_plan(int T, int d, int f, bool bf16, bool bias) {
  GatedBackPlan p = {};
  Take take;
  const size_t n = (size_t)T * f * (bf16 ? 2 : 4);
  p.dg = take(n);
  p.du = take(n);
  p.h = take(n);
  p.dh = split_of(bf16, kAlong, false, f, T, d, 1);
  p.dx = split_of(bf16, kAcross, false, d, T, 2 * (int64_t)f, 1);
  p.dw = split_of(bf16, kBoth, false, d, f, T, 3);
  if (bias) p.sums = take((size_t)sum_blocks(bf16, kAlong, p.dh, T) * 2 * f * 4);
  size_t part = p.dh.ws;
  if (p.dx.ws > part) part = p.dx.ws;
  if (p.dw.ws > part) part = p.dw.ws;
  p.part = take(part);
  p.bytes = take.at;
  return p;
}

template <typename T> hipError_t gated_fwd_run(const GatedArgs &a, hipStream_t s) {
  const GatedPlan p = gated_plan(a.T, a.d, a.f, !std::is_same<T, float>::value);
  char *ws = (char *)a.ws;
  EpiGlu<T> eu = {};
  eu.bg = a.bg; eu.bu = a.bu;
  eu.h = (T *)(ws + p.h); eu.g = (T *)a.g; eu.u = (T *)a.u;
  eu.ldy = a.f; eu.act = a.act;
  Prod q = prod_of(a.f, a.T, a.d);
  q.A[0] = a.wg; q.A2 = a.wu; q.lda[0] = a.d;
  q.B[0] = a.x; q.ldb = a.ldx;
  TW_TRY_HIP((product<T, kAlong>(q, p.up, ws + p.part, eu, s)));
  q = prod_of(a.d, a.T, a.f);
  q.A[0] = a.w2; q.lda[0] = a.d;
  q.B[0] = eu.h; q.ldb = a.f;
  return with_linear<T>(nullptr, a.res, a.ldr, a.y, a.d, a.y_bf16, nullptr, kActNone,
                        [&](const auto &e) { return product<T, kAcross>(q, p.down, ws + p.part, e, s); });
}

template <typename T> hipError_t gated_bwd_run(const GatedBackArgs &a, hipStream_t s) {
  constexpr bool bf16 = !std::is_same<T, float>::value;
  const bool bias = a.dbg || a.dbu;
  const GatedBackPlan p = gated_back_plan(a.T, a.d, a.f, bf16, bias);
  char *ws = (char *)a.ws;
  T *dg = (T *)(ws + p.dg), *du = (T *)(ws + p.du), *h = (T *)(ws + p.h);
  Prod q = prod_of(a.f, a.T, a.d);
  q.A[0] = a.w2; q.lda[0] = a.d;
  q.B[0] = a.dy; q.ldb = a.lddy;
  auto back = [&](auto sums) {
    EpiGluBack<T, decltype(sums)::value> e = {};
    e.g = (const T *)a.g; e.u = (const T *)a.u;
    e.dg = dg; e.du = du; e.h = h;
    e.ldy = a.f; e.act = a.act;
    if (bias) e.sums = (float *)(ws + p.sums);
    e.out[0] = a.dbg;
    e.out[1] = a.dbu;
    return product<T, kAlong>(q, p.dh, ws + p.part, e, s);
  };
  if (bias) {
    TW_TRY_HIP(back(std::true_type()));
    if (p.dh.S == 1 || row_strips(a.T, true, true) > 1)
      TW_TRY_HIP(add_sums((const float *)(ws + p.sums), sum_blocks(bf16, kAlong, p.dh, a.T), a.f, 2, a.dbg, a.dbu, s));
  } else {
    TW_TRY_HIP(back(std::false_type()));
  }
  q = prod_of(a.d, a.T, a.f);
  q.segs = 2;
  q.A[0] = a.wg; q.A[1] = a.wu; q.lda[0] = q.lda[1] = a.d;
  q.B[0] = dg; q.B[1] = du; q.ldb = a.f;
  TW_TRY_HIP((product<T, kAcross>(q, p.dx, ws + p.part, store_epi<T>(a.dx, a.d), s)));
  q = prod_of(a.d, a.f, a.T);
  q.batch = 3;
  q.A[0] = q.A[1] = a.x; q.A[2] = a.dy;
  q.lda[0] = q.lda[1] = a.ldx; q.lda[2] = a.lddy;
  q.B[0] = dg; q.B[1] = du; q.B[2] = h; q.ldb = a.f;
  auto ew = store_epi<T>(a.dwg, a.d);
  ew.y1 = (T *)a.dwu;
  ew.y2 = (T *)a.dw2;
  return product<T, kBoth>(q, p.dw, ws + p.part, ew, s);
}

}  // namespace

size_t linear_fwd_workspace(int T, int K, int N, int bf16, bool kn) {
  return split_of(bf16, kn ? kAcross : kAlong, false, N, T, K, 1).ws;
}
size_t linear_bwd_workspace(int T, int K, int N, int bf16, bool kn, int act, bool dx, bool dw, bool db) {
  return linear_back_plan(T, K, N, bf16, kn, act, dx, dw, db).bytes;
}
size_t gated_fwd_workspace(int T, int d, int f, int bf16) { return gated_plan(T, d, f, bf16).bytes; }
size_t gated_bwd_workspace(int T, int d, int f, int bf16, bool bias) { return gated_back_plan(T, d, f, bf16, bias).bytes; }

hipError_t launch_linear_fwd(const LinearArgs &a, hipStream_t s) {
  return a.bf16 ? linear_fwd_run<bf16_t>(a, s) : linear_fwd_run<float>(a, s);
}
hipError_t launch_linear_bwd(const LinearBackArgs &a, hipStream_t s) {
  const size_t e = a.bf16 ? 2 : 4;
  if (a.T == 0) {                           // no rows: the sums over them are zero
    if (a.dw) TW_TRY_HIP(zero(a.dw, (size_t)a.K * a.N * e, s));
    if (a.db) TW_TRY_HIP(zero(a.db, (size_t)a.N * 4, s));
    return hipSuccess;
  }
  return a.bf16 ? linear_bwd_run<bf16_t>(a, s) : linear_bwd_run<float>(a, s);
}
hipError_t launch_gated_fwd(const GatedArgs &a, hipStream_t s) {
  return a.bf16 ? gated_fwd_run<bf16_t>(a, s) : gated_fwd_run<float>(a, s);
}
hipError_t launch_gated_bwd(const GatedBackArgs &a, hipStream_t s) {
  const size_t n = (size_t)a.d * a.f * (a.bf16 ? 2 : 4);
  if (a.T == 0) {
    TW_TRY_HIP(zero(a.dwg, n, s));
    TW_TRY_HIP(zero(a.dwu, n, s));
    TW_TRY_HIP(zero(a.dw2, n, s));
    if (a.dbg) TW_TRY_HIP(zero(a.dbg, (size_t)a.f * 4, s));
    if (a.dbu) TW_TRY_HIP(zero(a.dbu, (size_t)a.f * 4, s));
    return hipSuccess;
  }
  return a.bf16 ? gated_bwd_run<bf16_t>(a, s) : gated_bwd_run<float>(a, s);
}

}  // namespace tw
