// Softmax cross entropy of a large vocabulary, straight from the hidden states x [T][d] and the
// head's weights w [V][d], forward and with its gradients, on gfx950 matrix cores.
//
//   z = x w^T;  lse = log sum_j exp z_j;  loss = lse - z_target
//   G = (exp(z - lse) - onehot(target)) dloss;  dx = G w;  dw = G^T x
//
// The three products (2 T V d operations each) bound it. The logits live in accumulators only:
// the first product's epilogue reduces a tile's block of PW vocabulary columns to (max, sum of
// exp) per token, and for a gradient leaves e = exp(z - block max) in the operand type. In bf16 that
// and G, which the next products need in bf16, are two roundings of up to 2^-8 each, whatever the size
// of z (a bf16 z would be off by 2^-8 |z|); dx and dw are then off by 1.4 times what rounding them to
// bf16 leaves by itself (in the norm, 0.0024 against 0.0017). G in two bf16 parts would double those
// products. fp32 operands keep 24 bits of both. Once a row's blocks are joined, one pass turns e into
// G in place; the target's element is formed from the sum without the target instead, so that p - 1 of
// a token the model is sure of keeps its digits.
//
// Tokens without a target (negative) take no part: the rows with one are gathered first, in
// order, and all products run over that list (its length stays on the device; workgroups beyond
// it leave at once). Whatever such rows hold, also NaN, reaches nothing. The forward of at most 512
// bf16 tokens makes the list in every workgroup instead and reads the rows of x where they lie,
// which saves a launch (one pass alone, T = 333, d = 2048, V = 50021: 85 -> 82 us).
//
// Tokens are taken in pieces of R rows, so that e needs R x V elements whatever T is (one piece as long
// as that costs no more memory than dw's sums over pieces would, see rows_of); dw is summed over the
// pieces in fp32. fp32 operands are split into three bf16 planes (mm.h) where the products are
// large, and multiplied as they are where they are small or few rows make them a stream of w; in the
// kernels' NP, the products of planes, these are 6 and 0, and bf16 is 1.
#include "launch.h"
#include "mm.h"
#include "row8.h"

namespace tw {
namespace {

typedef uint16_t bf16_t;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kFarLogit = 1024.f;                       // up to it the exponent is off by 2^-14 at most

// ------------------------------------------------------------------------------ rows, planes

// list[i] = i-th token with a target, tgt[i] = its target (V where that is V or more), pos[t] = its
// place or -1, *n_act = their number. One workgroup: every thread counts a contiguous run of
// tokens, the counts are scanned.
__global__ __launch_bounds__(1024) void k_xent_rows(const int64_t *__restrict__ y, int T, int V,
                                                    int32_t *__restrict__ list, int32_t *__restrict__ tgt,
                                                    int32_t *__restrict__ pos, int32_t *__restrict__ n_act) {
  __shared__ int wsum[16];
  const int per = (T + 1023) / 1024, t0 = min(T, (int)threadIdx.x * per), t1 = min(T, t0 + per);
  int c = 0;
  for (int t = t0; t < t1; ++t) c += y[t] >= 0;
  int total;
  int at = wave_excl_scan(c, &total);
  if ((threadIdx.x & 63) == 0) wsum[threadIdx.x >> 6] = total;
  __syncthreads();
  int all = 0;
  for (int i = 0; i < 16; ++i) {
    if (i < (int)(threadIdx.x >> 6)) at += wsum[i];
    all += wsum[i];
  }
  for (int t = t0; t < t1; ++t) {
    const int64_t v = y[t];
    pos[t] = v >= 0 ? at : -1;
    if (v >= 0) {
      tgt[at] = v < V ? (int)v : V;
      list[at++] = t;
    }
  }
  if (threadIdx.x == 0) *n_act = all;
}

// Splits 8 fp32 values into three bf16 planes, hi + mid + lo = v (24 bits; rounded to nearest,
// so mid and lo are at most 2^-8 and 2^-17 of v). The largest finite values would round to infinity
// and leave inf - inf: their hi is cut off instead. An infinite v has NaN in mid and lo.
TW_DEV void split8(const float (&v)[8], bf16_t *p, int64_t plane) {
  float h[8], r[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    h[k] = rounded<bf16_t>(v[k]);
    if (__builtin_isinf(h[k])) h[k] = __uint_as_float(__float_as_uint(v[k]) & 0xFFFF0000u);
    r[k] = v[k] - h[k];
  }
  store8(p, h);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    h[k] = rounded<bf16_t>(r[k]);
    r[k] -= h[k];
  }
  store8(p + plane, h);
  store8(p + 2 * plane, r);
}

// Workgroup t = first + blockIdx.x, token t < T: with a target, its row of x into the gathered operand
// (three planes or as it is); without, zeros to its loss, lse and row of dx. pos == NULL: the token's
// place is counted here (and list, tgt and n_act written), which for few tokens costs less than the
// launch of k_xent_rows. fp32 planes: the workgroups past T split w (wp == NULL: x is only gathered, as
// fp32).
template <typename T, typename DXT>
__global__ __launch_bounds__(256) void k_xent_stage(const T *__restrict__ x, int64_t ldx, int tokens, int d, int V,
                                                    const int64_t *__restrict__ y, const int32_t *__restrict__ pos,
                                                    int32_t *__restrict__ list, int32_t *__restrict__ tgt,
                                                    int32_t *__restrict__ n_act, bf16_t *__restrict__ xc, int64_t plane,
                                                    float *__restrict__ loss, float *__restrict__ lse,
                                                    DXT *__restrict__ dx, const T *__restrict__ w, size_t wn,
                                                    bf16_t *__restrict__ wp, int first) {
  const int t = first + (int)blockIdx.x;
  if constexpr (std::is_same<T, float>::value) {
    if (t >= tokens) {
      const size_t i = ((size_t)(t - tokens) * 256 + threadIdx.x) * 8;
      if (i >= wn) return;
      float v[8];
      load8(w + i, v);
      split8(v, wp + i, (int64_t)wn);
      return;
    }
  }
  int p;
  if (pos) {
    p = pos[t];
  } else {
    __shared__ int red[4];
    int c = 0;
    for (int i = threadIdx.x; i < t; i += 256) c += y[i] >= 0;
    c = wave_sum(c);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = c;
    __syncthreads();
    c = (red[0] + red[1]) + (red[2] + red[3]);
    const int64_t v = y[t];
    p = v >= 0 ? c : -1;
    if (threadIdx.x == 0) {
      if (p >= 0) {
        list[p] = t;
        tgt[p] = v < V ? (int)v : V;
      }
      if (t == tokens - 1) *n_act = c + (v >= 0);
    }
  }
  if (p < 0) {
    if (threadIdx.x == 0) {
      loss[t] = 0.f;
      lse[t] = 0.f;
    }
    const float z[8] = {};
    if (dx)
      for (int i = threadIdx.x * 8; i < d; i += 256 * 8) store8(dx + (size_t)t * d + i, z);
    return;
  }
  for (int i = threadIdx.x * 8; i < d; i += 256 * 8) {
    if constexpr (std::is_same<T, float>::value) {
      float v[8];
      load8(x + t * ldx + i, v);
      if (wp) split8(v, xc + (size_t)p * d + i, plane);
      else store8((float *)xc + (size_t)p * d + i, v);
    } else {
      *(uint4 *)(xc + (size_t)p * d + i) = *(const uint4 *)(x + t * ldx + i);
    }
  }
}

// ------------------------------------------------------------------------------------ logits

// Tokens [row0, row0 + R) of the list that exist.
TW_DEV int piece_rows(const int32_t *n_act, int row0, int R) { return min(max(*n_act - row0, 0), R); }

constexpr int kDirectRows = 512;                          // tokens of the forward without a gather

// The list of T <= kDirectRows tokens, made by a workgroup of NT threads in LDS (list: kDirectRows + 8
// ints, to be read after a barrier); returns its length, in every thread.
template <int NT> TW_DEV int block_list(const int64_t *y, int T, int *list) {
  constexpr int PER = kDirectRows / NT, NW = NT / 64;     // tokens of a thread, NT apart
  const int wave = threadIdx.x >> 6;
  uint64_t act[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int t = i * NT + threadIdx.x;
    act[i] = ballot64(t < T && y[t] >= 0);
    if ((threadIdx.x & 63) == 0) list[kDirectRows + i * NW + wave] = __popcll(act[i]);
  }
  __syncthreads();
  int n = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int c = list[kDirectRows + i * NW + w];
      if (w == wave && (act[i] >> (threadIdx.x & 63) & 1)) list[n + mbcnt64(act[i])] = i * NT + threadIdx.x;
      n += c;
    }
  return n;
}

// D[vocabulary][token] = w x^T: a lane holds 4 consecutive logits of a token per block, so that a
// token's maximum and sum are taken over a lane's registers and two exchanges, and e is stored 4
// elements at a time. part[token][block of WM columns] = (max, sum of exp(z - max) over all but the
// target), zt[token] = the target's logit.
// DIRECT: xc is x itself with rows ldx apart, y the targets of its R <= kDirectRows tokens; the list
// is made here.
template <class G, int NP, typename ET, bool KEEP, bool DIRECT>
__global__ __launch_bounds__(G::NT) void k_xent_logits(const bf16_t *__restrict__ w, int64_t wplane,
                                                       const bf16_t *__restrict__ xc, int64_t ldx, int64_t xplane,
                                                       const int64_t *__restrict__ y, const int32_t *__restrict__ tgt,
                                                       const int32_t *__restrict__ n_act, int row0, int R, int V, int d,
                                                       int mt, int nt, ET *__restrict__ e, int64_t lde,
                                                       float2 *__restrict__ part, int nblk, float *__restrict__ zt) {
  // The list of DIRECT lies in the same LDS object: next to a second one the compiler takes the
  // fragment reads for users of the loads in flight, and waits.
  __shared__ __attribute__((aligned(16))) char smem[G::SMEM];
  static_assert(G::SMEM >= (kDirectRows + 8) * 4 && kDirectRows / G::NT * (G::NT / 64) <= 8, "list");
  const int t = mm_xcd_tile(blockIdx.x, mt * nt);
  if (t < 0) return;
  int m, n, rows;
  mm_tile_mn<4>(t, mt, nt, m, n);
  const int m0 = m * G::BM, n0 = n * G::BN;
  int *rowl = (int *)smem;
  if constexpr (DIRECT) rows = block_list<G::NT>(y, R, rowl);
  else rows = piece_rows(n_act, row0, R);
  if (n0 >= rows) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, grp = lane >> 4;
  const int wm = wave / G::NWN, wn = wave % G::NWN;
  const int v0 = m0 + wm * G::WM, blk = v0 / G::WM;       // this wave's block of the vocabulary
  int toff[G::FN];                                        // each row's target as a column of the block
  auto targets = [&]() {
#pragma unroll
    for (int fn = 0; fn < G::FN; ++fn) {
      const int r = n0 + wn * G::WN + fn * 16 + (lane & 15);          // row of the piece
      toff[fn] = -1;
      if (r < rows) {
        if constexpr (DIRECT) {
          const int64_t v = y[rowl[r]];
          toff[fn] = (v < V ? (int)v : V) - v0;
        } else {
          toff[fn] = tgt[row0 + r] - v0;
        }
      }
    }
  };
  if constexpr (DIRECT) {                                 // before the loads take the list's place
    __syncthreads();
    targets();
  }
  f32x4_t acc[G::FM][G::FN];
#pragma unroll
  for (int i = 0; i < G::FM; ++i)
#pragma unroll
    for (int j = 0; j < G::FN; ++j) acc[i][j] = f32x4_t{};
  if constexpr (NP == 0) {
    const MmfOperand A = {(const float *)w + (size_t)m0 * d, d, min(V - m0, G::BM)};
    const MmfOperand B = {(const float *)xc + (size_t)(row0 + n0) * d, ldx, min(rows - n0, G::BN)};
    mmf_loop<G>(A, B, d, acc, smem);
  } else {
    const MmOperand A = {w + (size_t)m0 * d, d, wplane, min(V - m0, G::BM)};
    const MmOperand B = {xc + (DIRECT ? 0 : (size_t)(row0 + n0) * d), ldx, xplane, min(rows - n0, G::BN),
                         DIRECT ? rowl + n0 : nullptr};
    mm_loop64<G, NP>(A, B, d, acc, smem);
  }

  if constexpr (!DIRECT) targets();
  if (v0 + G::WM > V)                                     // the last block ends inside the vocabulary
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (v0 + fm * 16 + grp * 4 + i >= V)
#pragma unroll
          for (int fn = 0; fn < G::FN; ++fn) acc[fm][fn][i] = -INFINITY;
#pragma unroll
  for (int fn = 0; fn < G::FN; ++fn) {
    const int r = n0 + wn * G::WN + fn * 16 + (lane & 15);
    const bool ok = r < rows;
    // rare: one block in nblk holds a row's target
    const bool hit = ballot64((uint32_t)toff[fn] < (uint32_t)G::WM) != 0;
    if (hit) {
#pragma unroll
      for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (fm * 16 + grp * 4 + i == toff[fn]) zt[row0 + r] = acc[fm][fn][i];
    }
    float mx = -INFINITY;
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = fmaxf(mx, acc[fm][fn][i]);
    mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
    const float ref = mx == -INFINITY ? 0.f : mx;         // a block past the vocabulary: e = 0
    float refl = ref * kLog2e;
    if constexpr (NP == 1) {
      // The fused product below rounds ref log2 e, which puts 2^-24 |ref| log2 e in the exponent: as much
      // as the logits' own rounding near them, but a block that a mask of 1e30 or the type's lowest value
      // fills would come to infinity. Rare: rows far from zero take their reference off first.
      const bool far = fabsf(ref) > kFarLogit;
      if (ballot64(far)) {
        const float off = far ? ref : 0.f;
#pragma unroll
        for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[fm][fn][i] -= off;
        refl = far ? 0.f : refl;
      }
    }
    auto ex = [&](float z) {
      if constexpr (NP == 1) return __builtin_amdgcn_exp2f(fmaf(z, kLog2e, -refl));
      else return expf(z - ref);
    };
    float s = 0.f;
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = ex(acc[fm][fn][i]);
        s += v[i];
      }
      if constexpr (KEEP) {
        if (ok) {
          ET *p = e + (size_t)r * lde + v0 + fm * 16 + grp * 4;
          if constexpr (std::is_same<ET, float>::value) *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]);
          else *(uint2 *)p = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        }
      }
    }
    if (hit) {                                            // the same without the target
      s = 0.f;
#pragma unroll
      for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
        for (int i = 0; i < 4; ++i) s += fm * 16 + grp * 4 + i == toff[fn] ? 0.f : ex(acc[fm][fn][i]);
    }
    s += __shfl_xor(s, 16, 64);
    s += __shfl_xor(s, 32, 64);
    if (ok && grp == 0) part[(size_t)r * nblk + blk] = make_float2(mx, s);
  }
}

// Row of a piece: joins its blocks (of 1 << pw columns) to lse and loss; for a gradient turns its e
// into G (zero in the padding, where e is 0). With R the sum of exp(z - max) over all but the target
// and E the target's: loss = log(1 + R / E) and p - 1 = -R / (R + E), which keep the digits of a token
// that the model is sure of (R << E), where lse - z and exp(z - lse) - 1 have none left. A target
// beyond the vocabulary makes loss and G NaN.
// GRAD: `split` workgroups per row share its columns (each joins the blocks by itself); without, row
// first + blockIdx.x.
// DIRECT: a workgroup per token of y instead, zeros for one without a target.
template <typename ET, bool GRAD, bool DIRECT>
__global__ __launch_bounds__(256) void k_xent_join(const float2 *__restrict__ part, int nblk, int pw,
                                                   const float *__restrict__ zt, const int64_t *__restrict__ y,
                                                   const int32_t *__restrict__ tgts, const int32_t *__restrict__ list,
                                                   const int32_t *__restrict__ n_act, int row0, int R, int V,
                                                   const float *__restrict__ dloss, ET *__restrict__ e, int64_t lde,
                                                   bf16_t *__restrict__ g, int64_t gplane, int split,
                                                   float *__restrict__ loss, float *__restrict__ lse, int first) {
  __shared__ float red[8];
  const int wave = threadIdx.x >> 6;
  const int part_of = GRAD ? blockIdx.x % split : 0;
  int r = GRAD ? blockIdx.x / split : first + blockIdx.x, t, tgt;
  if constexpr (DIRECT) {
    t = r;
    const int64_t v = y[t];
    if (v < 0) {
      if (threadIdx.x == 0) loss[t] = lse[t] = 0.f;
      return;
    }
    int c = 0;                                            // tokens of the list before this one
    for (int i = threadIdx.x; i < t; i += 256) c += y[i] >= 0;
    c = wave_sum(c);
    if ((threadIdx.x & 63) == 0) red[wave] = __int_as_float(c);
    __syncthreads();
    r = 0;
    for (int i = 0; i < 4; ++i) r += __float_as_int(red[i]);
    __syncthreads();
    tgt = v < V ? (int)v : V;
  } else {
    if (r >= piece_rows(n_act, row0, R)) return;
    t = list[row0 + r];
    tgt = tgts[row0 + r];
  }
  const float2 *p = part + (size_t)r * nblk;
  // a thread's first blocks stay in registers between the two passes
  constexpr int kB = 8;
  float2 b[kB];
#pragma unroll
  for (int k = 0; k < kB; ++k) b[k] = threadIdx.x + k * 256 < nblk ? p[threadIdx.x + k * 256] : make_float2(-INFINITY, 0.f);
  float mx = -INFINITY;
#pragma unroll
  for (int k = 0; k < kB; ++k) mx = fmaxf(mx, b[k].x);
  for (int i = threadIdx.x + kB * 256; i < nblk; i += 256) mx = fmaxf(mx, p[i].x);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, 64));
  if ((threadIdx.x & 63) == 0) red[wave] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float ref = mx == -INFINITY ? 0.f : mx;
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < kB; ++k)
    if (threadIdx.x + k * 256 < nblk) s += b[k].y * expf(b[k].x - ref);
  for (int i = threadIdx.x + kB * 256; i < nblk; i += 256) s += p[i].y * expf(p[i].x - ref);
  s = wave_sumf(s);
  if ((threadIdx.x & 63) == 0) red[4 + wave] = s;
  __syncthreads();
  const float rest = (red[4] + red[5]) + (red[6] + red[7]);
  const bool bad = tgt >= V;                              // then rest is the sum over all
  const float z = bad ? NAN : zt[row0 + r], et = bad ? 0.f : expf(z - ref), all = rest + et;
  const float ls = logf(all), l = ref + ls;
  if (threadIdx.x == 0 && part_of == 0) {
    lse[t] = l;
    loss[t] = et > 0.5f ? log1pf(rest / et) : (ref - z) + ls;
  }
  if constexpr (GRAD) {
    // exp(z - lse) as exp(z - max) / sum: lse itself has lost the sum's digits in a row far from zero
    const float dl = bad ? NAN : dloss[t], at_target = -rest / all * dl, scale = dl / all;
    constexpr int kAt = 4;                                // units in flight: loads before any store
    const int step = split * 256 * 8;
    for (int i0 = (part_of * 256 + threadIdx.x) * 8; i0 < lde; i0 += kAt * step) {
      Raw8<ET> raw[kAt];
      float f[kAt];
#pragma unroll
      for (int q = 0; q < kAt; ++q) {
        const int i = i0 + q * step, b = i >> pw;         // one block covers the 8 columns
        if (i < lde) raw[q].load(e + (size_t)r * lde + i);
        f[q] = b < nblk ? p[b].x : 0.f;
      }
#pragma unroll
      for (int q = 0; q < kAt; ++q) {
        const int i = i0 + q * step;
        if (i >= lde) break;
        f[q] = expf(f[q] - ref) * scale;
        float v[8];
        raw[q].to(v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= f[q];
        if ((uint32_t)(tgt - i) < 8u)
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = i + k == tgt ? at_target : v[k];
        if (i + 8 > V)
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = i + k < V ? v[k] : 0.f;
        if constexpr (std::is_same<ET, float>::value) {
          if (g) split8(v, g + (size_t)r * lde + i, gplane);
          else store8(e + (size_t)r * lde + i, v);
        } else {
          store8(e + (size_t)r * lde + i, v);
        }
      }
    }
  }
}

// --------------------------------------------------------------------------------- gradients

// What the gradients' products read and write, for rows [row0, row0 + R) of the list.
template <typename T> struct GradPiece {
  const bf16_t *w, *xc, *g;
  int64_t wplane, xplane, gplane, lde;
  const int32_t *list, *n_act;
  int row0, R, V, d;
  int S, ks;                                              // dx: splits of the vocabulary, columns in each
  T *dx;
  float *part;                                            // dx's partial sums [S][R][d] (S > 1)
  bool add;                                               // dw: to the sums of earlier pieces
  float *sum;                                             // which are here
  T *dw;                                                  // NULL until the last piece
  int Sw, rs;                                             // dw: splits of the tokens, rows in each
  float *partw;                                           // dw's partial sums [Sw][V][d] (Sw > 1)
};

// dx: D[column of d][token] = w^T G^T over the vocabulary range of split b / tiles (w across k, G
// along k), workgroup b. One split: to the token's row of dx; several: fp32 partial sums.
template <class G, int NP, typename T> TW_DEV void dx_tile(const GradPiece<T> &a, int b, char *smem) {
  const int mt = (a.d + G::BM - 1) / G::BM, nt = (a.R + G::BN - 1) / G::BN, t = mm_xcd_tile(b, mt * nt * a.S);
  if (t < 0) return;
  int m, n;
  const int sp = t / (mt * nt);
  mm_tile_mn<8>(t % (mt * nt), mt, nt, m, n);
  const int m0 = m * G::BM, n0 = n * G::BN, rows = piece_rows(a.n_act, a.row0, a.R);
  if (n0 >= rows) return;
  f32x4_t acc[G::FM][G::FN];
#pragma unroll
  for (int i = 0; i < G::FM; ++i)
#pragma unroll
    for (int j = 0; j < G::FN; ++j) acc[i][j] = f32x4_t{};
  const int k0 = sp * a.ks, k1 = min(a.V, k0 + a.ks);
  if constexpr (NP == 0) {
    const MmfOperand A = {(const float *)a.w + (size_t)k0 * a.d + m0, a.d, min(a.d - m0, G::BM)};
    const MmfOperand B = {(const float *)a.g + (size_t)n0 * a.lde + k0, a.lde, min(rows - n0, G::BN)};
    if (k0 < k1) mmf_loop<G>(A, B, k1 - k0, acc, smem);
  } else {
    const MmOperand A = {a.w + (size_t)k0 * a.d + m0, a.d, a.wplane, min(a.d - m0, G::BM)};
    const MmOperand B = {a.g + (size_t)n0 * a.lde + k0, a.lde, a.gplane, min(rows - n0, G::BN)};
    if (k0 < k1) mm_loop<G, NP>(A, B, k1 - k0, acc, smem);
  }

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / G::NWN, wn = wave % G::NWN;
#pragma unroll
  for (int fn = 0; fn < G::FN; ++fn) {
    const int r = n0 + wn * G::WN + fn * 16 + (lane & 15);
    if (r >= rows) continue;
    const size_t at = a.S == 1 ? (size_t)a.list[a.row0 + r] * a.d : ((size_t)sp * a.R + r) * a.d;
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm) {
      const int c = m0 + wm * G::WM + fm * 16 + (lane >> 4) * 4;
      if (c >= a.d) continue;                             // d is a multiple of 8
      const f32x4_t v = acc[fm][fn];
      if (a.S > 1) *(f32x4_t *)(a.part + at + c) = v;
      else if constexpr (std::is_same<T, float>::value) *(f32x4_t *)(a.dx + at + c) = v;
      else *(uint2 *)(a.dx + at + c) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    }
  }
}

// Adds dx's S partial sums, 8 elements per thread, workgroup b of NT threads.
template <int NT, typename T> TW_DEV void dx_sum(const GradPiece<T> &a, int b) {
  const size_t i = ((size_t)b * NT + threadIdx.x) * 8;
  const int r = (int)(i / a.d), c = (int)(i % a.d);       // d is a multiple of 8
  if (r >= piece_rows(a.n_act, a.row0, a.R)) return;
  float v[8] = {};
#pragma unroll 4
  for (int s = 0; s < a.S; ++s) {
    float u[8];
    load8(a.part + (size_t)s * a.R * a.d + i, u);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += u[k];
  }
  store8(a.dx + (size_t)a.list[a.row0 + r] * a.d + c, v);
}

// dw's elements [at, at + 4) from a piece's sum u: with the sums of the pieces so far, to those sums or,
// rounded, to dw.
template <typename T> TW_DEV void dw_out(const GradPiece<T> &a, size_t at, f32x4_t u) {
  if (a.add) u += *(const f32x4_t *)(a.sum + at);
  if (!a.dw) *(f32x4_t *)(a.sum + at) = u;
  else if constexpr (std::is_same<T, float>::value) *(f32x4_t *)(a.dw + at) = u;
  else *(uint2 *)(a.dw + at) = make_uint2(pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]));
}

// Adds dw's Sw partial sums, 4 elements per thread, workgroup b of NT threads.
template <int NT, typename T> TW_DEV void dw_sum(const GradPiece<T> &a, int b) {
  const size_t n = (size_t)a.V * a.d, i = ((size_t)b * NT + threadIdx.x) * 4;
  if (i >= n) return;
  f32x4_t u = {};
#pragma unroll 4
  for (int s = 0; s < a.Sw; ++s) u += *(const f32x4_t *)(a.partw + s * n + i);
  dw_out(a, i, u);
}

// dw: D[column of d][vocabulary] = x^T G over the tokens of split b / tiles of the piece (both across k),
// workgroup b. A small dw of many tokens would occupy few CUs without the splits.
template <class G, int NP, typename T> TW_DEV void dw_tile(const GradPiece<T> &a, int b, char *smem) {
  const int mt = (a.d + G::BM - 1) / G::BM, nt = (a.V + G::BN - 1) / G::BN, t = mm_xcd_tile(b, mt * nt * a.Sw);
  if (t < 0) return;
  int m, n;
  const int sp = t / (mt * nt);
  mm_tile_mn<8>(t % (mt * nt), mt, nt, m, n);
  const int m0 = m * G::BM, n0 = n * G::BN, rows = piece_rows(a.n_act, a.row0, a.R);
  const int r0 = sp * a.rs, K = max(min(rows - r0, a.rs), 0);
  f32x4_t acc[G::FM][G::FN];
#pragma unroll
  for (int i = 0; i < G::FM; ++i)
#pragma unroll
    for (int j = 0; j < G::FN; ++j) acc[i][j] = f32x4_t{};
  const int cols = (int)min(a.lde - n0, (int64_t)G::BN);  // the padding of G's rows up to lde is zero
  if constexpr (NP == 0) {
    const MmfOperand A = {(const float *)a.xc + (size_t)(a.row0 + r0) * a.d + m0, a.d, min(a.d - m0, G::BM)};
    const MmfOperand B = {(const float *)a.g + (size_t)r0 * a.lde + n0, a.lde, cols};
    mmf_loop<G>(A, B, K, acc, smem);
  } else {
    const MmOperand A = {a.xc + (size_t)(a.row0 + r0) * a.d + m0, a.d, a.xplane, min(a.d - m0, G::BM)};
    const MmOperand B = {a.g + (size_t)r0 * a.lde + n0, a.lde, a.gplane, cols};
    mm_loop<G, NP>(A, B, K, acc, smem);
  }

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / G::NWN, wn = wave % G::NWN;
#pragma unroll
  for (int fn = 0; fn < G::FN; ++fn) {
    const int v = n0 + wn * G::WN + fn * 16 + (lane & 15);
    if (v >= a.V) continue;
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm) {
      const int c = m0 + wm * G::WM + fm * 16 + (lane >> 4) * 4;
      if (c >= a.d) continue;
      const size_t at = (size_t)v * a.d + c;
      if (a.Sw > 1) *(f32x4_t *)(a.partw + (size_t)sp * a.V * a.d + at) = acc[fm][fn];
      else dw_out(a, at, acc[fm][fn]);
    }
  }
}

template <class X, int NP, typename T> __global__ __launch_bounds__(X::NT) void k_xent_dx(GradPiece<T> a) {
  __shared__ __attribute__((aligned(16))) char smem[X::SMEM];
  dx_tile<X, NP>(a, blockIdx.x, smem);
}

// The workgroups from `tiles` on add dx's partial sums, which are complete when this launch begins.
template <class W, int NP, typename T> __global__ __launch_bounds__(W::NT) void k_xent_dw(GradPiece<T> a, int tiles) {
  __shared__ __attribute__((aligned(16))) char smem[W::SMEM];
  if ((int)blockIdx.x < tiles) dw_tile<W, NP>(a, blockIdx.x, smem);
  else dx_sum<W::NT>(a, blockIdx.x - tiles);
}

// Both products in one launch (dw's workgroups from `tiles` on), where each alone is too small to
// fill the GPU: T = 128, d = 256, V = 1009 in fp32 planes 30 us one after the
// other, 18 together and 4 for the sum of dx.
template <class X, class W, int NP, typename T>
__global__ __launch_bounds__(X::NT) void k_xent_dx_dw(GradPiece<T> a, int tiles) {
  static_assert(X::NT == W::NT, "threads");
  __shared__ __attribute__((aligned(16))) char smem[X::SMEM > W::SMEM ? X::SMEM : W::SMEM];
  if ((int)blockIdx.x < tiles) dx_tile<X, NP>(a, blockIdx.x, smem);
  else dw_tile<W, NP>(a, blockIdx.x - tiles, smem);
}

// The partial sums of dx (the first nx workgroups) and of dw.
template <typename T> __global__ __launch_bounds__(256) void k_xent_sums(GradPiece<T> a, int nx) {
  if ((int)blockIdx.x < nx) dx_sum<256>(a, blockIdx.x);
  else dw_sum<256>(a, blockIdx.x - nx);
}

__global__ __launch_bounds__(256) void k_xent_zero(uint4 *__restrict__ p, size_t n) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------------------------- plan

// The products' tiles. Large: 8 waves of 64 x 128 (logits: 128 x 64, and groups of 4 tiles of the
// vocabulary: 6.74 ms against 6.90 at T = 8192, d = 4096, V = 128000), one workgroup per CU, the least
// traffic per operation. The smaller ones, two workgroups per CU, are for calls whose large tiles would leave CUs
// idle or hold mostly rows that do not exist. The smallest logits tile's ring of four 64-k stages
// keeps 24 KB of w per workgroup in flight, for few tokens, where the stream of w is all there is.
enum { kSmall, kMid, kLarge, kStream };
template <int C> struct Tiles;
template <> struct Tiles<kSmall> {
  typedef MM64<64, 64, 16, 64, 4, 4> Z;                   // logits
  typedef MM<256, 64, 64, 64, 3, true, false> X;          // dx
  typedef MM<256, 64, 64, 64, 3, true, true> W;           // dw
};
template <> struct Tiles<kMid> {
  typedef MM64<128, 128, 64, 64, 3, 2> Z;
};
template <> struct Tiles<kLarge> {
  typedef MM64<256, 256, 128, 64, 3, 2> Z;
  typedef MM<256, 256, 64, 128, 4, true, false> X;
  typedef MM<256, 256, 64, 128, 4, true, true> W;
};

// Logits of at most 32 bf16 tokens with more than one such tile per CU: T = 20, d = 2048, V = 128000 112 us
// (128 x 128: 128), T = 1, d = 1024, V = 50000 26 (28). Up to one per CU, two 64 x 64 workgroups stream
// better than one of these (T = 1, d = 4096, V = 32000: 55 us against 59).
template <> struct Tiles<kStream> {
  typedef MM64<128, 32, 32, 32, 4, 4> Z;
};
struct TilesF {                                           // fp32 as it is
  typedef MMF<64, 64, false, false> Z;
  // logits of at most 32 tokens: T = 1, d = 2136, V = 80008 145 us, with 64 x 64 228; T = 16, d = 4096, V = 8000
  // 62 and 86
  typedef MMF<128, 32, false, false> ZFew;
  typedef MMF<64, 64, true, false> X;
  typedef MMF<64, 64, true, true> W;
};

struct TilesFew {
  typedef TilesF::ZFew Z;
};

constexpr int kCUs = 256;
constexpr int kCountT = 2048;                             // tokens up to which k_xent_stage counts
constexpr size_t kPieceBytes = (size_t)1 << 30;

// Nanoseconds of `tiles` tiles of a class over `stages` stages: rounds of resident workgroups, each
// with its stages (all workgroups of a CU together) and its start and epilogue. Measured per kernel
// with every class forced, T x d x V in bf16 (small / mid / large, us): logits 100 x 1024 x 8000: 11 / 15
// / 32, 1000 x 4096 x 8000: 108 / 66 / 92, 4096 x 1024 x 16000: 293 / 153 / 140; dx 500 x 512 x 2000: 15 / 17
// (small / large), 1000 x 4096 x 8000: 98 / 63; dw 128 x 256 x 1009 in fp32: 16 / 25, 4096 x 1024 x 16000:
// 203 / 118. (Tiles of 256 x 128 for dx and dw were slower than either everywhere.) fp32 in planes /
// as it is, a whole call with gradients: 128 x 256 x 1009 44 / 29, 64 x 1024 x 32000 303 / 184, 16 x 4096 x 8000
// 299 / 182, 600 x 1024 x 5000 235 / 246, 2255 x 1648 x 6125 876 / 1298.
struct Cost {
  int per_cu, stage, alone, start;                        // alone: a stage where no CU has two workgroups
};
constexpr Cost kCostZ[3] = {{2, 450, 450, 2500}, {2, 1000, 750, 4000}, {1, 1450, 1450, 9000}};      // 64-k stages
constexpr int kSums = 3000;                                                       // the launch that adds partial sums
constexpr Cost kCostF = {2, 1050, 550, 3000};                                    // fp32 as it is: 32-k stages
constexpr Cost kCostG[3] = {{2, 750, 700, 4500}, {}, {1, 850, 850, 10000}};       // dx, dw: 32-k stages
int64_t cost_of(const Cost &c, int64_t tiles, int64_t stages) {
  if (tiles <= kCUs) return stages * c.alone + c.start;
  const int64_t slots = kCUs * c.per_cu;
  return (tiles + slots - 1) / slots * (stages * c.stage + c.start);
}
// Whether a smaller tile's cost n is to be preferred: near ties go to the larger, whose tiles of
// tokens without a target cost nothing.
bool cheaper(int64_t n, int64_t best) { return n * 10 < best * 9; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The logits tile of class c: columns, and log2 of the columns per wave.
int block_m(int c) { return c == kStream ? Tiles<kStream>::Z::BM : 64 << c; }
int block_log(int c) { return c == kSmall ? 4 : c == kMid ? 6 : c == kStream ? 5 : 7; }
constexpr int kBlockLogF = 5;
static_assert(TilesF::Z::WM == 32 && TilesF::ZFew::WM == 32 && Tiles<kSmall>::Z::WM == 16 && Tiles<kMid>::Z::WM == 64 &&
                  Tiles<kLarge>::Z::WM == 128 && Tiles<kStream>::Z::WM == 32,
              "block_log");

struct Plan {
  int R, pieces, nblk, S, ks, Sw, rs, zc, dc, wc;                 // zc, dc, wc: classes of logits, dx, dw
  int64_t lde;
  bool direct, sums, plain;                               // plain: fp32 as it is
  size_t list, tgt, pos, zt, xc, wp, part, e, g, dxp, dwp, sum, bytes;   // offsets of the workspace
};

Plan plan_of(int T, int d, int V, int bf16, bool grad) {
  Plan p = {};
  const int np = bf16 ? 1 : 6;
  p.lde = ceil_div(V, 256) * 256;
  p.direct = bf16 && !grad && T <= kDirectRows;
  int64_t z = 0, dx = 0, dw = 0;                          // the products' costs
  for (int c = kLarge; c >= kSmall; --c) {
    const int b = 64 << c;
    const int64_t n = cost_of(kCostZ[c], ceil_div(V, b) * ceil_div(T, b), ceil_div(d, 64) * np);
    if (!z || cheaper(n, z)) {
      z = n;
      p.zc = c;
    }
  }
  if (bf16 && T <= 32 && ceil_div(V, block_m(kStream)) > kCUs) p.zc = kStream;
  // (both splits are chosen for all R rows; where most tokens have no target, dx's remaining tiles each walk
  // a long range of the vocabulary on few CUs)
  // dx in R rows by tiles of m columns of d and b tokens: the vocabulary split 1, 2, 4, .. 64 times; the
  // partial sums cost their traffic (about 5 bytes per ps)
  auto split_dx = [&](const Cost &c, int m, int b, int R, int products, int64_t &best, int cls) {
    const int64_t tiles = ceil_div(d, m) * ceil_div(R, b);
    for (int S0 = 1; S0 <= 64 && (S0 == 1 || tiles * S0 <= kCUs * c.per_cu); S0 *= 2) {
      const int64_t ks = ceil_div(ceil_div(V, S0), 64) * 64, S = ceil_div(V, ks);
      const int64_t n = cost_of(c, tiles * S, ks / 32 * products) + (S > 1 ? kSums + S * R * d * 8 / 5000 : 0);
      if (!best || cheaper(n, best)) {
        best = n;
        p.dc = cls;
        p.S = (int)S;
        p.ks = (int)ks;
      }
    }
  };
  // dw over R tokens by tiles of m columns of d and b of the vocabulary: the tokens split likewise, in
  // partial sums of at most 64 MB
  auto split_dw = [&](const Cost &c, int m, int b, int R, int products, int64_t &best, int cls) {
    const int64_t tiles = ceil_div(d, m) * ceil_div(V, b);
    for (int S0 = 1; S0 <= 64 && (S0 == 1 || (tiles * S0 <= kCUs * c.per_cu && (int64_t)S0 * V * d <= 16 << 20)); S0 *= 2) {
      const int64_t rs = ceil_div(ceil_div(R, S0), 32) * 32, S = ceil_div(R, rs);
      const int64_t n = cost_of(c, tiles * S, rs / 32 * products) + (S > 1 ? kSums + S * V * d * 8 / 5000 : 0);
      if (!best || cheaper(n, best)) {
        best = n;
        p.wc = cls;
        p.Sw = (int)S;
        p.rs = (int)rs;
      }
    }
  };
  const size_t planes = bf16 ? 1 : 3;
  // rows of a piece: as many as kPieceBytes hold of what a row keeps between the launches. bf16
  // gradients of several pieces need dw's sums in fp32; where all rows at once take no more
  // memory than that, there is one piece.
  auto rows_of = [&](int blocks, size_t element) {
    p.nblk = blocks;
    const size_t row = (size_t)p.nblk * 8 + (grad ? (size_t)p.lde * element : 0);
    const size_t sums = grad && bf16 ? (size_t)V * d * 4 : 0;
    const int64_t all = ceil_div(T, 64) * 64;
    int64_t R = (int64_t)(kPieceBytes / row) / 256 * 256;
    if (R < 256) R = 256;
    if (R >= all || (size_t)all * row <= kPieceBytes + sums) R = all;
    p.R = (int)R;
    p.pieces = (T + p.R - 1) / p.R;
    p.sums = sums && p.pieces > 1;
  };
  // blocks of all columns that the tiles cover (with e kept, its padding too)
  rows_of((int)((grad ? p.lde : ceil_div(V, block_m(p.zc)) * block_m(p.zc)) >> block_log(p.zc)), bf16 ? 2 : 10);
  if (grad) {
    for (int c = kLarge; c >= kSmall; c -= kLarge) split_dx(kCostG[c], 256, 64 << c, p.R, np, dx, c);
    for (int c = kLarge; c >= kSmall; c -= kLarge) split_dw(kCostG[c], 256, 64 << c, p.R, np, dw, c);
  }
  if (!bf16) {
    // the planes of w are written and read again
    const int64_t split = (int64_t)V * d * 10 / 5000, by_planes = split + z + (dx + dw) * p.pieces;
    Plan q = p;
    p.zc = T <= 32 ? kStream : kSmall;
    const int b = T <= 32 ? TilesF::ZFew::BM : TilesF::Z::BM;
    rows_of((int)((grad ? p.lde : ceil_div(V, b) * b) >> kBlockLogF), 4);
    int64_t fx = 0, fw = 0;
    const int64_t fz = cost_of(kCostF, ceil_div(V, b) * ceil_div(T, 64), ceil_div(d, 32));
    if (grad) {
      split_dx(kCostF, 64, 64, p.R, 1, fx, kSmall);
      split_dw(kCostF, 64, 64, p.R, 1, fw, kSmall);
    }
    p.plain = fz + (fx + fw) * p.pieces < by_planes;
    if (!p.plain) p = q;
  }
  size_t at = 256;                                        // n_act
  auto take = [&](size_t n) {
    const size_t o = at;
    at += align256(n);
    return o;
  };
  p.list = take((size_t)T * 4);
  p.tgt = take((size_t)T * 4);
  p.pos = p.zt = take((size_t)T * 4);                     // pos is done with before zt begins
  p.xc = take((size_t)T * d * (p.plain ? 4 : 2 * planes));
  if (!bf16 && !p.plain) p.wp = take((size_t)V * d * 2 * planes);
  p.part = take((size_t)p.R * p.nblk * 8);
  if (grad) {
    p.e = take((size_t)p.R * p.lde * (bf16 ? 2 : 4));
    if (!bf16 && !p.plain) p.g = take((size_t)p.R * p.lde * 6);
    if (p.S > 1) p.dxp = take((size_t)p.S * p.R * d * 4);
    if (p.Sw > 1) p.dwp = take((size_t)p.Sw * V * d * 4);
    if (p.sums) p.sum = take((size_t)V * d * 4);
  }
  p.bytes = at;
  return p;
}

// f(first, workgroups) over `total` workgroups of 256 threads, in as many launches as it takes: HIP
// counts the threads of one in 32 bits, which 2^24 tokens reach.
constexpr int64_t kLaunch = 1 << 23;
template <typename F> hipError_t in_launches(int64_t total, F &&f) {
  for (int64_t first = 0; first < total; first += kLaunch) {
    f(first, (unsigned)(total - first < kLaunch ? total - first : kLaunch));
    TW_TRY_HIP(hipGetLastError());
  }
  return hipSuccess;
}

int grid8(int64_t tiles) { return (int)((tiles + 7) / 8 * 8); }

// f(Tiles<c>()) for dx and dw
template <typename F> hipError_t with_tiles(int c, F &&f) {
  return c == kSmall ? f(Tiles<kSmall>()) : f(Tiles<kLarge>());
}

// and for the logits (kStream: bf16 only)
template <int NP, typename F> hipError_t with_logits(int c, F &&f) {
  if constexpr (NP == 1)
    if (c == kStream) return f(Tiles<kStream>());
  return c == kMid ? f(Tiles<kMid>()) : with_tiles(c, f);
}

// T: type of the operands and results; ET: of e
template <typename T, typename ET, int NP>
hipError_t xent_run(const XentArgs &a, const Plan &p, hipStream_t s) {
  char *ws = (char *)a.ws;
  int32_t *n_act = (int32_t *)ws, *list = (int32_t *)(ws + p.list), *tgt = (int32_t *)(ws + p.tgt);
  int32_t *pos = (int32_t *)(ws + p.pos);
  float *zt = (float *)(ws + p.zt);
  bf16_t *xc = (bf16_t *)(ws + p.xc);
  float2 *part = (float2 *)(ws + p.part);
  ET *e = (ET *)(ws + p.e);
  bf16_t *g = NP <= 1 ? (bf16_t *)e : (bf16_t *)(ws + p.g), *wp = NP <= 1 ? nullptr : (bf16_t *)(ws + p.wp);
  const int64_t xplane = (int64_t)a.T * a.d, wplane = (int64_t)a.V * a.d, gplane = (int64_t)p.R * p.lde;
  const bool grad = a.dw != nullptr;
  const int pw = NP == 0 ? kBlockLogF : block_log(p.zc);
  const bf16_t *w = NP <= 1 ? (const bf16_t *)a.w : wp;
  if constexpr (NP == 1) {
    // rows are addressed with 32-bit byte offsets
    if (p.direct && (a.T == 1 || a.ldx <= (1 << 20))) {
      auto logits = [&](auto C) {
        typedef typename decltype(C)::Z Z;
        const int mt = (int)ceil_div(a.V, Z::BM), nt = (int)ceil_div(a.T, Z::BN);
        k_xent_logits<Z, 1, ET, false, true><<<grid8((int64_t)mt * nt), Z::NT, 0, s>>>(
            w, 0, (const bf16_t *)a.x, a.ldx, 0, a.y, nullptr, nullptr, 0, a.T, a.V, a.d, mt, nt, nullptr, 0, part, p.nblk,
            zt);
        return hipGetLastError();
      };
      TW_TRY_HIP(with_logits<NP>(p.zc, logits));
      k_xent_join<ET, false, true><<<a.T, 256, 0, s>>>(part, p.nblk, pw, zt, a.y, nullptr, nullptr, nullptr, 0, a.T, a.V,
                                                       nullptr, nullptr, 0, nullptr, 0, 1, a.loss, a.lse, 0);
      return hipGetLastError();
    }
  }
  if (a.T > kCountT) {
    k_xent_rows<<<1, 1024, 0, s>>>(a.y, a.T, a.V, list, tgt, pos, n_act);
    TW_TRY_HIP(hipGetLastError());
  }
  const int64_t split = NP <= 1 ? 0 : ceil_div(wplane, 256 * 8);
  TW_TRY_HIP(in_launches(a.T + split, [&](int64_t first, unsigned n) {
    k_xent_stage<T, T><<<n, 256, 0, s>>>((const T *)a.x, a.ldx, a.T, a.d, a.V, a.y, a.T > kCountT ? pos : nullptr, list,
                                         tgt, n_act, xc, xplane, a.loss, a.lse, (T *)a.dx, (const T *)a.w,
                                         (size_t)wplane, wp, (int)first);
  }));
  for (int q = 0; q < p.pieces; ++q) {
    const int row0 = q * p.R, R = a.T - row0 < p.R ? a.T - row0 : p.R;
    auto logits = [&](auto C) {
      typedef typename decltype(C)::Z Z;
      // with e kept, the tiles cover its padding too
      const int mt = (int)ceil_div(grad ? p.lde : a.V, Z::BM), nt = (int)ceil_div(R, Z::BN);
      auto go = [&](auto keep) {
        k_xent_logits<Z, NP, ET, decltype(keep)::value, false><<<grid8((int64_t)mt * nt), Z::NT, 0, s>>>(
            w, wplane, xc, a.d, xplane, nullptr, tgt, n_act, row0, R, a.V, a.d, mt, nt, e, p.lde, part, p.nblk, zt);
      };
      if (grad) go(std::integral_constant<bool, true>());
      else go(std::integral_constant<bool, false>());
      return hipGetLastError();
    };
    if constexpr (NP == 0) TW_TRY_HIP(p.zc == kStream ? logits(TilesFew()) : logits(TilesF()));
    else TW_TRY_HIP(with_logits<NP>(p.zc, logits));
    // a row's columns go to several workgroups where rows alone would leave CUs idle
    int split = 1;
    while (grad && R * split < 4 * kCUs && split * 8192 < p.lde) split *= 2;
    auto join = [&](auto G, int64_t first, unsigned n) {
      k_xent_join<ET, decltype(G)::value, false><<<n, 256, 0, s>>>(part, p.nblk, pw, zt, nullptr, tgt, list, n_act, row0,
                                                                   R, a.V, a.dloss, e, p.lde, NP > 1 ? g : nullptr,
                                                                   gplane, split, a.loss, a.lse, (int)first);
    };
    if (grad) {                             // R < 2^22: a row keeps 512 bytes or more
      join(std::integral_constant<bool, true>(), 0, R * split);
      TW_TRY_HIP(hipGetLastError());
    } else {
      TW_TRY_HIP(in_launches(R, [&](int64_t first, unsigned n) { join(std::integral_constant<bool, false>(), first, n); }));
    }
    if (!grad) continue;
    const bool last = q + 1 == p.pieces, f32 = NP != 1;
    GradPiece<T> gp;
    gp.w = w; gp.xc = xc; gp.g = g;
    gp.wplane = wplane; gp.xplane = xplane; gp.gplane = gplane; gp.lde = p.lde;
    gp.list = list; gp.n_act = n_act;
    gp.row0 = row0; gp.R = R; gp.V = a.V; gp.d = a.d;
    gp.S = p.S; gp.ks = p.ks;
    gp.dx = (T *)a.dx; gp.part = p.S > 1 ? (float *)(ws + p.dxp) : nullptr;
    gp.add = q > 0;
    gp.sum = f32 ? (float *)a.dw : (float *)(ws + p.sum);
    gp.dw = last || f32 ? (T *)a.dw : nullptr;
    gp.Sw = p.Sw; gp.rs = p.rs; gp.partw = p.Sw > 1 ? (float *)(ws + p.dwp) : nullptr;
    auto dx_grid = [&](auto X) { return grid8(ceil_div(a.d, decltype(X)::BM) * ceil_div(R, decltype(X)::BN) * p.S); };
    auto dw_grid = [&](auto W) { return grid8(ceil_div(a.d, decltype(W)::BM) * ceil_div(a.V, decltype(W)::BN) * p.Sw); };
    auto sum_grid = [&](int nt) { return p.S > 1 ? (int)ceil_div((int64_t)R * a.d, nt * 8) : 0; };
    auto sums = [&](int nx) {
      const int nw = p.Sw > 1 ? (int)ceil_div(wplane, 256 * 4) : 0;
      if (nx + nw) k_xent_sums<<<nx + nw, 256, 0, s>>>(gp, nx);
      return hipGetLastError();
    };
    if (NP == 0 || (p.dc == kSmall && p.wc == kSmall)) {
      typedef typename std::conditional<NP == 0, TilesF, Tiles<kSmall>>::type C;
      typedef typename C::X X;
      typedef typename C::W W;
      const int tiles = dx_grid(X());
      k_xent_dx_dw<X, W, NP><<<tiles + dw_grid(W()), X::NT, 0, s>>>(gp, tiles);
      TW_TRY_HIP(hipGetLastError());
      TW_TRY_HIP(sums(sum_grid(256)));
      continue;
    }
    if constexpr (NP > 0) {
      TW_TRY_HIP(with_tiles(p.dc, [&](auto C) {
        typedef typename decltype(C)::X X;
        k_xent_dx<X, NP><<<dx_grid(X()), X::NT, 0, s>>>(gp);
        return hipGetLastError();
      }));
      TW_TRY_HIP(with_tiles(p.wc, [&](auto C) {
        typedef typename decltype(C)::W W;
        const int tiles = dw_grid(W());
        k_xent_dw<W, NP><<<tiles + sum_grid(W::NT), W::NT, 0, s>>>(gp, tiles);
        return hipGetLastError();
      }));
      TW_TRY_HIP(sums(0));
    }
  }
  return hipSuccess;
}

}  // namespace

size_t xent_workspace_bytes(int T, int d, int V, int bf16, bool grad) { return plan_of(T, d, V, bf16, grad).bytes; }

hipError_t launch_xent(const XentArgs &a, hipStream_t s) {
  if (a.T == 0) {                           // no tokens: dw is zero
    const size_t n16 = (size_t)a.V * a.d * (a.bf16 ? 2 : 4) / 16;
    return in_launches((n16 + 255) / 256, [&](int64_t first, unsigned n) {
      k_xent_zero<<<n, 256, 0, s>>>((uint4 *)a.dw + first * 256, n16 - first * 256);
    });
  }
  const Plan p = plan_of(a.T, a.d, a.V, a.bf16, a.dw != nullptr);
  if (a.bf16) return xent_run<bf16_t, bf16_t, 1>(a, p, s);
  return p.plain ? xent_run<float, float, 0>(a, p, s) : xent_run<float, float, 6>(a, p, s);
}

}  // namespace tw
