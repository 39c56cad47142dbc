// Layer norm of token rows on gfx950, forward and backward, with the residual add of a
// pre-norm block on either side.
//
//   s = x + r (rounded to x's type);  mu = mean(s);  rstd = 1 / sqrt(mean((s - mu)^2) + eps)
//   y = (s - mu) rstd w + b
//   xh = (s - mu) rstd;  g = dy w
//   dx = rstd (g - mean(g) - xh mean(g xh)) + dres;  dw = sum_t dy xh;  db = sum_t dy
//
// Both passes do about ten operations per element read, so HBM bounds them. A workgroup holds
// a whole row in registers (8-element units, VPT of them per thread), so that every operand is
// read once whatever the number of passes over the row: the mean, the centred squares and the
// output all come from the registers. Measured: forward with residual at T = 4096, d = 2048 in bf16
// 12.5 us where the 67 MB lie in the last-level cache, 17.7 with inputs that come from HBM; backward at
// T = 16384, d = 4096 with fp32 dy and bf16 s and dres 121 + 5 us (5.3 TB/s; a 2 GiB copy reaches 4.7 -
// 4.9). The statistics and the sums over tokens are fp32; the variance is summed from centred values,
// which keeps it exact for rows far from zero.
#include "common.h"
#include "launch.h"
#include "row8.h"

namespace tw {
namespace {

constexpr int kU = 8;                       // elements of a unit: 16 bytes of bf16, 32 of fp32

// Sums of the NV values of every thread over the workgroup, the same bits in every thread.
// `red` holds 2 x 16 x NV floats; `turn` alternates between its halves from call to call, so
// that one barrier per call is enough.
template <int NV> TW_DEV void block_sum(float (&v)[NV], float *red, int &turn) {
#pragma unroll
  for (int k = 0; k < NV; ++k) v[k] = wave_sumf(v[k]);
  const int nw = blockDim.x >> 6;
  if (nw == 1) return;
  float *r = red + turn * 16 * NV;
  turn ^= 1;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int k = 0; k < NV; ++k) r[(threadIdx.x >> 6) * NV + k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float t = 0.f;
    for (int i = 0; i < nw; ++i) t += r[i * NV + k];
    v[k] = t;
  }
}

template <typename T, typename YT, int VPT>
__global__ __launch_bounds__(1024) void k_norm_fwd(const T *__restrict__ x, int64_t ldx, const T *__restrict__ res,
                                                   int64_t ldr, const float *__restrict__ w,
                                                   const float *__restrict__ b, int rows, int d, float eps,
                                                   YT *__restrict__ y, T *__restrict__ s, float *__restrict__ mean,
                                                   float *__restrict__ rstd) {
  __shared__ float red[32];
  int turn = 0;
  const int units = d / kU, nt = blockDim.x;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {        // beyond 2^31 in its last step
    float v[VPT][kU];
    float sum[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = threadIdx.x + i * nt;
      if (u >= units) continue;
      load8(x + row * ldx + (size_t)u * kU, v[i]);
      if (res) {
        float r[kU];
        load8(res + row * ldr + (size_t)u * kU, r);
#pragma unroll
        for (int k = 0; k < kU; ++k) v[i][k] = rounded<T>(v[i][k] + r[k]);
        store8(s + row * d + (size_t)u * kU, v[i]);
      }
#pragma unroll
      for (int k = 0; k < kU; ++k) sum[0] += v[i][k];
    }
    block_sum(sum, red, turn);
    const float mu = sum[0] / (float)d;
    float sq[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (threadIdx.x + i * nt >= units) continue;
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        v[i][k] -= mu;
        sq[0] += v[i][k] * v[i][k];
      }
    }
    block_sum(sq, red, turn);
    const float rs = 1.f / sqrtf(sq[0] / (float)d + eps);
    if (threadIdx.x == 0) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = rs;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = threadIdx.x + i * nt;
      if (u >= units) continue;
      float wv[kU], bv[kU], o[kU];
      load8(w + u * kU, wv);
      if (b) load8(b + u * kU, bv);
#pragma unroll
      for (int k = 0; k < kU; ++k) o[k] = v[i][k] * rs * wv[k] + (b ? bv[k] : 0.f);
      store8(y + row * d + (size_t)u * kU, o);
    }
  }
}

// A row's operands of the backward on their way.
template <typename T, typename DYT, typename DXT, int VPT> struct BwdRow {
  Raw8<T> s[VPT];
  Raw8<DYT> dy[VPT];
  Raw8<DXT> dres[VPT];
  float mu, rs;
};

// One workgroup takes rows blockIdx.x, blockIdx.x + gridDim.x, ... and keeps its columns' sums
// of dy xh and dy in registers; they end in part[blockIdx.x][2][d] (or straight in dw and db
// where it is the only workgroup), so no atomics, and the same bits on every call. With one unit
// per thread (d <= 8192) w stays in registers over the rows, and the next row's operands are loaded
// before the sums of this one, so that the loads do not stop at the barrier; with two, 1024 threads
// leave no registers for that.
template <typename T, typename DYT, typename DXT, int VPT>
__global__ __launch_bounds__(1024) void k_norm_bwd(const DYT *__restrict__ dy, int64_t lddy, const T *__restrict__ s,
                                                   int64_t lds, const float *__restrict__ w,
                                                   const float *__restrict__ mean, const float *__restrict__ rstd,
                                                   const DXT *__restrict__ dres, int64_t lddr, int rows, int d,
                                                   DXT *__restrict__ dx, float *__restrict__ dw,
                                                   float *__restrict__ db, float *__restrict__ part) {
  __shared__ float red[64];
  constexpr bool kAhead = VPT == 1;
  int turn = 0;
  const int units = d / kU, nt = blockDim.x;
  float aw[VPT][kU], ab[VPT][kU], wv[VPT][kU];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
#pragma unroll
    for (int k = 0; k < kU; ++k) aw[i][k] = ab[i][k] = 0.f;
    const int u = threadIdx.x + i * nt;
    if (kAhead && u < units) load8(w + u * kU, wv[i]);
  }
  typedef BwdRow<T, DYT, DXT, VPT> Row;
  auto fetch = [&](int64_t row, Row &r) {
    r.mu = mean[row];
    r.rs = rstd[row];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = threadIdx.x + i * nt;
      if (u >= units) continue;
      r.s[i].load(s + row * lds + (size_t)u * kU);
      r.dy[i].load(dy + row * lddy + (size_t)u * kU);
      if (kAhead && dres) r.dres[i].load(dres + row * lddr + (size_t)u * kU);
    }
  };
  Row cur, next;
  int64_t row = blockIdx.x;                               // beyond 2^31 in its last step
  if (kAhead && row < rows) fetch(row, cur);
  for (; row < rows; row += gridDim.x) {
    if (!kAhead) fetch(row, cur);
    else if (row + gridDim.x < rows) fetch(row + gridDim.x, next);
    float xh[VPT][kU], g[VPT][kU];
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = threadIdx.x + i * nt;
      if (u >= units) continue;
      if (!kAhead) load8(w + u * kU, wv[i]);
      cur.s[i].to(xh[i]);
      cur.dy[i].to(g[i]);
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        xh[i][k] = (xh[i][k] - cur.mu) * cur.rs;
        aw[i][k] += g[i][k] * xh[i][k];
        ab[i][k] += g[i][k];
        g[i][k] *= wv[i][k];
        sum[0] += g[i][k];
        sum[1] += g[i][k] * xh[i][k];
      }
    }
    block_sum(sum, red, turn);
    const float mg = sum[0] / (float)d, mx = sum[1] / (float)d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = threadIdx.x + i * nt;
      if (u >= units) continue;
      float o[kU];
#pragma unroll
      for (int k = 0; k < kU; ++k) o[k] = cur.rs * (g[i][k] - mg - xh[i][k] * mx);
      if (dres) {
        float r[kU];
        if (!kAhead) cur.dres[i].load(dres + row * lddr + (size_t)u * kU);
        cur.dres[i].to(r);
#pragma unroll
        for (int k = 0; k < kU; ++k) o[k] += r[k];
      }
      store8(dx + row * d + (size_t)u * kU, o);
    }
    if (kAhead) cur = next;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int u = threadIdx.x + i * nt;
    if (u >= units) continue;
    float *pw = gridDim.x == 1 ? dw : part + (size_t)blockIdx.x * 2 * d;
    float *pb = gridDim.x == 1 ? db : pw + d;
#pragma unroll
    for (int k = 0; k < kU; k += 4) {
      *(float4 *)(pw + u * kU + k) = make_float4(aw[i][k], aw[i][k + 1], aw[i][k + 2], aw[i][k + 3]);
      if (pb) *(float4 *)(pb + u * kU + k) = make_float4(ab[i][k], ab[i][k + 1], ab[i][k + 2], ab[i][k + 3]);
    }
  }
}

// dw and db from the P partial rows of 2 d sums: a workgroup takes 32 of the 2 d columns, its 128
// groups of 8 lanes every 128th row, and the groups' sums are added in order.
__global__ __launch_bounds__(1024) void k_norm_bwd_sum(const float *__restrict__ part, int P, int d,
                                                       float *__restrict__ dw, float *__restrict__ db) {
  __shared__ float4 red[128][8];
  __shared__ float red2[8][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 7) * 4, grp = threadIdx.x >> 3;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < 2 * d)
#pragma unroll 4
    for (int p = grp; p < P; p += 128) {
      const float4 v = *(const float4 *)(part + (size_t)p * 2 * d + col);
      a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
    }
  red[grp][threadIdx.x & 7] = a;
  __syncthreads();
  if (threadIdx.x < 256) {
    const int at = threadIdx.x & 31, g = threadIdx.x >> 5;
    float t = 0.f;
    for (int i = 0; i < 16; ++i) t += ((const float *)&red[g * 16 + i][at >> 2])[at & 3];
    red2[g][at] = t;
  }
  __syncthreads();
  const int c = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x >= 32 || c >= 2 * d) return;
  float t = 0.f;
  for (int i = 0; i < 8; ++i) t += red2[i][threadIdx.x];
  if (c < d) dw[c] = t;
  else if (db) db[c - d] = t;
}

// Threads of a workgroup that holds a row of d in VPT units per thread.
int row_threads(int d, int vpt) { return ((d / kU + vpt - 1) / vpt + 63) / 64 * 64; }
int norm_vpt(int d) { return d <= 1024 * kU ? 1 : 2; }

template <typename T, typename YT>
hipError_t norm_fwd(const NormFwd &a, hipStream_t s) {
  const int vpt = norm_vpt(a.d), nt = row_threads(a.d, vpt);
  const int grid = a.rows < 8192 ? a.rows : 8192;
  auto go = [&](auto V) {
    k_norm_fwd<T, YT, decltype(V)::value><<<grid, nt, 0, s>>>((const T *)a.x, a.ldx, (const T *)a.res, a.ldr, a.w, a.b,
                                                              a.rows, a.d, a.eps, (YT *)a.y, (T *)a.s, a.mean, a.rstd);
  };
  if (vpt == 1) go(std::integral_constant<int, 1>());
  else go(std::integral_constant<int, 2>());
  return hipGetLastError();
}

template <typename T, typename DYT, typename DXT>
hipError_t norm_bwd(const NormBwd &a, hipStream_t s) {
  const int vpt = norm_vpt(a.d), nt = row_threads(a.d, vpt), P = norm_bwd_strips(a.rows, a.d);
  auto go = [&](auto V) {
    k_norm_bwd<T, DYT, DXT, decltype(V)::value><<<P, nt, 0, s>>>(
        (const DYT *)a.dy, a.lddy, (const T *)a.s, a.lds, a.w, a.mean, a.rstd, (const DXT *)a.dres, a.lddr, a.rows, a.d,
        (DXT *)a.dx, a.dw, a.db, a.part);
  };
  if (vpt == 1) go(std::integral_constant<int, 1>());
  else go(std::integral_constant<int, 2>());
  TW_TRY_HIP(hipGetLastError());
  if (P == 1) return hipSuccess;
  k_norm_bwd_sum<<<(2 * a.d + 31) / 32, 1024, 0, s>>>(a.part, P, a.d, a.dw, a.db);
  return hipGetLastError();
}

}  // namespace

// Workgroups of the backward, each with its partial sums: one for a few rows (their sums then
// need no second launch), one per row up to 512 (two per CU); beyond, one for eight rows as long as
// all fit the GPU at 1024 threads per CU, at least 512. With 512 for every d, T = 16384 and d = 64
// took 38.6 us, now 14.9; more at large d would add to the partial sums' traffic, and 256 for rows
// of more than 512 threads leaves loads waiting (T = 4000, d = 12288: 151 us against 126).
int norm_bwd_strips(int rows, int d) {
  if (rows <= 512) return rows <= 4 ? 1 : rows;
  const int most = 256 * 1024 / row_threads(d, norm_vpt(d)), p = rows / 8 < most ? rows / 8 : most;
  return p > 512 ? p : 512;
}

hipError_t launch_norm_fwd(const NormFwd &a, hipStream_t s) {
  if (a.x_bf16) return a.y_bf16 ? norm_fwd<uint16_t, uint16_t>(a, s) : norm_fwd<uint16_t, float>(a, s);
  return a.y_bf16 ? norm_fwd<float, uint16_t>(a, s) : norm_fwd<float, float>(a, s);
}

hipError_t launch_norm_bwd(const NormBwd &a, hipStream_t s) {
  auto dx = [&](auto X, auto DY) {
    typedef decltype(X) XT;
    typedef decltype(DY) DYT;
    return a.dx_bf16 ? norm_bwd<XT, DYT, uint16_t>(a, s) : norm_bwd<XT, DYT, float>(a, s);
  };
  if (a.x_bf16) return a.dy_bf16 ? dx(uint16_t(), uint16_t()) : dx(uint16_t(), float());
  return a.dy_bf16 ? dx(float(), uint16_t()) : dx(float(), float());
}

}  // namespace tw
