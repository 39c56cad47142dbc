// The global L2 norm of many gradient tensors and clipping by it, on gfx950.
//
//   n = sqrt(sum over all tensors of g^2);  c = min(1, max_norm / (n + 1e-6));  out = c g
//
// Bound by HBM: the norm reads every gradient once, the clip reads and writes it once more. The
// tensors are cut into chunks of one size; a workgroup finds its chunk's tensor in a table that
// travels in the kernel arguments (no device copy of pointers, so a call can be captured), and
// takes every gridDim.x-th chunk. Squares are summed in fp64: an fp32 square overflows from
// 1.8e19 on and vanishes below 1e-23, and the conversions cost less than the loads. A workgroup's
// sum goes to its own place in the workspace, and the places are added in one fixed order, so
// the norm has the same bits on every call.
#include "common.h"
#include "launch.h"
#include "row8.h"

namespace tw {
namespace {

constexpr int kNT = 256;
constexpr int kGridMax = 2048;              // workgroups of a launch (8 per CU)
constexpr float kClipEps = 1e-6f;

struct Table {
  int n;                                    // tensors
  int chunk;                                // elements of a chunk, a multiple of 8 kNT
  uint32_t first[kGradTab + 1];             // first chunk of each tensor
  int64_t len[kGradTab];
  const void *g[kGradTab];
  void *out[kGradTab];
  uint8_t bf16[kGradTab], out_bf16[kGradTab], vec[kGradTab];
};

TW_DEV int tensor_of(const Table &t, uint32_t chunk) {
  int lo = 0, hi = t.n;                     // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The workgroup's sum of v, in thread 0 (fixed order).
TW_DEV double block_sum64(double v, double *red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

template <typename T> TW_DEV void sum_chunk(const T *g, int n, bool vec, double &acc) {
  if (vec) {
    const int n8 = n & ~7;
    for (int i = threadIdx.x * 8; i < n8; i += kNT * 8) {
      float v[8];
      load8(g + i, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc = fma((double)v[k], (double)v[k], acc);
    }
    for (int i = n8 + threadIdx.x; i < n; i += kNT) {
      const double v = Elem<T>::load(g, i);
      acc = fma(v, v, acc);
    }
  } else {
    for (int i = threadIdx.x; i < n; i += kNT) {
      const double v = Elem<T>::load(g, i);
      acc = fma(v, v, acc);
    }
  }
}

__global__ __launch_bounds__(kNT) void k_grad_sq(Table t, double *__restrict__ part) {
  __shared__ double red[4];
  double acc = 0.0;
  const uint32_t total = t.first[t.n];
  for (uint32_t c = blockIdx.x; c < total; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = (int64_t)(c - t.first[i]) * t.chunk;
    const int n = (int)(t.len[i] - at < t.chunk ? t.len[i] - at : t.chunk);
    if (t.bf16[i]) sum_chunk((const uint16_t *)t.g[i] + at, n, t.vec[i], acc);
    else sum_chunk((const float *)t.g[i] + at, n, t.vec[i], acc);
  }
  const double s = block_sum64(acc, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// sqrt of the sum of the n partial sums, in every thread.
TW_DEV float total_norm(const double *part, int n, double *red) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += kNT) v += part[i];
  return (float)sqrt(block_sum64(v, red));
}

__global__ __launch_bounds__(kNT) void k_grad_norm(const double *__restrict__ part, int n, float *__restrict__ norm) {
  __shared__ double red[4];
  const float v = total_norm(part, n, red);
  if (threadIdx.x == 0) *norm = v;
}

template <typename T, typename OT> TW_DEV void scale_chunk(const T *g, OT *o, int n, bool vec, float c) {
  if (vec) {
    const int n8 = n & ~7;
    for (int i = threadIdx.x * 8; i < n8; i += kNT * 8) {
      float v[8];
      load8(g + i, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= c;
      store8(o + i, v);
    }
    for (int i = n8 + threadIdx.x; i < n; i += kNT) store1(o + i, Elem<T>::load(g, i) * c);
  } else {
    for (int i = threadIdx.x; i < n; i += kNT) store1(o + i, Elem<T>::load(g, i) * c);
  }
}

// Every workgroup adds the partial sums itself (a few KB from L2), which saves a launch between
// the sums and the scaling.
__global__ __launch_bounds__(kNT) void k_grad_scale(Table t, const double *__restrict__ part, int n, float max_norm,
                                                    float *__restrict__ norm) {
  __shared__ double red[4];
  const float nv = total_norm(part, n, red);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = nv;
  float c = max_norm / (nv + kClipEps);
  c = c > 1.f ? 1.f : c;                    // a NaN stays one
  const uint32_t total = t.first[t.n];
  for (uint32_t b = blockIdx.x; b < total; b += gridDim.x) {
    // backwards: what the sums read last is still in the last-level cache (537 MB of fp32
    // gradients, sums and scaling: 302 us, forwards 317)
    const uint32_t k = total - 1 - b;
    const int i = tensor_of(t, k);
    if (c == 1.f && t.out[i] == t.g[i]) continue;      // in place and below the limit
    const int64_t at = (int64_t)(k - t.first[i]) * t.chunk;
    const int m = (int)(t.len[i] - at < t.chunk ? t.len[i] - at : t.chunk);
    const float *gf = (const float *)t.g[i] + at;
    const uint16_t *gb = (const uint16_t *)t.g[i] + at;
    float *of = (float *)t.out[i] + at;
    uint16_t *ob = (uint16_t *)t.out[i] + at;
    if (t.bf16[i]) {
      if (t.out_bf16[i]) scale_chunk(gb, ob, m, t.vec[i], c);
      else scale_chunk(gb, of, m, t.vec[i], c);
    } else {
      if (t.out_bf16[i]) scale_chunk(gf, ob, m, t.vec[i], c);
      else scale_chunk(gf, of, m, t.vec[i], c);
    }
  }
}

// Elements per chunk: 2048 (one vector per thread) as long as the launch has workgroups for
// every chunk, up to 16384 for large sets.
int chunk_of(int64_t total) {
  int c = 8 * kNT;
  while (c < 8 * 8 * kNT && total > (int64_t)c * kGridMax) c *= 2;
  return c;
}

// Fills t with tensors [from, from + kGradTab) and returns the workgroups to launch.
int fill(Table &t, const GradArgs &a, int from, int chunk) {
  t.n = 0;
  t.chunk = chunk;
  uint32_t first = 0;
  for (int i = from; i < a.n && i < from + kGradTab; ++i) {
    if (a.len[i] == 0) continue;
    const int k = t.n++;
    t.first[k] = first;
    first += (uint32_t)((a.len[i] + chunk - 1) / chunk);
    t.len[k] = a.len[i];
    t.g[k] = a.g[i];
    t.out[k] = a.out ? a.out[i] : nullptr;
    t.bf16[k] = a.dtype[i] != 0;
    t.out_bf16[k] = a.out_dtype ? a.out_dtype[i] != 0 : 0;
    t.vec[k] = (((uintptr_t)t.g[k] | (uintptr_t)t.out[k]) & 15) == 0;
  }
  t.first[t.n] = first;
  return first < (uint32_t)kGridMax ? (int)first : kGridMax;
}

int64_t elements(const GradArgs &a) {
  int64_t n = 0;
  for (int i = 0; i < a.n; ++i) n += a.len[i];
  return n;
}

}  // namespace

// Bytes of the partial sums: one per workgroup of each table's launch.
size_t grad_workspace_bytes(int n) { return (size_t)((n + kGradTab - 1) / kGradTab) * kGridMax * sizeof(double); }

hipError_t launch_grad(const GradArgs &a, hipStream_t s) {
  const int chunk = chunk_of(elements(a));
  int parts = 0;
  Table t;
  for (int from = 0; from < a.n; from += kGradTab) {
    const int grid = fill(t, a, from, chunk);
    if (!grid) continue;
    k_grad_sq<<<grid, kNT, 0, s>>>(t, a.part + parts);
    TW_TRY_HIP(hipGetLastError());
    parts += grid;
  }
  if (!a.out || parts == 0) {
    k_grad_norm<<<1, kNT, 0, s>>>(a.part, parts, a.norm);
    return hipGetLastError();
  }
  float *norm = a.norm;
  for (int from = (a.n - 1) / kGradTab * kGradTab; from >= 0; from -= kGradTab) {
    const int grid = fill(t, a, from, chunk);
    if (!grid) continue;
    k_grad_scale<<<grid, kNT, 0, s>>>(t, a.part, parts, a.max_norm, norm);
    TW_TRY_HIP(hipGetLastError());
    norm = nullptr;
  }
  return hipSuccess;
}

}  // namespace tw
