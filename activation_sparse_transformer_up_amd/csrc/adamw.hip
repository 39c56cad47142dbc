// The AdamW step over many tensors, states in 32 or in 8 bits, on gfx950.
//
//   g' = c g,  c = min(1, max_norm / (norm + 1e-6)) where a norm is given
//   m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Bound by HBM: p, g, m and v are read once, p, m, v (and a bf16 copy of p) written once, 28 bytes per
// element in 32 bits, 14 with 8-bit states and bf16 gradients. As for the gradient norm, the tensors are
// cut into chunks of one size, a workgroup finds its chunk's tensor in a table that travels in the kernel
// arguments, and takes every gridDim.x-th chunk. A thread takes 8 neighbouring elements.
//
// The 8-bit states: a block of 256 elements, 32 lanes, shares a scale s = (largest of the block) / (top
// code's value).
//   m = q |q| s, q in -127 .. 127;  v = q^4 s, q in 0 .. 255
// Roots, not straight steps: the square keeps m's relative error at 1 / q and sqrt(v)'s, by which m is
// divided, at 1 / q as well, down to 2^-16 of the block's largest. A v above zero takes q = 1 at
// least: it may come back larger, which shortens the step, but never as zero under an m that is not. A scale
// is at least 2^-126, so its reciprocal is finite.
// The step itself uses the unrounded m and v; only what is kept for the next one is rounded. Products
// and sums are rounded one by one (no contraction), so that codes, which one last bit may move over a
// border, do not depend on the compiler.
#include "common.h"
#include "launch.h"
#include "row8.h"

namespace tw {
namespace {

constexpr int kNT = 256;
constexpr int kGridMax = 2048;              // workgroups of a launch (8 per CU)
constexpr float kClipEps = 1e-6f;
constexpr float kTiny = 0x1p-126f;
constexpr double kMaxRate = 1e30;           // as the host's check of lr
constexpr float kStepM = (float)(1.0 / 16129.0), kStepV = (float)(1.0 / 4228250625.0);    // 127^-2, 255^-4

struct Table {
  int n;                                    // tensors
  int chunk;                                // elements of a chunk, a multiple of 8 kNT
  uint32_t first[kAdamTab + 1];             // first chunk of each tensor
  int64_t len[kAdamTab];
  void *p[kAdamTab], *m[kAdamTab], *v[kAdamTab], *copy[kAdamTab];
  const void *g[kAdamTab];
  float *ms[kAdamTab], *vs[kAdamTab];
  double decay[kAdamTab];
  uint8_t p_bf16[kAdamTab], g_bf16[kAdamTab], vec[kAdamTab];
};
static_assert(sizeof(Table) < 3600, "kernel arguments");

// The step's factors, each rounded once from 64 bits.
struct Hyper {
  double lr, beta1, beta2, eps;
  int64_t step;
  const float *lr_dev;
  const int64_t *step_dev;
  const float *norm;
  float max_norm;
  // from the host where lr and step are, else made by every workgroup
  float root2, rate;                        // 1 / sqrt(1 - b2^t), lr / (1 - b1^t)
};

template <typename TAB> TW_DEV int tensor_of(const TAB &t, uint32_t chunk) {
  int lo = 0, hi = t.n;                     // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

TW_DEV double pow_int(double b, int64_t n) {
  double r = 1.0;
  for (; n > 0; n >>= 1) {
    if (n & 1) r *= b;
    b *= b;
  }
  return r;
}

// 8 elements at i of n (beyond them zeros), whole vectors where vec.
template <typename T> TW_DEV void get8(const T *p, int i, int n, bool vec, float (&o)[8]) {
  if (vec && i + 8 <= n) {
    load8(p + i, o);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = i + k < n ? Elem<T>::load(p, i + k) : 0.f;
  }
}
template <typename T> TW_DEV void put8(T *p, int i, int n, bool vec, const float (&v)[8]) {
  if (vec && i + 8 <= n) {
    store8(p + i, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) store1(p + i + k, v[k]);
  }
}
// The same for codes, one byte each.
TW_DEV uint2 get_codes(const uint8_t *p, int i, int n, bool vec) {
  if (vec && i + 8 <= n) return *(const uint2 *)(p + i);
  uint2 u = make_uint2(0, 0);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (i + k < n) (k < 4 ? u.x : u.y) |= (uint32_t)p[i + k] << (8 * (k & 3));
  return u;
}
TW_DEV void put_codes(uint8_t *p, int i, int n, bool vec, uint2 u) {
  if (vec && i + 8 <= n) {
    *(uint2 *)(p + i) = u;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) p[i + k] = (uint8_t)((k < 4 ? u.x : u.y) >> (8 * (k & 3)));
  }
}
TW_DEV uint32_t byte_of(uint2 u, int k) { return ((k < 4 ? u.x : u.y) >> (8 * (k & 3))) & 0xFFu; }

TW_DEV float value_m(uint2 u, int k, float s) {
#pragma clang fp contract(off)
  const float q = (float)(int8_t)byte_of(u, k);
  return q * fabsf(q) * s;
}
TW_DEV float value_v(uint2 u, int k, float s) {
#pragma clang fp contract(off)
  const float q = (float)byte_of(u, k), q2 = q * q;
  return q2 * q2 * s;
}

// The scale of a block of 32 lanes' 8 values each, the largest magnitude times k. Magnitudes are
// compared as their bits, by which a NaN is above all.
TW_DEV float block_scale(const float (&x)[8], float k) {
  uint32_t b = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) b = max(b, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) b = max(b, (uint32_t)__shfl_xor((int)b, o, 64));
  const float s = __uint_as_float(b) * k;
  return s < kTiny ? kTiny : s;
}

// q[i] = rint(sqrt(t[i])), FOURTH: rint(sqrt(sqrt(t[i]))), of correctly rounded roots (t up to 255^4). The
// hardware's root is off by an ulp, 2^-14 of a code after two: only lanes with a root that close to a border between
// two codes take their roots again. Correct roots throughout, and a quotient for the step, made the step of 366M
// elements wait for its arithmetic: 1344 us, with hardware roots 1170.
template <bool FOURTH> TW_DEV void codes_of(const float (&t)[8], float (&q)[8]) {
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a = __builtin_amdgcn_sqrtf(t[i]);
    if constexpr (FOURTH) a = __builtin_amdgcn_sqrtf(a);
    q[i] = rintf(a);
    far = fmaxf(far, fabsf(a - q[i]));
  }
  if (far > 0.4999f)
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = rintf(FOURTH ? sqrtf(sqrtf(t[i])) : sqrtf(t[i]));
}

// The low bytes of four numbers.
TW_DEV uint32_t bytes4(int a, int b, int c, int d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400u), __builtin_amdgcn_perm(b, a, 0x0c0c0400u), 0x05040100u);
}

// eps from which FAST takes m / (sqrt(v) r + eps) with the hardware's root and reciprocal, 8 2^-24 at most off
// (below, the root of a tiny v, which the hardware may flush, would count); 8-bit states only: with fp32 ones
// the step waits for HBM either way.
constexpr double kFastEps = 1e-12;

template <typename PT, typename GT, bool EIGHT, bool FAST>
TW_DEV void step_chunk(const Table &t, int i, int64_t at, int n, float c, bool clip, const Hyper &h, float keep, float root2,
                       float rate) {
#pragma clang fp contract(off)
  const bool vec = t.vec[i];
  PT *p = (PT *)t.p[i] + at;
  const GT *g = (const GT *)t.g[i] + at;
  uint16_t *copy = t.copy[i] ? (uint16_t *)t.copy[i] + at : nullptr;
  const float b1 = (float)h.beta1, a1 = (float)(1.0 - h.beta1), b2 = (float)h.beta2, a2 = (float)(1.0 - h.beta2);
  const float eps = (float)h.eps;
  // whole blocks of threads, so that every lane of an 8-bit block takes part in its scale
  const int steps = (n + kNT * 8 - 1) / (kNT * 8);
  for (int k = 0; k < steps; ++k) {
    const int j = (k * kNT + threadIdx.x) * 8;
    float pv[8], gv[8], m[8], v[8];
    get8(p, j, n, vec, pv);
    get8(g, j, n, vec, gv);
    const int64_t blk = (at + j) / kAdamBlock;
    if constexpr (EIGHT) {
      const uint2 qm = get_codes((const uint8_t *)t.m[i] + at, j, n, vec), qv = get_codes((const uint8_t *)t.v[i] + at, j, n, vec);
      const float sm = j < n ? t.ms[i][blk] : 0.f, sv = j < n ? t.vs[i][blk] : 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m[e] = value_m(qm, e, sm);
        v[e] = value_v(qv, e, sv);
      }
    } else {
      get8((const float *)t.m[i] + at, j, n, vec, m);
      get8((const float *)t.v[i] + at, j, n, vec, v);
    }
    if (clip)
#pragma unroll
      for (int e = 0; e < 8; ++e) gv[e] *= c;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = gv[e];
      m[e] = m[e] * b1 + x * a1;
      v[e] = v[e] * b2 + x * x * a2;
      float d;
      if constexpr (FAST) d = m[e] * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(v[e]) * root2 + eps);
      else d = m[e] / (sqrtf(v[e]) * root2 + eps);
      pv[e] = pv[e] * keep - d * rate;
    }
    if (j + 8 > n)                          // elements that are not the tensor's are not of the block
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e >= n) m[e] = v[e] = 0.f;
    put8(p, j, n, vec, pv);
    if (copy) put8(copy, j, n, vec, pv);
    if constexpr (EIGHT) {
      const float sm = block_scale(m, kStepM), sv = block_scale(v, kStepV);
      const float im = 1.f / sm, iv = 1.f / sv;
      float r[8], q[8];
      int o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = fabsf(m[e]) * im;
      codes_of<false>(r, q);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = (int)copysignf(fminf(q[e], 127.f), m[e]);
      put_codes((uint8_t *)t.m[i] + at, j, n, vec, make_uint2(bytes4(o[0], o[1], o[2], o[3]), bytes4(o[4], o[5], o[6], o[7])));
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = v[e] * iv;
      codes_of<true>(r, q);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = (int)fminf(v[e] > 0.f ? fmaxf(q[e], 1.f) : q[e], 255.f);
      put_codes((uint8_t *)t.v[i] + at, j, n, vec, make_uint2(bytes4(o[0], o[1], o[2], o[3]), bytes4(o[4], o[5], o[6], o[7])));
      if ((threadIdx.x & 31) == 0 && j < n) {
        t.ms[i][blk] = sm;
        t.vs[i][blk] = sv;
      }
    } else {
      put8((float *)t.m[i] + at, j, n, vec, m);
      put8((float *)t.v[i] + at, j, n, vec, v);
    }
  }
}

template <bool EIGHT, bool FAST> __global__ __launch_bounds__(kNT) void k_adamw(Table t, Hyper h) {
#pragma clang fp contract(off)
  float c = 1.f;
  if (h.norm) {
    const float nv = *h.norm;
    if (!(nv >= 0.f && nv < INFINITY)) return;      // no step from gradients that overflowed
    c = h.max_norm / (nv + kClipEps);
    c = c > 1.f ? 1.f : c;
  }
  double lr = h.lr;
  float root2 = h.root2, rate = h.rate;
  if (h.lr_dev || h.step_dev) {
    if (h.lr_dev) lr = (double)*h.lr_dev;
    const int64_t step = h.step_dev ? *h.step_dev : h.step;
    if (!(lr >= 0.0 && lr <= kMaxRate) || step < 1) return;         // what the host refuses would spoil every parameter
    root2 = (float)(1.0 / sqrt(1.0 - pow_int(h.beta2, step)));
    rate = (float)(lr / (1.0 - pow_int(h.beta1, step)));
  }
  const uint32_t total = t.first[t.n];
  for (uint32_t b = blockIdx.x; b < total; b += gridDim.x) {
    const int i = tensor_of(t, b);
    const int64_t at = (int64_t)(b - t.first[i]) * t.chunk;
    const int n = (int)(t.len[i] - at < t.chunk ? t.len[i] - at : t.chunk);
    const float keep = (float)(1.0 - lr * t.decay[i]);
    const bool clip = h.norm != nullptr;
    if (t.p_bf16[i]) {
      if (t.g_bf16[i]) step_chunk<uint16_t, uint16_t, EIGHT, FAST>(t, i, at, n, c, clip, h, keep, root2, rate);
      else step_chunk<uint16_t, float, EIGHT, FAST>(t, i, at, n, c, clip, h, keep, root2, rate);
    } else {
      if (t.g_bf16[i]) step_chunk<float, uint16_t, EIGHT, FAST>(t, i, at, n, c, clip, h, keep, root2, rate);
      else step_chunk<float, float, EIGHT, FAST>(t, i, at, n, c, clip, h, keep, root2, rate);
    }
  }
}

struct ValueTable {
  int n, chunk;
  uint32_t first[kAdamTab + 1];
  int64_t len[kAdamTab];
  const uint8_t *q[kAdamTab];
  const float *s[kAdamTab];
  void *out[kAdamTab];
  uint8_t second[kAdamTab], vec[kAdamTab];
};

template <typename OT> __global__ __launch_bounds__(kNT) void k_adamw8_values(ValueTable t) {
  const uint32_t total = t.first[t.n];
  for (uint32_t b = blockIdx.x; b < total; b += gridDim.x) {
    const int i = tensor_of(t, b);
    const int64_t at = (int64_t)(b - t.first[i]) * t.chunk;
    const int n = (int)(t.len[i] - at < t.chunk ? t.len[i] - at : t.chunk);
    for (int j = threadIdx.x * 8; j < n; j += kNT * 8) {
      const uint2 u = get_codes(t.q[i] + at, j, n, t.vec[i]);
      const float s = t.s[i][(at + j) / kAdamBlock];
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = t.second[i] ? value_v(u, e, s) : value_m(u, e, s);
      put8((OT *)t.out[i] + at, j, n, t.vec[i], o);
    }
  }
}

// Elements per chunk: 2048 (one unit per thread) as long as the launch has workgroups for every
// chunk, up to 16384 for large sets.
int chunk_of(const int64_t *len, int n) {
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += len[i];
  int c = 8 * kNT;
  while (c < 8 * 8 * kNT && total > (int64_t)c * kGridMax) c *= 2;
  return c;
}

// Tensors [from, from + kAdamTab) of n: f(k, i) fills entry k from tensor i; returns the workgroups.
template <typename TAB, typename F> int fill(TAB &t, const int64_t *len, int n, int from, int chunk, F &&f) {
  t.n = 0;
  t.chunk = chunk;
  uint32_t first = 0;
  for (int i = from; i < n && i < from + kAdamTab; ++i) {
    if (len[i] == 0) continue;
    const int k = t.n++;
    t.first[k] = first;
    first += (uint32_t)((len[i] + chunk - 1) / chunk);
    t.len[k] = len[i];
    f(k, i);
  }
  t.first[t.n] = first;
  return first < (uint32_t)kGridMax ? (int)first : kGridMax;
}

}  // namespace

hipError_t launch_adamw(const AdamArgs &a, hipStream_t s) {
  Hyper h = {};
  h.lr = a.lr; h.beta1 = a.beta1; h.beta2 = a.beta2; h.eps = a.eps;
  h.step = a.step;
  h.lr_dev = a.lr_dev; h.step_dev = a.step_dev;
  h.norm = a.norm; h.max_norm = a.max_norm;
  if (!a.lr_dev && !a.step_dev) {
    h.root2 = (float)(1.0 / sqrt(1.0 - pow(a.beta2, (double)a.step)));
    h.rate = (float)(a.lr / (1.0 - pow(a.beta1, (double)a.step)));
  }
  const int chunk = chunk_of(a.len, a.n);
  Table t;
  for (int from = 0; from < a.n; from += kAdamTab) {
    const int grid = fill(t, a.len, a.n, from, chunk, [&](int k, int i) {
      t.p[k] = a.p[i]; t.g[k] = a.g[i]; t.m[k] = a.m[i]; t.v[k] = a.v[i];
      t.copy[k] = a.copy ? a.copy[i] : nullptr;
      t.ms[k] = a.eight ? a.ms[i] : nullptr;
      t.vs[k] = a.eight ? a.vs[i] : nullptr;
      t.decay[k] = a.decay[i];
      t.p_bf16[k] = a.p_dtype[i] != 0;
      t.g_bf16[k] = a.g_dtype[i] != 0;
      t.vec[k] = (((uintptr_t)t.p[k] | (uintptr_t)t.g[k] | (uintptr_t)t.copy[k] | (uintptr_t)t.m[k] | (uintptr_t)t.v[k]) & 15) == 0;
    });
    if (!grid) continue;
    if (!a.eight) k_adamw<false, false><<<grid, kNT, 0, s>>>(t, h);
    else if (a.eps >= kFastEps) k_adamw<true, true><<<grid, kNT, 0, s>>>(t, h);
    else k_adamw<true, false><<<grid, kNT, 0, s>>>(t, h);
    TW_TRY_HIP(hipGetLastError());
  }
  return hipSuccess;
}

hipError_t launch_adamw8_values(const AdamValuesArgs &a, hipStream_t s) {
  const int chunk = chunk_of(a.len, a.n);
  ValueTable t;
  for (int from = 0; from < a.n; from += kAdamTab) {
    const int grid = fill(t, a.len, a.n, from, chunk, [&](int k, int i) {
      t.q[k] = (const uint8_t *)a.codes[i];
      t.s[k] = a.scales[i];
      t.out[k] = a.out[i];
      t.second[k] = a.second[i] != 0;
      t.vec[k] = (((uintptr_t)t.q[k] | (uintptr_t)t.out[k]) & 15) == 0;
    });
    if (!grid) continue;
    if (a.out_bf16) k_adamw8_values<uint16_t><<<grid, kNT, 0, s>>>(t);
    else k_adamw8_values<float><<<grid, kNT, 0, s>>>(t);
    TW_TRY_HIP(hipGetLastError());
  }
  return hipSuccess;
}

}  // namespace tw
