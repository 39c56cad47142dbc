// Rows in units of 8 elements (16 bytes of bf16, 32 of fp32), widened to fp32 and rounded back.
// The rounding is v_cvt_pk_bf16_f32's: to nearest even, infinities and NaN kept as such.
#pragma once
#include "common.h"

namespace tw {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

TW_DEV uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)a, (__bf16)b});
}

TW_DEV void load8(const uint16_t *p, float (&o)[8]) { Vec16<uint16_t>::load(p, o); }
TW_DEV void load8(const float *p, float (&o)[8]) {
  const float4 a = *(const float4 *)p, b = *(const float4 *)(p + 4);
  o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
  o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
}

// The same 8 elements as loaded, widened later: a load in flight then takes 4 registers of bf16.
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> {
  uint4 u;
  TW_DEV void load(const uint16_t *p) { u = *(const uint4 *)p; }
  TW_DEV void to(float (&o)[8]) const { Vec16<uint16_t>::load((const uint16_t *)&u, o); }
};
template <> struct Raw8<float> {
  float4 a, b;
  TW_DEV void load(const float *p) {
    a = *(const float4 *)p;
    b = *(const float4 *)(p + 4);
  }
  TW_DEV void to(float (&o)[8]) const {
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  }
};

// Nontemporal: outputs that the writing kernel never reads again.
TW_DEV void store8(float *p, const float (&v)[8]) {
  __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, (f32x4_t *)p);
  __builtin_nontemporal_store(f32x4_t{v[4], v[5], v[6], v[7]}, (f32x4_t *)(p + 4));
}
TW_DEV void store8(uint16_t *p, const float (&v)[8]) {
  __builtin_nontemporal_store(u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                      pack_bf16(v[6], v[7])},
                              (u32x4_t *)p);
}

TW_DEV void store1(float *p, float v) { *p = v; }
TW_DEV void store1(uint16_t *p, float v) { *p = (uint16_t)pack_bf16(v, 0.f); }

// v as T stores it
template <typename T> TW_DEV float rounded(float v) {
  if constexpr (std::is_same<T, float>::value) return v;
  else return __uint_as_float(pack_bf16(0.f, v) & 0xFFFF0000u);
}

}  // namespace tw
