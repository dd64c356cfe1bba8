// Row helpers of the bandwidth-bound token kernels: 8 consecutive elements of a
// row moved between memory (16 bytes of bf16 or 32 bytes of float32, aligned)
// and float32 registers.
#pragma once

#include "common.h"

namespace moe {

// 8 consecutive elements kept as loaded (one or two 16-byte loads) and converted
// element by element where they are used: half the registers of a float32 copy
// for 16-bit rows, so more row loads fit in flight.
template <typename T> struct Raw16;
template <> struct Raw16<bf16> {
  typedef bf16x8 type;
  __device__ __forceinline__ static type load(const bf16* p) { return *reinterpret_cast<const bf16x8*>(p); }
  __device__ __forceinline__ static float get(const type& v, int i) { return static_cast<float>(v[i]); }
};
template <> struct Raw16<float> {
  struct type { f32x4 a, b; };
  __device__ __forceinline__ static type load(const float* p) {
    return {*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4)};
  }
  __device__ __forceinline__ static float get(const type& v, int i) { return i < 4 ? v.a[i] : v.b[i - 4]; }
};

__device__ __forceinline__ void load8(const bf16* p, float* v) {
  const bf16x8 q = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(q[i]);
}
__device__ __forceinline__ void store8(bf16* p, const float* v) {
  bf16x8 q;
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = static_cast<bf16>(v[i]);
  *reinterpret_cast<bf16x8*>(p) = q;
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p);
  const f32x4 b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[i + 4] = b[i]; }
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  f32x4 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) { a[i] = v[i]; b[i] = v[i + 4]; }
  *reinterpret_cast<f32x4*>(p) = a;
  *reinterpret_cast<f32x4*>(p + 4) = b;
}

// Eight elements as loaded, in whole registers (a vector of 16-bit values that lives across a
// loop's turns is taken apart into one register a value).
template <typename T> struct Row8;
template <> struct Row8<bf16> {
  u32x4 v;
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i & 1 ? v[i >> 1] & 0xffff0000u : v[i >> 1] << 16);
  }
  // as if newly loaded: values converted before are not kept
  __device__ __forceinline__ void renew() { asm volatile("" : "+v"(v)); }
};
template <> struct Row8<float> {
  f32x4 a, b;
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i] : b[i - 4]; }
  __device__ __forceinline__ void renew() {}
};

// Loads and stores of them; NT: past the caches, for rows that are read or written once and
// are too many to be found in a cache again.
template <bool NT> __device__ __forceinline__ void load_row8(Row8<bf16>& q, const bf16* p) {
  const u32x4* s = reinterpret_cast<const u32x4*>(p);
  if constexpr (NT) q.v = __builtin_nontemporal_load(s);
  else q.v = *s;
}
template <bool NT> __device__ __forceinline__ void load_row8(Row8<float>& q, const float* p) {
  const f32x4* s = reinterpret_cast<const f32x4*>(p);
  if constexpr (NT) q = {__builtin_nontemporal_load(s), __builtin_nontemporal_load(s + 1)};
  else q = {s[0], s[1]};
}
template <bool NT> __device__ __forceinline__ void store_row8(bf16* p, const float* v) {
  if constexpr (NT) {
    bf16x8 q;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = static_cast<bf16>(v[i]);
    __builtin_nontemporal_store(q, reinterpret_cast<bf16x8*>(p));
  } else {
    store8(p, v);
  }
}
template <bool NT> __device__ __forceinline__ void store_row8(float* p, const float* v) {
  if constexpr (NT) {
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(p));
    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, reinterpret_cast<f32x4*>(p + 4));
  } else {
    store8(p, v);
  }
}

// Sum over the 64 lanes of a wavefront; every lane ends with the same bits.
__device__ __forceinline__ float wave_sum64(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// The same sum in registers only: shifts inside each row of 16 lanes, then the rows' totals
// passed on to the last lane, and from there to all (in a scalar register).  Six steps of a few
// cycles, where a step through the LDS crossbar takes some sixty.
__device__ __forceinline__ float wave_total(float v) {
#define MOE_SUM_STEP(ctrl, rows) \
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, rows, 0xf, false))
  MOE_SUM_STEP(0x111, 0xf);   // row_shr:1
  MOE_SUM_STEP(0x112, 0xf);   // row_shr:2
  MOE_SUM_STEP(0x114, 0xf);   // row_shr:4
  MOE_SUM_STEP(0x118, 0xf);   // row_shr:8
  MOE_SUM_STEP(0x142, 0xa);   // row_bcast:15
  MOE_SUM_STEP(0x143, 0xc);   // row_bcast:31
#undef MOE_SUM_STEP
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sums over LANES lanes next to one another (8, 16, 32: each such group its own, with the
// others' lanes on or off; 64: wave_total).  Each step adds a lane's mirror image, so all
// lanes end with the same bits.
template <int LANES> __device__ __forceinline__ float lanes_total(float v) {
  if constexpr (LANES == 64) {
    return wave_total(v);
  } else {
#define MOE_SUM_STEP(ctrl) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, false))
    MOE_SUM_STEP(0xb1);                          // quad_perm 1,0,3,2
    MOE_SUM_STEP(0x4e);                          // quad_perm 2,3,0,1
    MOE_SUM_STEP(0x141);                         // row_half_mirror: the eight lanes' two quads
    if (LANES > 8) MOE_SUM_STEP(0x140);          // row_mirror: the sixteen's two halves
#undef MOE_SUM_STEP
    if (LANES > 16) v += __shfl_xor(v, 16, 64);
    return v;
  }
}

}  // namespace moe
