// 4-bit weights: quantisation, packing of given codes, and the values back.
//
// Wavefronts work on tiles (w4.h); lane l owns row l%16 and, for i = 0..3, the eight
// columns i*32 + (l/16)*8, which is both a 16-byte load of bf16 weights and one
// packed word.  A group's largest magnitude is then a maximum over the four lanes of
// a row (two shuffles) and, for groups of 64 or 128, over the lane's own words.
#include "common.h"
#include "kernels.h"
#include "rows.h"
#include "w4.h"

namespace moe {

namespace {

// Eight codes (their low four bits) as a packed word.
__device__ __forceinline__ uint32_t pack8(const int* q) {
  uint32_t u = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    u |= (__builtin_amdgcn_perm((uint32_t)q[2 * j + 1], (uint32_t)q[2 * j], 0x05040100u) & 0x000f000fu) << (4 * j);
  return u;
}
__device__ __forceinline__ int code_at(uint32_t u, int c) { return (int)(u >> (4 * (c >> 1) + 16 * (c & 1))) & 15; }

__device__ __forceinline__ float scale_f32(uint16_t s) { return __uint_as_float((uint32_t)s << 16); }

// 8 + w/s rounded to the nearest integer, halves to even, from the exact quotient (a division
// a weight took 52 us for four experts' 6,144 x 1,792 bf16 weights; the first way below 33, the second 26).
//
// The product with the rounded reciprocal is at most one off, and the remainder w - q s
// (exact in one fused step: q has 4 bits, s 8) says where.  Groups of tiny weights are
// scaled up first, so that the reciprocal is finite.
struct Quotient {
  float up, s, inv;
  __device__ __forceinline__ explicit Quotient(float scale) {
    const bool some = scale > 0.f;             // scale 0: every quotient 0
    up = some ? (scale < 0x1p-60f ? 0x1p64f : 1.f) : 0.f;
    s = some ? scale * up : 1.f;
    inv = some ? 1.f / s : 0.f;
  }
  __device__ __forceinline__ int operator()(float w) const {
    w *= up;
    const float n = rintf(w * inv);
    const float r = fmaf(-n, s, w), over = fmaf(2.f, fabsf(r), -s);
    // past the half (over's bits are then a positive integer), or on it (zero) with an odd n: one further
    const int q = (int)n, on = (__float_as_int(r) >> 31) | 1;
    const int to = q + (__float_as_int(over) + (q & 1) > 0 ? on : 0);
    return 8 + (to < -8 ? -8 : to > 7 ? 7 : to);
  }
};
// bf16 weights whose scale is a normal number: both are whole numbers below 2^8 times powers of two,
// so a quotient that is not on a half is at least 2^-14 of itself away from one.  Rounded
// 2^-18 below and above it, it gives the same integer twice, or the two next to the half:
// then the even one.  (Adding 1.5 * 2^23 + 8 rounds to an integer, which the sum's low bits hold.)
struct NearQuotient {
  float below, above;
  __device__ __forceinline__ explicit NearQuotient(float scale) {
    const float inv = scale > 0.f ? 1.f / scale : 0.f;
    below = inv * (1.f - 0x1p-18f);
    above = inv * (1.f + 0x1p-18f);
  }
  __device__ __forceinline__ int operator()(float w) const {
    const int a = __float_as_int(fmaf(w, below, 12582920.f)), b = __float_as_int(fmaf(w, above, 12582920.f));
    const int odd = (a << 31) >> 31;
    return (b & odd) | (a & ~odd);
  }
};

// Where the scale of row l%16 and group g of a tile's row tile lies.  The wavefront of the
// last column tile also clears what pads the row.
__device__ __forceinline__ int64_t scale_slot(int64_t mat, int RT, int rt, int NG, int lane, int g) {
  return ((mat * RT + rt) * 16 + (lane & 15)) * NG + g;
}
template <int GPT>
__device__ __forceinline__ void clear_padding(bf16* scales, int64_t mat, int RT, int rt, int KT, int kt, int NG, int lane) {
  if (kt != KT - 1 || lane >= 16) return;
  for (int g = KT * GPT; g < NG; ++g) scales[scale_slot(mat, RT, rt, NG, lane, g)] = from_f32<bf16>(0.f);
}

struct TileAt {
  int64_t mat;     // matrix
  int rt, kt;      // tile in it
};
__device__ __forceinline__ TileAt tile_at(int64_t tile, int RT, int KT) {
  const int64_t per = (int64_t)RT * KT, m = tile / per;
  const int l = (int)(tile - m * per);
  return {m, l / KT, l % KT};
}

// s = bf16(max|w| * (1/7 in float32)), q = rint(w / s) + 8 clamped to 0..15; a group whose scale is 0
// has code 8 throughout.  Reads 2 or 4 bytes and writes half a byte a weight.  A wavefront
// takes two column tiles of a row tile: eight loads in flight (four tiles: 57.7 us for the
// round trip of four experts against 54.0, and 14.4 against 10.1 for one small matrix).
constexpr int kTurn = 2;
template <typename T, int GPT>
__global__ __launch_bounds__(256) void w4_quantize_kernel(int64_t turns, int R, int C, int RT, int KT, int NG,
                                                          const T* __restrict__ w, uint32_t* __restrict__ codes,
                                                          bf16* __restrict__ scales) {
  const int64_t turn = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (turn >= turns) return;
  const int lane = threadIdx.x & 63, quad = lane >> 4;
  const TileAt at = tile_at(turn, RT, (KT + kTurn - 1) / kTurn);
  const int row = at.rt * kW4Rows + (lane & 15), k0 = at.kt * kTurn, c0 = k0 * kW4Cols + quad * 8;
  const T* src = w + (at.mat * R + row) * (int64_t)C + c0;
  Row8<T> v[kTurn][4];
#pragma unroll
  for (int u = 0; u < kTurn; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[u][i] = {};
      if (row < R && c0 + u * kW4Cols + i * 32 < C) load_row8<true>(v[u][i], src + u * kW4Cols + i * 32);
    }
  bf16 scale[kTurn * GPT];
  u32x4* dst = reinterpret_cast<u32x4*>(codes + (((at.mat * RT + at.rt) * KT + k0) * 64 + lane) * 4);
#pragma unroll
  for (int u = 0; u < kTurn; ++u) {
    float amax[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[u][i].get(j)));
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      amax[i] = fmaxf(m, __shfl_xor(m, 32, 64));
    }
    if (GPT <= 2) {
      amax[0] = amax[1] = fmaxf(amax[0], amax[1]);
      amax[2] = amax[3] = fmaxf(amax[2], amax[3]);
    }
    if (GPT == 1) amax[0] = amax[1] = amax[2] = amax[3] = fmaxf(amax[0], amax[2]);
    u32x4 words;
#pragma unroll
    for (int g = 0; g < GPT; ++g) {
      const bf16 sb = from_f32<bf16>(amax[g * (4 / GPT)] * (1.f / 7.f));
      scale[u * GPT + g] = sb;
      auto round = [&](auto quotient) {
#pragma unroll
        for (int i = g * (4 / GPT); i < (g + 1) * (4 / GPT); ++i) {
          int q[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) q[j] = quotient(v[u][i].get(j));
          words[i] = pack8(q);
        }
      };
      const float s = to_f32(sb);
      if (sizeof(T) == 2 && !__any(s < 0x1p-120f && amax[g * (4 / GPT)] > 0.f)) round(NearQuotient(s));
      else round(Quotient(s));
    }
    if (k0 + u < KT) dst[u * 64] = words;
  }
  // what pads the row is zero: its columns were
  if (quad == 0) {
    bf16* to = scales + scale_slot(at.mat, RT, at.rt, NG, lane, k0 * GPT);
#pragma unroll
    for (int g = 0; g < kTurn * GPT; g += 2)   // (NG is a multiple of four)
      if (k0 * GPT + g < NG) {
        typedef __attribute__((__vector_size__(2 * sizeof(bf16)))) bf16 bf16x2;
        *reinterpret_cast<bf16x2*>(to + g) = bf16x2{scale[g], scale[g + 1]};
      }
    if (kTurn * GPT == 2 && k0 + kTurn >= KT && (k0 * GPT) % 4 == 0 && k0 * GPT + 2 < NG)
      *reinterpret_cast<uint32_t*>(to + 2) = 0u;              // the row's padding that no turn covers
  }
}

// Codes given row by row (two a byte, the even column in the low half) and scales
// [R, ceil(C/group)].
template <int GPT>
__global__ __launch_bounds__(256) void w4_pack_kernel(int64_t tiles, int R, int C, int RT, int KT, int NG,
                                                      const uint8_t* __restrict__ q, const bf16* __restrict__ s,
                                                      uint32_t* __restrict__ codes, bf16* __restrict__ scales) {
  const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (tile >= tiles) return;
  const int lane = threadIdx.x & 63, quad = lane >> 4;
  const TileAt at = tile_at(tile, RT, KT);
  const int row = at.rt * kW4Rows + (lane & 15), c0 = at.kt * kW4Cols + quad * 8;
  constexpr int group = kW4Cols / GPT;
  const int ng = (C + group - 1) / group;
  u32x4 words;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u = 0x88888888u;
    if (row < R && c0 + i * 32 < C) {
      const uint32_t b = *reinterpret_cast<const uint32_t*>(q + ((at.mat * R + row) * (int64_t)C + c0 + i * 32) / 2);
      int qs[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) qs[j] = (int)(b >> (4 * j)) & 15;
      u = pack8(qs);
    }
    words[i] = u;
    if (quad == 0 && i % (4 / GPT) == 0) {
      const int g = at.kt * GPT + i / (4 / GPT);
      scales[scale_slot(at.mat, RT, at.rt, NG, lane, g)] =
          row < R && g < ng ? s[(at.mat * R + row) * (int64_t)ng + g] : from_f32<bf16>(0.f);
    }
  }
  clear_padding<GPT>(scales, at.mat, RT, at.rt, KT, at.kt, NG, lane);
  *reinterpret_cast<u32x4*>(codes + (tile * 64 + lane) * 4) = words;
}

// w = s (q - 8): exact in float32 (12 bits), rounded once for bf16.
template <typename T, int GPT>
__global__ __launch_bounds__(256) void w4_dequantize_kernel(int64_t tiles, int R, int C, int RT, int KT, int NG,
                                                            const uint32_t* __restrict__ codes,
                                                            const uint16_t* __restrict__ scales, T* __restrict__ w) {
  const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (tile >= tiles) return;
  const int lane = threadIdx.x & 63, quad = lane >> 4;
  const TileAt at = tile_at(tile, RT, KT);
  const int row = at.rt * kW4Rows + (lane & 15), c0 = at.kt * kW4Cols + quad * 8;
  const u32x4 words = *reinterpret_cast<const u32x4*>(codes + (tile * 64 + lane) * 4);
  T* dst = w + (at.mat * R + row) * (int64_t)C + c0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (row >= R || c0 + i * 32 >= C) continue;
    const float s = scale_f32(scales[scale_slot(at.mat, RT, at.rt, NG, lane, at.kt * GPT + i / (4 / GPT))]);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = s * (float)(code_at(words[i], j) - 8);
    store8(dst + i * 32, v);
  }
}

template <typename F> void by_group(int group, F f) {
  if (group == 32) f(std::integral_constant<int, 4>{});
  else if (group == 64) f(std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 1>{});
}

}  // namespace

hipError_t launch_w4_quantize(int dtype, int64_t n, int64_t R, int64_t C, int group, const void* w, void* codes,
                              void* scales, hipStream_t stream) {
  const int RT = (int)w4_row_tiles(R), KT = (int)w4_col_tiles(C);
  const int64_t turns = n * RT * ((KT + kTurn - 1) / kTurn);
  const dim3 grid((unsigned)((turns + 3) / 4)), block(256);
  by_group(group, [&](auto gpt) {
    constexpr int G = decltype(gpt)::value;
    if (dtype == 1)
      hipLaunchKernelGGL((w4_quantize_kernel<bf16, G>), grid, block, 0, stream, turns, (int)R, (int)C, RT, KT, w4_row_scales(C, group),
                         (const bf16*)w, (uint32_t*)codes, (bf16*)scales);
    else
      hipLaunchKernelGGL((w4_quantize_kernel<float, G>), grid, block, 0, stream, turns, (int)R, (int)C, RT, KT, w4_row_scales(C, group),
                         (const float*)w, (uint32_t*)codes, (bf16*)scales);
  });
  return hipGetLastError();
}

hipError_t launch_w4_pack(int64_t n, int64_t R, int64_t C, int group, const void* q, const void* s, void* codes,
                          void* scales, hipStream_t stream) {
  const int RT = (int)w4_row_tiles(R), KT = (int)w4_col_tiles(C);
  const int64_t tiles = n * RT * KT;
  const dim3 grid((unsigned)((tiles + 3) / 4)), block(256);
  by_group(group, [&](auto gpt) {
    hipLaunchKernelGGL((w4_pack_kernel<decltype(gpt)::value>), grid, block, 0, stream, tiles, (int)R, (int)C, RT, KT, w4_row_scales(C, group),
                       (const uint8_t*)q, (const bf16*)s, (uint32_t*)codes, (bf16*)scales);
  });
  return hipGetLastError();
}

hipError_t launch_w4_dequantize(int dtype, int64_t n, int64_t R, int64_t C, int group, const void* codes,
                                const void* scales, void* w, hipStream_t stream) {
  const int RT = (int)w4_row_tiles(R), KT = (int)w4_col_tiles(C);
  const int64_t tiles = n * RT * KT;
  const dim3 grid((unsigned)((tiles + 3) / 4)), block(256);
  by_group(group, [&](auto gpt) {
    constexpr int G = decltype(gpt)::value;
    if (dtype == 1)
      hipLaunchKernelGGL((w4_dequantize_kernel<bf16, G>), grid, block, 0, stream, tiles, (int)R, (int)C, RT, KT, w4_row_scales(C, group),
                         (const uint32_t*)codes, (const uint16_t*)scales, (bf16*)w);
    else
      hipLaunchKernelGGL((w4_dequantize_kernel<float, G>), grid, block, 0, stream, tiles, (int)R, (int)C, RT, KT, w4_row_scales(C, group),
                         (const uint32_t*)codes, (const uint16_t*)scales, (float*)w);
  });
  return hipGetLastError();
}

}  // namespace moe
