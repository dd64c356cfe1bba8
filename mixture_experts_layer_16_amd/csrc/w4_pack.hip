// 4-bit weights: quantisation, packing of given codes, and the values back.
//
// One wavefront per tile (w4.h); lane l owns row l%16 and, for i = 0..3, the eight
// columns i*32 + (l/16)*8, which is both a 16-byte load of bf16 weights and one
// packed word.  A group's largest magnitude is then a maximum over the four lanes of
// a row (two shuffles) and, for groups of 64 or 128, over the lane's own words.
#include "common.h"
#include "kernels.h"
#include "rows.h"
#include "w4.h"

namespace moe {

namespace {

__device__ __forceinline__ uint32_t pack8(const int* q) {
  uint32_t u = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) u |= (uint32_t)q[2 * j] << (4 * j) | (uint32_t)q[2 * j + 1] << (4 * j + 16);
  return u;
}
__device__ __forceinline__ int code_at(uint32_t u, int c) { return (int)(u >> (4 * (c >> 1) + 16 * (c & 1))) & 15; }

__device__ __forceinline__ float scale_f32(uint16_t s) { return __uint_as_float((uint32_t)s << 16); }

// Round w/s to the nearest integer, halves to even, from the exact quotient: the
// rounded quotient decides first, and where it came to lie on the wrong side of a
// half the remainder w - q s (exact in one fused step: q has 4 bits, s 8) says so.
__device__ __forceinline__ float round_quotient(float w, float s) {
  float q = rintf(w / s);
  const float r = fmaf(-q, s, w);
  if (2.f * fabsf(r) > s) q += r > 0.f ? 1.f : -1.f;
  return q;
}

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

// s = bf16(max|w| / 7), q = rint(w / s) + 8 clamped to 0..15; a group whose scale is 0
// has code 8 throughout.  Reads 2 or 4 bytes and writes half a byte a weight.
template <typename T, int GPT>
__global__ __launch_bounds__(256) void w4_quantize_kernel(int64_t tiles, int R, int C, int RT, int KT, int NG,
                                                          const T* __restrict__ w, uint32_t* __restrict__ codes,
                                                          bf16* __restrict__ scales) {
  const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (tile >= tiles) return;
  const int lane = threadIdx.x & 63, quad = lane >> 4;
  const TileAt at = tile_at(tile, RT, KT);
  const int row = at.rt * kW4Rows + (lane & 15), c0 = at.kt * kW4Cols + quad * 8;
  const T* src = w + (at.mat * R + row) * (int64_t)C + c0;
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (row < R && c0 + i * 32 < C) {
      load8(src + i * 32, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
  float amax[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[i][j]));
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
  for (int i = 0; i < 4; ++i) {
    const bf16 sb = from_f32<bf16>(amax[i] / 7.f);
    const float s = to_f32(sb);
    int q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      q[j] = s > 0.f ? 8 + (int)fminf(fmaxf(round_quotient(v[i][j], s), -8.f), 7.f) : 8;
    words[i] = pack8(q);
    if (quad == 0 && i % (4 / GPT) == 0)
      scales[scale_slot(at.mat, RT, at.rt, NG, lane, at.kt * GPT + i / (4 / GPT))] = sb;
  }
  clear_padding<GPT>(scales, at.mat, RT, at.rt, KT, at.kt, NG, lane);
  *reinterpret_cast<u32x4*>(codes + (tile * 64 + lane) * 4) = words;
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
  const int64_t tiles = n * RT * KT;
  const dim3 grid((unsigned)((tiles + 3) / 4)), block(256);
  by_group(group, [&](auto gpt) {
    constexpr int G = decltype(gpt)::value;
    if (dtype == 1)
      hipLaunchKernelGGL((w4_quantize_kernel<bf16, G>), grid, block, 0, stream, tiles, (int)R, (int)C, RT, KT, w4_row_scales(C, group),
                         (const bf16*)w, (uint32_t*)codes, (bf16*)scales);
    else
      hipLaunchKernelGGL((w4_quantize_kernel<float, G>), grid, block, 0, stream, tiles, (int)R, (int)C, RT, KT, w4_row_scales(C, group),
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
