// Products of few rows with 4-bit weights (w4.h): y[r] = W[e] x[r] for the rows r of
// expert e, plain or as the gate/up pair of a SwiGLU expert.
//
// With few rows an expert the time is the weights' bytes.  A wavefront streams tiles
// of 16 weight rows x 128 columns; the weights are the A operand of 16x16x32 bf16
// MFMAs and up to 16 token rows the B operand, so one pass over the weights serves
// 16 rows.  Per code there is then no multiply on the vector unit, only the unpacking:
//
//   a bf16 with exponent 2^p holds p' = 7 fraction bits, so OR-ing a 4-bit code into
//   its fraction adds the code in steps of 2^(p - 7 + bit): 0x4300 | q = 128 + q and,
//   with the code three bits higher, 0x4180 | q << 3 = 16 + q.  One shift and one
//   and-or make two operands (v_and_or_b32).
//
// The offsets (136 or 24 with the code's own 8) are taken out by the matrix unit too:
// a group's accumulators start at (-136 | -24) . x, one MFMA with a constant A operand
// shared by every tile of the wavefront, instead of at zero.  What is then left per
// group is total += s * acc, one FMA a result.  All sums are float32.
//
// B operands are bf16 planes whose sum is the float32 activation: one plane for bf16
// activations, three for float32 ones (24 bits), two for the hidden activations of a
// bf16 expert, which so keep 16 bits instead of being rounded to 8 between the two
// products (the weight stream, not the MFMAs, is what bounds the kernel).
//
// The wavefronts of a workgroup split the columns and add their totals in LDS in a
// fixed order; there are no atomics, results are bit-reproducible.
#include "common.h"
#include "kernels.h"
#include "tile_walk.h"
#include "w4.h"

namespace moe {

namespace {

constexpr int kWaves = 4;      // wavefronts of a workgroup, each a share of the columns
constexpr int kDepth = 3;      // column tiles a wavefront has in flight
constexpr int kTok = 16;       // token rows of a workgroup

struct W4Args {
  const bf16* x;               // [planes][n_in, C]
  int64_t x_plane;             // elements between planes
  int64_t n_in;
  const int32_t* a_rows;       // row r reads x[a_rows[r]], or nullptr
  const int32_t* offsets;      // [E + 1] device, or nullptr: rows 0 .. n_max-1 of one matrix
  int64_t n_max;
  int E, C, R, KT, RT;
  const uint32_t* codes[2];
  const uint16_t* scales[2];
  void* y;                     // [n_max, R], or bf16 planes [planes][n_max, R]
  int64_t y_plane;
};

struct TokenTile {
  int e;                       // expert, or -1: no such tile
  int64_t row0;
  int rows;                    // 1 .. kTok
};

// The slot-th tile of kTok rows over the experts' segments (tile_walk.h's bounds: the
// offsets are not trusted).  Every wavefront scans for itself: 64 experts a step, a
// running maximum and a running sum over the lanes.
__device__ __forceinline__ TokenTile find_tile(const int32_t* offsets, int E, int64_t n_max, int slot) {
  const int lane = threadIdx.x & 63;
  int prev = offsets[0];
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int top = e < E ? offsets[e + 1] : prev;
    top = top > prev ? top : prev;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(top, o, 64);
      if (lane >= o && v > top) top = v;
    }
    int below = __shfl_up(top, 1, 64);
    if (lane == 0) below = prev;
    const int hi = (int)clamp64(top, 0, n_max), lo = (int)clamp64(below, 0, n_max);
    int sum = e < E ? (hi - lo + kTok - 1) / kTok : 0;
    const int own = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(sum, o, 64);
      if (lane >= o) sum += v;
    }
    const unsigned long long past = __ballot(base + sum > slot);
    if (past != 0) {
      const int src = __ffsll(past) - 1;
      const int t = slot - base - __shfl(sum - own, src, 64);
      const int l = __shfl(lo, src, 64), h = __shfl(hi, src, 64);
      const int left = h - l - t * kTok;
      return {e0 + src, (int64_t)l + (int64_t)t * kTok, left < kTok ? left : kTok};
    }
    base += __shfl(sum, 63, 64);
    prev = __shfl(top, 63, 64);
  }
  return {-1, 0, 0};
}

// Eight codes -> eight bf16: 128 + q in elements 0 and 1, 16 + q in the others; FINE:
// 16 + q throughout (one shift more; the smaller offset keeps four times less rounding
// of the group sums, which float32 results show and bf16 ones do not).
template <bool FINE> __device__ __forceinline__ bf16x8 unpack(uint32_t u) {
  u32x4 v;
  v[0] = FINE ? ((u << 3) & 0x00780078u) | 0x41804180u : (u & 0x000f000fu) | 0x43004300u;
  v[1] = ((u >> 1) & 0x00780078u) | 0x41804180u;
  v[2] = ((u >> 5) & 0x00780078u) | 0x41804180u;
  v[3] = ((u >> 9) & 0x00780078u) | 0x41804180u;
  return __builtin_bit_cast(bf16x8, v);
}
template <bool FINE> __device__ __forceinline__ bf16x8 offset_operand() {
  constexpr uint32_t m136 = 0xc308c308u, m24 = 0xc1c0c1c0u;   // -136, -24 in both halves
  const u32x4 v = {FINE ? m24 : m136, m24, m24, m24};
  return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// GPT scales of four rows each
template <int GPT> struct Scales {
  uint2 v[GPT];
};

// PLANES bf16 planes of x; GPT groups a tile; SWIGLU: the two streams are the same
// rows of the gate and up matrices and y gets silu(g) * u in OUT planes; otherwise
// they are two adjacent row tiles of one matrix and y gets the products as TO.
template <int PLANES, int GPT, bool SWIGLU, int OUT, typename TO>
__global__ __launch_bounds__(64 * kWaves) void w4_matvec_kernel(W4Args a) {
  __shared__ float red[kWaves][2][16][kTok + 1];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int col = lane & 15, quad = lane >> 4;
  constexpr bool FINE = PLANES == 3;

  TokenTile tt;
  if (a.offsets) {
    tt = find_tile(a.offsets, a.E, a.n_max, (int)blockIdx.y);
    if (tt.e < 0) return;
  } else {
    const int64_t r0 = (int64_t)blockIdx.y * kTok, left = a.n_max - r0;
    tt = {0, r0, left < kTok ? (int)left : kTok};
  }
  const int e = __builtin_amdgcn_readfirstlane(tt.e), rows = __builtin_amdgcn_readfirstlane(tt.rows);
  const int64_t row0 = tt.row0;

  // the streams' row tiles; a second tile past the matrix reads the first again and is not stored
  const int rt0 = SWIGLU ? (int)blockIdx.x : 2 * (int)blockIdx.x;
  const int rt1 = SWIGLU ? rt0 : (rt0 + 1 < a.RT ? rt0 + 1 : rt0);
  const int64_t t0 = ((int64_t)e * a.RT + rt0) * a.KT, t1 = ((int64_t)e * a.RT + rt1) * a.KT;
  const uint32_t* codes[2] = {a.codes[0] + t0 * 256 + lane * 4, a.codes[SWIGLU ? 1 : 0] + t1 * 256 + lane * 4};
  const uint16_t* scales[2] = {a.scales[0] + t0 * (16 * GPT) + quad * (4 * GPT),
                               a.scales[SWIGLU ? 1 : 0] + t1 * (16 * GPT) + quad * (4 * GPT)};
  // lanes past the last row repeat it: a column of the result depends on its own column of B only
  const int64_t r = row0 + (col < rows ? col : rows - 1);
  const int64_t src = a.a_rows ? clamp_row(a.a_rows[r], a.n_in) : r;
  const bf16* x = a.x + src * (int64_t)a.C + quad * 8;

  f32x4 total[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  const bf16x8 minus = offset_operand<FINE>();
  for (int k0 = wave; k0 < a.KT; k0 += kWaves * kDepth) {
    u32x4 w[kDepth][2];
    Scales<GPT> s[kDepth][2];
    bf16x8 b[kDepth][PLANES][4];
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      const int kt = k0 + u * kWaves < a.KT ? k0 + u * kWaves : k0;
#pragma unroll
      for (int n = 0; n < 2; ++n) w[u][n] = *reinterpret_cast<const u32x4*>(codes[n] + (int64_t)kt * 256);
    }
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      const int kt = k0 + u * kWaves < a.KT ? k0 + u * kWaves : k0;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int g = 0; g < GPT; ++g)
          s[u][n].v[g] = *reinterpret_cast<const uint2*>(scales[n] + (int64_t)kt * (16 * GPT) + g * 4);
#pragma unroll
      for (int p = 0; p < PLANES; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // columns past the row: any in-bounds value; their scale is 0 or their MFMA is skipped
          const int c = kt * kW4Cols + i * 32 < a.C ? kt * kW4Cols + i * 32 : 0;
          b[u][p][i] = *reinterpret_cast<const bf16x8*>(x + p * a.x_plane + c);
        }
    }
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      const int kt = k0 + u * kWaves;
      if (kt >= a.KT) break;
#pragma unroll
      for (int g = 0; g < GPT; ++g) {
        constexpr int M = 4 / GPT;      // MFMAs of a group
        f32x4 c0 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const int i = g * M + m;
          if (kt * kW4Cols + i * 32 >= a.C) break;
#pragma unroll
          for (int p = 0; p < PLANES; ++p) c0 = mfma(minus, b[u][p][i], c0);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          f32x4 acc = c0;
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const int i = g * M + m;
            if (kt * kW4Cols + i * 32 >= a.C) break;
            const bf16x8 wf = unpack<FINE>(w[u][n][i]);
#pragma unroll
            for (int p = 0; p < PLANES; ++p) acc = mfma(wf, b[u][p][i], acc);
          }
          const uint2 sv = s[u][n].v[g];
          total[n][0] = fmaf(__uint_as_float(sv.x << 16), acc[0], total[n][0]);
          total[n][1] = fmaf(__uint_as_float(sv.x & 0xffff0000u), acc[1], total[n][1]);
          total[n][2] = fmaf(__uint_as_float(sv.y << 16), acc[2], total[n][2]);
          total[n][3] = fmaf(__uint_as_float(sv.y & 0xffff0000u), acc[3], total[n][3]);
        }
      }
    }
  }

#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][n][quad * 4 + i][col] = total[n][i];
  __syncthreads();

  const int ro = tid & 15, tok = tid >> 4;      // one result (of each stream) a thread
  float v[2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    v[n] = red[0][n][ro][tok];
#pragma unroll
    for (int q = 1; q < kWaves; ++q) v[n] += red[q][n][ro][tok];
  }
  if (tok >= rows) return;
  if constexpr (SWIGLU) {
    const int f = rt0 * kW4Rows + ro;
    if (f >= a.R) return;
    float h = v[0] / (1.f + expf(-v[0])) * v[1];
    bf16* y = static_cast<bf16*>(a.y) + (row0 + tok) * (int64_t)a.R + f;
#pragma unroll
    for (int p = 0; p < OUT; ++p) {
      const bf16 part = from_f32<bf16>(h);
      y[p * a.y_plane] = part;
      h -= to_f32(part);
    }
  } else {
    TO* y = static_cast<TO*>(a.y) + (row0 + tok) * (int64_t)a.R;
    const int n0 = rt0 * kW4Rows + ro, n1 = (rt0 + 1) * kW4Rows + ro;
    if (n0 < a.R) y[n0] = from_f32<TO>(v[0]);
    if (n1 < a.R) y[n1] = from_f32<TO>(v[1]);
  }
}

// float32 x as three bf16 planes that sum to it (24 bits)
__global__ __launch_bounds__(256) void split3_kernel(int64_t n, const float* __restrict__ x, bf16* __restrict__ p) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const f32x4 v = *reinterpret_cast<const f32x4*>(x + i);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float h = v[j];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const bf16 part = from_f32<bf16>(h);
      p[q * n + i + j] = part;
      h -= to_f32(part);
    }
  }
}

template <int PLANES, bool SWIGLU, int OUT, typename TO>
hipError_t launch(const W4Args& a, int group, int64_t token_tiles, hipStream_t stream) {
  const dim3 grid((unsigned)(SWIGLU ? a.RT : (a.RT + 1) / 2), (unsigned)token_tiles), block(64 * kWaves);
  if (group == 32)
    hipLaunchKernelGGL((w4_matvec_kernel<PLANES, 4, SWIGLU, OUT, TO>), grid, block, 0, stream, a);
  else if (group == 64)
    hipLaunchKernelGGL((w4_matvec_kernel<PLANES, 2, SWIGLU, OUT, TO>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((w4_matvec_kernel<PLANES, 1, SWIGLU, OUT, TO>), grid, block, 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_split3(int64_t n, const void* x, void* planes, hipStream_t stream) {
  hipLaunchKernelGGL(split3_kernel, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, stream, n, (const float*)x,
                     (bf16*)planes);
  return hipGetLastError();
}

}  // namespace

int64_t w4_token_tiles(int64_t n_max, int64_t E) {
  // each expert with rows has one last, perhaps partial tile
  return n_max / kTok + (n_max < E ? n_max : E);
}

hipError_t launch_w4_matvec(int dtype, int64_t T, int64_t C, int64_t R, int group, const void* x, const void* codes,
                            const void* scales, void* y, void* x_planes, hipStream_t stream) {
  W4Args a{};
  a.n_in = a.n_max = T;
  a.E = 1;
  a.C = (int)C; a.R = (int)R; a.KT = (int)w4_col_tiles(C); a.RT = (int)w4_row_tiles(R);
  a.codes[0] = (const uint32_t*)codes; a.scales[0] = (const uint16_t*)scales;
  a.y = y;
  const int64_t tiles = (T + kTok - 1) / kTok;
  if (dtype == 1) {
    a.x = (const bf16*)x;
    return launch<1, false, 1, bf16>(a, group, tiles, stream);
  }
  hipError_t err = launch_split3(T * C, x, x_planes, stream);
  if (err != hipSuccess) return err;
  a.x = (const bf16*)x_planes;
  a.x_plane = T * C;
  return launch<3, false, 1, float>(a, group, tiles, stream);
}

hipError_t launch_w4_grouped_ffn(int dtype, int64_t n_max, int64_t d, int64_t E, int64_t F, int group, const void* x,
                                 int64_t n_in, const int32_t* a_rows, const int32_t* offsets, const void* const* codes,
                                 const void* const* scales, void* y_perm, void* x_planes, void* h_planes,
                                 hipStream_t stream) {
  const int64_t tiles = w4_token_tiles(n_max, E);
  W4Args g{};
  g.n_in = n_in; g.a_rows = a_rows; g.offsets = offsets; g.n_max = n_max;
  g.E = (int)E;
  g.C = (int)d; g.R = (int)F; g.KT = (int)w4_col_tiles(d); g.RT = (int)w4_row_tiles(F);
  for (int n = 0; n < 2; ++n) { g.codes[n] = (const uint32_t*)codes[n]; g.scales[n] = (const uint16_t*)scales[n]; }
  g.y = h_planes;
  g.y_plane = n_max * F;
  W4Args w = g;
  w.x = (const bf16*)h_planes;
  w.x_plane = n_max * F;
  w.n_in = n_max; w.a_rows = nullptr;
  w.C = (int)F; w.R = (int)d; w.KT = (int)w4_col_tiles(F); w.RT = (int)w4_row_tiles(d);
  w.codes[0] = (const uint32_t*)codes[2]; w.scales[0] = (const uint16_t*)scales[2];
  w.y = y_perm;
  hipError_t err;
  if (dtype == 1) {
    g.x = (const bf16*)x;
    if ((err = launch<1, true, 2, bf16>(g, group, tiles, stream)) != hipSuccess) return err;
    return launch<2, false, 1, bf16>(w, group, tiles, stream);
  }
  if ((err = launch_split3(n_in * d, x, x_planes, stream)) != hipSuccess) return err;
  g.x = (const bf16*)x_planes;
  g.x_plane = n_in * d;
  if ((err = launch<3, true, 3, bf16>(g, group, tiles, stream)) != hipSuccess) return err;
  return launch<3, false, 1, float>(w, group, tiles, stream);
}

}  // namespace moe
