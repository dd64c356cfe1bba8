// Products of few rows with 4-bit weights (w4.h): y[r] = W[e] x[r] for the rows r of
// expert e, plain or as the gate/up pair of a SwiGLU expert.
//
// With few rows an expert the time is the weights' bytes.  A wavefront streams tiles
// of 16 weight rows x 128 columns; up to 16 token rows are the A operand of 16x16x32 bf16
// MFMAs and the weights the B operand, so one pass over the weights serves 16 rows, and a
// lane's results all belong to one weight row: a group's scale is one number a lane.  Per
// code there is then no multiply on the vector unit, only the unpacking:
//
//   a bf16 with exponent 2^p holds 7 fraction bits, so OR-ing a 4-bit code into its
//   fraction adds the code in steps of 2^(p - 7 + bit): 0x4300 | q = 128 + q and, with
//   the code three bits higher, 0x4180 | q << 3 = 16 + q.  One shift and one and-or make
//   two operands (v_and_or_b32).
//
// The offsets (136 or 24 with the code's own 8) are taken out by the matrix unit too:
// a group's accumulators start at x . (-136 | -24), one MFMA with a constant B operand
// shared by every tile of the wavefront, instead of at zero.  What is then left per
// group is total += s * acc, one FMA a result.  All sums are float32.  Float32 results
// take codes without an offset instead (unpack_exact).
//
// A operands are bf16 planes whose sum is the float32 activation: one plane for bf16
// activations, three for float32 ones (24 bits), two for the hidden activations of a
// bf16 expert, which so keep 16 bits instead of being rounded to 8 between the two
// products (the weight stream, not the MFMAs, is what bounds the kernel).
//
// The wavefronts that share a tile split its columns and add their totals in LDS in a
// fixed order; there are no atomics, results are bit-reproducible.
#include "common.h"
#include "kernels.h"
#include "tile_walk.h"
#include "w4.h"

namespace moe {

namespace {

constexpr int kWaves = 4;      // wavefronts of a workgroup
constexpr int kTok = 16;       // token rows of an MFMA
constexpr int kStreamed = 2;   // weights pass through the caches without staying (nt)

struct W4Args {
  const bf16* x;               // [planes][n_in, C]
  int64_t n_in;
  const int32_t* a_rows;       // row r reads x[a_rows[r]], or nullptr
  const int32_t* offsets;      // [E + 1] device, or nullptr: rows 0 .. n_max-1 of one matrix
  int64_t n_max;
  int E, C, R, KT, RT, NG;     // NG: scales of a weight row, padded (w4.h)
  const uint32_t* codes[2];
  const uint16_t* scales[2];
  void* y;                     // [n_max, R], or bf16 planes [planes][n_max, R]
  int64_t y_plane;
};

struct TokenTile {
  int e;                       // expert, or -1: no such tile
  int row0, rows;              // rows: 1 .. kTok
};

// Inclusive scans over the 64 lanes in registers: shifts inside each row of 16 lanes,
// then the rows' last values passed on.
template <typename F> __device__ __forceinline__ int lane_scan(int v, int identity, F f) {
  v = f(v, __builtin_amdgcn_update_dpp(identity, v, 0x111, 0xf, 0xf, false));   // row_shr:1
  v = f(v, __builtin_amdgcn_update_dpp(identity, v, 0x112, 0xf, 0xf, false));   // row_shr:2
  v = f(v, __builtin_amdgcn_update_dpp(identity, v, 0x114, 0xf, 0xf, false));   // row_shr:4
  v = f(v, __builtin_amdgcn_update_dpp(identity, v, 0x118, 0xf, 0xf, false));   // row_shr:8
  v = f(v, __builtin_amdgcn_update_dpp(identity, v, 0x142, 0xa, 0xf, false));   // row_bcast:15
  v = f(v, __builtin_amdgcn_update_dpp(identity, v, 0x143, 0xc, 0xf, false));   // row_bcast:31
  return v;
}

// The slot-th tile of 16 rows over the experts' segments (tile_walk.h's bounds: the
// offsets are not trusted).  Every wavefront scans for itself, 64 experts a step: a
// running maximum of the offsets and a running sum of the experts' tiles.
__device__ __forceinline__ TokenTile find_tile(const int32_t* offsets, int E, int64_t n_max, int slot) {
  const int lane = threadIdx.x & 63;
  int prev = offsets[0], base = 0;
  int ahead = lane < E ? offsets[lane + 1] : 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    const int raw = e < E ? ahead : prev;
    if (e + 64 < E) ahead = offsets[e + 65];
    const int top = lane_scan(raw > prev ? raw : prev, INT32_MIN, [](int a, int b) { return a > b ? a : b; });
    int below = __shfl_up(top, 1, 64);
    if (lane == 0) below = prev;
    const int hi = (int)clamp64(top, 0, n_max), lo = (int)clamp64(below, 0, n_max);
    const int own = e < E ? (hi - lo + kTok - 1) / kTok : 0;
    const int sum = lane_scan(own, 0, [](int a, int b) { return a + b; });
    const unsigned long long past = __ballot(base + sum > slot);
    if (past != 0) {
      const int src = __ffsll(past) - 1;
      const int t = slot - base - (__builtin_amdgcn_readlane(sum, src) - __builtin_amdgcn_readlane(own, src));
      const int row0 = __builtin_amdgcn_readlane(lo, src) + t * kTok;
      const int left = __builtin_amdgcn_readlane(hi, src) - row0;
      return {e0 + src, row0, left < kTok ? left : kTok};
    }
    base += __builtin_amdgcn_readlane(sum, 63);
    prev = __builtin_amdgcn_readlane(top, 63);
  }
  return {-1, 0, 0};
}

// Eight codes -> eight bf16: 128 + q in elements 0 and 1, 16 + q in the others.  The
// constants are registers (as literals, of which an instruction holds one, each and-or
// became two instructions): the masks vector ones, the exponents scalar ones.
struct UnpackConstants {
  uint32_t mask0, mask3, exp7, exp4;
  __device__ __forceinline__ UnpackConstants() : mask0(0x000f000fu), mask3(0x00780078u), exp7(0x43004300u), exp4(0x41804180u) {
    asm("" : "+v"(mask0), "+v"(mask3), "+s"(exp7), "+s"(exp4));
  }
};
__device__ __forceinline__ bf16x8 unpack(uint32_t u, const UnpackConstants& k) {
  const u32x4 v = {(u & k.mask0) | k.exp7, ((u >> 1) & k.mask3) | k.exp4, ((u >> 5) & k.mask3) | k.exp4,
                   ((u >> 9) & k.mask3) | k.exp4};
  return __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ bf16x8 offset_operand() {
  constexpr uint32_t m136 = 0xc308c308u, m24 = 0xc1c0c1c0u;   // -136, -24 in both halves
  const u32x4 v = {m136, m24, m24, m24};
  return __builtin_bit_cast(bf16x8, v);
}

// The same without an offset, (q - 8) / 16 in every element, for float32 results: sums
// that carry an offset round to the offset's size, which bf16 results do not show.  (With
// 16 + q throughout, float32 products of 4,800 columns were off by 1.5e-6 of their norm;
// so by 1.4e-7, a plain float32 product by 5.6e-7, and as fast: 33 x 4096 x 4096 in 22.2 us
// against 21.7.)  v_cvt_off_f32_i4 takes a signed code, so q with its top bit the other
// way, to that sixteenth, whose high half is a bf16; the 16 is put back a group at a time.
__device__ __forceinline__ bf16x8 unpack_exact(uint32_t u) {
  u ^= 0x88888888u;
  u32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = __builtin_amdgcn_perm(__float_as_uint(__builtin_amdgcn_cvt_off_f32_i4((int)(u >> (4 * j + 16)))),
                                 __float_as_uint(__builtin_amdgcn_cvt_off_f32_i4((int)(u >> (4 * j)))), 0x07060302u);
  return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// A buffer whose loads at offsets of `bytes` and more give zero and touch no memory.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t bounded(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}
constexpr uint32_t kNowhere = 0xfffffff0u;   // an offset past every buffer
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t more) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, (int)more, 0));
}

// `bytes` (2, 4 or 8) at offset `at` of a buffer, in a pair of words
template <int BYTES> __device__ __forceinline__ uint2 load_scales(__amdgpu_buffer_rsrc_t r, int at) {
  if constexpr (BYTES == 8) return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0));
  else if constexpr (BYTES == 4) return uint2{__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0), 0u};
  else return uint2{(uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0), 0u};
}
__device__ __forceinline__ float scale_at(const uint2& v, int i) {
  const uint32_t u = i < 2 ? v.x : v.y;
  return __uint_as_float(i & 1 ? u & 0xffff0000u : u << 16);
}

// A wavefront's LDS accesses are carried out in order; this keeps the compiler to it.
__device__ __forceinline__ void lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
// How the planes of a tile's rows are laid over MFMA rows.  Where SLOT rows of each plane
// fit 16 together they share one MFMA (plane p of row r is MFMA row p * SLOT + r, and the
// planes' results are added at the end); with SLOT 16 each plane has MFMAs of its own, which
// follow one another into the same accumulators.  (Two tiles of 16 rows a wavefront, so
// that 17 to 32 rows unpack a weight once, measured no faster: 30.4 us against 27.7 for 96
// rows of a 6,144 x 6,144 matrix.)
template <int PLANES, int SLOT> struct Rows {
  static constexpr bool kPacked = PLANES * SLOT <= 16;
  static constexpr int kUnits = kPacked ? 1 : PLANES;         // load units of a column tile: planes that follow one another
  static constexpr int kGroups = kPacked ? PLANES * SLOT / 4 : 4;        // groups of four rows of a load unit
  static constexpr int kTile = kUnits * 4096;                 // LDS bytes of 128 columns
};

// Activations go through LDS: a lane's MFMA operand is 16 bytes of row lane%16, and loaded
// like that straight into registers every load instruction touches 64 separate pieces,
// which costs the address unit as much as 1 KB of weights (measured at 5 rows an expert:
// 210 us against 182 without these loads).  Instead a load takes 256 contiguous bytes of
// each of four rows, one write puts them down and four reads pick the operands up.  Piece j
// of row r lies at j ^ r, so that the 16 rows of a read are in 16 different bank groups.
template <int PLANES, int SLOT> struct RowLoads {
  using L = Rows<PLANES, SLOT>;
  static constexpr int RG = L::kGroups;
  __amdgpu_buffer_rsrc_t xr;
  uint32_t off[RG], last[RG];                  // in the last column tile, columns past the row are not there either
  uint32_t plane;                              // bytes between planes
  int put[RG], KT;
  // the rows' numbers; whoever comes next can be on its way before they arrive
  __device__ __forceinline__ RowLoads(const W4Args& a, int row0, int rows) : KT(a.KT) {
    const int quad = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      const int r = L::kPacked ? (g * 4 + quad) % SLOT : g * 4 + quad;
      off[g] = r < rows ? (a.a_rows ? a.a_rows[row0 + r] : row0 + r) : 0;
    }
  }
  __device__ __forceinline__ void place(const W4Args& a, int rows) {
    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const bool cut = (a.KT - 1) * kW4Cols + col * 8 >= a.C;
    plane = (uint32_t)a.n_in * (uint32_t)(a.C * 2);
    xr = bounded(a.x, plane * PLANES);
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      const int v = g * 4 + quad, r = L::kPacked ? v % SLOT : v;
      const uint32_t at = (uint32_t)clamp_row((int)off[g], a.n_in) * (uint32_t)(a.C * 2) + col * 16 +
                          (L::kPacked ? v / SLOT * plane : 0u);
      off[g] = r < rows ? at : kNowhere;       // rows that are not there load nothing, and so zeros
      last[g] = cut ? kNowhere : off[g];
      put[g] = v * 256 + ((col ^ v) * 16);
    }
  }
  // unit u of column tile k, clamped to the row's
  __device__ __forceinline__ void load(u32x4 (&x)[RG], int u, int k) const {
    const int kc = k < KT ? k : KT - 1;
#pragma unroll
    for (int g = 0; g < RG; ++g) x[g] = load16(xr, kc == KT - 1 ? last[g] : off[g], u * plane + kc * (kW4Cols * 2));
  }
  __device__ __forceinline__ void store(const u32x4 (&x)[RG], char* unit) const {
#pragma unroll
    for (int g = 0; g < RG; ++g) *reinterpret_cast<u32x4*>(unit + put[g]) = x[g];
  }
};

// One column tile of NT streams of weights against an LDS tile of rows.  s holds the scales
// of the streams' groups, this tile's from group s_at on.
template <int MP, bool EXACT, int GPT, int NT>
__device__ __forceinline__ void multiply_tile(const char* tile, const u32x4 (&w)[NT], const uint2 (&s)[NT], int s_at,
                                              bf16x8 minus, const UnpackConstants& consts, f32x4 (&total)[NT]) {
  constexpr int M = 4 / GPT;         // MFMAs of a group
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  bf16x8 b[MP][4];
#pragma unroll
  for (int p = 0; p < MP; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      b[p][i] = *reinterpret_cast<const bf16x8*>(tile + p * 4096 + col * 256 + (((i * 4 + quad) ^ col) * 16));
#pragma unroll
  for (int g = 0; g < GPT; ++g) {
    f32x4 c0 = {0.f, 0.f, 0.f, 0.f};
    if constexpr (!EXACT) {
#pragma unroll
      for (int i = g * M; i < (g + 1) * M; ++i)
#pragma unroll
        for (int p = 0; p < MP; ++p) c0 = mfma(b[p][i], minus, c0);
    }
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      f32x4 acc = c0;
#pragma unroll
      for (int i = g * M; i < (g + 1) * M; ++i) {
        const bf16x8 wf = EXACT ? unpack_exact(w[m][i]) : unpack(w[m][i], consts);
#pragma unroll
        for (int p = 0; p < MP; ++p) acc = mfma(b[p][i], wf, acc);
      }
      const float sc = scale_at(s[m], s_at + g);
#pragma unroll
      for (int i = 0; i < 4; ++i) total[m][i] = fmaf(sc, EXACT ? acc[i] * 16.f : acc[i], total[m][i]);
    }
  }
  // the sums are due here: moved behind the loop's other tiles they would keep every
  // group's accumulators alive
#pragma unroll
  for (int m = 0; m < NT; ++m) asm volatile("" : "+v"(total[m]));
}

// The buffers of one set of NT streams.  SWIGLU: row tiles of the gate and up matrices in
// turn; otherwise adjacent row tiles of one matrix.  A stream past the matrix has no bytes:
// it loads zeros, and its scales with them.
template <int NT, int GPT, bool SWIGLU> struct Streams {
  __amdgpu_buffer_rsrc_t codes[NT], scales[NT];
  int n, NG;
  // from column tile k0 on, n of them
  __device__ __forceinline__ Streams(const W4Args& a, int64_t e, int first, int k0, int n_) : n(n_), NG(a.NG) {
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      const int rt = first + (SWIGLU ? m / 2 : m), mat = SWIGLU ? m % 2 : 0;
      const bool in = rt < a.RT;
      const int64_t t = e * a.RT + (in ? rt : 0);
      codes[m] = bounded(a.codes[mat] + (t * a.KT + k0) * 256, in ? n * 1024 : 0);
      scales[m] = bounded(a.scales[mat] + t * 16 * NG + k0 * GPT, in ? (16 * NG - k0 * GPT) * 2 : 0);
    }
  }
  __device__ __forceinline__ void load(u32x4 (&w)[NT], int k) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int m = 0; m < NT; ++m)
      w[m] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(codes[m], lane * 16 + k * 1024, 0, kStreamed));
  }
  // of SB column tiles from k on; zeros past the n-th
  template <int SB> __device__ __forceinline__ void load_scales_of(uint2 (&s)[NT], int k) const {
    const int col = threadIdx.x & 15;
#pragma unroll
    for (int m = 0; m < NT; ++m)
      s[m] = load_scales<SB * GPT * 2>(scales[m], k < n ? col * (NG * 2) + k * (GPT * 2) : (int)kNowhere);
  }
};

// The products of a set of streams' n column tiles from k0 on, DEPTH of them in flight (a
// multiplication past the n-th adds zero: its scales are).
//
// SHARED: the workgroup's wavefronts go over the same columns, and each puts down one load
// unit of the next kWaves for all: a quarter of the loads, and one barrier for them (it waits
// for LDS only, the weights stay in flight).  Otherwise a wavefront has columns and LDS of
// its own.
template <int PLANES, int SLOT, int GPT, int NT, int DEPTH, bool SHARED, bool SWIGLU>
__device__ __forceinline__ void stream(const W4Args& a, const Streams<NT, GPT, SWIGLU>& from, int k0, int row0, int rows,
                                       char* lds, f32x4 (&total)[NT]) {
  using L = Rows<PLANES, SLOT>;
  constexpr bool EXACT = PLANES == 3;
  constexpr int SB = 4 / GPT < DEPTH ? 4 / GPT : DEPTH;       // column tiles of a scale load
  RowLoads<PLANES, SLOT> rl(a, row0, rows);
  const bf16x8 minus = offset_operand();
  const UnpackConstants consts;
  u32x4 w[DEPTH][NT];
  uint2 s[DEPTH / SB][NT];
  if constexpr (SHARED) {
    constexpr int CH = kWaves / L::kUnits, U = DEPTH > CH ? DEPTH : CH;     // column tiles of a chunk, of a turn
    static_assert(U % CH == 0 && U % DEPTH == 0);
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int tile = wave / L::kUnits, unit = wave % L::kUnits;
    u32x4 x[L::kGroups];
    auto put = [&](int half) {
      if (tile < CH) rl.store(x, lds + (half * CH + tile) * L::kTile + unit * 4096);
      lds_barrier();
    };
#pragma unroll
    for (int u = 0; u < DEPTH; ++u) {
      from.load(w[u], u);
      if (u % SB == 0) from.template load_scales_of<SB>(s[u / SB], u);
    }
    rl.place(a, rows);
    rl.load(x, unit, tile);
    put(0);
    int half = 0;
    for (int k = 0; k < from.n; k += U) {
#pragma unroll
      for (int v = 0; v < U; ++v) {
        const int u = v % DEPTH;
        if (v % CH == 0) rl.load(x, unit, k + v + CH + tile);
        multiply_tile<L::kUnits, EXACT, GPT, NT>(lds + (half * CH + v % CH) * L::kTile, w[u], s[u / SB], u % SB * GPT,
                                                minus, consts, total);
        from.load(w[u], k + v + DEPTH);
        if (u % SB == SB - 1) from.template load_scales_of<SB>(s[u / SB], k + v + 1 - SB + DEPTH);
        if (v % CH == CH - 1) put(half ^= 1);  // the other half was last read before the last barrier
        __builtin_amdgcn_sched_barrier(0);     // tiles interleaved by the scheduler need the registers of a whole turn
      }
    }
  } else {
    u32x4 x[DEPTH][L::kUnits][L::kGroups];
    auto load_x = [&](int u, int k) {
#pragma unroll
      for (int q = 0; q < L::kUnits; ++q) rl.load(x[u][q], q, k);
    };
#pragma unroll
    for (int u = 0; u < DEPTH; ++u) {
      from.load(w[u], u);
      if (u % SB == 0) from.template load_scales_of<SB>(s[u / SB], u);
    }
    rl.place(a, rows);
#pragma unroll
    for (int u = 0; u < DEPTH; ++u) load_x(u, k0 + u);
    for (int k = 0; k < from.n; k += DEPTH) {
#pragma unroll
      for (int u = 0; u < DEPTH; ++u) {
        lds_order();                           // the operands before these have been read
#pragma unroll
        for (int q = 0; q < L::kUnits; ++q) rl.store(x[u][q], lds + q * 4096);
        lds_order();
        multiply_tile<L::kUnits, EXACT, GPT, NT>(lds, w[u], s[u / SB], u % SB * GPT, minus, consts, total);
        from.load(w[u], k + u + DEPTH);
        load_x(u, k0 + k + u + DEPTH);
        if (u % SB == SB - 1) from.template load_scales_of<SB>(s[u / SB], k + u + 1 - SB + DEPTH);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // planes that shared MFMAs: their results are SLOT rows apart
  if constexpr (L::kPacked && PLANES > 1) {
    const int quad = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = quad * 4 < PLANES * SLOT ? total[m][i] : 0.f;
        if (SLOT == 4) v += __shfl_xor(v, 16, 64);
        if (PLANES * SLOT > 8) v += __shfl_xor(v, 32, 64);
        total[m][i] = v;
      }
  }
}

// The results of one set of streams and 16 token rows.
template <int NT, bool SWIGLU, int OUT, typename TO>
__device__ __forceinline__ void store_results(const W4Args& a, const f32x4 (&v)[NT], int first, int64_t row0, int rows) {
  constexpr int kRows = SWIGLU ? NT / 2 : NT;
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (quad * 4 + i >= rows) continue;
    const int64_t row = (row0 + quad * 4 + i) * a.R;
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
      const int f = (first + m) * kW4Rows + col;
      if (f >= a.R) continue;
      if constexpr (SWIGLU) {
        const float g = v[2 * m][i];
        float h = g / (1.f + expf(-g)) * v[2 * m + 1][i];
#pragma unroll
        for (int p = 0; p < OUT; ++p) {
          const bf16 part = from_f32<bf16>(h);
          static_cast<bf16*>(a.y)[p * a.y_plane + row + f] = part;
          h -= to_f32(part);
        }
      } else {
        static_cast<TO*>(a.y)[row + f] = from_f32<TO>(v[m][i]);
      }
    }
  }
}

// Up to 16 token rows a workgroup (blockIdx.y) and some of the weight rows: KS wavefronts
// share a set of NT streams, each a run of their column tiles.
template <int PLANES, int GPT, int KS, int NT, bool SWIGLU, int OUT, typename TO>
__global__ __launch_bounds__(64 * kWaves, 3) void w4_matvec_kernel(W4Args a) {
  constexpr bool kShared = KS == 1;
  constexpr int DEPTH = kShared || PLANES == 1 ? 4 : 2;       // private activations take registers ahead of time too
  constexpr int kRows = SWIGLU ? NT / 2 : NT;                 // row tiles of a set
  // LDS: two chunks of column tiles (at most kWaves load units each), or a column tile a wavefront
  constexpr int kTile = Rows<PLANES, 16>::kTile, kLds = (kShared ? 2 : PLANES) * kWaves * 4096;
  constexpr int kRed = KS > 1 ? kWaves * NT * 1024 : 0;
  __shared__ __attribute__((aligned(16))) char lds[kLds > kRed ? kLds : kRed];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;

  TokenTile tt;
  if (a.offsets) {
    tt = find_tile(a.offsets, a.E, a.n_max, (int)blockIdx.y);
    if (tt.e < 0) return;
  } else {
    const int r0 = (int)blockIdx.y * kTok, left = (int)a.n_max - r0;
    tt = {0, r0, left < kTok ? left : kTok};
  }
  const int64_t e = __builtin_amdgcn_readfirstlane(tt.e);
  const int row0 = __builtin_amdgcn_readfirstlane(tt.row0), rows = __builtin_amdgcn_readfirstlane(tt.rows);

  const int first = ((int)blockIdx.x * (kWaves / KS) + wave / KS) * kRows;      // row tile of stream 0
  // this wavefront's run of column tiles: whole scale loads
  constexpr int SB = 4 / GPT < DEPTH ? 4 / GPT : DEPTH;
  const int run = ((a.KT + KS - 1) / KS + SB - 1) / SB * SB, k0 = (wave % KS) * run;
  const int n = (!kShared && first >= a.RT) || k0 >= a.KT ? 0 : (a.KT - k0 < run ? a.KT - k0 : run);
  f32x4 total[NT];
#pragma unroll
  for (int m = 0; m < NT; ++m) total[m] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (n > 0) {
    const Streams<NT, GPT, SWIGLU> from(a, e, first, k0, n);
    char* mine = kShared ? lds : lds + wave * kTile;
    constexpr int kSlot8 = PLANES < 3 ? 8 : 16;
    if (rows <= 4) stream<PLANES, 4, GPT, NT, DEPTH, kShared>(a, from, k0, row0, rows, mine, total);
    else if (rows <= kSlot8) stream<PLANES, kSlot8, GPT, NT, DEPTH, kShared>(a, from, k0, row0, rows, mine, total);
    else stream<PLANES, 16, GPT, NT, DEPTH, kShared>(a, from, k0, row0, rows, mine, total);
  }

  if constexpr (KS > 1) {
    f32x4* red = reinterpret_cast<f32x4*>(lds);               // [wave][NT][lane]
    __syncthreads();
#pragma unroll
    for (int m = 0; m < NT; ++m) red[(wave * NT + m) * 64 + lane] = total[m];
    __syncthreads();
    if (wave % KS != 0) return;
#pragma unroll
    for (int q = 1; q < KS; ++q)
#pragma unroll
      for (int m = 0; m < NT; ++m) total[m] += red[((wave + q) * NT + m) * 64 + lane];
  }
  if (first < a.RT) store_results<NT, SWIGLU, OUT, TO>(a, total, first, row0, rows);
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

template <int PLANES, int GPT, int KS, int NT, bool SWIGLU, int OUT, typename TO>
void launch_one(const W4Args& a, hipStream_t stream, int64_t token_tiles) {
  const int per = kWaves / KS * (SWIGLU ? NT / 2 : NT);       // row tiles of a workgroup
  hipLaunchKernelGGL((w4_matvec_kernel<PLANES, GPT, KS, NT, SWIGLU, OUT, TO>),
                     dim3((unsigned)((a.RT + per - 1) / per), (unsigned)token_tiles), dim3(64 * kWaves), 0, stream, a);
}

// How many wavefronts share the columns: as few as still fill the card, since longer runs
// lose less to their start and end.  A CU holds 12 wavefronts; measured (bf16, columns
// 6,144 and 1,792, 96 experts): one token, 7 and 6 wavefronts a CU at KS 2, 32.7 us (36.2 at
// KS 4, 36.4 with the down product at KS 1); two tokens, 7 at KS 1, 53.6 us (56.0 at KS 2).
// Fuller tiles, whose activations cost more, gain earlier from sharing them: 16 rows of 8
// experts (4,096 and 1,536) with 3 at KS 1 33.4 us, 39.5 at KS 2.  One matrix and one
// token, 6,144 x 6,144: a stream of its own for each of four wavefronts 6.8 us, two 7.7.
template <int PLANES, int GPT, bool SWIGLU, int OUT, typename TO>
void launch_group(const W4Args& a, int num_cu, hipStream_t stream) {
  const int64_t tiles = w4_token_tiles(a.n_max, a.offsets ? a.E : 0);
  const int64_t used = a.n_max < a.E ? a.n_max : a.E, most = a.n_max / kTok;
  const int64_t busy = used > most ? used : most;             // token tiles with rows, about
  const int64_t waves = (SWIGLU ? a.RT : (a.RT + 1) / 2) * busy, enough = a.n_max >= 8 * busy ? 3 : 7;
  if (waves >= num_cu * enough) launch_one<PLANES, GPT, 1, 2, SWIGLU, OUT, TO>(a, stream, tiles);
  else if (waves >= num_cu * 3) launch_one<PLANES, GPT, 2, 2, SWIGLU, OUT, TO>(a, stream, tiles);
  else if (SWIGLU || waves * 2 >= num_cu * 3) launch_one<PLANES, GPT, 4, 2, SWIGLU, OUT, TO>(a, stream, tiles);
  else launch_one<PLANES, GPT, 4, SWIGLU ? 2 : 1, SWIGLU, OUT, TO>(a, stream, tiles);
}

template <int PLANES, bool SWIGLU, int OUT, typename TO>
hipError_t launch(const W4Args& a, int group, int num_cu, hipStream_t stream) {
  if (group == 32) launch_group<PLANES, 4, SWIGLU, OUT, TO>(a, num_cu, stream);
  else if (group == 64) launch_group<PLANES, 2, SWIGLU, OUT, TO>(a, num_cu, stream);
  else launch_group<PLANES, 1, SWIGLU, OUT, TO>(a, num_cu, stream);
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
  return E == 0 ? (n_max + kTok - 1) / kTok : n_max / kTok + (n_max < E ? n_max : E);
}

hipError_t launch_w4_matvec(int dtype, int64_t T, int64_t C, int64_t R, int group, const void* x, const void* codes,
                            const void* scales, void* y, void* x_planes, int num_cu, hipStream_t stream) {
  W4Args a{};
  a.n_in = a.n_max = T;
  a.E = 1;
  a.C = (int)C; a.R = (int)R; a.KT = (int)w4_col_tiles(C); a.RT = (int)w4_row_tiles(R);
  a.NG = w4_row_scales(C, group);
  a.codes[0] = (const uint32_t*)codes; a.scales[0] = (const uint16_t*)scales;
  a.y = y;
  if (dtype == 1) {
    a.x = (const bf16*)x;
    return launch<1, false, 1, bf16>(a, group, num_cu, stream);
  }
  hipError_t err = launch_split3(T * C, x, x_planes, stream);
  if (err != hipSuccess) return err;
  a.x = (const bf16*)x_planes;
  return launch<3, false, 1, float>(a, group, num_cu, stream);
}

hipError_t launch_w4_grouped_ffn(int dtype, int64_t n_max, int64_t d, int64_t E, int64_t F, int group, const void* x,
                                 int64_t n_in, const int32_t* a_rows, const int32_t* offsets, const void* const* codes,
                                 const void* const* scales, void* y_perm, void* x_planes, void* h_planes,
                                 int num_cu, hipStream_t stream) {
  W4Args g{};
  g.n_in = n_in; g.a_rows = a_rows; g.offsets = offsets; g.n_max = n_max;
  g.E = (int)E;
  g.C = (int)d; g.R = (int)F; g.KT = (int)w4_col_tiles(d); g.RT = (int)w4_row_tiles(F);
  for (int n = 0; n < 2; ++n) { g.codes[n] = (const uint32_t*)codes[n]; g.scales[n] = (const uint16_t*)scales[n]; }
  g.NG = w4_row_scales(d, group);
  g.y = h_planes;
  g.y_plane = n_max * F;
  W4Args w = g;
  w.x = (const bf16*)h_planes;
  w.n_in = n_max; w.a_rows = nullptr;
  w.C = (int)F; w.R = (int)d; w.KT = (int)w4_col_tiles(F); w.RT = (int)w4_row_tiles(d);
  w.NG = w4_row_scales(F, group);
  w.codes[0] = (const uint32_t*)codes[2]; w.scales[0] = (const uint16_t*)scales[2];
  w.y = y_perm;
  hipError_t err;
  if (dtype == 1) {
    g.x = (const bf16*)x;
    if ((err = launch<1, true, 2, bf16>(g, group, num_cu, stream)) != hipSuccess) return err;
    return launch<2, false, 1, bf16>(w, group, num_cu, stream);
  }
  if ((err = launch_split3(n_in * d, x, x_planes, stream)) != hipSuccess) return err;
  g.x = (const bf16*)x_planes;
  if ((err = launch<3, true, 3, bf16>(g, group, num_cu, stream)) != hipSuccess) return err;
  return launch<3, false, 1, float>(w, group, num_cu, stream);
}

}  // namespace moe
