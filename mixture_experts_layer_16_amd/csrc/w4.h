// 4-bit weights with group scales: W[r, c] = s[r, c / group] * (q[r, c] - 8), q in
// 0..15, s in bf16, groups of 32, 64 or 128 columns.
//
// A matrix [R, C] is laid out once in tiles of 16 rows x 128 columns, row tile by
// row tile, so that a wavefront loads a tile with one 16-byte load a lane and the
// loaded words are, after the unpacking below, MFMA operands as they are:
//
//   codes  [RT, KT] tiles of 1,024 bytes: lane l holds the 32-bit words i = 0..3 of
//          row rt*16 + l%16, columns kt*128 + i*32 + (l/16)*8 + 0..7; in a word,
//          nibble j is column 2j and nibble j + 4 column 2j + 1 (j = 0..3), so
//          that nibbles j and j + 4 sit 16 bits apart, as a bf16 pair does
//   scales [RT, 16, NG] bf16: the scales of each row in order, so that a lane loads
//          those of several column tiles at once
//
// with RT = ceil(R/16), KT = ceil(C/128), NG = KT * 128/group rounded up to 4.  Rows and
// columns past the matrix have code 8 and scale 0.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kW4Rows = 16;      // rows of a tile
constexpr int kW4Cols = 128;     // columns of a tile
constexpr int kW4TileBytes = kW4Rows * kW4Cols / 2;

inline int64_t w4_row_tiles(int64_t R) { return (R + kW4Rows - 1) / kW4Rows; }
inline int64_t w4_col_tiles(int64_t C) { return (C + kW4Cols - 1) / kW4Cols; }
inline int w4_row_scales(int64_t C, int64_t group) { return (int)((w4_col_tiles(C) * (kW4Cols / group) + 3) / 4 * 4); }

}  // namespace moe
