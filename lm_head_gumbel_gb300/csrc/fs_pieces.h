// fs_pieces.h -- how quantisation reads rows: in pieces of 8 elements from a row's start,
// whole (16 bytes at a time) where that stays inside the matrix, else element by element.
// Host code too, so that the rule can be checked without a GPU.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FS_BOTH __host__ __device__
#else
#define FS_BOTH
#endif

namespace fs {
namespace fp8 {

constexpr int kPiece = 8;

// A piece of which n elements exist (0 or fewer: none), of the matrix's last row or another
// one.  Past a row's end lies the next row, so only the last row's pieces have to be full.
FS_BOTH constexpr bool whole_piece(int n, bool last) { return last ? n >= kPiece : n > 0; }

// Whether whole pieces are read at all: x [N, d] of `size` bytes an element with row stride ldx
// (0 of a single row).  Their 16-byte loads are aligned, and no piece that begins inside a row
// passes the next one's first element: fp32 rows 4 elements apart are read element by element,
// whose last but one row's piece would end behind the last row.
constexpr bool whole_pieces(uintptr_t x, int64_t N, int64_t ldx, int size) {
  return x % 16 == 0 && ldx * size % 16 == 0 && (N == 1 || ldx >= kPiece);
}

}  // namespace fp8
}  // namespace fs
