// row_reads.hpp -- which aligned vectors a warp reads of a row of bf16 that begins anywhere, and which
// of them lie whole in the matrix's memory.  Host and device code; it compiles without CUDA.
#pragma once

#include <cstdint>

#ifndef ZERO_HD
#ifdef __CUDACC__
#define ZERO_HD __host__ __device__
#else
#define ZERO_HD
#endif
#endif

namespace zeroadam {
namespace {

// A matrix's memory, [begin, end): nothing outside is read.
struct Extents {
  uintptr_t begin, end;
  ZERO_HD bool whole(uintptr_t p) const { return p >= begin && p + 16 <= end; }
};

// The 8 columns a lane of those from `row` on, n of which there are (256 at most looked at), come
// from the aligned vector that the lane's first one lies in and the next lane's; lane 31 reads its
// next one itself.
struct LaneReads {
  uintptr_t first, next;
  bool has_first, has_next;
  ZERO_HD LaneReads(uintptr_t row, int64_t n, int lane) {
    const int s = shift(row);
    first = row + 2 * (8 * lane - s);
    next = row + 2 * (256 - s);
    has_first = 8 * lane - s < n;
    has_next = lane == 31 && s > 0 && 256 - s < n;
  }
  // Elements from the boundary before `row` to it.
  ZERO_HD static int shift(uintptr_t row) { return static_cast<int>(row % 16 / 2); }
};

// The rows [first, end) of a matrix whose vectors are all whole in its memory: a vector begins up to 7
// elements before a row and ends up to 7 behind it.  aligned: every row begins on a 16-byte boundary.
struct WholeRows {
  int32_t first, end;
  WholeRows() = default;
  ZERO_HD WholeRows(int64_t rows, int64_t width, int64_t ld, bool aligned) {
    const int64_t near = (6 + ld) / ld;  // rows that begin less than 7 elements from the memory's end
    const int64_t least = aligned ? 0 : near, most = rows - (aligned && width % 8 == 0 ? 0 : near);
    first = static_cast<int32_t>(least < rows ? least : rows);
    end = static_cast<int32_t>(most > first ? most : first);
  }
  ZERO_HD bool has(int32_t row) const { return row >= first && row < end; }
};

// A vector that is not whole in the matrix's memory, element by element from `at(address)`; what
// is not there is 0.
template <typename At>
ZERO_HD inline void read_cut(uintptr_t p, const Extents& in, uint64_t w[2], At at) {
  w[0] = w[1] = 0;
#ifdef __CUDACC__
#pragma unroll 1  // (rare, and short in the kernel's code)
#endif
  for (int c = 0; c < 8; ++c) {
    const uintptr_t q = p + 2 * c;
    const uint64_t x = q >= in.begin && q < in.end ? static_cast<uint64_t>(at(q)) << (16 * (c % 4)) : 0;
    if (c < 4) w[0] |= x;
    else w[1] |= x;
  }
}

}  // namespace
}  // namespace zeroadam
