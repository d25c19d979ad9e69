// Reads rows of small matrices as the embedding gradient's warps do, at every width, pitch and
// address, from memory that is theirs alone, and counts elements that come out wrong and reads
// outside of the matrix.  With "whole" every vector is read as if it were whole.
#include <cstdio>
#include <cstring>
#include <vector>

#include "row_reads.hpp"

using namespace zeroadam;

int main(int argc, char** argv) {
  const bool whole = argc > 1 && std::strcmp(argv[1], "whole") == 0;
  alignas(16) static uint16_t memory[8192];
  for (int k = 0; k < 8192; ++k) memory[k] = static_cast<uint16_t>(k + 1);
  long outside = 0, wrong = 0, vectors = 0, cut = 0, unsafe = 0, most = 0;
  for (int width : {1, 2, 3, 7, 8, 9, 15, 16, 100, 247, 248, 249, 255, 256, 257, 263, 264, 300})
    for (int pitch = width; pitch < width + 9; ++pitch)
      for (int rows : {1, 2, 3, 9})
        for (int offset = 8; offset < 16; ++offset) {
          const uint16_t* dy = memory + offset;
          const uintptr_t begin = reinterpret_cast<uintptr_t>(dy);
          const bool aligned = offset % 8 == 0 && (rows == 1 || pitch % 8 == 0);
          const WholeRows safe(rows, width, pitch, aligned);
          most = rows > 3 && safe.end - safe.first > most ? safe.end - safe.first : most;
          const Extents in{begin, begin + 2 * ((rows - 1) * pitch + width)};
          const auto at = [&](uintptr_t p) {
            if (p < in.begin || p + 2 > in.end) ++outside;
            return *reinterpret_cast<const uint16_t*>(p);
          };
          for (int r = 0; r < rows; ++r)
            for (int col = 0; col < width; col += 256) {
              const uintptr_t row = begin + 2 * (r * pitch + col);
              const int64_t n = width - col;
              std::vector<uint16_t> got(33 * 8, 0);  // from the first lane's aligned vector on
              const auto read = [&](bool has, uintptr_t p, int k) {
                if (!has) return;
                if (p % 16 != 0) ++wrong;
                ++vectors;
                uint64_t w[2];
                if (safe.has(r) && !in.whole(p)) ++unsafe;
                if (whole || in.whole(p)) {
                  std::memcpy(w, reinterpret_cast<const void*>(p), 16);
                  for (int c = 0; c < 8; ++c) at(p + 2 * c);
                } else {
                  ++cut;
                  read_cut(p, in, w, at);
                }
                std::memcpy(&got[8 * k], w, 16);
              };
              for (int lane = 0; lane < 32; ++lane) {
                const LaneReads v(row, n, lane);
                read(v.has_first, v.first, lane);
                read(v.has_next, v.next, 32);
              }
              const int s = LaneReads::shift(row);
              for (int j = 0; j < 256 && j < n; ++j)
                if (got[s + j] != reinterpret_cast<const uint16_t*>(row)[j]) ++wrong;
            }
        }
  std::printf("vectors %ld\ncut %ld\noutside %ld\nwrong %ld\nunsafe %ld\nmost %ld\n", vectors, cut, outside, wrong,
              unsafe, most);
  return 0;
}
