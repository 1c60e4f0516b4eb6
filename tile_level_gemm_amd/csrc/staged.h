// Where the register-staged blocks load from: 16-byte chunks that never leave their operand, whatever the
// edge.  Plain integer arithmetic, so it is the same on the host, where a test walks every chunk.
//
// An operand is `lines` runs of `width` elements, ld apart: K-major the rows from the block's first to the
// operand's last by this part's K, M/N-major this part's K rows by the columns from the block's first to
// the operand's last.  ve: elements of a chunk.  Internal header.
#pragma once

#include <stdint.h>

namespace tg {

constexpr int staged_min(int a, int b) { return a < b ? a : b; }
constexpr int staged_max(int a, int b) { return a > b ? a : b; }

// Chunk `chunk` of line `row` of a block's stage of bk K: its line and its first element.
struct StagedPlace {
  int line, first;
};
template <bool MN>
constexpr StagedPlace staged_place(int stage, int bk, int ve, int row, int chunk) {
  return MN ? StagedPlace{stage * bk + row, chunk * ve} : StagedPlace{row, stage * bk + chunk * ve};
}
// The element the load starts at, from the block's first element at k = 0 of its part.  A chunk that would
// pass the end of its line is moved back to the line's last `ve` elements (into earlier columns or K of the
// same line where fewer are left), a line past the end repeats the last one.
constexpr int64_t staged_offset(StagedPlace p, int64_t ld, int lines, int width, int ve) {
  return (int64_t)staged_min(p.line, lines - 1) * ld + staged_min(p.first, width - ve);
}
// Elements to shift the loaded chunk down by, zeros from above: how far it was moved, all of it for K past
// the end (a row or column past the end feeds only outputs that are not stored).
template <bool MN>
constexpr int staged_back(StagedPlace p, int kl, int width, int ve) {
  return MN && p.line >= kl ? ve : staged_min(staged_max(0, p.first - (width - ve)), ve);
}

}  // namespace tg
