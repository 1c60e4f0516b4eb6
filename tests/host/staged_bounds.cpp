// Walks every chunk that the register-staged blocks load (csrc/staged.h): each 16 bytes lie inside one line of
// the operand, and after the shift each element is the operand's, or zero for K past the end.
//
// argv: kind (0 K-major, 1 M/N-major), bytes of an element, block size, extent (rows or columns), K, leading
// dimension beyond the packed one, K of a part.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../tile_level_gemm_amd/csrc/staged.h"

using namespace tg;

static int bad(const char* what, long a, long b, long c, long d) {
  std::printf("%s: block %ld part %ld stage %ld line %ld\n", what, a, b, c, d);
  return 1;
}

template <bool MN>
static int walk(int eb, int bs, int extent, int K, int gap, int kps) {
  const int ve = 16 / eb, bk = 128 / eb;
  const int cols = MN ? extent : K, rows = MN ? K : extent;   // the operand as it is stored
  const int64_t ld = cols + gap;
  // element (row, col) is its own name; the gaps hold none
  auto name = [&](int64_t at, int64_t* row, int64_t* col) {
    *row = at / ld;
    *col = at % ld;
    return at >= 0 && *row < rows && *col < cols;
  };
  for (int m0 = 0; m0 < extent; m0 += bs)
    for (int k0 = 0; k0 < K; k0 += kps) {
      const int kl = staged_min(K - k0, kps), left = extent - m0, KT = (kl + bk - 1) / bk;
      const int lines = MN ? kl : left, width = MN ? left : kl;
      const int64_t base = MN ? (int64_t)k0 * ld + m0 : (int64_t)m0 * ld + k0;
      for (int s = 0; s < KT + 2; ++s) {   // the loads run two stages past the last
        const bool fixed = (MN && left < bs) || s + 1 >= KT;
        for (int line = 0; line < (MN ? bk : bs); ++line)
          for (int chunk = 0; chunk < (MN ? bs : bk) / ve; ++chunk) {
            const StagedPlace p = staged_place<MN>(s, bk, ve, line, chunk);
            const int64_t from = base + staged_offset(p, ld, lines, width, ve);
            int64_t r0, c0, r1, c1;
            if (!name(from, &r0, &c0) || !name(from + ve - 1, &r1, &c1) || r0 != r1)
              return bad("outside the operand", m0, k0, s, line);
            if (s >= KT) continue;
            const int back = fixed ? staged_back<MN>(p, kl, width, ve) : 0;
            if (back < 0 || back > ve) return bad("shift", m0, k0, s, line);
            for (int e = 0; e < ve; ++e) {
              // what the stage wants here: K index and row or column, from the block's first
              const int k = MN ? s * bk + line : s * bk + chunk * ve + e, i = MN ? chunk * ve + e : line;
              if (i >= left) continue;   // feeds outputs that are not stored
              const bool zero = e + back >= ve;
              if (k >= kl) {
                if (!zero) return bad("K past the end is not zero", m0, k0, s, line);
                continue;
              }
              const int64_t want = MN ? (int64_t)(k0 + k) * ld + m0 + i : (int64_t)(m0 + i) * ld + k0 + k;
              if (zero || from + back + e != want) return bad("not the operand's element", m0, k0, s, line);
            }
          }
      }
    }
  return 0;
}

int main(int argc, char** argv) {
  int v[7], n = 0;
  if (argc < 8 || (argc - 1) % 7) return 2;
  for (int a = 1; a < argc; a += 7) {
    for (int i = 0; i < 7; ++i) v[i] = std::atoi(argv[a + i]);
    if (v[0] ? walk<true>(v[1], v[2], v[3], v[4], v[5], v[6]) : walk<false>(v[1], v[2], v[3], v[4], v[5], v[6])) {
      std::printf("kind %d bytes %d block %d extent %d K %d gap %d part %d\n", v[0], v[1], v[2], v[3], v[4], v[5], v[6]);
      return 1;
    }
    ++n;
  }
  std::printf("%d operands\n", n);
  return 0;
}
