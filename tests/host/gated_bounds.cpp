// Walks every chunk that gated blocks load of their weights (csrc/staged.h): through registers each 16 bytes lie
// inside one line of the operand and hold, after the shift, the element of the projection, row or column and K
// that its place in the block stands for, or zero for K past the end; the direct loads' chunks that the buffer
// check lets through lie inside the operand and hold the same.
//
// argv: kind (0 [2N][K], 1 [K][2N]), bytes of an element, block size, columns of a group, N, K, leading dimension
// beyond the packed one, K of a part.
#include <cstdio>
#include <cstdlib>

#include "../../tile_level_gemm_amd/csrc/staged.h"

using namespace tg;

static int bad(const char* what, long a, long b, long c, long d) {
  std::printf("%s: block %ld part %ld stage %ld line %ld\n", what, a, b, c, d);
  return 1;
}

template <bool MN>
static int walk(int eb, int bs, int r, int N, int K, int gap, int kps) {
  const int ve = 16 / eb, bk = 128 / eb, waves = bs == 64 ? 4 : 8, per = bs / 8 / waves;
  const int cols = MN ? 2 * N : K, rows = MN ? K : 2 * N;
  const int64_t ld = cols + gap;
  const bool direct = (ld * eb) % 16 == 0 && (MN ? (int64_t)N * eb : (int64_t)K * eb) % 16 == 0;
  // a place of the block: projection and column of D behind the block's first
  auto half = [&](int i) { return i / r % 2; };
  auto behind = [&](int i) { return i / (2 * r) * r + i % r; };
  for (int n0 = 0; n0 < N; n0 += bs / 2)
    for (int k0 = 0; k0 < K; k0 += kps) {
      const int kl = staged_min(K - k0, kps), left = 2 * N - n0, KT = (kl + bk - 1) / bk;
      const int lines = MN ? kl : left, width = MN ? left : kl;
      const int64_t base = MN ? (int64_t)k0 * ld + n0 : (int64_t)n0 * ld + k0;
      auto at = [&](int i, int k) {   // the element that place i and K index k of the part stand for
        const int64_t n = (int64_t)half(i) * N + n0 + behind(i);
        return MN ? (int64_t)(k0 + k) * ld + n : n * ld + k0 + k;
      };
      auto inside = [&](int64_t a) { return a >= 0 && a / ld < rows && a % ld < cols; };
      for (int s = 0; s < KT + 2; ++s) {
        const bool fixed = (MN && 2 * (N - n0) < bs) || s + 1 >= KT;
        for (int line = 0; line < (MN ? bk : bs); ++line)
          for (int chunk = 0; chunk < (MN ? bs : bk) / ve; ++chunk) {
            const StagedPlace b = staged_place<MN>(s, bk, ve, line, chunk), p = gated_place<MN>(b, r, N);
            const int64_t from = base + staged_offset(p, ld, lines, width, ve);
            if (!inside(from) || !inside(from + ve - 1) || from / ld != (from + ve - 1) / ld) return bad("outside", n0, k0, s, line);
            const int back = fixed ? staged_back<MN>(p, kl, width, ve) : 0;
            for (int e = 0; e < ve && s < KT; ++e) {
              const int k = MN ? s * bk + line : s * bk + chunk * ve + e, i = MN ? chunk * ve + e : line;
              if (n0 + behind(i) >= N) continue;   // feeds results that are not stored
              const bool zero = e + back >= ve;
              if (k >= kl) {
                if (!zero) return bad("K past the end is not zero", n0, k0, s, line);
              } else if (zero || from + back + e != at(i, k)) {
                return bad("not the operand's element", n0, k0, s, line);
              }
            }
            if (!direct) continue;
            // direct loads: byte offset from the descriptor's base, its records; a chunk past them is zeros
            const int64_t row = line;
            int64_t start, off, records;
            if (MN) {
              start = base;
              off = (((int64_t)s * bk + line) * ld + gated_index(chunk * ve, r, N)) * eb;
              records = ((int64_t)(kl - 1) * ld + left) * eb;
            } else {
              const int wave = (int)(row / (8 * per));   // whose instruction loads this row
              const int own = 8 * per, place = wave * own, first = n0 + gated_index(place, r, 0), have = N - first;
              if (r % own) return bad("rows of a wave", n0, k0, s, line);
              start = ((int64_t)(place / r % 2) * N + staged_min(first, N - 1)) * ld + k0;
              const bool past = chunk * 16 >= staged_max(0, staged_min(128, kl * eb - s * 128));
              off = past ? (int64_t)1 << 31 : (row % own) * ld * eb + (int64_t)s * 128 + chunk * 16;
              records = have <= 0 ? 0 : ((int64_t)(staged_min(have, own) - 1) * ld + kl) * eb;
            }
            for (int e = 0; e < ve; ++e) {
              const int k = MN ? s * bk + line : s * bk + chunk * ve + e, i = MN ? chunk * ve + e : line;
              const bool loads = off + 16 <= records;
              if (!loads && off < records) return bad("a chunk across the records' end", n0, k0, s, line);
              const int64_t a = start + off / eb + e;
              if (loads && a / ld >= rows) return bad("direct: outside", n0, k0, s, line);
              if (n0 + behind(i) >= N) continue;
              if (k >= kl ? loads : (!loads || a != at(i, k))) return bad("direct: not the operand's element", n0, k0, s, line);
            }
          }
      }
    }
  return 0;
}

int main(int argc, char** argv) {
  int v[8], n = 0;
  if (argc < 9 || (argc - 1) % 8) return 2;
  for (int a = 1; a < argc; a += 8) {
    for (int i = 0; i < 8; ++i) v[i] = std::atoi(argv[a + i]);
    if (v[0] ? walk<true>(v[1], v[2], v[3], v[4], v[5], v[6], v[7]) : walk<false>(v[1], v[2], v[3], v[4], v[5], v[6], v[7])) {
      std::printf("kind %d bytes %d block %d group %d N %d K %d gap %d part %d\n", v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
      return 1;
    }
    ++n;
  }
  std::printf("%d operands\n", n);
  return 0;
}
