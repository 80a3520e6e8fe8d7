// Host check of the 8-bit attention's schedule: the spans that the CTAs record from
// their walks alone, and the rule that keeps a merge inside its records.  No kernel
// is launched.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "tt_attn_q8.cuh"

using namespace tt;

static int check(const std::vector<int>& len, int L_cap, int U, int P, std::vector<int>& seen) {
  const int B = (int)len.size();
  std::vector<int> tiles;  // of each unit
  for (int b = 0; b < B; ++b)
    for (int k = 0; k < U; ++k)
      tiles.push_back(1 + (std::min(std::max(len[b], 0), L_cap) + kAttnBN - 1) / kAttnBN);
  const int units = (int)tiles.size();
  int T = 0;
  for (int n : tiles) T += n;
  std::vector<int2> span(units, make_int2(-1, 1 << 30)), want(units, make_int2(1 << 30, -1));
  std::vector<char> slot(units + P - 1, 0);
  for (int c = 0; c < P; ++c) {
    const int lo = cta_first(c, T, P), hi = cta_first(c + 1, T, P);
    int u = 0, first = 0;
    while (first + tiles[u] <= lo) first += tiles[u++];
    TileWalk w;
    w.ctx_len = len.data();
    w.left = hi - lo;
    w.B = B;
    w.L_cap = L_cap;
    w.U = U;
    w.b = u / U;
    w.k = u % U;
    w.off = lo - first;
    w.len = len[w.b];
    put_spans(span.data(), w, c);
    for (int t = lo; t < hi; ++u) {
      const int to = std::min(hi, first + tiles[u]);
      want[u].x = std::min(want[u].x, c);
      want[u].y = std::max(want[u].y, c);
      if (u + c >= units + P - 1 || slot[u + c]++) return std::printf("slot of unit %d, CTA %d\n", u, c);
      first += tiles[u];
      t = to;
    }
  }
  for (int u = 0; u < units; ++u) {
    if (span[u].x != want[u].x || span[u].y != want[u].y)
      return std::printf("unit %d: %d..%d, not %d..%d\n", u, span[u].x, span[u].y, want[u].x, want[u].y);
    if (!span_in_range(span[u], P)) return std::printf("unit %d refused\n", u);
    seen.push_back(span[u].y - span[u].x);
  }
  return 0;
}

int main() {
  std::srand(1);
  std::vector<int> seen;
  for (int i = 0; i < 400; ++i) {
    const int B = 1 + std::rand() % 40, L_cap = std::rand() % 3000, U = 1 + std::rand() % 8;
    std::vector<int> len(B);
    for (int& x : len) x = std::rand() % 4 ? std::rand() % (L_cap + 1) : std::rand() % 5 * 2000 - 4000;
    for (int P : {1, 3, 148, 1024})
      if (check(len, L_cap, U, P, seen)) return 1;
  }
  bool wide = false;
  for (int n : seen) wide |= n > 20;
  if (!wide) return std::printf("no unit over many CTAs\n"), 1;
  // what an older or a foreign workspace may hold
  const int bad[][2] = {{-1, 0}, {0, 148}, {5, 4}, {1 << 30, (1 << 30) + 1}, {0, 0x7fffffff},
                        {(int)0xA5A5A5A5, (int)0xA5A5A5A5}, {3, -2147483647 - 1}, {148, 148}};
  for (auto& s : bad)
    if (span_in_range(make_int2(s[0], s[1]), 148)) return std::printf("%d..%d taken\n", s[0], s[1]), 1;
  for (int x : {0, 7, 147})
    if (!span_in_range(make_int2(x, 147), 148)) return 1;
  std::printf("q8_spans: ok\n");
  return 0;
}
