// Grids of the rotary and 4-bit calls (host code of csrc/kvq_paged4.cuh): CTAs
// cover all tokens, none is empty, their number fits a launch.
#include <cstdio>

#include "kvq_paged4.cuh"

using namespace kvq;

static int failures = 0;

static void covers(const char* what, int n, long long ctas, long long tokens) {
  if (ctas >= 1 && ctas <= 0x7fffffffLL && tokens >= 1 && ctas * tokens >= n && (ctas - 1) * tokens < n) return;
  if (++failures <= 20) std::printf("%s: %d tokens, %lld CTAs of %lld\n", what, n, ctas, tokens);
}

int main() {
  int checked = 0;
  for (long long base : {1LL, 2LL, 255LL, 1000LL, 40000LL, 1LL << 20, (1LL << 30) + 1, 0x7fffffffLL - 513, 0x7fffffffLL - 300,
                         0x7fffffffLL - 200, 0x7fffffffLL - 100, 0x7fffffffLL - 3}) {
    for (int more = 0; more < 4; ++more) {
      const int n = static_cast<int>(base + more > 0x7fffffffLL ? 0x7fffffffLL : base + more);
      for (int lanes = 1; lanes <= 128; ++lanes) {
        const int rows = 256 / lanes;
        const long long ctas = angles_ctas(n, rows);  // (each goes round: every row has one, none more than it takes)
        if (ctas < 1 || ctas > ctas_of(n, rows) || ctas_of(n, rows) * rows < n) covers("angles", n, -1, rows);
        ++checked;
      }
      for (int heads : {1, 3, 8, 40, 1000}) {
        for (int D : {8, 64, 96, 128, 256}) {
          for (int rot : {2, 8, 16, 24, 64, 90, 256}) {
            for (int inter = 0; inter < 2; ++inter) {
              if (rot > D) continue;
              for (int threads : {256, 512}) {
                RotateParams p = {};
                p.n_tokens = n;
                p.n_heads = heads;
                p.D = D;
                p.rot = rot;
                p.interleaved = inter;
                p.units.d = rotate_units(D, rot, inter);
                const long long ctas = rotate_ctas(&p, threads);
                covers("rotate", n, ctas, p.tokens);
                ++checked;
              }
            }
          }
        }
        for (int per : {4, 8, 16}) {
          for (int rounds : {2, 16}) {
            const Grid4 g = grid4(n, 2LL * heads * per, rounds, 256);
            covers("4-bit", n, g.kv_ctas, g.tokens);
            ++checked;
          }
        }
      }
    }
  }
  std::printf("checked %d failures %d\n", checked, failures);
  return failures != 0;
}
