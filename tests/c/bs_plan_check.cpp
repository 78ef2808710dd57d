// The device-planned grid of the block-scaled decode (csrc/bs_plan.h).
#include <cstdio>
#include <initializer_list>

#include "bs_plan.h"

static int bad = 0;
static void expect(long long got, long long want, const char* what, int a, int b, int c) {
  if (got == want) return;
  std::printf("%s (%d, %d, %d): %lld, not %lld\n", what, a, b, c, got, want);
  bad = 1;
}

int main() {
  const int wave = 304, warps = 4;
  auto grid = [&](int B, int H, int n_z, int tiles_each) {
    const int zg = n_z == 2 || n_z == 4 ? n_z : 1;
    return pd::bs_device_grid(B, H, n_z, zg, (long long)tiles_each * B, wave, warps, wave);
  };
  for (int B = 1; B <= 400; ++B)
    for (int H : {1, 2, 8, 40})
      for (int t : {0, 1, 13, 40, 63, 125, 1000}) {
        // up to 8 columns a KV head: a block per (sequence, KV head), within ten tiles a warp
        const bool few = (long long)B * H < wave && t / warps <= (long long)t * B * H / (wave * warps) + 10;
        expect(grid(B, H, 1, t), few ? B * H : wave, "one slice", B, H, t);
        for (int n_z : {2, 3, 4, 5, 6, 9, 12, 16}) {
          const int zg = n_z == 2 || n_z == 4 ? n_z : 1, g = grid(B, H, n_z, t);
          if (g == wave) continue;
          // the blocks hold whole lines: a divisor of the lines of a (sequence, KV head)
          if (g > wave || g < B * H || g % (B * H) != 0 || (n_z / zg) % (g / (B * H)) != 0)
            expect(g, -1, "blocks that cut lines", B, H, n_z);
          // and a warp's tiles are near its equal share
          const long long each = (long long)t * B * H * n_z / g / warps;
          if (each > (long long)t * B * H * n_z / (wave * warps) + 41) expect(each, 0, "tiles a warp", B, H, n_z);
        }
      }
  // one short sequence of 40 query columns a KV head: 40 segments over 40 blocks, not over 8
  expect(grid(1, 8, 5, 40), 40, "five slices", 1, 8, 40);
  expect(grid(4, 8, 5, 40), 160, "five slices", 4, 8, 40);
  expect(grid(8, 8, 5, 40), wave, "five slices, 320 segments", 8, 8, 40);
  expect(grid(16, 8, 3, 13), 128, "three slices, three a block", 16, 8, 13);
  expect(grid(1, 8, 2, 40), 8, "two slices side by side", 1, 8, 40);
  expect(grid(32, 1, 16, 40), 256, "sixteen slices, two a block", 32, 1, 40);
  if (!bad) std::printf("block-scaled plan ok\n");
  return bad;
}
