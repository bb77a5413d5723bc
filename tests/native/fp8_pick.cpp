// Host-only driver of the FP8 product's choice of a tile
// (rotated_bit_amd/csrc/fp8_pick.hpp), for tests/test_fp8_pick.py.
//
//   fp8_pick            lines "bf16|f32 M N K experts grouped" from standard
//                       input -> "index bn bm threads workgroups"
//   fp8_pick tables     the number of entries of each table
//   fp8_pick launches   the most threads of any launch over sizes up to the
//                       largest, with the tables' costs and with costs that
//                       make the smallest tiles look free
#include <cstdio>
#include <cstring>

#include "../../rotated_bit_amd/csrc/fp8_pick.hpp"

using namespace harp;

template <int T>
static int64_t threads(const Fp8Tile (&tiles)[T], int i, int M, int N, int live) {
  return fp8_n_tiles(tiles[i], N) * fp8_m_tiles(tiles[i], M, live) * tiles[i].threads;
}

template <int T>
static int64_t most(const Fp8Tile (&tiles)[T], float output) {
  const int experts[] = {1, 2, 8, 64, 255, 256, 900, 1023, 1024};
  const int ks[] = {16, 128, 144, 1024, 4096, 8192, 65536, 262144};
  int64_t top = 0;
  for (int N = 262144; N >= 1; N = N > 64 ? N - N / 9 : N - 1)
    for (int E : experts)
      for (int M = 65536; M >= 1; M = M > 256 ? M - M / 40 : M - 1)
        for (int K : ks)
          for (int grouped = E > 1; grouped < 2; ++grouped) {
            const int live = fp8_live(M, E, grouped != 0);
            const int i = fp8_pick(tiles, output, M, N, K, live, grouped != 0);
            const int64_t t = threads(tiles, i, M, N, live);
            if (t > top) top = t;
          }
  return top;
}

template <int T>
static int64_t most_if_small_were_free(const Fp8Tile (&tiles)[T]) {
  Fp8Tile doctored[T];
  for (int i = 0; i < T; ++i) {
    doctored[i] = tiles[i];
    const float c = static_cast<float>(tiles[i].bn) * static_cast<float>(tiles[i].bm);
    doctored[i].lone = doctored[i].round = c * c * c;
    doctored[i].lone_run = doctored[i].round_run = 0.0f;
  }
  return most(doctored, 0.0f);
}

int main(int argc, char** argv) {
  if (argc > 1 && std::strcmp(argv[1], "launches") == 0) {
    std::printf("bf16 %lld %lld\nf32 %lld %lld\n",
                static_cast<long long>(most(kBf16Tiles, kBf16Output)),
                static_cast<long long>(most_if_small_were_free(kBf16Tiles)),
                static_cast<long long>(most(kF32Tiles, kF32Output)),
                static_cast<long long>(most_if_small_were_free(kF32Tiles)));
    return 0;
  }
  if (argc > 1 && std::strcmp(argv[1], "tables") == 0) {
    std::printf("bf16 %zu\nf32 %zu\n", sizeof(kBf16Tiles) / sizeof(Fp8Tile),
                sizeof(kF32Tiles) / sizeof(Fp8Tile));
    return 0;
  }
  char dt[8];
  int M, N, K, E, grouped;
  while (std::scanf("%7s %d %d %d %d %d", dt, &M, &N, &K, &E, &grouped) == 6) {
    const int live = fp8_live(M, E, grouped != 0);
    const bool bf16 = std::strcmp(dt, "bf16") == 0;
    const int i = bf16 ? fp8_pick(kBf16Tiles, kBf16Output, M, N, K, live, grouped != 0)
                       : fp8_pick(kF32Tiles, kF32Output, M, N, K, live, grouped != 0);
    const Fp8Tile& t = bf16 ? kBf16Tiles[i] : kF32Tiles[i];
    std::printf("%d %d %d %d %lld\n", i, t.bn, t.bm, t.threads,
                static_cast<long long>(fp8_n_tiles(t, N) * fp8_m_tiles(t, M, live)));
  }
  return 0;
}
