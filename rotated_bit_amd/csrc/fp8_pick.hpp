// Which tile the FP8 product works in (fp8_gemm.hip).  Plain C++, so that the
// choice can be looked at without a GPU.
#pragma once

#include <cmath>
#include <cstdint>

namespace harp {

// The tiles, largest first, with what they take in us, from least squares
// over 1200 products (16 .. 65536 rows and outputs, K 1024 .. 8192; residual
// 6 %): up to 256 tiles, one per CU, `lone` and `lone_run` for each run of 128
// inputs; beyond, `round` and `round_run` for each round of `per` tiles (512
// where two workgroups fit a CU and hide each other's waits); and on top
// kF32Output or kBf16Output for each 2^20 outputs and run, the matrix pipe's
// power and the shared bandwidth.  The estimate picks the tile: large ones do
// the most work per time, small ones leave no CU idle where there are few
// outputs, and what a round takes before and behind its runs counts where K
// is small.  Over 78 products of drawn sizes the picked tile is within 1 %
// (float32 y) and 2 % (bf16) of the fastest on average, 22 % at worst; a
// cost per run alone left 3.5 %, 44 % at worst.  It ranks the tiles and is no
// forecast: the time that weights take from memory is not in it (16 x 28672 x
// 8192 bf16: 20 us estimated, 45 measured).
struct Fp8Tile {
  int bn, bm, threads, per;   // outputs x rows, threads of a workgroup
  float lone, lone_run, round, round_run;
};
constexpr float kBf16Output = 0.064f, kF32Output = 0.081f;
constexpr Fp8Tile kBf16Tiles[] = {
    {256, 256, 512, 256, 6.3f, 0.861f, 6.3f, 0.861f},
    {256, 128, 256, 256, 4.8f, 0.525f, 4.8f, 0.525f},
    {128, 128, 256, 256, 3.3f, 0.362f, 3.3f, 0.362f},
    {128, 128, 256, 512, 2.0f, 0.588f, 3.2f, 0.606f},
    {128, 64, 256, 512, 2.5f, 0.265f, 2.2f, 0.428f},
    {64, 64, 256, 256, 2.8f, 0.171f, 2.8f, 0.171f},
    {64, 32, 128, 512, 2.9f, 0.146f, 2.9f, 0.225f},
    {32, 32, 128, 512, 2.3f, 0.094f, 2.4f, 0.162f},
    {32, 16, 256, 512, 2.3f, 0.060f, 2.3f, 0.105f},
    {16, 16, 256, 512, 2.1f, 0.044f, 2.3f, 0.077f},
};
constexpr Fp8Tile kF32Tiles[] = {
    {128, 128, 512, 256, 5.1f, 0.572f, 5.1f, 0.572f},
    {128, 128, 256, 512, 4.9f, 0.707f, 3.7f, 1.004f},
    {128, 64, 256, 512, 3.7f, 0.501f, 3.0f, 0.690f},
    {64, 64, 256, 512, 2.3f, 0.340f, 2.8f, 0.384f},
    {64, 32, 128, 512, 2.8f, 0.281f, 3.4f, 0.247f},
    {64, 32, 256, 256, 3.5f, 0.126f, 3.5f, 0.126f},
    {32, 32, 256, 512, 2.0f, 0.137f, 2.3f, 0.168f},
    {32, 16, 256, 512, 2.3f, 0.073f, 2.3f, 0.114f},
    {16, 16, 256, 512, 2.2f, 0.055f, 2.3f, 0.082f},
};

// Experts with rows, at most.
inline int fp8_live(int M, int experts, bool grouped) {
  return !grouped ? 1 : experts < M ? experts : M;
}
inline int64_t fp8_n_tiles(const Fp8Tile& t, int N) { return (int64_t{N} + t.bn - 1) / t.bn; }
// Row tiles of any routing, at most: sum_e ceil(c_e / bm) <= (M + live (bm - 1)) / bm.
inline int64_t fp8_m_tiles(const Fp8Tile& t, int M, int live) {
  return (M + int64_t{live} * (t.bm - 1)) / t.bm;
}
// A launch has fewer than 2^32 threads.  With these costs no tile that is left
// out by that would be picked (the most are 3.55e9 threads: float32 y, 11750
// rows of 1024 experts, 262144 outputs); the tiles from 128 x 128 on always
// fit.
inline bool fp8_fits(const Fp8Tile& t, int M, int N, int live) {
  return fp8_n_tiles(t, N) * fp8_m_tiles(t, M, live) * t.threads < int64_t{1} << 32;
}

// Index of the tile with the least estimate among those that fit a launch.
template <int TILES>
int fp8_pick(const Fp8Tile (&tiles)[TILES], float output, int M, int N, int K, int live,
             bool grouped) {
  int best = 0;
  double least = INFINITY;
  const double rows = static_cast<double>(M) / live;   // of an expert, on average
  const int runs = (K + 127) / 128;
  for (int i = 0; i < TILES; ++i) {
    const Fp8Tile& c = tiles[i];
    if (!fp8_fits(c, M, N, live)) continue;
    // an expert's last tile is half empty on average; dense rows are known
    double m_tiles = rows / c.bm + 0.5;
    if (m_tiles < 1.0) m_tiles = 1.0;
    m_tiles = grouped ? live * m_tiles : (M + c.bm - 1) / c.bm;
    const double count = m_tiles * static_cast<double>(fp8_n_tiles(c, N));
    double cost = output * runs * count * (c.bn * c.bm / 1048576.0);
    if (count <= 256.0)
      cost += c.lone + runs * c.lone_run;
    else
      cost += std::ceil(count / c.per) * (c.round + runs * c.round_run);
    if (cost < least) {
      least = cost;
      best = i;
    }
  }
  return best;
}

}  // namespace harp
