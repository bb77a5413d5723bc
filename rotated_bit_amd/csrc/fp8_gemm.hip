// The FP8 (e4m3) product with a float32 scale per 1 x 128 run of a and per
// 128 x 128 block of w, dense and grouped by expert:
//
//     y[m][n] = sum_b sa[m][b] sw[n/128][b] P_b[m][n],
//     P_b[m][n] = sum_{k in run b} a[m][k] w[n][k].
//
// For a bf16 y one v_mfma_f32_16x16x128_f8f6f4 forms P_b of 16 x 16 outputs (its 128
// inputs are one run), so the scales enter once per matrix instruction as
// four fused multiply-adds per lane.  The weights are the row operand and a
// the column operand: lane l holds the four consecutive outputs
// n0 + 4 (l / 16) + 0..3 of row m0 + l % 16, which share one factor sa sw.
#include "fp8_common.hpp"
#include "launch.hpp"

namespace harp {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Fp8Args {
  const uint8_t* w;
  const float* ws;
  const uint8_t* a;
  const float* as;
  const int32_t* rows;      // null: rows[i] = i
  const int32_t* offsets;   // null: one matrix, all M rows
  void* y;
  int N, K, KB, E, M, a_rows;
};

// The rows [row0, row0 + count) of expert e that slot `slot` works on:
// every expert's rows are cut into tiles of BM, counted in expert order.
// Each wave computes it on its own: 64 experts at a time, an inclusive scan
// of their tile counts.  False: the slot has no tile.
struct Tile {
  int e, row0, count;
};
template <int BM>
__device__ __forceinline__ bool find_tile(const Fp8Args& p, int slot, Tile& t) {
  if (p.offsets == nullptr) {
    t.e = 0;
    t.row0 = slot * BM;
    t.count = min(BM, p.M - t.row0);
    return t.count > 0;
  }
  const int lane = threadIdx.x & (kWave - 1);
  int before = 0;   // tiles of the experts already passed
  for (int e0 = 0; e0 < p.E; e0 += kWave) {
    const int e = e0 + lane;
    int start = 0, end = 0;
    if (e < p.E) {
      start = min(max(p.offsets[e], 0), p.M);
      end = min(max(p.offsets[e + 1], 0), p.M);
    }
    const int tiles = (max(end - start, 0) + BM - 1) / BM;
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int u = __shfl_up(upto, o, kWave);
      if (lane >= o) upto += u;
    }
    const int first = before + upto - tiles;
    const unsigned long long hit = __ballot(slot >= first && slot < first + tiles);
    if (hit != 0) {
      const int src = __ffsll(hit) - 1;
      t.e = e0 + src;
      t.row0 = __shfl(start, src, kWave) + BM * (slot - __shfl(first, src, kWave));
      t.count = min(BM, __shfl(end, src, kWave) - t.row0);
      return true;
    }
    before += __shfl(upto, kWave - 1, kWave);
  }
  return false;
}

// The a row of output row i (< M), -1 for one that reads nothing.
__device__ __forceinline__ int source_row(const Fp8Args& p, int i) {
  const int r = p.rows == nullptr ? i : p.rows[i];
  return r >= 0 && r < p.a_rows ? r : -1;
}

// 32 codes of a row at inputs k .. k+31 (zeros from K on, and for !in).
__device__ __forceinline__ i32x8 load_codes(const uint8_t* row, int k, int K, bool in) {
  u32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
  if (in && k + 16 <= K) lo = *reinterpret_cast<const u32x4*>(row + k);
  if (in && k + 32 <= K) hi = *reinterpret_cast<const u32x4*>(row + k + 16);
  return i32x8{static_cast<int>(lo[0]), static_cast<int>(lo[1]), static_cast<int>(lo[2]),
               static_cast<int>(lo[3]), static_cast<int>(hi[0]), static_cast<int>(hi[1]),
               static_cast<int>(hi[2]), static_cast<int>(hi[3])};
}

// Eight codes as bf16 (exact).
__device__ __forceinline__ bf16x8 codes_bf16(int lo, int hi) {
  const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// P_b of 16 x 16 outputs.  The FP8 matrix instruction aligns the products
// of eight consecutive inputs to the largest of them and drops what lies
// 2^-13 below it (measured: a product of 2^16 next to one of 2^2 loses the
// latter, inputs eight apart keep it), which leaves y within 5e-5 of itself
// on rows with outlier columns: a thirtieth of a bf16 y's own rounding, but
// too much for a float32 one.  EXACT converts the codes to bf16 (exact) and
// sums the run with four bf16 matrix instructions, at half the rate.
template <bool EXACT>
__device__ __forceinline__ floatx4 mfma_run(i32x8 w, i32x8 a) {
  floatx4 d = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (!EXACT) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, d, 0, 0, 0, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(w[2 * i], w[2 * i + 1]),
                                                  codes_bf16(a[2 * i], a[2 * i + 1]), d, 0, 0,
                                                  0);
    return d;
  }
}

// Outputs n .. n+3 of a row of N (one store where rows keep its alignment).
__device__ __forceinline__ void store4(float* row, int n, int N, floatx4 v) {
  if (N % 4 == 0) {
    if (n < N) *reinterpret_cast<floatx4*>(row + n) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) row[n + i] = v[i];
  }
}
__device__ __forceinline__ void store4(uint16_t* row, int n, int N, floatx4 v) {
  if (N % 4 == 0) {
    if (n < N)
      *reinterpret_cast<u32x2*>(row + n) =
          u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) row[n + i] = f32_to_bf16(v[i]);
  }
}

// One workgroup: 16 outputs of up to 16 rows; wave v sums the runs v, v + 8,
// ..., and the eight sums meet in LDS.
template <typename YT>
__global__ __launch_bounds__(512) void fp8_stream_kernel(Fp8Args p) {
  constexpr bool kExact = sizeof(YT) == 4;
  __shared__ floatx4 part[8][kWave];
  Tile t;
  if (!find_tile<16>(p, blockIdx.y, t)) return;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int n0 = blockIdx.x * 16, g = lane >> 4, c = lane & 15;
  const int src = c < t.count ? source_row(p, t.row0 + c) : -1;
  const size_t arow = src < 0 ? 0 : src;
  const uint8_t* a = p.a + arow * p.K;
  const float* sa = p.as + arow * p.KB;
  const bool w_in = n0 + c < p.N;
  const uint8_t* w = p.w + (static_cast<size_t>(t.e) * p.N + (w_in ? n0 + c : 0)) * p.K;
  const float* sw = p.ws + (static_cast<size_t>(t.e) * fp8_runs(p.N) + n0 / kFp8Run) * p.KB;
  floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb = wave; kb < p.KB; kb += 8) {
    const int k = kb * kFp8Run + 32 * g;
    const floatx4 P = mfma_run<kExact>(load_codes(w, k, p.K, w_in), load_codes(a, k, p.K, src >= 0));
    const float s = src >= 0 ? sa[kb] * sw[kb] : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(s, P[i], acc[i]);
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int v = 1; v < 8; ++v) acc += part[v][lane];
  if (c < t.count)
    store4(static_cast<YT*>(p.y) + static_cast<size_t>(t.row0 + c) * p.N, n0 + 4 * g, p.N, acc);
}

// ---- tiles through LDS --------------------------------------------------------
//
// BN outputs x BM rows per workgroup, WN x WM per wave, one run (128 inputs,
// a 128-byte row of LDS) per step.  Two LDS buffers: while the waves work on
// one, the next run's codes and row scales come in with buffer_load ... lds
// (16 bytes per lane, no registers in between); one barrier per step.  A
// buffer load past its descriptor's end writes zeros, which covers rows past
// the tile and, with the offset pushed out of range, the inputs from K on.
//
// LDS rows hold their eight 16-byte chunks at chunk ^ key(row), so that the
// 16 lanes that read 16 bytes each at a time, from 16 rows, hit all 64 banks
// (two rows' chunk slots): rows of one parity have eight keys.  Matrix tile
// i of 64 outputs takes the LDS rows 16 (r / 4) + 4 i + r % 4 (r = 0..15), so
// that a lane's results over the four tiles are 16 consecutive outputs and
// a row of y is written in whole 128-byte lines.
__device__ __forceinline__ int w_key(int row) { return ((row >> 1) & 1) | ((row >> 3) & 6); }
__device__ __forceinline__ int a_key(int row) { return (row >> 1) & 7; }

// Descriptor of `bytes` bytes at address v (raw, no stride); wave-uniform.
__device__ __forceinline__ u32x4 buffer_of(uint64_t v, uint32_t bytes) {
  return u32x4{static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v))),
               static_cast<uint32_t>(
                   __builtin_amdgcn_readfirstlane(static_cast<int>((v >> 32) & 0xffff))),
               static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(bytes))),
               0x00020000u};
}
// 16 (4) bytes per lane from descriptor r at off to LDS address
// lds + 16 (4) lane.  The s_nop covers the wait states between a vector
// write of the descriptor's scalars, or the write of m0, and the load.
__device__ __forceinline__ void load_lds16(u32x4 r, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds),
               "v"(off), "s"(r)
               : "memory");
}
__device__ __forceinline__ void load_lds4(u32x4 r, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds),
               "v"(off), "s"(r)
               : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (const __attribute__((address_space(3))) void*)p));
}

// Sixteen consecutive outputs n .. n+15 of a row.
__device__ __forceinline__ void store16(float* row, int n, int N, const floatx4 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) store4(row, n + 4 * i, N, v[i]);
}
__device__ __forceinline__ void store16(uint16_t* row, int n, int N, const floatx4 (&v)[4]) {
  if (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < 4; i += 2)
      if (n + 4 * i < N)
        *reinterpret_cast<u32x4*>(row + n + 4 * i) =
            u32x4{pack_bf16x2(v[i][0], v[i][1]), pack_bf16x2(v[i][2], v[i][3]),
                  pack_bf16x2(v[i + 1][0], v[i + 1][1]), pack_bf16x2(v[i + 1][2], v[i + 1][3])};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) store4(row, n + 4 * i, N, v[i]);
  }
}

// XCD-aware order: workgroup ids go round the 8 XCDs, so each XCD gets a
// contiguous run of the tile order, in which panels of 4 output tiles run
// over the row tiles: the 32 tiles an XCD works on at a time share 4 weight
// and 8 row tiles in its L2.
__device__ __forceinline__ void tile_of(int id, int n_tiles, int m_tiles, int& nt, int& mt) {
  constexpr int kXcds = 8, kPanel = 4;
  const int total = n_tiles * m_tiles;
  const int per = total / kXcds, more = total % kXcds;
  const int xcd = id % kXcds;
  const int t = xcd * per + min(xcd, more) + id / kXcds;
  const int panel = t / (kPanel * m_tiles);
  const int width = min(kPanel, n_tiles - panel * kPanel);
  const int r = t - panel * kPanel * m_tiles;
  nt = panel * kPanel + r % width;
  mt = r / width;
}

template <int BN, int BM, int WN, int WM, int STAGES, typename YT>
__global__ __launch_bounds__(BN / WN * (BM / WM) * kWave) void fp8_tile_kernel(Fp8Args p,
                                                                               int n_tiles,
                                                                               int m_tiles) {
  constexpr bool kExact = sizeof(YT) == 4;
  constexpr int kWaves = BN / WN * (BM / WM);
  constexpr int kRowsPerLoad = 8 * kWaves;      // 8 LDS rows per wave instruction
  constexpr int kWLoads = BN / kRowsPerLoad, kALoads = BM / kRowsPerLoad;
  static_assert(kWLoads == 4 && kALoads == 4 && kRowsPerLoad % 32 == 0, "four loads each");
  static_assert(WN % 64 == 0 && kFp8Run % WN == 0 && WM % 16 == 0, "");
  constexpr int kABase = BN * kFp8Run, kSBase = kABase + BM * kFp8Run;
  constexpr int kSwWave = BM / kWave;           // the wave that loads the weight scales
  constexpr int kStage = kSBase + kWaves * kWave * 4;
  constexpr int kAhead = STAGES - 1;            // runs in flight
  constexpr int kLoads = kWLoads + kALoads + 1;   // of a wave per run
  static_assert(kSwWave < kWaves && BN / kFp8Run <= kWave, "");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES][kStage];
  int nt, mt;
  tile_of(blockIdx.x, n_tiles, m_tiles, nt, mt);
  Tile t;
  if (!find_tile<BM>(p, mt, t)) return;
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
  t.count = __builtin_amdgcn_readfirstlane(t.count);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n0 = nt * BN;
  const int K = p.K, KB = p.KB;

  // what this thread loads: LDS row lr + i kRowsPerLoad, chunk lane % 8
  const int lr = 8 * wave + (lane >> 3);
  const int ac = 16 * ((lane & 7) ^ a_key(lr));
  auto wc = [&](int i) { return 16 * ((lane & 7) ^ w_key(lr + i * kRowsPerLoad)); };
  uint32_t woff[kWLoads], aoff[kALoads];
#pragma unroll
  for (int i = 0; i < kWLoads; ++i) woff[i] = (lr + i * kRowsPerLoad) * K + wc(i);
  const uint8_t* abase = p.a;
  const float* sabase = p.as;
  uint32_t abytes, sabytes;
  constexpr uint32_t kOut = 0x80000000u;
  // the first waves load the row scales, wave kSwWave a scale per 128
  // outputs, the others zeros (every wave counts the same loads)
  uint32_t soff = kOut;
  if (p.rows == nullptr) {
    abase += static_cast<size_t>(t.row0) * K;
    sabase += static_cast<size_t>(t.row0) * KB;
    abytes = t.count * K;
    sabytes = t.count * KB * 4;
#pragma unroll
    for (int i = 0; i < kALoads; ++i) aoff[i] = (lr + i * kRowsPerLoad) * K + ac;
    if (wave < kSwWave) soff = threadIdx.x * KB * 4;
  } else {
    abytes = static_cast<uint32_t>(p.a_rows) * K;       // below 2^31 (host)
    sabytes = static_cast<uint32_t>(p.a_rows) * KB * 4;
#pragma unroll
    for (int i = 0; i < kALoads; ++i) {
      const int r = lr + i * kRowsPerLoad;
      const int src = r < t.count ? source_row(p, t.row0 + r) : -1;
      aoff[i] = src < 0 ? kOut : static_cast<uint32_t>(src) * K + ac;
    }
    if (static_cast<int>(threadIdx.x) < min(BM, t.count)) {
      const int src = source_row(p, t.row0 + threadIdx.x);
      if (src >= 0) soff = static_cast<uint32_t>(src) * KB * 4;
    }
  }
  const uint8_t* wbase = p.w + (static_cast<size_t>(t.e) * p.N + n0) * K;
  const uint32_t wbytes = min(BN, p.N - n0) * K;
  if (wave == kSwWave) {
    const int blocks = fp8_runs(p.N), b0 = n0 / kFp8Run;
    sabase = p.ws + (static_cast<size_t>(t.e) * blocks + b0) * KB;
    sabytes = min(BN / kFp8Run, blocks - b0) * KB * 4;
    soff = lane < BN / kFp8Run ? lane * KB * 4 : kOut;
  }
  const int tail = K % kFp8Run;      // inputs of the last run, 0: all 128

  const uint32_t lds_base = __builtin_amdgcn_readfirstlane(lds_address(lds)) + wave * 1024;
  const uint32_t lds_scales = lds_base - wave * 1024 + kSBase + wave * 256;
  // the next run to load: its bases and the bytes behind them
  uint64_t wp = reinterpret_cast<uint64_t>(wbase), ap = reinterpret_cast<uint64_t>(abase),
           sp = reinterpret_cast<uint64_t>(sabase);
  uint32_t wleft = wbytes, aleft = abytes, sleft = sabytes;
  auto cut = [&]() {   // the last run: inputs from K on read as zeros
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      woff[i] = wc(i) >= tail ? kOut : woff[i];
      aoff[i] = ac >= tail ? kOut : aoff[i];
    }
  };
  // load n (0 .. kLoads - 1) of the next run into `stage`
  auto load = [&](int n, int stage) {
    const uint32_t at = stage * kStage;
    if (n < kWLoads)
      load_lds16(buffer_of(wp, wleft), woff[n],
                 lds_base + at + n * (kRowsPerLoad * kFp8Run));
    else if (n < kWLoads + kALoads)
      load_lds16(buffer_of(ap, aleft), aoff[n - kWLoads],
                 lds_base + at + kABase + (n - kWLoads) * (kRowsPerLoad * kFp8Run));
    else
      load_lds4(buffer_of(sp, sleft), soff, lds_scales + at);
  };
  // moves on to run kb; from KB on the descriptors are empty and the loads
  // only write zeros
  auto advance = [&](int kb) {
    wp += kFp8Run;
    ap += kFp8Run;
    sp += 4;
    wleft = kb < KB ? wleft - kFp8Run : 0;
    aleft = kb < KB ? aleft - kFp8Run : 0;
    sleft = kb < KB ? sleft - 4 : 0;
    if (tail != 0 && kb == KB - 1) cut();
  };

  const int wn = (wave % (BN / WN)) * WN, wm = (wave / (BN / WN)) * WM;
  const int g = lane >> 4, c = lane & 15;
  floatx4 acc[WN / 16][WM / 16];
#pragma unroll
  for (int i = 0; i < WN / 16; ++i)
#pragma unroll
    for (int j = 0; j < WM / 16; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  // fragment of LDS row `row` (16-byte chunks 2 g and 2 g + 1)
  auto fragment = [&](const uint8_t* base, int row, int key) {
    const u32x4 lo = *reinterpret_cast<const u32x4*>(base + row * kFp8Run + 16 * ((2 * g) ^ key));
    const u32x4 hi =
        *reinterpret_cast<const u32x4*>(base + row * kFp8Run + 16 * ((2 * g + 1) ^ key));
    return i32x8{static_cast<int>(lo[0]), static_cast<int>(lo[1]), static_cast<int>(lo[2]),
                 static_cast<int>(lo[3]), static_cast<int>(hi[0]), static_cast<int>(hi[1]),
                 static_cast<int>(hi[2]), static_cast<int>(hi[3])};
  };

  constexpr int TI = WN / 16, TJ = WM / 16;
  auto w_fragment = [&](const uint8_t* st, int i) {
    const int row = wn + 64 * (i / 4) + 16 * (c >> 2) + 4 * (i % 4) + (c & 3);
    return fragment(st, row, w_key(row));
  };
  if (tail != 0 && KB == 1) cut();
  for (int kb = 0; kb < kAhead; ++kb) {
#pragma unroll
    for (int n = 0; n < kLoads; ++n) load(n, kb);
    advance(kb + 1);
  }
  // Step kb: the products of run kb - 1 that are left (its last two weight
  // rows of tiles), under which the first operands of run kb are read, then
  // run kb up to its own last two rows.  All reads of a run are thus done
  // before the barrier that ends the step it began in, the loads of a run
  // have that whole step to arrive, and the matrix pipe does not wait for
  // LDS behind the barrier.
  constexpr int kRows = 2, kRest = kRows * TJ, kProducts = TI * TJ;
  // the scaled addition of a product comes kLag products after its issue: by
  // then the matrix pipe has finished it and works on the later ones
  constexpr int kLag = kExact ? 1 : 3;
  // a load per kEvery products: issued in one go the loads fill the address
  // queue and hold up the wave's matrix instructions
  constexpr int kEvery = kProducts >= 2 * kLoads ? 2 : 1;
  static_assert(kProducts >= kEvery * kLoads && TI % 4 == 0, "every load has a place");
  i32x8 fa[TJ], fw[4];       // row i of weight tiles in fw[i % 4]
  float s_old[TJ], s[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    fa[j] = i32x8{};
    s[j] = 0.0f;
  }
  fw[2] = fw[3] = i32x8{};
  int stage = 0;
  floatx4 P[kLag + 1];
  // product n of a step: the remaining rows column by column, so that each
  // column's fa is free for the next run early, then the rows in order
  auto row_of = [](int n) { return n < kRest ? TI - kRows + n % kRows : (n - kRest) / TJ; };
  auto col_of = [](int n) { return n < kRest ? n / kRows : (n - kRest) % TJ; };
  auto add = [&](int n) {
    const int i = row_of(n), j = col_of(n);
    const float f = n < kRest ? s_old[j] : s[j];
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(f, P[n % (kLag + 1)][r], acc[i][j][r]);
    asm volatile("" : "+v"(acc[i][j]));   // here, not at the end of the step
  };
  for (int kb = 0; kb < KB; ++kb) {
    // this wave's loads of run kb have arrived (later runs' may still be in
    // flight) and its reads of run kb - 1 are done; after the barrier that
    // holds for every wave
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kAhead - 1) * kLoads) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const uint8_t* st = lds[stage];
    const int next = stage == 0 ? STAGES - 1 : stage - 1;
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    const float* sc = reinterpret_cast<const float*>(st + kSBase);
    const float swk = sc[BM + wn / kFp8Run];
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      s_old[j] = s[j];
      s[j] = sc[wm + 16 * j + c];
    }
#pragma unroll
    for (int n = 0; n < kProducts; ++n) {
      const int i = row_of(n), j = col_of(n);
      if (n < 2) fw[n] = w_fragment(st, n);
      if (n >= kRest && j == 0) fw[(i + 2) % 4] = w_fragment(st, i + 2);
      P[n % (kLag + 1)] = mfma_run<kExact>(fw[i % 4], fa[j]);
      if (n < kRest && n % kRows == kRows - 1) {
        const int row = wm + 16 * j + c;
        fa[j] = fragment(st + kABase, row, a_key(row));
      }
      if (n == kRest) {
#pragma unroll
        for (int u = 0; u < TJ; ++u) s[u] *= swk;
      }
      if (n % kEvery == kEvery - 1 && n / kEvery < kLoads) load(n / kEvery, next);
      if constexpr (!kExact) __builtin_amdgcn_sched_barrier(0);
      if (n >= kLag) add(n - kLag);
      if constexpr (!kExact) __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int n = kProducts - kLag; n < kProducts; ++n) add(n);
    advance(kb + kAhead + 1);
  }
#pragma unroll
  for (int n = 0; n < kRest; ++n) {
    const int i = row_of(n), j = col_of(n);
    const floatx4 D = mfma_run<kExact>(fw[i % 4], fa[j]);
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(s[j], D[r], acc[i][j][r]);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load outlives its LDS
#pragma unroll
  for (int j = 0; j < WM / 16; ++j) {
    const int m = wm + 16 * j + c;
    if (m >= t.count) continue;
    YT* row = static_cast<YT*>(p.y) + static_cast<size_t>(t.row0 + m) * p.N;
#pragma unroll
    for (int i = 0; i < WN / 16; i += 4) {
      const floatx4 v[4] = {acc[i][j], acc[i + 1][j], acc[i + 2][j], acc[i + 3][j]};
      store16(row, n0 + wn + 16 * i + 16 * g, p.N, v);
    }
  }
}

template <int BN, int BM, int WN, int WM, int STAGES, typename YT>
hipError_t launch_tile(const Fp8Args& p, int live, hipStream_t stream) {
  const int n_tiles = (p.N + BN - 1) / BN;
  const int m_tiles = static_cast<int>((p.M + static_cast<int64_t>(live) * (BM - 1)) / BM);
  fp8_tile_kernel<BN, BM, WN, WM, STAGES, YT>
      <<<dim3(n_tiles * m_tiles), BN / WN * (BM / WM) * kWave, 0, stream>>>(p, n_tiles, m_tiles);
  return hipGetLastError();
}

}  // namespace

namespace {

template <typename YT>
hipError_t launch_by_size(const Fp8Args& p, hipStream_t stream) {
  // experts with rows; sum_e ceil(c_e / BM) <= (M + live (BM - 1)) / BM
  const int live = p.offsets == nullptr ? 1 : (p.E < p.M ? p.E : p.M);
  // the tiles' buffer offsets reach 2^31 bytes into a where rows are gathered
  const bool reach = p.rows == nullptr || static_cast<int64_t>(p.a_rows) * p.K < (int64_t{1} << 31);
  if (p.M > 64 * live && reach) {
    if constexpr (sizeof(YT) == 2) {
      if (p.M > 512 * live) return launch_tile<256, 256, 128, 64, 2, YT>(p, live, stream);
    }
    return launch_tile<128, 128, 64, 64, 4, YT>(p, live, stream);
  }
  const dim3 grid((p.N + 15) / 16, (p.M + live * 15) / 16);
  fp8_stream_kernel<YT><<<grid, 512, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_gemm(const harp_fp8_weight& W, const uint8_t* a, const float* a_scale,
                           int a_rows, const int32_t* rows, const int32_t* offsets, void* y,
                           int y_dt, int M, hipStream_t stream) {
  const Fp8Args p{W.w, W.scale, a,   a_scale,        rows,      offsets, y,
                  W.N, W.K,     fp8_runs(W.K), W.experts, M,       a_rows};
  return y_dt == HARP_BF16 ? launch_by_size<uint16_t>(p, stream)
                           : launch_by_size<float>(p, stream);
}

}  // namespace harp
