// The FP8 (e4m3) product with a float32 scale per 1 x 128 run of a and per
// 128 x 128 block of w, dense and grouped by expert:
//
//     y[m][n] = sum_b sa[m][b] sw[n/128][b] P_b[m][n],
//     P_b[m][n] = sum_{k in run b} a[m][k] w[n][k].
//
// For a bf16 y one v_mfma_f32_16x16x128_f8f6f4 forms P_b of 16 x 16 outputs
// (its 128 inputs are one run), so the scales enter once per matrix
// instruction as four fused multiply-adds per lane.  The weights are the row
// operand and a the column operand: a lane holds four consecutive outputs of
// one row of y, which share one factor sa sw.
//
// What bounds it (MI355X): with few rows the pass over the weights (16 x
// 28672 x 8192: 44.8 us, 5.3 TB/s; 64 rows over 64 experts of 4096 x 4096:
// 84 us, 5.4 TB/s; 1 x 4096 x 4096: 5.4 us, latency); with many rows power
// (4096 x 28672 x 8192: 784 to 827 us, 2.33 PFLOP/s and more, matrix pipe
// 68 % busy; 631 us with zeros as inputs); in between how many tiles there
// are for 256 CUs (512 x 4096 x 4096: 15.7 us, 1.09 PFLOP/s).
#include <type_traits>

#include "fp8_common.hpp"
#include "fp8_pick.hpp"
#include "launch.hpp"
#include "validate.hpp"

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

// The tile a workgroup works on: outputs from nt BN on of the rows
// [row0, row0 + count) of expert e.  near_rows row tiles next to each other in
// the order work on its weights, it is the row_at-th of them; and near_outs
// output tiles on its rows, out_at.
struct Tile {
  int e, nt, row0, count;
  int row_at, near_rows, out_at, near_outs;
};

// Order of the tiles: expert after expert; an expert's k row tiles x n_tiles
// output tiles in panels of w = max(4, 32 / k) output tiles, a panel in
// blocks of 8 row tiles, in which the row tiles of one output tile follow
// each other.  Workgroup ids go round the 8 XCDs; each XCD takes a contiguous
// eighth of the order, so that the 32 tiles it works on at a time are up to
// 8 row tiles x w output tiles that share weights and rows in its L2.
// (64 rows over 64 experts 105 -> 96 us, 8192 over 32 441 -> 423 us against
// output panels over all experts per XCD.)
// Each wave computes its place on its own: 64 experts at a time, an
// inclusive scan of their row tiles.  False: there is no such tile (grids
// are sized for the worst routing; m_tiles: row tiles they have room for).
template <int BM>
__device__ __forceinline__ bool find_tile(const Fp8Args& p, int id, int n_tiles, int m_tiles,
                                          Tile& t) {
  constexpr int kXcds = 8, kAtOnce = 32, kPanel = 4, kBlock = 8;
  const int lane = threadIdx.x & (kWave - 1);
  int start = 0, end = p.M, tiles = m_tiles, upto = m_tiles, all = m_tiles;
  auto look = [&](int e) {   // expert e of this lane: its rows and the scan
    start = end = 0;
    if (e < p.E) {
      start = min(max(p.offsets[e], 0), p.M);
      end = min(max(p.offsets[e + 1], 0), p.M);
    }
    tiles = (max(end - start, 0) + BM - 1) / BM;
    upto = tiles;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int u = __shfl_up(upto, o, kWave);
      if (lane >= o) upto += u;
    }
  };
  if (p.offsets != nullptr) {
    all = 0;
    for (int e0 = (p.E - 1) / kWave * kWave; e0 >= 0; e0 -= kWave) {
      look(e0 + lane);   // the last look is at experts 0 .. 63
      all = min(all + __shfl(upto, kWave - 1, kWave), m_tiles);
    }
  }
  const int total = all * n_tiles, per = total / kXcds, more = total % kXcds;
  const int xcd = id % kXcds, nth = id / kXcds;
  if (nth >= per + (xcd < more ? 1 : 0)) return false;
  const int place = xcd * per + min(xcd, more) + nth, slot = place / n_tiles;
  int first = 0, k = tiles;
  t.e = 0;
  t.row0 = 0;
  if (p.offsets != nullptr) {
    int before = 0;
    for (int e0 = 0;;) {
      const unsigned long long hit = __ballot(slot < before + upto);
      if (hit != 0) {
        const int src = __ffsll(hit) - 1;
        t.e = e0 + src;
        k = __shfl(tiles, src, kWave);
        first = before + __shfl(upto, src, kWave) - k;
        t.row0 = __shfl(start, src, kWave);
        end = __shfl(end, src, kWave);
        break;
      }
      before += __shfl(upto, kWave - 1, kWave);
      e0 += kWave;
      if (e0 >= p.E) return false;
      look(e0 + lane);
    }
  }
  const int w = max(kPanel, kAtOnce / k);
  const int r = place - first * n_tiles, panel = r / (w * k);
  const int width = min(w, n_tiles - panel * w), in = r - panel * w * k;
  const int block = in / (kBlock * width), rest = in - block * kBlock * width;
  const int height = min(kBlock, k - block * kBlock);
  t.row_at = rest % height;
  t.near_rows = height;
  t.out_at = rest / height;
  t.near_outs = width;
  t.nt = panel * w + t.out_at;
  t.row0 += BM * (block * kBlock + t.row_at);
  t.count = min(BM, end - t.row0);
  return true;
}

// The a row of output row i (< M), -1 for one that reads nothing.
__device__ __forceinline__ int source_row(const Fp8Args& p, int i) {
  const int r = p.rows == nullptr ? i : p.rows[i];
  return r >= 0 && r < p.a_rows ? r : -1;
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
// A buffer offset past the end of every descriptor used here: those are at
// most kFp8MaxGather bytes (gathered rows) or 256 rows of K.
constexpr uint32_t kOut = kFp8MaxGather;

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi) {
  return i32x8{static_cast<int>(lo[0]), static_cast<int>(lo[1]), static_cast<int>(lo[2]),
               static_cast<int>(lo[3]), static_cast<int>(hi[0]), static_cast<int>(hi[1]),
               static_cast<int>(hi[2]), static_cast<int>(hi[3])};
}

// ---- tiles through LDS --------------------------------------------------------
//
// BN outputs x BM rows per workgroup, WN x WM per wave, one run (128 inputs,
// a 128-byte row of LDS) per step of a group of waves.  KG groups take the
// runs in turn and meet at the end (for few tiles: more waves per tile and
// fewer steps).  STAGES LDS buffers per group: while the waves work on one,
// the next runs' codes and scales come in with buffer_load ... lds (16 bytes
// per lane, no registers in between); one barrier per step.  A buffer load
// past its descriptor's end writes zeros, which covers rows past the tile
// and, with the offset pushed out of range, the inputs from K on.
//
// With S = up to 4 matrix tiles of 16 outputs side by side in a wave, tile i
// takes the LDS rows 4 S (r / 4) + 4 i + r % 4 (r = 0..15), so that a lane's
// results over the S tiles are 4 S consecutive outputs and a row of y is
// written in long pieces (whole 128-byte lines for S = 4).
// LDS rows hold their eight 16-byte chunks at chunk ^ key(row).  A 16-byte
// read serves 16 lanes at a time, each from a row r of its own: lanes 0-3,
// 12-15 and 20-27, then 4-11, 16-19 and 28-31, and so on from 32 (measured).
// Both hold every r, but r = 4..11 in the other half of 32 lanes than the
// rest, which reads the chunk two places off: bit 1 of its place is r2 ^ r3
// (bits of r) or the complement.  With key = r1 + 6 r3 the place after the
// exclusive or has r1, r2 and r3 as its bits, up to constants, and r0 tells
// between two rows' slots, so the 16 reads fall on all 64 banks (4096 x
// 28672 x 8192: LDS busy 27 % of the time, against 51 % with the conflicts of
// key = r / 2; 820 -> 812 us, power binds there).
template <int S>
__device__ __forceinline__ int w_key(int row) {
  return ((row >> 1) & 1) | (6 * ((row >> (S == 4 ? 5 : S == 2 ? 4 : 3)) & 1));
}
__device__ __forceinline__ int a_key(int row) { return w_key<1>(row); }

// Descriptor of `bytes` bytes at p (raw, no stride); wave-uniform.
__device__ __forceinline__ u32x4 buffer_of(const void* p, uint32_t bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return u32x4{static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v))),
               static_cast<uint32_t>(
                   __builtin_amdgcn_readfirstlane(static_cast<int>((v >> 32) & 0xffff))),
               static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(bytes))),
               0x00020000u};
}
// 16 (4) bytes per lane from descriptor r at off to LDS address
// lds + 16 (4) lane.  The s_nop is the wait state between the write of m0 and
// the load.  A load also needs five behind a vector instruction's write of a
// scalar that it reads, which the compiler does not see to for inline
// assembly: settle() stands in front of the first load of all, whose r comes
// from v_readfirstlane; later r are scalar arithmetic's, but where the compiler
// spills scalars, v_readlane brings them back, and the build looks through the
// machine code and refuses a load that follows too closely (build.py).  Five
// wait states in each block would do as well, at up to 2 % of the large
// products and 8 % of 64 x 4096 x 4096 (6.5 -> 7.0 us).
__device__ __forceinline__ void load_lds16(u32x4 r, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds),
               "v"(off), "s"(r)
               : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(u32x4 r, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds),
               "v"(off), "s"(r)
               : "memory", "m0");
}
// The wait states between a vector write of a scalar and a load that uses it.
__device__ __forceinline__ void settle() { asm volatile("s_nop 7" ::: "memory"); }
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (const __attribute__((address_space(3))) void*)p));
}

// 4 S consecutive outputs from n on of a row whose length keeps 16 bytes'
// alignment.
template <int S>
__device__ __forceinline__ void store_outputs(float* row, int n, int N, const floatx4 (&v)[S]) {
#pragma unroll
  for (int i = 0; i < S; ++i)
    if (n + 4 * i < N) *reinterpret_cast<floatx4*>(row + n + 4 * i) = v[i];
}
template <int S>
__device__ __forceinline__ void store_outputs(uint16_t* row, int n, int N,
                                              const floatx4 (&v)[S]) {
  if constexpr (S == 1) {
    if (n < N)
      *reinterpret_cast<u32x2*>(row + n) =
          u32x2{pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3])};
  } else {
#pragma unroll
    for (int i = 0; i < S; i += 2)
      if (n + 4 * i < N)
        *reinterpret_cast<u32x4*>(row + n + 4 * i) =
            u32x4{pack_bf16x2(v[i][0], v[i][1]), pack_bf16x2(v[i][2], v[i][3]),
                  pack_bf16x2(v[i + 1][0], v[i + 1][1]), pack_bf16x2(v[i + 1][2], v[i + 1][3])};
  }
}

template <int BN, int BM, int WN, int WM, int KG, int STAGES, typename YT>
__global__ __launch_bounds__(KG* BN / WN * (BM / WM) * kWave) void fp8_tile_kernel(Fp8Args p,
                                                                                   int n_tiles,
                                                                                   int m_tiles) {
  constexpr bool kExact = sizeof(YT) == 4;
  constexpr int G = BN / WN * (BM / WM);        // waves of a group
  constexpr int TI = WN / 16, TJ = WM / 16;     // a wave's matrix tiles
  constexpr int S = TI < 4 ? TI : 4;            // of them side by side
  constexpr int kRowsPerLoad = 8 * G;           // 8 LDS rows per wave instruction
  constexpr int kARows = (BM + kRowsPerLoad - 1) / kRowsPerLoad * kRowsPerLoad;
  constexpr int kWLoads = BN / kRowsPerLoad, kALoads = kARows / kRowsPerLoad;
  static_assert(BN % kRowsPerLoad == 0 && TI % S == 0 && S != 3, "");
  static_assert(BN <= kFp8Run ? kFp8Run % BN == 0 : BN % kFp8Run == 0, "");
  static_assert(kFp8Run % WN == 0 && WM % 16 == 0, "");
  // scales: 64 to a slot; first the rows', then one per 128 outputs
  constexpr int kRowSlots = (BM + kWave - 1) / kWave, kBlocks = (BN + kFp8Run - 1) / kFp8Run;
  constexpr int kSLoads = (kRowSlots + 1 + G - 1) / G, kSlots = kSLoads * G;
  constexpr int kAhead = STAGES - 1;            // runs in flight
  constexpr int kLoads = kWLoads + kALoads + kSLoads;   // of a wave per run
  // The 256 x 256 tile has room for two runs in LDS only, so a run's loads
  // have at most one step to arrive, less than a line from beyond L2 takes
  // at times.  Its waves therefore also ask for one dword of each line three
  // runs further on, which brings the line into L2; each workgroup asks for
  // its share of the lines it has in common with its neighbours.  These two
  // loads are a step's last and may stay in flight over the barrier (4096 x
  // 28672 x 8192: 812 -> 793 us on one card, 847 -> 826 on another, there 721 ->
  // 631 with zeros as inputs; 512 rows 134 -> 126).  Tiles with three stages or two workgroups a CU lose by it
  // (256 x 128 grouped 426 -> 479 us, 128 x 128 1024 -> 1112).
  constexpr bool kTouch = BN + BM > 384;
  constexpr int kTouches = kTouch ? 2 : 0, kTouchAhead = 2;
  static_assert(kAhead * kTouches + (kAhead - 1) * kLoads < 64, "the counter of loads in flight");
  static_assert(!kTouch || (KG == 1 && TI >= 4 && !kExact), "touch() stands there only");
  // one array: the stages' w rows, their a rows, their scales, so that a
  // stage is an immediate offset of the reads
  constexpr int kWRun = BN * kFp8Run, kARun = kARows * kFp8Run, kSRun = kSlots * kWave * 4;
  constexpr int kABase = STAGES * KG * kWRun, kSBase = kABase + STAGES * KG * kARun;
  constexpr int kTBase = kSBase + STAGES * KG * kSRun;   // 256 bytes per wave, never read
  constexpr int kLds = kTBase + (kTouch ? G * kWave * 4 : 0);
  static_assert(kLds <= 160 * 1024 && (KG - 1) * G * TI * TJ * 1024 <= kLds, "");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  Tile t;
  if (!find_tile<BM>(p, blockIdx.x, n_tiles, m_tiles, t)) return;
  t.nt = __builtin_amdgcn_readfirstlane(t.nt);
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
  t.count = __builtin_amdgcn_readfirstlane(t.count);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int group = KG == 1 ? 0 : wave / G, gw = KG == 1 ? wave : wave % G;
  const int n0 = t.nt * BN;
  const int K = p.K, KB = p.KB;

  // what this lane loads: LDS rows lr + i kRowsPerLoad, chunk lane % 8
  const int lr = 8 * gw + (lane >> 3);
  auto wc = [&](int i) { return 16 * ((lane & 7) ^ w_key<S>(lr + i * kRowsPerLoad)); };
  auto ac = [&](int i) { return 16 * ((lane & 7) ^ a_key(lr + i * kRowsPerLoad)); };
  uint32_t woff[kWLoads], aoff[kALoads], soff[kSLoads];
#pragma unroll
  for (int i = 0; i < kWLoads; ++i) woff[i] = (lr + i * kRowsPerLoad) * K + wc(i);
  const uint8_t* abase = p.a;
  const float* asbase = p.as;
  uint32_t abytes, asbytes;
  if (p.rows == nullptr) {
    abase += static_cast<size_t>(t.row0) * K;
    asbase += static_cast<size_t>(t.row0) * KB;
    abytes = t.count * K;
    asbytes = t.count * KB * 4;
#pragma unroll
    for (int i = 0; i < kALoads; ++i) aoff[i] = (lr + i * kRowsPerLoad) * K + ac(i);
  } else {
    abytes = static_cast<uint32_t>(p.a_rows) * K;
    asbytes = static_cast<uint32_t>(p.a_rows) * KB * 4;
#pragma unroll
    for (int i = 0; i < kALoads; ++i) {
      const int r = lr + i * kRowsPerLoad;
      const int src = r < t.count ? source_row(p, t.row0 + r) : -1;
      aoff[i] = src < 0 ? kOut : static_cast<uint32_t>(src) * K + ac(i);
    }
  }
  const uint8_t* wbase = p.w + (static_cast<size_t>(t.e) * p.N + n0) * K;
  const uint32_t wbytes = min(BN, p.N - n0) * K;
  const int blocks = fp8_runs(p.N), b0 = n0 / kFp8Run;
  const float* wsbase = p.ws + (static_cast<size_t>(t.e) * blocks + b0) * KB;
  const uint32_t wsbytes = min(kBlocks, blocks - b0) * KB * 4;
  const int tail = K % kFp8Run;      // inputs of the last run, 0: all 128

  const uint32_t lds_base = __builtin_amdgcn_readfirstlane(lds_address(lds));
  const uint32_t lds_w = lds_base + group * kWRun + gw * 1024,
                 lds_a = lds_base + kABase + group * kARun + gw * 1024,
                 lds_s = lds_base + kSBase + group * kSRun + gw * (kWave * 4);
  // descriptors of the group's next run to load: its bases and the bytes
  // behind them
  auto first = [&](const void* base, uint32_t bytes, int by) {
    return buffer_of(static_cast<const uint8_t*>(base) + group * by,
                     group < KB ? bytes - group * by : 0);
  };
  u32x4 dw = first(wbase, wbytes, kFp8Run), da = first(abase, abytes, kFp8Run), ds[kSLoads];
#pragma unroll
  for (int u = 0; u < kSLoads; ++u) {
    const int slot = gw + u * G;
    const bool of_rows = slot < kRowSlots;
    ds[u] = of_rows ? first(asbase, asbytes, 4) : first(wsbase, wsbytes, 4);
    soff[u] = of_rows ? (slot * kWave + lane) * KB * 4 : lane * KB * 4;
    if (slot > kRowSlots || (!of_rows && lane >= kBlocks)) soff[u] = kOut;
    if (of_rows && p.rows != nullptr) {
      const int r = slot * kWave + lane;
      const int src = r < min(BM, t.count) ? source_row(p, t.row0 + r) : -1;
      soff[u] = src < 0 ? kOut : static_cast<uint32_t>(src) * KB * 4;
    }
  }
  auto cut = [&]() {   // the last run: inputs from K on read as zeros
#pragma unroll
    for (int i = 0; i < kWLoads; ++i) woff[i] = wc(i) >= tail ? kOut : woff[i];
#pragma unroll
    for (int i = 0; i < kALoads; ++i) aoff[i] = ac(i) >= tail ? kOut : aoff[i];
  };
  // Load n (0 .. kLoads - 1) of the next run into `stage`.  The last load
  // through a descriptor moves it on to the group's run after that; where
  // there is none (keep == 0) it is left empty, and the loads through it
  // write zeros and read nothing.
  uint32_t keep = 0;
  auto move = [&](u32x4& d, uint32_t by) {
    const uint64_t v = (static_cast<uint64_t>(d[1]) << 32 | d[0]) + by;
    d[0] = static_cast<uint32_t>(v);
    d[1] = static_cast<uint32_t>(v >> 32);
    d[2] = (d[2] - by) & keep;
  };
  auto load = [&](int n, int stage) {
    if (n < kWLoads) {
      load_lds16(dw, woff[n], lds_w + stage * (KG * kWRun) + n * (kRowsPerLoad * kFp8Run));
      if (n == kWLoads - 1) move(dw, KG * kFp8Run);
    } else if (n < kWLoads + kALoads) {
      const int i = n - kWLoads;
      load_lds16(da, aoff[i], lds_a + stage * (KG * kARun) + i * (kRowsPerLoad * kFp8Run));
      if (i == kALoads - 1) move(da, KG * kFp8Run);
    } else {
      const int u = n - kWLoads - kALoads;
      load_lds4(ds[u], soff[u], lds_s + stage * (KG * kSRun) + u * (G * kWave * 4));
      move(ds[u], KG * 4);
    }
  };
  // lane 8 r + i touches row r of the wave's load i, if that row is in its share
  uint32_t touch_w = kOut, touch_a = kOut, past = 0;
  if constexpr (kTouch) {
    static_assert(kWLoads <= 8 && kALoads <= 8, "");
    const int i = lane & 7, row = lr + i * kRowsPerLoad;
    if (i < kWLoads && row % t.near_rows == t.row_at) touch_w = row * K + kTouchAhead * kFp8Run;
    uint32_t at = kOut;
#pragma unroll
    for (int u = 0; u < kALoads; ++u)
      if (i == u && aoff[u] < kOut) at = aoff[u] - ac(u);
    if (at < kOut && row % t.near_outs == t.out_at) touch_a = at + kTouchAhead * kFp8Run;
  }
  // after the loads of a run, whose descriptors then stand at the next one
  auto touch = [&]() {
    if constexpr (kTouch) {
      load_lds4(dw, touch_w | past, lds_base + kTBase + gw * (kWave * 4));
      load_lds4(da, touch_a | past, lds_base + kTBase + gw * (kWave * 4));
    }
  };
  // before the loads of step s's run
  auto ready = [&](int s) {
    const int kb = s * KG + group;
    if (tail != 0 && kb == KB - 1) cut();
    keep = kb + KG < KB ? ~0u : 0u;
    if constexpr (kTouch) past = kb + 1 + kTouchAhead < KB ? 0u : kOut;
  };

  const int wn = (gw % (BN / WN)) * WN, wm = (gw / (BN / WN)) * WM;
  const int g = lane >> 4, c = lane & 15;
  floatx4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  // fragments: 16-byte chunks 2 g and 2 g + 1 of an LDS row.  All rows a
  // lane reads have one key, so a fragment is two addresses and an offset.
  const int wrow = wn + 4 * S * (c >> 2) + (c & 3), arow = wm + c;
  const uint8_t* wl = lds + group * kWRun + wrow * kFp8Run;
  const uint8_t* al = lds + kABase + group * kARun + arow * kFp8Run;
  const uint8_t *wlo = wl + 16 * ((2 * g) ^ w_key<S>(wrow)),
                *whi = wl + 16 * ((2 * g + 1) ^ w_key<S>(wrow));
  const uint8_t *alo = al + 16 * ((2 * g) ^ a_key(arow)),
                *ahi = al + 16 * ((2 * g + 1) ^ a_key(arow));
  auto w_fragment = [&](int stage, int i) {   // tile i: rows wrow + 16 S (i / S) + 4 (i % S)
    const int off = stage * (KG * kWRun) + (16 * S * (i / S) + 4 * (i % S)) * kFp8Run;
    return join(*reinterpret_cast<const u32x4*>(wlo + off),
                *reinterpret_cast<const u32x4*>(whi + off));
  };
  auto a_fragment = [&](int stage, int j) {
    const int off = stage * (KG * kARun) + 16 * j * kFp8Run;
    return join(*reinterpret_cast<const u32x4*>(alo + off),
                *reinterpret_cast<const u32x4*>(ahi + off));
  };
  const float* sc = reinterpret_cast<const float*>(lds + kSBase + group * kSRun);
  auto row_scale = [&](int stage, int j) { return sc[stage * (KG * kSRun / 4) + arow + 16 * j]; };
  auto weight_scale = [&](int stage) {
    return sc[stage * (KG * kSRun / 4) + kRowSlots * kWave + wn / kFp8Run];
  };
  // this wave's loads of the step's run have arrived (later ones, and the
  // touches behind each run's, may still be in flight) and its reads of the
  // step before are done; after the barrier that holds for every wave.  A group
  // of one wave loads for itself.
  auto arrive = [&]() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kAhead - 1) * kLoads + kAhead * kTouches)
                 : "memory");
    if constexpr (G > 1) __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  asm volatile("" : "+s"(dw), "+s"(da));
#pragma unroll
  for (int u = 0; u < kSLoads; ++u) asm volatile("" : "+s"(ds[u]));
  settle();
  for (int s = 0; s < kAhead; ++s) {
    ready(s);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) load(n, s);
    touch();
  }
  const int steps = (KB + KG - 1) / KG;
  auto all_steps = [&](auto step) {
    for (int s = 0; s < steps; s += STAGES) {
      step(s, std::integral_constant<int, 0>{});
      if (s + 1 < steps) step(s + 1, std::integral_constant<int, 1 % STAGES>{});
      if constexpr (STAGES > 2)
        if (s + 2 < steps) step(s + 2, std::integral_constant<int, 2 % STAGES>{});
      if constexpr (STAGES > 3)
        if (s + 3 < steps) step(s + 3, std::integral_constant<int, 3 % STAGES>{});
      if constexpr (STAGES > 4)
        if (s + 4 < steps) step(s + 4, std::integral_constant<int, 4 % STAGES>{});
      static_assert(STAGES >= 2 && STAGES <= 5, "");
    }
  };

  constexpr int kProducts = TI * TJ;
  // A wave with no row or no output of its own does its share of the loads
  // and leaves the matrix pipe to the others (8192 rows unevenly over 32
  // experts 439 -> 425 us, over 64 of 2048 x 4096 166 -> 162 us).
  const bool idle = (BM > WM && wm >= t.count) || (BN > WN && n0 + wn >= p.N);
  if (idle) {
    all_steps([&](int s, auto at) {
      arrive();
      ready(s + kAhead);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) load(n, (decltype(at)::value + kAhead) % STAGES);
      touch();
    });
  } else if constexpr (TI < 4) {
    all_steps([&](int s, auto at) {
      constexpr int stage = decltype(at)::value, next = (stage + kAhead) % STAGES;
      arrive();
      i32x8 fw[TI], fa[TJ];
      float f[TJ];
#pragma unroll
      for (int i = 0; i < TI; ++i) fw[i] = w_fragment(stage, i);
#pragma unroll
      for (int j = 0; j < TJ; ++j) fa[j] = a_fragment(stage, j);
      const float swk = weight_scale(stage);
#pragma unroll
      for (int j = 0; j < TJ; ++j) f[j] = row_scale(stage, j) * swk;
      ready(s + kAhead);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) load(n, next);
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int i = 0; i < TI; ++i) {
          const floatx4 P = mfma_run<kExact>(fw[i], fa[j]);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(f[j], P[r], acc[i][j][r]);
        }
    });
  } else if constexpr (kExact) {
    // The order of the branch below (there it is explained), with the
    // operands as bf16.  A sum is four matrix instructions; two sums, a pair,
    // are formed in turn.  The vector ALU's work is laid between them, two
    // conversions and one scaled addition to a matrix instruction (in turn
    // with another wave's those take 23 cycles, 17 without any), so that no
    // matrix instruction waits for an operand just converted: a fragment is
    // read a pair before its conversion, which is at least a pair before its
    // first use, and a sum is added a pair after it (200 x 11008 x 4096:
    // 37.8 -> 33.4 us against conversions in front of the sums).
    constexpr int kRest = TJ, kPairs = TI * TJ / 2, kHalf = TJ / 2;   // in pairs
    constexpr int kPer = (kLoads + kPairs - 1) / kPairs;
    static_assert(TJ % 2 == 0, "");
    // pair p's two outputs: of the last two rows of weight tiles column by
    // column, then of the other rows in order
    auto row_of = [](int p, int u) { return p < kRest ? TI - 2 + u : (p - kRest) / kHalf; };
    auto col_of = [](int p, int u) { return p < kRest ? p : (p - kRest) % kHalf * 2 + u; };
    // the pair in which a fragment is converted: after the last use of the
    // registers of the run before where there is room for that, and always
    // before the fragment's first use
    auto w_at = [](int i) { return i < TI - 2 ? kRest + i * kHalf - 1 : kPairs - TI + i; };
    auto a_at = [](int j) { return j + 1 < kRest + j / 2 - 1 ? j + 1 : kRest + j / 2 - 1; };
    i32x8 rw[TI], ra[TJ];                  // as read
    bf16x8 xw[TI][4], xa[TJ][4], na[TJ][4];
    floatx4 P[2][2];
    float f_old[TJ], f[TJ];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      xw[TI - 2][q] = xw[TI - 1][q] = bf16x8{};
#pragma unroll
      for (int j = 0; j < TJ; ++j) xa[j][q] = bf16x8{};
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) f[j] = 0.0f;
    P[1][0] = P[1][1] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    auto add = [&](int p, int u, const float (&by)[TJ]) {
      floatx4& to = acc[row_of(p, u)][col_of(p, u)];
#pragma unroll
      for (int r = 0; r < 4; ++r) to[r] = fmaf(by[col_of(p, u)], P[p % 2][u][r], to[r]);
      asm volatile("" : "+v"(to));   // here, not at the end of the step
    };
    all_steps([&](int s, auto at) {
      constexpr int stage = decltype(at)::value, next = (stage + kAhead) % STAGES;
      arrive();
      ready(s + kAhead);
      const float swk = weight_scale(stage);
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        f_old[j] = f[j];
        f[j] = row_scale(stage, j);
      }
#pragma unroll
      for (int p = 0; p < kPairs; ++p) {
#pragma unroll
        for (int i = 0; i < TI; ++i)
          if (w_at(i) - 1 == p) rw[i] = w_fragment(stage, i);
#pragma unroll
        for (int j = 0; j < TJ; ++j)
          if (a_at(j) - 1 == p) ra[j] = a_fragment(stage, j);
        if (p == kRest) {
#pragma unroll
          for (int u = 0; u < TJ; ++u) f[u] *= swk;
        }
#pragma unroll
        for (int u = p * kPer; u < (p + 1) * kPer && u < kLoads; ++u) load(u, next);
        __builtin_amdgcn_sched_barrier(0);
        P[p % 2][0] = P[p % 2][1] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
            P[p % 2][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                xw[row_of(p, u)][q], xa[col_of(p, u)][q], P[p % 2][u], 0, 0, 0);
#pragma unroll
          for (int i = 0; i < TI; ++i)
            if (w_at(i) == p) xw[i][q] = codes_bf16(rw[i][2 * q], rw[i][2 * q + 1]);
#pragma unroll
          for (int j = 0; j < TJ; ++j)
            if (a_at(j) == p) na[j][q] = codes_bf16(ra[j][2 * q], ra[j][2 * q + 1]);
          if (q >= 2) {
            if (p == 0)
              add(kPairs - 1, q - 2, f_old);
            else
              add(p - 1, q - 2, p - 1 < kRest ? f_old : f);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < TJ; ++j)
          if (a_at(j) == p) {
#pragma unroll
            for (int q = 0; q < 4; ++q) xa[j][q] = na[j][q];
          }
      }
    });
    static_assert(kPairs % 2 == 0, "the last pair's sums are in P[1]");
    add(kPairs - 1, 0, f);
    add(kPairs - 1, 1, f);
#pragma unroll
    for (int p = 0; p < kRest; ++p) {
      P[p % 2][0] = P[p % 2][1] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          P[p % 2][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              xw[row_of(p, u)][q], xa[col_of(p, u)][q], P[p % 2][u], 0, 0, 0);
      add(p, 0, f);
      add(p, 1, f);
    }
  } else {
    // Step s: the products of the run before that are left (its last two
    // rows of weight tiles), under which the first operands of this run are
    // read, then this run up to its own last two rows.  All reads of a run
    // are thus done before the barrier that ends the step it began in, the
    // loads of a run have that whole step to arrive, and the matrix pipe
    // does not wait for LDS behind the barrier.
    constexpr int kRows = 2, kRest = kRows * TJ;
    // the scaled addition of a product comes kLag products after its issue:
    // by then the matrix pipe has finished it and works on the later ones.
    constexpr int kLag = 3;
    constexpr int kPer = (kLoads + kProducts - 1) / kProducts;
    i32x8 fa[TJ], fw[4];       // row i of weight tiles in fw[i % 4]
    float f_old[TJ], f[TJ];
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      fa[j] = i32x8{};
      f[j] = 0.0f;
    }
    fw[2] = fw[3] = i32x8{};
    floatx4 P[4];
    // product n of a step: the remaining rows column by column, so that each
    // column's fa is free for this run early, then the rows in order
    auto row_of = [](int n) { return n < kRest ? TI - kRows + n % kRows : (n - kRest) / TJ; };
    auto col_of = [](int n) { return n < kRest ? n / kRows : (n - kRest) % TJ; };
    auto add = [&](int n) {
      const int i = row_of(n), j = col_of(n);
      const float by = n < kRest ? f_old[j] : f[j];
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(by, P[n % 4][r], acc[i][j][r]);
      asm volatile("" : "+v"(acc[i][j]));   // here, not at the end of the step
    };
    all_steps([&](int s, auto at) {
      constexpr int stage = decltype(at)::value, next = (stage + kAhead) % STAGES;
      arrive();
      ready(s + kAhead);
      const float swk = weight_scale(stage);
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        f_old[j] = f[j];
        f[j] = row_scale(stage, j);
      }
#pragma unroll
      for (int n = 0; n < kProducts; ++n) {
        const int i = row_of(n), j = col_of(n);
        if (n < 2) fw[n] = w_fragment(stage, n);
        if (n >= kRest && j == 0) fw[(i + 2) % 4] = w_fragment(stage, i + 2);
        P[n % 4] = mfma_run<false>(fw[i % 4], fa[j]);
        if (n < kRest && n % kRows == kRows - 1) fa[j] = a_fragment(stage, j);
        if (n == kRest) {
#pragma unroll
          for (int u = 0; u < TJ; ++u) f[u] *= swk;
        }
        // the next run's loads a few per product: issued in one go they fill
        // the address queue and hold up the wave's matrix instructions
#pragma unroll
        for (int u = n * kPer; u < (n + 1) * kPer && u < kLoads; ++u) load(u, next);
        __builtin_amdgcn_sched_barrier(0);
        if (n >= kLag) add(n - kLag);
        __builtin_amdgcn_sched_barrier(0);
      }
      touch();
#pragma unroll
      for (int n = kProducts - kLag; n < kProducts; ++n) add(n);
    });
#pragma unroll
    for (int n = 0; n < kRest; ++n) {
      const int i = row_of(n), j = col_of(n);
      const floatx4 D = mfma_run<false>(fw[i % 4], fa[j]);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(f[j], D[r], acc[i][j][r]);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load outlives its LDS
  if constexpr (KG > 1) {   // the groups' sums, in order
    __syncthreads();
    floatx4* part = reinterpret_cast<floatx4*>(lds) + gw * (TI * TJ * kWave) + lane;
    if (group > 0) {
#pragma unroll
      for (int n = 0; n < kProducts; ++n)
        part[((group - 1) * G * kProducts + n) * kWave] = acc[n / TJ][n % TJ];
    }
    __syncthreads();
    if (group == 0) {
      for (int u = 0; u < KG - 1; ++u)
#pragma unroll
        for (int n = 0; n < kProducts; ++n)
          acc[n / TJ][n % TJ] += part[(u * G * kProducts + n) * kWave];
    }
  }

  // Rows of y that keep the alignment of 16 bytes are written from the
  // registers.  Other rows go through LDS, each at the place in 16 bytes that
  // its first output has in memory, and from there in aligned pieces of 16
  // bytes (2772 x 28631 x 576: 132 us against 270 with a store per output,
  // and 96 for 28632 outputs).
  constexpr int V = 16 / sizeof(YT), kPitch = BN + V, kPieces = kPitch / V;
  constexpr int kThreads = KG * G * kWave;
  static_assert(BM * kPitch * static_cast<int>(sizeof(YT)) <= kLds, "");
  const bool direct = p.N % V == 0;
  YT* stage = reinterpret_cast<YT*>(lds);
  auto place_of = [&](int m) {   // of row m's first output, in outputs of y
    return static_cast<size_t>(t.row0 + m) * p.N + n0;
  };
  if (!direct) __syncthreads();
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int m = wm + 16 * j + c;
    if (m >= t.count || group > 0) continue;
    const bool none = p.rows != nullptr && source_row(p, t.row0 + m) < 0;
    YT* row = static_cast<YT*>(p.y) + static_cast<size_t>(t.row0 + m) * p.N;
    YT* staged = stage + m * kPitch + static_cast<int>(place_of(m) % V);
#pragma unroll
    for (int i = 0; i < TI; i += S) {
      floatx4 v[S];
#pragma unroll
      for (int u = 0; u < S; ++u) v[u] = none ? floatx4{0.0f, 0.0f, 0.0f, 0.0f} : acc[i + u][j];
      const int n = wn + 16 * i + 4 * S * g;
      if (direct) {
        store_outputs<S>(row, n0 + n, p.N, v);
      } else {
#pragma unroll
        for (int u = 0; u < 4 * S; ++u) put(staged + n + u, v[u / 4][u % 4]);
      }
    }
  }
  if (direct) return;
  __syncthreads();
  const int width = min(BN, p.N - n0);
  for (int q = threadIdx.x; q < t.count * kPieces; q += kThreads) {
    const int m = q / kPieces, at = q % kPieces * V;   // outputs at .. at + V - 1 of the place
    const size_t place = place_of(m);
    const int shift = static_cast<int>(place % V);
    YT* to = static_cast<YT*>(p.y) + (place - shift) + at;
    const YT* from = stage + m * kPitch + at;
    if (at >= shift && at + V <= shift + width) {
      *reinterpret_cast<u32x4*>(to) = *reinterpret_cast<const u32x4*>(from);
    } else {
#pragma unroll
      for (int u = 0; u < V; ++u)
        if (at + u >= shift && at + u < shift + width) to[u] = from[u];
    }
  }
}

// ---- launch -----------------------------------------------------------------------

// The tile of entry I of the table for YT (fp8_pick.hpp).
template <int I, int BN, int BM, int WN, int WM, int KG, int STAGES, typename YT>
hipError_t launch_tile(const Fp8Args& p, int live, hipStream_t stream) {
  constexpr int kThreads = KG * BN / WN * (BM / WM) * kWave;
  constexpr Fp8Tile tile = sizeof(YT) == 2 ? kBf16Tiles[I] : kF32Tiles[I];
  static_assert(tile.bn == BN && tile.bm == BM && tile.threads == kThreads, "");
  const int n_tiles = static_cast<int>(fp8_n_tiles(tile, p.N));
  const int m_tiles = static_cast<int>(fp8_m_tiles(tile, p.M, live));
  fp8_tile_kernel<BN, BM, WN, WM, KG, STAGES, YT>
      <<<dim3(n_tiles * m_tiles), kThreads, 0, stream>>>(p, n_tiles, m_tiles);
  return hipGetLastError();
}

hipError_t launch_by_size(const Fp8Args& p, int live, uint16_t*, hipStream_t stream) {
  using T = uint16_t;
  switch (fp8_pick(kBf16Tiles, kBf16Output, p.M, p.N, p.K, live, p.offsets != nullptr)) {
    case 0: return launch_tile<0, 256, 256, 128, 64, 1, 2, T>(p, live, stream);
    case 1: return launch_tile<1, 256, 128, 128, 64, 1, 3, T>(p, live, stream);
    case 2: return launch_tile<2, 128, 128, 64, 64, 1, 4, T>(p, live, stream);
    case 3: return launch_tile<3, 128, 128, 64, 64, 1, 2, T>(p, live, stream);
    case 4: return launch_tile<4, 128, 64, 64, 32, 1, 3, T>(p, live, stream);
    case 5: return launch_tile<5, 64, 64, 64, 32, 2, 4, T>(p, live, stream);
    case 6: return launch_tile<6, 64, 32, 64, 32, 2, 3, T>(p, live, stream);
    case 7: return launch_tile<7, 32, 32, 32, 32, 2, 4, T>(p, live, stream);
    case 8: return launch_tile<8, 32, 16, 32, 16, 4, 3, T>(p, live, stream);
    default: return launch_tile<9, 16, 16, 16, 16, 4, 4, T>(p, live, stream);
  }
}
hipError_t launch_by_size(const Fp8Args& p, int live, float*, hipStream_t stream) {
  using T = float;
  switch (fp8_pick(kF32Tiles, kF32Output, p.M, p.N, p.K, live, p.offsets != nullptr)) {
    case 0: return launch_tile<0, 128, 128, 64, 64, 2, 2, T>(p, live, stream);
    case 1: return launch_tile<1, 128, 128, 64, 64, 1, 2, T>(p, live, stream);
    case 2: return launch_tile<2, 128, 64, 64, 32, 1, 3, T>(p, live, stream);
    case 3: return launch_tile<3, 64, 64, 64, 32, 2, 2, T>(p, live, stream);
    case 4: return launch_tile<4, 64, 32, 64, 32, 2, 3, T>(p, live, stream);
    case 5: return launch_tile<5, 64, 32, 64, 32, 4, 3, T>(p, live, stream);
    case 6: return launch_tile<6, 32, 32, 32, 32, 4, 2, T>(p, live, stream);
    case 7: return launch_tile<7, 32, 16, 32, 16, 4, 3, T>(p, live, stream);
    default: return launch_tile<8, 16, 16, 16, 16, 4, 4, T>(p, live, stream);
  }
}

}  // namespace

hipError_t launch_fp8_gemm(const harp_fp8_weight& W, const uint8_t* a, const float* a_scale,
                           int a_rows, const int32_t* rows, const int32_t* offsets, void* y,
                           int y_dt, int M, hipStream_t stream) {
  const Fp8Args p{W.w, W.scale, a,   a_scale,        rows,      offsets, y,
                  W.N, W.K,     fp8_runs(W.K), W.experts, M,       a_rows};
  const int live = fp8_live(M, p.E, offsets != nullptr);
  return y_dt == HARP_BF16 ? launch_by_size(p, live, static_cast<uint16_t*>(nullptr), stream)
                           : launch_by_size(p, live, static_cast<float*>(nullptr), stream);
}

}  // namespace harp
