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

}  // namespace

hipError_t launch_fp8_gemm(const harp_fp8_weight& W, const uint8_t* a, const float* a_scale,
                           int a_rows, const int32_t* rows, const int32_t* offsets, void* y,
                           int y_dt, int M, hipStream_t stream) {
  const Fp8Args p{W.w, W.scale, a,   a_scale,        rows,      offsets, y,
                  W.N, W.K,     fp8_runs(W.K), W.experts, M,       a_rows};
  // sum_e ceil(c_e / BM) <= (M + live (BM - 1)) / BM with live <= min(E, M)
  const int live = offsets == nullptr ? 1 : (W.experts < M ? W.experts : M);
  const dim3 grid((W.N + 15) / 16, (M + live * 15) / 16);
  if (y_dt == HARP_BF16)
    fp8_stream_kernel<uint16_t><<<grid, 512, 0, stream>>>(p);
  else
    fp8_stream_kernel<float><<<grid, 512, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace harp
