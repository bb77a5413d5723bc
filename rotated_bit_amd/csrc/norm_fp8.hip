// Residual addition and RMS norm, and the gated activation, with their
// output in float32 / bf16 or as e4m3 codes with a scale per 128 values.
//
//     h = x + r,  y = h / sqrt(mean(h^2) + eps) w;      v = g / (1 + exp(-g)) u
//
// One workgroup per row for the norm: the row is read once and stays in
// registers (float32) over the sum of squares, so a row moves x, r in and
// r', y out and nothing else.  A row whose squares leave float32's range is
// scaled in its registers and summed again (scaled_mean).  A thread holds chunks of 8 consecutive
// values; the 16 lanes of a DPP row hold one run of 128, whose maximum is
// four lane rotations.  Both are bound by memory (MI355X: norm of 8192 x
// 8192 bf16 to codes 82.7 us, 5.7 TB/s; activation of 2000 x 28672 55.4 us,
// 5.2 TB/s) down to a few hundred rows (333 x 5120 float32: 6.8 us, 3.5
// TB/s: three trips to memory one behind the other, x, the residual, and
// the weight behind the sum, then the stores); one row of 4096 takes 2.5 us.
#include "fp8_common.hpp"
#include "launch.hpp"

namespace harp {
namespace {

constexpr int kNormThreads = 1024;   // at most

// Values d .. d+7 of a row of D; VEC: whole chunks, 16-byte aligned.
template <bool VEC, typename T>
__device__ __forceinline__ void load_chunk(const T* row, int d, int D, float (&v)[8]) {
  if constexpr (VEC) {
    load8(row + d, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = d + i < D ? as_f32(row[d + i]) : 0.0f;
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_chunk(T* row, int d, int D, const float (&v)[8]) {
  if constexpr (VEC) {
    store8(row + d, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (d + i < D) put(row + d + i, v[i]);
  }
}

// Sum / maximum of v over the workgroup, the same bits in every thread.  All
// threads call; part is free again after the next barrier.
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += shfl_xor(v, o);
  if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  v = 0.0f;
  for (int i = 0; i < static_cast<int>(blockDim.x) / kWave; ++i) v += part[i];
  return v;
}
__device__ __forceinline__ float block_max(float v, float* part) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, shfl_xor(v, o));
  if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  v = 0.0f;
  for (int i = 0; i < static_cast<int>(blockDim.x) / kWave; ++i) v = fmaxf(v, part[i]);
  return v;
}

// mean(h^2) + eps below which the squares may have lost bits as subnormal
// numbers: those are off by 2^-150 each, so the mean by as much, 2^-50 of it.
constexpr float kLeastMean = 0x1p-100f;
constexpr int kScaledExponent = 50;   // 2^100 per square, 32768 of them

// The mean of a row whose squares leave float32's range: the row in h is
// taken times the power of two that brings the largest of |h| and sqrt(eps)
// just below 2^50, and its mean and eps are that power's square larger, which
// h / sqrt(mean + eps) does not see.  Rows of zeros without eps, of NaN and of
// infinities keep `mean`.  The whole workgroup calls, or none of it.
template <int C>
__device__ __forceinline__ float scaled_mean(float (&h)[C][8], float mean, float eps, int D,
                                             float* part) {
  float m = sqrtf(eps);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(h[c][i]));
  __syncthreads();
  m = block_max(m, part);
  if (m == 0.0f || m == INFINITY) return mean;
  const int by = kScaledExponent - __builtin_amdgcn_frexp_expf(m);
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[c][i] = ldexpf(h[c][i], by);
      ss = fmaf(h[c][i], h[c][i], ss);
    }
  __syncthreads();
  return block_sum(ss, part) / static_cast<float>(D) + ldexpf(eps, 2 * by);
}

// Codes and scale of the chunk's run; all 16 lanes of the run's row call.
__device__ __forceinline__ void store_codes(uint8_t* qrow, float* srow, int d, bool in,
                                            const float (&v)[8], int lane) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  const float s = fp8_scale(row16_max(m));
  if (in) {
    *reinterpret_cast<u32x2*>(qrow + d) = fp8_pack8(v, 1.0f / s);
    if ((lane & 15) == 0) srow[d / kFp8Run] = s;
  }
}

// XT: float or uint16_t (bf16).  YT: float, uint16_t, or uint8_t (codes).
// C chunks per thread: chunk c of thread t is chunk c * blockDim.x + t of
// the row, so that a DPP row holds one run.
template <typename XT, typename YT, int C, bool VEC>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_kernel(
    const XT* __restrict__ x, const XT* residual, XT* residual_out, const void* __restrict__ w,
    int w_bf16, float eps, YT* __restrict__ y, float* __restrict__ q_scale, int D) {
  __shared__ float part[kNormThreads / kWave];
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const size_t row = blockIdx.x;
  const size_t at = row * D;
  float h[C][8];
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int d = 8 * (c * blockDim.x + t);
    if (d < D) {
      load_chunk<VEC>(x + at, d, D, h[c]);
      if (residual != nullptr) {
        float r[8];
        load_chunk<VEC>(residual + at, d, D, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] += r[i];
      }
      if (residual_out != nullptr) store_chunk<VEC>(residual_out + at, d, D, h[c]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(h[c][i], h[c][i], ss);
  }
  float mean = block_sum(ss, part) / static_cast<float>(D) + eps;
  if (mean < kLeastMean || mean == INFINITY) mean = scaled_mean<C>(h, mean, eps, D, part);
  const float r = 1.0f / sqrtf(mean);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int d = 8 * (c * blockDim.x + t);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (d < D) {
      if (w_bf16)
        load_chunk<VEC>(static_cast<const uint16_t*>(w), d, D, v);
      else
        load_chunk<VEC>(static_cast<const float*>(w), d, D, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= h[c][i] * r;
    }
    if constexpr (sizeof(YT) == 1) {
      store_codes(y + at, q_scale + row * fp8_runs(D), d, d < D, v, lane);
    } else {
      if (d < D) store_chunk<VEC>(y + at, d, D, v);
    }
  }
}

template <typename XT, typename YT, bool VEC>
hipError_t norm_launch(const void* x, const void* residual, void* residual_out, const void* w,
                       int w_dt, float eps, void* y, float* q_scale, int M, int D,
                       hipStream_t stream) {
  const int chunks = (D + 7) / 8;
  const int C = chunks <= kNormThreads ? 1 : chunks <= 2 * kNormThreads ? 2 : 4;
  const int threads = ((chunks + C - 1) / C + kWave - 1) / kWave * kWave;
  const auto go = [&](auto kernel) {
    kernel<<<dim3(M), dim3(threads), 0, stream>>>(
        static_cast<const XT*>(x), static_cast<const XT*>(residual),
        static_cast<XT*>(residual_out), w, w_dt == HARP_BF16, eps, static_cast<YT*>(y), q_scale,
        D);
    return hipGetLastError();
  };
  if (C == 1) return go(rmsnorm_kernel<XT, YT, 1, VEC>);
  if (C == 2) return go(rmsnorm_kernel<XT, YT, 2, VEC>);
  return go(rmsnorm_kernel<XT, YT, 4, VEC>);
}

template <typename XT>
hipError_t norm_by_output(const void* x, const void* residual, void* residual_out, const void* w,
                          int w_dt, float eps, void* y, int y_dt, float* q_scale, int M, int D,
                          hipStream_t stream) {
  const auto go = [&](auto launch) {
    return launch(x, residual, residual_out, w, w_dt, eps, y, q_scale, M, D, stream);
  };
  if (q_scale != nullptr) return go(norm_launch<XT, uint8_t, true>);   // D a multiple of 16
  const bool vec = D % 8 == 0;
  if (y_dt == HARP_BF16)
    return vec ? go(norm_launch<XT, uint16_t, true>) : go(norm_launch<XT, uint16_t, false>);
  return vec ? go(norm_launch<XT, float, true>) : go(norm_launch<XT, float, false>);
}

// One DPP row of 16 lanes per run of 128 outputs.
template <typename XT>
__global__ __launch_bounds__(256) void silu_mul_fp8_kernel(const XT* __restrict__ gu,
                                                           uint8_t* __restrict__ q,
                                                           float* __restrict__ q_scale,
                                                           unsigned runs, int D) {
  const unsigned run = blockIdx.x * 16 + threadIdx.x / 16;   // row * B + b
  const unsigned B = fp8_runs(D);
  const bool any = run < runs;
  const size_t row = any ? run / B : 0;
  const int d = static_cast<int>((any ? run % B : 0) * kFp8Run + 8 * (threadIdx.x & 15));
  const bool in = any && d < D;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  if (in) {
    float g[8];
    load8(gu + row * 2 * D + d, g);
    load8(gu + row * 2 * D + D + d, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= g[i] / (1.0f + __expf(-g[i]));
  }
  store_codes(q + row * D, q_scale + row * B, d, in, v, threadIdx.x);
}

}  // namespace

hipError_t launch_rmsnorm(const void* x, int x_dt, const void* residual, void* residual_out,
                          const void* weight, int w_dt, float eps, void* y, int y_dt,
                          float* q_scale, int M, int D, hipStream_t stream) {
  return x_dt == HARP_BF16 ? norm_by_output<uint16_t>(x, residual, residual_out, weight, w_dt,
                                                      eps, y, y_dt, q_scale, M, D, stream)
                           : norm_by_output<float>(x, residual, residual_out, weight, w_dt, eps,
                                                   y, y_dt, q_scale, M, D, stream);
}

hipError_t launch_silu_mul_fp8(const void* gate_up, int x_dt, uint8_t* q, float* q_scale, int M,
                               int D, hipStream_t stream) {
  const unsigned runs = static_cast<unsigned>(M) * fp8_runs(D);
  const dim3 grid((runs + 15) / 16);
  if (x_dt == HARP_BF16)
    silu_mul_fp8_kernel<<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(gate_up), q,
                                                  q_scale, runs, D);
  else
    silu_mul_fp8_kernel<<<grid, 256, 0, stream>>>(static_cast<const float*>(gate_up), q, q_scale,
                                                  runs, D);
  return hipGetLastError();
}

}  // namespace harp
