// Residual addition, root-mean-square norm and int8 quantization in one pass.
//
// Row m: h = fp16_rn(x + r) (h = x without a residual), y = h * rstd * w with
// rstd = 1 / sqrt(mean(h^2) + eps) (fp32, IEEE square root and divide), then
// the per-token quantization of quantize_act.cuh on the fp32 values of y (no
// rounding to fp16 in between): sA = fp16_rn(max |y| / 127), A8 =
// clamp(rint(y / sA), -127, 127), rowsum = sum A8. What w4a8_gemm takes, so
// that the norm in front of a linear layer ("QServe/QoQ" abstract: W4A8
// serving) costs one read of its input instead of a write and two reads more.
//
// The norm is taken of the rounded h, the value that the residual stream
// keeps: a later call on h alone gives the same codes.
//
// HBM-bound (2 + 2 bytes read, 2 + 1 written per element). One CTA per row,
// the row in registers from the first read to the codes.
#pragma once
#include "quantize_act.cuh"

namespace w4a8 {

// Sum (or maximum) over the CTA, the same value in every thread: one barrier.
// `red` must not be written again before every thread has passed a later
// barrier.
template <int THREADS, bool MAX>
__device__ __forceinline__ float block_all(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < THREADS / 32; ++i) v = MAX ? fmaxf(v, red[i]) : v + red[i];
  return v;
}

// VPT: 16-byte vectors (8 halves) per thread; K <= THREADS * VPT * 8.
template <int THREADS, int VPT, bool RES>
__global__ void __launch_bounds__(THREADS) rmsnorm_quantize_kernel(const __half* X, const __half* R,
                                                                   const __half* __restrict__ W, float eps,
                                                                   int64_t K, __half* H, int8_t* __restrict__ A8,
                                                                   __half* __restrict__ sA,
                                                                   int32_t* __restrict__ rowsum, int early_release) {
  __shared__ float s_sum[32], s_max[32];
  __shared__ int s_cnt[32];
  if (early_release) grid_launch_dependents();  // as in quantize_act_kernel
  grid_dependency_wait();
  if (!early_release) grid_launch_dependents();
  const int64_t m = blockIdx.x;
  const int nvec = static_cast<int>(K >> 3);
  const uint4* x = reinterpret_cast<const uint4*>(X + m * K);
  const uint4* r = reinterpret_cast<const uint4*>(R + m * K);
  const uint4* w = reinterpret_cast<const uint4*>(W);
  uint4 v[VPT];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int idx = threadIdx.x + i * THREADS;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (idx < nvec) {
      v[i] = x[idx];
      if constexpr (RES) {
        const uint4 rv = r[idx];
        __half2* a = reinterpret_cast<__half2*>(&v[i]);
        const __half2* b = reinterpret_cast<const __half2*>(&rv);
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = __hadd2_rn(a[j], b[j]);  // one rounding of the exact sum
        reinterpret_cast<uint4*>(H + m * K)[idx] = v[i];
      }
    }
    const __half2* h = reinterpret_cast<const __half2*>(&v[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(h[j]);
      sum = fmaf(f.x, f.x, sum);
      sum = fmaf(f.y, f.y, sum);
    }
  }
  sum = block_all<THREADS, false>(sum, s_sum);
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(K)), eps)));
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int idx = threadIdx.x + i * THREADS;
    if (idx < nvec) {
      const uint4 wv = __ldg(w + idx);
      const __half2* h = reinterpret_cast<const __half2*>(&v[i]);
      const __half2* g = reinterpret_cast<const __half2*>(&wv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(h[j]), q = __half22float2(g[j]);
        amax = fmaxf(amax, fmaxf(fabsf(f.x * rstd * q.x), fabsf(f.y * rstd * q.y)));
      }
    }
  }
  amax = block_all<THREADS, true>(amax, s_max);
  const __half s_h = __float2half_rn(__fdiv_rn(amax, 127.0f));
  const float sf = __half2float(s_h);
  int local = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int idx = threadIdx.x + i * THREADS;
    if (idx < nvec) {
      const uint4 wv = __ldg(w + idx);
      const __half2* h = reinterpret_cast<const __half2*>(&v[i]);
      const __half2* g = reinterpret_cast<const __half2*>(&wv);
      int q[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (sf != 0.0f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = __half22float2(h[j]), u = __half22float2(g[j]);
          q[2 * j] = quant_code<127>(f.x * rstd * u.x, sf);
          q[2 * j + 1] = quant_code<127>(f.y * rstd * u.y, sf);
          local += q[2 * j] + q[2 * j + 1];
        }
      }
      CodeOut<8>::store(A8 + m * K, idx, q);
    }
  }
  if (rowsum != nullptr) {
    const int total = block_sum<THREADS>(local, s_cnt);
    if (threadIdx.x == 0) rowsum[m] = total;
  }
  if (threadIdx.x == 0) sA[m] = s_h;
}

}  // namespace w4a8
