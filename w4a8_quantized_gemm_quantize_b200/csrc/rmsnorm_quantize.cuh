// Residual addition, root-mean-square norm and int8 quantization in one pass.
//
// Row m: h = fp16_rn(x + r) (h = x without a residual), y = h * rstd * w with
// rstd = 1 / sqrt(mean(h^2) + eps) (fp32, IEEE square root and divide), then
// the per-token quantization of quantize_act.cuh on the fp32 values of y (no
// rounding to fp16 in between): sA = fp16_rn(min(max |y| / 127, 65504)), A8 =
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
#include "codes.cuh"
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

// VPT: 16-byte vectors (8 halves) per thread; K <= THREADS * VPT * 8. KEEP: the
// weights and y stay in registers too; with 8 vectors a thread and 1024 threads
// (64 registers each) only the row does, and y is worked out twice.
//
// Measured, replayed graphs: 8192 x 4096 with residual 39.0 us (6.0 TB/s), 1024 x
// 14336 17.7 us (its 103 MB partly in L2; with 512 threads of 4 vectors a quarter
// more: more vectors a thread keep more of the row under way), 1 x 4096 2.0 us. The
// codes' quotients corrected by their remainder cost 0.8 of the 39.0.
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
  constexpr bool KEEP = VPT <= 4 || THREADS <= 256;
  constexpr int kKeep = KEEP ? VPT : 1;
  uint4 v[VPT], rv[kKeep], wv[kKeep];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {  // every read of the row under way at once
      const int idx = threadIdx.x + i * THREADS;
      v[i] = rv[i] = wv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (idx < nvec) {
        v[i] = __ldcs(x + idx);
        if constexpr (RES) rv[i] = __ldcs(r + idx);
        wv[i] = __ldg(w + idx);
      }
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int idx = threadIdx.x + i * THREADS;
    uint4 rr = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (KEEP) {
      rr = rv[i];
    } else {
      v[i] = idx < nvec ? __ldcs(x + idx) : rr;
      if (RES && idx < nvec) rr = __ldcs(r + idx);
    }
    __half2* h = reinterpret_cast<__half2*>(&v[i]);
    if constexpr (RES) {
      const __half2* b = reinterpret_cast<const __half2*>(&rr);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = __hadd2_rn(h[j], b[j]);  // one rounding of the exact sum
      if (idx < nvec) reinterpret_cast<uint4*>(H + m * K)[idx] = v[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(h[j]);
      sum = fmaf(f.x, f.x, sum);
      sum = fmaf(f.y, f.y, sum);
    }
  }
  sum = block_all<THREADS, false>(sum, s_sum);
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(K)), eps)));
  const auto norm_of = [&](int i, float (&y)[8]) {
    const int idx = threadIdx.x + i * THREADS;
    uint4 ww = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (KEEP) {
      ww = wv[i];
    } else if (idx < nvec) {
      ww = __ldg(w + idx);
    }
    const __half2* h = reinterpret_cast<const __half2*>(&v[i]);
    const __half2* g = reinterpret_cast<const __half2*>(&ww);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(h[j]), q = __half22float2(g[j]);
      y[2 * j] = f.x * rstd * q.x;
      y[2 * j + 1] = f.y * rstd * q.y;
    }
  };
  float y[kKeep][8];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float(&yy)[8] = y[KEEP ? i : 0];
    norm_of(i, yy);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(yy[e]));
  }
  amax = block_all<THREADS, true>(amax, s_max);
  const __half s_h = __float2half_rn(fminf(__fdiv_rn(amax, 127.0f), 65504.0f));
  const float sf = __half2float(s_h);
  const float inv = sf > 0.0f ? __fdiv_rn(1.0f, sf) : 0.0f;
  // A normal scale is within 2^-11 of amax / 127, so that no code passes 127;
  // a subnormal one may be half of it, and the largest stands for all beyond it.
  const bool clamp = sf < 6.2e-5f || sf == 65504.0f;
  const float top = 127.0f * sf;
  int local = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int idx = threadIdx.x + i * THREADS;
    float(&yy)[8] = y[KEEP ? i : 0];
    if constexpr (!KEEP) norm_of(i, yy);
    if (clamp) {
#pragma unroll
      for (int e = 0; e < 8; ++e) yy[e] = fminf(fmaxf(yy[e], -top), top);
    }
    if (idx < nvec) {
#pragma unroll
      for (int e = 0; e < 8; ++e) yy[e] = quotient(yy[e], sf, inv);
      const uint2 c = make_uint2(pack_codes(yy, 1.0f), pack_codes(yy + 4, 1.0f));
      reinterpret_cast<uint2*>(A8 + m * K)[idx] = c;
      local = __dp4a(static_cast<int>(c.x), 0x01010101, local);
      local = __dp4a(static_cast<int>(c.y), 0x01010101, local);
    }
  }
  if (threadIdx.x == 0) sA[m] = s_h;
  if (rowsum != nullptr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) local += __shfl_xor_sync(0xffffffffu, local, o);
    if ((threadIdx.x & 31) == 0) s_cnt[threadIdx.x >> 5] = local;
    __syncthreads();
    if (threadIdx.x < 32) {
      local = threadIdx.x < THREADS / 32 ? s_cnt[threadIdx.x] : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) local += __shfl_xor_sync(0xffffffffu, local, o);
      if (threadIdx.x == 0) rowsum[m] = local;
    }
  }
}

}  // namespace w4a8
