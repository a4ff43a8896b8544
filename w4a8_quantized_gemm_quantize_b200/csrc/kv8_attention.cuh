// Attention over the paged 8-bit KV cache (kv8_cache.cuh): one new token per
// sequence (decode) or several (prefill, causal).
//
//   s_j = scale * sK_page(j) * sum_d q[d] cK[j, d],   j < the row's limit
//   Y = fp16_rn(sum_j softmax(s)_j sV_page(j) cV[j, d])
//
// Row i of a sequence's n new tokens sees its first len - n + i + 1 tokens. A
// row that sees nothing gives zeros.
#pragma once
#include "kv8_cache.cuh"

namespace w4a8 {

struct Kv8AttnArgs {
  const __half* q;  // [T, Hq, 128]
  Kv8Cache c;
  Kv8Batch s;
  __half* out;  // [T, Hq, 128]
  int Hq;
  float scale;
  int* err;
};

constexpr int kKv8SimpleWarps = 8;

// One warp per (row, query head): lane l holds dimensions 4 l .. 4 l + 3; one
// pass over the tokens with the running maximum and sum.
__global__ void __launch_bounds__(kKv8SimpleWarps * 32) kv8_attention_simple_kernel(Kv8AttnArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kKv8SimpleWarps + (threadIdx.x >> 5);
  if (item >= static_cast<int64_t>(a.s.T) * a.Hq) return;
  const int row = static_cast<int>(item / a.Hq), h = static_cast<int>(item % a.Hq);
  const int b = a.s.q_start == nullptr ? row : kv8_find(a.s, row, 1, 1, 0);
  if (b < 0) return;
  const int64_t capacity = static_cast<int64_t>(a.c.max_blocks) * a.c.P;
  const Kv8Seq sq = kv8_sequence(a.s, b, capacity, lane == 0 ? a.err : nullptr);
  int limit = 0;
  if (a.s.q_start == nullptr) {
    limit = static_cast<int>(min(static_cast<int64_t>(max(sq.len, 0)), capacity));
  } else {
    const int n = kv8_row_start(a.s, b + 1) - sq.first;
    if (row - sq.first >= n) return;
    if (sq.n > 0) limit = sq.pos0 + row - sq.first + 1;
  }
  const int g = h / (a.Hq / a.c.Hkv);
  const uint2 qr = *reinterpret_cast<const uint2*>(a.q + item * kKv8D + 4 * lane);
  const float2 q01 = __half22float2(*reinterpret_cast<const __half2*>(&qr.x));
  const float2 q23 = __half22float2(*reinterpret_cast<const __half2*>(&qr.y));
  float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j0 = 0; j0 < limit; j0 += a.c.P) {
    const int page = __ldg(a.c.table + static_cast<int64_t>(b) * a.c.max_blocks + j0 / a.c.P);
    if (page < 0 || page >= a.c.num_pages) {
      if (lane == 0) atomicCAS(a.err, 0, kErrKv8Range);
      continue;
    }
    const int64_t bk = static_cast<int64_t>(page) * 2 * a.c.Hkv + g, bv = bk + a.c.Hkv;
    const float sk = __ldg(a.c.scales + bk) * a.scale, sv = __ldg(a.c.scales + bv);
    const int n = min(a.c.P, limit - j0);
    for (int j = 0; j < n; ++j) {
      const char4 k = *reinterpret_cast<const char4*>(a.c.codes + (bk * a.c.P + j) * kKv8D + 4 * lane);
      const char4 v = *reinterpret_cast<const char4*>(a.c.codes + (bv * a.c.P + j) * kKv8D + 4 * lane);
      float s = q01.x * k.x + q01.y * k.y + q23.x * k.z + q23.y * k.w;
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= sk;
      const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn), w = p * sv;
      m = mn;
      l = l * f + p;
      o[0] = o[0] * f + w * v.x;
      o[1] = o[1] * f + w * v.y;
      o[2] = o[2] * f + w * v.z;
      o[3] = o[3] * f + w * v.w;
    }
  }
  const float r = l > 0.0f ? 1.0f / l : 0.0f;
  uint2 y;
  *reinterpret_cast<__half2*>(&y.x) = __floats2half2_rn(o[0] * r, o[1] * r);
  *reinterpret_cast<__half2*>(&y.y) = __floats2half2_rn(o[2] * r, o[3] * r);
  *reinterpret_cast<uint2*>(a.out + item * kKv8D + 4 * lane) = y;
}

}  // namespace w4a8
