// The paged 8-bit KV cache: its layout, where a sequence's tokens lie in it,
// and the kernel that rotates q and k and appends k and v.
//
// Cache: pages of P tokens (16, 32, 64 or 128), codes int8 [num_pages, 2 (K,
// V), Hkv, P, 128], one fp32 scale per (page, K | V, head); value = code *
// scale. Token p of sequence b lies in page block_table[b, p / P] at place p %
// P. A scale for each block of tokens and head keeps the parameters at 1/2048
// of the codes' bytes (P = 64) and lets attention take the scale out of whole
// tiles of the products.
//
// Appending: the page's scale grows to s' = max(s, max |x| / 127) over the new
// tokens of the page, and where it grows the codes already in the page are
// carried over, c' = rint(c * (s / s')). A page whose first place is written
// by the call starts from s = 0, whatever its last owner left there.
#pragma once
#include "codes.cuh"
#include "ptx.cuh"

namespace w4a8 {

constexpr int kKv8D = 128;          // head dimension
constexpr int kErrKv8Range = 7;     // W4A8_DEVERR_KV_RANGE
constexpr int kErrKv8Wait = 11;     // W4A8_DEVERR_KV_WAIT

struct Kv8Cache {
  int8_t* codes;         // [num_pages, 2, Hkv, P, 128]
  float* scales;         // [num_pages, 2, Hkv]
  const int32_t* table;  // [B, max_blocks]
  int num_pages, max_blocks, Hkv, P;
};

// Which sequence a row of the batch belongs to, and where it stands in it.
struct Kv8Batch {
  const int32_t* seq_lens;  // [B] cached tokens, the new ones among them
  const int32_t* q_start;   // [B + 1] first new token of each sequence; null: one each
  int B;
  int T;  // rows
};

__device__ __forceinline__ int kv8_row_start(const Kv8Batch& s, int b) {
  return s.q_start == nullptr ? b : min(max(__ldg(s.q_start + b), 0), s.T);
}

// Largest b in [0, B) with start_b * mul / div + b * add <= x, or -1 (the left
// side does not fall in b). log2(B) dependent loads.
__device__ __forceinline__ int kv8_find(const Kv8Batch& s, int64_t x, int mul, int div, int add) {
  int lo = -1, hi = s.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const int64_t key = static_cast<int64_t>(kv8_row_start(s, mid)) * mul / div + static_cast<int64_t>(mid) * add;
    if (key <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Rows [first, first + n) of the batch are sequence b's new tokens, at
// positions [pos0, pos0 + n) of it. n < 0: nothing to do; a length or a start
// outside its range is reported.
struct Kv8Seq {
  int first, n, pos0, len;
};
__device__ __forceinline__ Kv8Seq kv8_sequence(const Kv8Batch& s, int b, int64_t capacity, int* err) {
  Kv8Seq q;
  q.first = kv8_row_start(s, b);
  q.n = s.q_start == nullptr ? 1 : kv8_row_start(s, b + 1) - q.first;
  q.len = __ldg(s.seq_lens + b);
  if (s.q_start == nullptr && q.len == 0) q.n = 0;  // a place of the batch that no sequence fills
  q.pos0 = q.len - q.n;
  if (q.n < 0 || q.len < 0 || q.len > capacity || q.pos0 < 0) {
    if (err != nullptr) atomicCAS(err, 0, kErrKv8Range);
    q.n = -1;
  }
  return q;
}

// --------------------------------------------------------------- append
struct Kv8AppendArgs {
  const __half* qkv;  // [T, (Hq + 2 Hkv) * 128]
  Kv8Cache c;
  Kv8Batch s;
  const float* inv_freq;  // [rotary / 2]
  __half* q_out;          // [T, Hq, 128]
  int Hq, rotary, q_rows, q_blocks;
  float rope_scale;
  int* err;
};

// Threads of an append block, by PAGE: the page's tokens, or 0 (below). Measured,
// 4 x 500 tokens, 32 + 2 x 8 heads: pages of 16 by 128 threads 10.7 us, by 256
// 14.9 (more of the blocks' short chains of dependent reads run at once); of 32
// by 128 9.5, by 256 12.1; of 64 by 256 11.2, by 128 12.1 (a thread holds too
// much); of 128 by 512 13.6, by 256 14.1 (all with the cheaper angles below).
__host__ __device__ constexpr int kv8_append_threads(int P) { return P <= 32 ? 128 : P == 64 ? 256 : 512; }
__host__ __device__ constexpr int kv8_append_blocks(int P) { return P <= 32 ? 8 : P == 64 ? 4 : 2; }  // of an SM

// The rotation of pair i at position pos: angle pos * f_i, taken in turns.
// f_i / (2 pi) is held as a 64-bit fraction of a turn, so that the product
// with the position wraps at whole turns by itself and is exact to 2^-29 of a
// turn at position 2^24 (an fp32 product is off by 2^-24 * pos * f radians,
// 0.008 at position 131072). Its top 32 bits give the quarter turn and the
// angle within it, in [-pi / 4, pi / 4], where the Taylor series' next terms are
// below 2^-25. The sine and cosine come out within 2^-23, so that an
// angle moves a code by 127 * 2^-23 of a step and few lie that near the middle
// between two. (The hardware's approximations, within 2^-20.5, took 37.1 us
// where these take 39.6, with an error bound six times as wide.)
__device__ __forceinline__ uint64_t kv8_turns(float f) {
  // 1 / (2 pi) in two terms, and the first product's remainder: what is left of
  // whole turns is within 2^-54 for a frequency of any size
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  const double x = static_cast<double>(f), t = x * kHi;
  const double part = (t - rint(t)) + fma(x, kLo, fma(x, kHi, -t));
  return static_cast<uint64_t>(__double2ll_rn(part * 18446744073709551616.0));
}
__device__ __forceinline__ void kv8_cos_sin(uint64_t turns, int pos, float scale, float* c, float* s) {
  const uint32_t top = static_cast<uint32_t>((turns * static_cast<uint64_t>(pos)) >> 32);
  const uint32_t quarter = (top + 0x20000000u) >> 30;
  const float a = static_cast<float>(static_cast<int32_t>(top - (quarter << 30))) * 1.4629180792671596e-9f;  // pi / 2^31
  const float a2 = a * a;
  const float sa = fmaf(a * a2, fmaf(a2, fmaf(a2, fmaf(a2, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), a);
  const float ca = fmaf(a2, fmaf(a2, fmaf(a2, fmaf(a2, 1.0f / 40320, -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  const bool odd = (quarter & 1u) != 0;
  // (the quarter's signs as the sign bits)
  *c = __uint_as_float(__float_as_uint((odd ? sa : ca) * scale) ^ (((quarter + 1u) & 2u) << 30));
  *s = __uint_as_float(__float_as_uint((odd ? ca : sa) * scale) ^ ((quarter & 2u) << 30));
}

// Which eight of a head's 128 values lane i of 16 takes: [lo, lo + 4) and [hi,
// hi + 4), whole pairs where that can be, so that each is rotated once.
//  kSplit: half layout, pairs (j, j + rotary / 2): j = 4 i .. in the first rotary
//    / 8 lanes, the values behind the rotated ones in the others;
//  kPairs: interleaved pairs, the eight in a row from 8 i;
//  kSingle: what fours do not divide (half layout with rotary % 8 != 0): the
//    eight in a row, each pair's other value read by itself (8200 tokens, rotary
//    50: 83 us where kSplit takes 40).
enum Kv8Layout { kSplit, kPairs, kSingle };
struct Kv8Lane {
  int lo, hi;
};
template <Kv8Layout L>
__device__ __forceinline__ Kv8Lane kv8_lane(int i, int rotary) {
  if constexpr (L == kSplit) {
    const int half = rotary >> 1;
    if (4 * i < half) return {4 * i, half + 4 * i};
    return {rotary + 8 * (i - half / 4), rotary + 8 * (i - half / 4) + 4};
  }
  return {8 * i, 8 * i + 4};
}
struct Kv8Vec {
  uint2 lo, hi;
};
__device__ __forceinline__ Kv8Vec kv8_load(const __half* vec, const Kv8Lane& n) {
  return {__ldcs(reinterpret_cast<const uint2*>(vec + n.lo)), __ldcs(reinterpret_cast<const uint2*>(vec + n.hi))};
}
__device__ __forceinline__ void kv8_to_float(const uint2& v, float* o) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
  o[0] = a.x;
  o[1] = a.y;
  o[2] = b.x;
  o[3] = b.y;
}
// Where a lane has the cosines and sines of its pairs from.
struct Kv8Table {  // a row's, in shared memory
  const float* c;
  const float* s;
  __device__ __forceinline__ void four(int i, float (&ca)[4], float (&sa)[4]) const {
    const float4 cv = *reinterpret_cast<const float4*>(c + 4 * i), sv = *reinterpret_cast<const float4*>(s + 4 * i);
    ca[0] = cv.x, ca[1] = cv.y, ca[2] = cv.z, ca[3] = cv.w;
    sa[0] = sv.x, sa[1] = sv.y, sa[2] = sv.z, sa[3] = sv.w;
  }
  __device__ __forceinline__ void one(int j, float* cj, float* sj) const {
    *cj = c[j];
    *sj = s[j];
  }
};
struct Kv8Direct {  // worked out
  const uint64_t* turns;
  int pos;
  float scale;
  __device__ __forceinline__ void four(int i, float (&ca)[4], float (&sa)[4]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) kv8_cos_sin(turns[4 * i + e], pos, scale, &ca[e], &sa[e]);
  }
  __device__ __forceinline__ void one(int j, float* cj, float* sj) const { kv8_cos_sin(turns[j], pos, scale, cj, sj); }
};
// The lane's values (o[0..3] from lo, o[4..7] from hi), rotated: (a, b) -> (a
// cos - b sin, a sin + b cos). vec: the vector (kSingle).
template <Kv8Layout L, typename Angles>
__device__ __forceinline__ void kv8_rotate(const Kv8Vec& r, const __half* vec, int i, const Angles& angles, int rotary,
                                           float (&o)[8]) {
  kv8_to_float(r.lo, o);
  kv8_to_float(r.hi, o + 4);
  const int half = rotary >> 1;
  if constexpr (L == kSingle) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = 8 * i + e;
      if (d < rotary) {
        const int j = d < half ? d : d - half;
        const float y = __half2float(vec[d < half ? d + half : j]);
        float c, s;
        angles.one(j, &c, &s);
        o[e] = d < half ? o[e] * c - y * s : y * s + o[e] * c;
      }
    }
  } else if (4 * i < half) {
    // (kPairs: a rotary that 8 does not divide ends inside a lane's pairs)
    float c[4], s[4];
    angles.four(i, c, s);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float& x = o[L == kSplit ? e : 2 * e];
      float& y = o[L == kSplit ? e + 4 : 2 * e + 1];
      const float u = x * c[e] - y * s[e], v = x * s[e] + y * c[e];
      if (L == kSplit || 4 * i + e < half) {
        x = u;
        y = v;
      }
    }
  }
}

// R rows of q, every head of them, so that the angles are worked out once a row.
// A thread's first reads are under way before the rows' positions are known.
template <int R, Kv8Layout L, int THREADS>
__device__ __forceinline__ void kv8_rotate_q(const Kv8AppendArgs& a, int64_t capacity, const uint64_t* s_turns,
                                             float (*s_cos)[kKv8D / 2], float (*s_sin)[kKv8D / 2]) {
  constexpr int kDepth = R == 1 ? 2 : 1;  // a row's vectors that a thread has under way at once
  const int t = threadIdx.x;
  const int i = t & 15;
  const int half = a.rotary >> 1;
  const int row0 = static_cast<int>(blockIdx.x) * R;
  const int rows = min(R, a.s.T - row0);
  const int vectors = a.Hq * 16;
  const int64_t row_elems = static_cast<int64_t>(a.Hq + 2 * a.c.Hkv) * kKv8D;
  const __half* src = a.qkv + row0 * row_elems;
  __half* dst = a.q_out + static_cast<int64_t>(row0) * vectors * 8;
  const Kv8Lane lane = kv8_lane<L>(i, a.rotary);
  Kv8Vec r[R][kDepth];
  const auto load = [&](int v0) {
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        const int v = v0 + u * THREADS;
        if (k < rows && v < vectors) r[k][u] = kv8_load(src + k * row_elems + (v >> 4) * kKv8D, lane);
      }
  };
  load(t);
  // every row's position, -1 for one that is left as it is
  int pos[R];
  Kv8Seq q = {0, -1, 0, 0};
#pragma unroll
  for (int k = 0; k < R; ++k) {
    pos[k] = -1;
    const int row = row0 + k;
    if (k >= rows) continue;
    if (k == 0 || row - q.first >= q.n) {
      const int b = a.s.q_start == nullptr ? row : kv8_find(a.s, row, 1, 1, 0);
      if (b < 0) continue;
      q = kv8_sequence(a.s, b, capacity, t == 0 ? a.err : nullptr);
    }
    if (row - q.first < q.n) pos[k] = q.pos0 + row - q.first;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < R; ++k)
    if (THREADS >= R * 64 ? (t >> 6) == k : (t >> 6) == k % (THREADS / 64))
      if ((t & 63) < half && pos[k] >= 0)
        kv8_cos_sin(s_turns[t & 63], pos[k], a.rope_scale, &s_cos[k][t & 63], &s_sin[k][t & 63]);
  __syncthreads();
  for (int v0 = t; v0 < vectors; v0 += kDepth * THREADS) {
    if (v0 != t) load(v0);
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        const int v = v0 + u * THREADS;
        if (pos[k] < 0 || v >= vectors) continue;
        float o[8];
        kv8_rotate<L>(r[k][u], src + k * row_elems + (v >> 4) * kKv8D, i, Kv8Table{s_cos[k], s_sin[k]}, a.rotary, o);
        uint2 w[2];
        __half2* h = reinterpret_cast<__half2*>(w);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = __floats2half2_rn(o[2 * j], o[2 * j + 1]);
        __half* to = dst + (k * a.Hq + (v >> 4)) * kKv8D;
        if (!in_bounds(row0 + k < a.s.T && (v >> 4) < a.Hq && lane.lo >= 0 && lane.lo + 4 <= kKv8D && lane.hi >= 0 &&
                           lane.hi + 4 <= kKv8D, a.err))
          continue;
        *reinterpret_cast<uint2*>(to + lane.lo) = w[0];
        *reinterpret_cast<uint2*>(to + lane.hi) = w[1];
      }
  }
}

// Blocks [0, q_blocks): q_rows (at most 4) rows of q each, every head of them,
// so that the angles are worked out once a row. The others: one (page of a
// sequence, K | V, head) each; P * 16 vectors of 8 values, in registers from
// the read to the codes, so that the maximum over the page comes before the
// first code.
//
// HBM-bound (2 bytes read per value, 2 or 1 written) for many rows: 8200 tokens,
// 32 + 2 x 8 heads, 184 MB, 40 us (4.6 TB/s); the rows of q alone run at 5.5
// TB/s, the pages are held up by the chain of reads in front of theirs (length,
// start, page). A decode step is that chain: 16 sequences 2.3 us. All of a thread's
// reads are under way before the angles are worked out, and a page's angles by
// the thread that rotates with them: sharing them among a block's threads
// through shared memory took a barrier a slab and 5 us more.
//
// PAGE: the page's tokens; 0: one new token per sequence in pages of any size,
// by the one slab that holds it. Measured, 64 such sequences, pages of 16 / 32 /
// 64 / 128: 3.1 us each; through the whole page 3.3 / 3.7 / 5.3 / 9.3.
template <int PAGE, Kv8Layout L>
__global__ void __launch_bounds__(kv8_append_threads(PAGE), kv8_append_blocks(PAGE)) kv8_append_kernel(Kv8AppendArgs a) {
  constexpr int kThreads = kv8_append_threads(PAGE);
  const int P = PAGE > 0 ? PAGE : a.c.P;
  constexpr int kSlab = kThreads / 16;  // tokens of the page a pass covers
  constexpr int kPasses = PAGE > 0 ? PAGE / kSlab : 1;
  __shared__ __align__(16) uint64_t s_turns[kKv8D / 2];
  __shared__ __align__(16) float s_cos[4][kKv8D / 2], s_sin[4][kKv8D / 2];  // of the rows of q
  __shared__ float s_red[kThreads / 32];
  const int t = threadIdx.x;
  const int i = t & 15;  // lane of a vector
  const int half = a.rotary >> 1;
  grid_dependency_wait();
  grid_launch_dependents();
  if (t < half) s_turns[t] = kv8_turns(__ldg(a.inv_freq + t));
  const int64_t capacity = static_cast<int64_t>(a.c.max_blocks) * P;
  const int64_t row_elems = static_cast<int64_t>(a.Hq + 2 * a.c.Hkv) * kKv8D;
  if (static_cast<int>(blockIdx.x) < a.q_blocks) {
    if (a.q_rows == 1)
      kv8_rotate_q<1, L, kThreads>(a, capacity, s_turns, s_cos, s_sin);
    else
      kv8_rotate_q<4, L, kThreads>(a, capacity, s_turns, s_cos, s_sin);
    return;
  }
  // item: a page that the call writes to. Sequence b's pages start at item
  // start_b / P + 2 b: n new tokens touch at most n / P + 2 pages.
  const int heads2 = 2 * a.c.Hkv;
  const int64_t flat = static_cast<int64_t>(blockIdx.x) - a.q_blocks;
  const int64_t item = flat / heads2;
  const int kh = static_cast<int>(flat - item * heads2);  // K | V, head
  int b, k;
  if (a.s.q_start == nullptr) {
    b = static_cast<int>(item);
    k = 0;
  } else {
    b = kv8_find(a.s, item, 1, P, 2);
    if (b < 0) return;
    k = static_cast<int>(item - (kv8_row_start(a.s, b) / P + 2 * static_cast<int64_t>(b)));
  }
  const Kv8Seq q = kv8_sequence(a.s, b, capacity, t == 0 ? a.err : nullptr);
  if (q.n <= 0) return;
  const int shift = PAGE > 0 ? 0 : __ffs(P) - 1;  // (a division by it costs 0.4 us)
  const int page_no = (PAGE > 0 ? q.pos0 / P : q.pos0 >> shift) + k;
  if (page_no > (PAGE > 0 ? (q.len - 1) / P : (q.len - 1) >> shift)) return;
  const int base = page_no * P;                                     // position of the page's first place
  const int lo = max(q.pos0 - base, 0), hi = min(q.len - base, P);  // places [lo, hi) are new
  const bool is_k = kh < a.c.Hkv;
  const int rotary = is_k ? a.rotary : 0;
  const __half* src = a.qkv + (static_cast<int64_t>(q.first) + base - q.pos0) * row_elems +
                      static_cast<int64_t>(a.Hq + kh) * kKv8D;  // place 0 of the page (read from place lo on)
  const Kv8Lane lane = kv8_lane<L>(i, rotary);
  const int slab0 = PAGE > 0 ? 0 : lo & ~(kSlab - 1);  // where the passes begin
  Kv8Vec raw[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int j = slab0 + p * kSlab + (t >> 4);
    if (j >= lo && j < hi) raw[p] = kv8_load(src + j * row_elems, lane);
  }
  const int page = __ldg(a.c.table + static_cast<int64_t>(b) * a.c.max_blocks + page_no);
  if (page < 0 || page >= a.c.num_pages) {
    if (t == 0) atomicCAS(a.err, 0, kErrKv8Range);
    return;
  }
  const int64_t block = static_cast<int64_t>(page) * heads2 + kh;
  int8_t* codes = a.c.codes + block * P * kKv8D;
  const float s_old = lo > 0 ? a.c.scales[block] : 0.0f;
  float x[kPasses][8];
  float amax = 0.0f;
  if (is_k) __syncthreads();  // s_turns
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int j = slab0 + p * kSlab + (t >> 4);
    if (j >= lo && j < hi) {
      kv8_rotate<L>(raw[p], src + j * row_elems, i, Kv8Direct{s_turns, base + j, a.rope_scale}, rotary, x[p]);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[p][e]));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((t & 31) == 0) s_red[t >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, s_red[w]);
  const float s_new = fmaxf(s_old, __fdiv_rn(amax, 127.0f));
  const float r = s_new > 1e-37f ? __fdiv_rn(1.0f, s_new) : 0.0f;  // (below it the reciprocal may not be finite)
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int j = slab0 + p * kSlab + (t >> 4);
    if (j >= lo && j < hi) {
      // (the correction in quotient() takes 1.5 us of 41, an IEEE division 7)
      float u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = quotient(x[p][e], s_new, r);
      if (!in_bounds(j >= 0 && j < P && block >= 0 && block < static_cast<int64_t>(a.c.num_pages) * heads2 &&
                         lane.lo >= 0 && lane.lo + 4 <= kKv8D && lane.hi >= 0 && lane.hi + 4 <= kKv8D, a.err))
        continue;
      // (|u| <= 127 (1 + 2^-22): no code is beyond 127)
      *reinterpret_cast<uint32_t*>(codes + j * kKv8D + lane.lo) = pack_codes(u, 1.0f);
      *reinterpret_cast<uint32_t*>(codes + j * kKv8D + lane.hi) = pack_codes(u + 4, 1.0f);
    }
  }
  if (lo > 0 && s_new > s_old) {  // the codes that were there, carried over to the larger scale
    const float ratio = __fdiv_rn(s_old, s_new);
    for (int v = t; v < lo * 16; v += kThreads) {
      if (!in_bounds(v < P * 16 && block < static_cast<int64_t>(a.c.num_pages) * heads2, a.err)) break;
      uint2* at = reinterpret_cast<uint2*>(codes) + v;
      const uint2 c = *at;
      uint32_t w[2] = {c.x, c.y}, u[2] = {0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int old = static_cast<int8_t>(w[e >> 2] >> (8 * (e & 3)));
        u[e >> 2] |= (static_cast<uint32_t>(__float2int_rn(static_cast<float>(old) * ratio)) & 0xFFu) << (8 * (e & 3));
      }
      *at = make_uint2(u[0], u[1]);
    }
  }
  if (t == 0 && in_bounds(block >= 0 && block < static_cast<int64_t>(a.c.num_pages) * heads2, a.err))
    a.c.scales[block] = s_new;
}

}  // namespace w4a8
