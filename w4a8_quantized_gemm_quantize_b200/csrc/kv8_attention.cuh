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

// --------------------------------------------------------------- decode
// Warp-level building blocks of the decode kernel.
//
// D += A B on the tensor cores, fp16 x fp16 -> fp32, 16 x 8 x 16. Lane (g = lane
// / 4, c = lane % 4) holds A rows g, g + 8 at columns 2c, 2c + 1 (+ 8), B
// column g at rows 2c, 2c + 1 (+ 8), D rows g, g + 8 at columns 2c, 2c + 1.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit values held two to a lane (lane (g, c):
// row g, columns 2c, 2c + 1).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Bytes (lo, hi) of w, biased by 128, as a pair of fp16 values without the
// bias: a byte u in the mantissa of 1024 is 1024 + u, and 1152 comes off
// exactly. SEL 0x4140: bytes 0, 1; 0x4342: bytes 2, 3.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t unbias_pair(uint32_t w) {
  const uint32_t x = __byte_perm(w, 0x64646464u, SEL);
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&x), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Arrives on the barrier once this thread's earlier cp.async copies are done.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// A warp's bounded wait for copies; false (in every lane) if they are not there
// after a second limit either.
__device__ __forceinline__ bool kv8_wait(uint64_t* bar, uint32_t parity, DevErr err) {
  const bool ok = mbar_wait_limit(bar, parity, nullptr, err, kErrKv8Wait, kWaitLimitNs) ||
                  mbar_wait_limit(bar, parity, nullptr, err, kErrKv8Wait, kWaitLimitNs);
  return __all_sync(0xffffffffu, ok) != 0;
}

// What bounds a decode step is reading the cache: 256 bytes per token and kv
// head against G = Hq / Hkv times 512 operations. So the kernel is built around
// loads in flight: 12 (or 8, below) warps per SM, each with its own ring of two (three)
// tiles of 32 tokens (K and V, 8 KB) that it fills by TMA and empties by itself, no
// warp waiting for another before the end. Measured, replayed graphs over caches
// larger than the L2: 64 kv heads' cache of 8 sequences of 2048 to 4096 tokens, 397
// MB in 77 us, 5.2 TB/s; 16 sequences with 8 kv heads, 106 MB, 34 us, of which 5
// to start and 8 for the last tiles and the joins (33 us where the L2 holds the
// cache). One sequence of 500 tokens: 10 us, the chain of one warp's reads, products
// and joins. The tensor-core part is small (16 +
// 16 products of 16 x 8 x 16 per tile and 8 columns) and stays in registers:
// S^T = K q^T has tokens as rows and query heads as its 8 columns, so that K
// goes from its bytes to the A operand without a shuffle (the order of the
// contraction is free: lane (g, c) takes dimensions 32c .. 32c + 31 of its
// tokens' rows), and O^T = V^T w^T takes each lane's 16 bytes of a token row as
// 16 rows of A. Bytes become fp16 integers, exactly, with about 1.3 operations
// each.
//
// Softmax weights carry their page's value scale: with z_j = x_j + log2 sV_j (x
// the score in powers of two) and a running maximum M over z, w_j = 2^(z_j - M
// + 14) is at most 2^14 and goes into the product as two fp16 terms (hi + lo:
// exact to 2^-22, and to 2^-38 of the largest), while the denominator sums w_j
// / sV_j in fp32. Up to four heads share the 8 columns as hi (0-3) and lo
// (4-7); up to eight take a second product for lo.
//
// The 8 columns are rows of a kv head's query group: row R = i G + h is head h
// at new token i, so that a handful of new tokens per sequence (a decode step's
// one, guesses to be checked) take the same path, each column with its own
// causal limit, more than 8 rows as further column groups.
//
// Work is dealt out by tiles: all (sequence, kv head, column group) pairs' tiles
// in one line, cut evenly over the CTAs and over their warps. What a warp
// finishes alone it writes; partial results of a pair meet in shared memory,
// then, where a pair crosses CTAs, in the workspace, where the last CTA to
// arrive (a counter, no waiting) adds them up in the order of the line.
constexpr int kDecTile = 32;
constexpr int kDecStageBytes = 2 * kDecTile * kKv8D;
constexpr int kDecCols = 8;
constexpr int kDecPart = kDecCols * (2 + kKv8D);  // floats of a partial result in the workspace: m[8], l[8], O[8][128]
constexpr int kDecMaxCtas = 256;

// One CTA per SM. Up to four columns (DUP): 12 warps with two stages each (8
// sequences of 2048 to 4096 tokens, 64 kv heads: 76 us, with 8 warps of three
// stages 81: the warps wait for their own chains of instructions more than for
// the copies). Up to eight, whose partial results take twice the room: 8 warps
// with three (16 sequences, 8 query heads a kv head: 37 us, with 10 of two 40).
template <bool DUP>
struct DecCfg {
  static constexpr int kWarps = DUP ? 12 : 8;
  static constexpr int kStages = DUP ? 2 : 3;
  static constexpr int kCols = DUP ? 4 : kDecCols;
  static constexpr int kRingBytes = kStages * kDecStageBytes;
  static constexpr int kPartBytes = kCols * (2 + kKv8D) * 4;  // m[], l[], O[][128]
  // Shared memory (offsets from a 1024-byte aligned base): the rings, each
  // warp's first partial result (its last one goes into its spent ring), what
  // the partial results are of, barriers, the tiles' scales.
  static constexpr int kOffPart = kWarps * kRingBytes;
  static constexpr int kOffPairs = kOffPart + kWarps * kPartBytes;
  static constexpr int kOffBars = kOffPairs + kWarps * 2 * 32;
  static constexpr int kOffMeta = kOffBars + kWarps * kStages * 8;
  static constexpr int kOffLast = kOffMeta + kWarps * kStages * 16;
  static constexpr int kBytes = kOffLast + 16 + 1024;  // + alignment slack
  static_assert(kBytes <= 232448, "shared memory of one CTA");
  static_assert(kPartBytes <= kRingBytes && kPartBytes % 16 == 0 && kOffMeta % 16 == 0, "layout");
  static_assert(2 * kWarps <= 32, "a lane for each partial result when they are joined");
};

struct Kv8DecodeArgs {
  Kv8AttnArgs a;
  int* count;   // [gridDim.x] arrivals of pairs that cross CTAs, zero between calls
  float* part;  // [gridDim.x][2][kDecPart]
  int max_rows; // sequences with more rows (new tokens times G) are another kernel's
};

// One pair's place in the line of tiles.
struct DecPair {
  int b, j;        // sequence (-1: none), (kv head, column group) within it
  int len, tiles;  // cached tokens, tiles of each of the sequence's pairs
  int row0, n;     // its first row of the batch, its new tokens
  int64_t first;   // the pair's first tile in the line
};
static_assert(sizeof(DecPair) == 32, "DecCfg");

// Sequence b's lengths; tiles == 0: it has no part in this kernel's work.
__device__ __forceinline__ DecPair dec_sequence(const Kv8AttnArgs& a, int b, int G, int max_rows, bool report) {
  DecPair p = {b, 0, 0, 0, 0, 0, 0};
  if (b >= a.s.B) return p;
  const int64_t capacity = static_cast<int64_t>(a.c.max_blocks) * a.c.P;
  p.row0 = kv8_row_start(a.s, b);
  p.n = a.s.q_start == nullptr ? 1 : kv8_row_start(a.s, b + 1) - p.row0;
  if (p.n < 0 && report) atomicCAS(a.err, 0, kErrKv8Range);
  if (p.n <= 0 || static_cast<int64_t>(p.n) * G > max_rows) return p;
  p.len = __ldg(a.s.seq_lens + b);
  const int least = a.s.q_start == nullptr ? 0 : p.n;
  if (p.len < least || p.len > capacity) {
    if (report) atomicCAS(a.err, 0, kErrKv8Range);
    p.len = a.s.q_start == nullptr && p.len > 0 ? static_cast<int>(capacity) : 0;
  }
  p.tiles = p.len > 0 ? (p.len + kDecTile - 1) / kDecTile : 1;
  return p;
}

// Adds partial result (m2, l2, o2) to (m, l, o), m in powers of two.
__device__ __forceinline__ void dec_join(float& m, float& l, float2& o, float m2, float l2, float2 o2) {
  const float mn = fmaxf(m, m2);
  const float f = m == -INFINITY ? 0.0f : ex2(m - mn), f2 = m2 == -INFINITY ? 0.0f : ex2(m2 - mn);
  m = mn;
  l = l * f + l2 * f2;
  o.x = o.x * f + o2.x * f2;
  o.y = o.y * f + o2.y * f2;
}
__device__ __forceinline__ __half2 dec_pack(float2 o, float l) {
  const float r = l > 0.0f ? 1.0f / l : 0.0f;
  return __floats2half2_rn(o.x * r, o.y * r);
}

// Debug builds: whether 128 values of q or out from offset `at` on are there.
__device__ __forceinline__ bool kv8_row_ok(const Kv8AttnArgs& a, int64_t at) {
  return in_bounds(at >= 0 && at <= (static_cast<int64_t>(a.s.T) * a.Hq - 1) * kKv8D, a.err);
}

// Where row R of a sequence's kv head lies in q and out.
__device__ __forceinline__ int64_t dec_row(const Kv8AttnArgs& a, const DecPair& p, int G, int kvh, int R) {
  return ((static_cast<int64_t>(p.row0) + R / G) * a.Hq + kvh * G + R % G) * kKv8D;
}

template <bool DUP>
__global__ void __launch_bounds__(DecCfg<DUP>::kWarps * 32, 1)
    kv8_decode_kernel(const __grid_constant__ CUtensorMap map, Kv8DecodeArgs args) {
  using C = DecCfg<DUP>;
  constexpr int kWarps = C::kWarps, kStages = C::kStages, kCols = C::kCols;
  extern __shared__ __align__(1024) uint8_t dec_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dec_smem_raw) + 1023) & ~uintptr_t(1023));
  const Kv8AttnArgs& a = args.a;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g = lane >> 2, c = lane & 3;
  uint8_t* ring = sm + warp * C::kRingBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kOffBars) + warp * kStages;
  float* meta = reinterpret_cast<float*>(sm + C::kOffMeta) + warp * kStages * 4;
  DecPair* s_pairs = reinterpret_cast<DecPair*>(sm + C::kOffPairs);  // [warp][2]
  int* s_last = reinterpret_cast<int*>(sm + C::kOffLast);
  const auto part_of = [&](int entry) {  // a warp's first or last partial result
    return reinterpret_cast<float*>(entry & 1 ? sm + (entry >> 1) * C::kRingBytes
                                              : sm + C::kOffPart + (entry >> 1) * C::kPartBytes);
  };
  const DevErr err{a.err};
  const int P = a.c.P, G = a.Hq / a.c.Hkv;
  const int shift = __ffs(P) - 1;
  const auto groups_of = [&](int n) { return DUP ? 1 : (n * G + kDecCols - 1) / kDecCols; };
  if (t == 0) prefetch_tensormap(&map);
  if (lane < kStages) mbar_init(bars + lane, 5);  // the bulk copies, and four scales
  fence_barrier_init();
  __syncwarp();
  grid_dependency_wait();
  grid_launch_dependents();

  // the line's length, and this CTA's and this warp's part of it (mine: of up to
  // 32 sequences, looked up once)
  const auto work_of = [&](const DecPair& p) { return static_cast<int64_t>(p.tiles) * (groups_of(p.n) * a.c.Hkv); };
  DecPair mine = dec_sequence(a, lane, G, args.max_rows, blockIdx.x == 0 && warp == 0);
  int64_t total = work_of(mine);
  for (int b = lane + 32; b < a.s.B; b += 32)
    total += work_of(dec_sequence(a, b, G, args.max_rows, blockIdx.x == 0 && warp == 0));
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (total == 0) return;
  // CTAs: a tile a warp at least; where that is fewer than there are, as many
  // for each pair, so that pairs of one length end with a CTA (joining across
  // CTAs costs 3 us of a call of 10)
  int ctas = gridDim.x;
  if (total < static_cast<int64_t>(kWarps) * ctas) {
    int pairs = mine.tiles > 0 ? groups_of(mine.n) * a.c.Hkv : 0;
    for (int o = 16; o > 0; o >>= 1) pairs += __shfl_xor_sync(0xffffffffu, pairs, o);
    const int want = (static_cast<int>(total) + kWarps - 1) / kWarps;
    ctas = a.s.B <= 32 && pairs <= static_cast<int>(gridDim.x) ? pairs * max(want / pairs, 1) : want;
  }
  if (static_cast<int>(blockIdx.x) >= ctas) return;
  // CTA i takes quot tiles, one more if i < rest
  const int64_t quot = total / ctas;
  const int rest = static_cast<int>(total - quot * ctas);
  const auto cta_start = [&](int i) { return i * quot + min(i, rest); };
  const int64_t cs = cta_start(blockIdx.x), ce = cta_start(blockIdx.x + 1);
  const int64_t ws = cs + (ce - cs) * warp / kWarps, we = cs + (ce - cs) * (warp + 1) / kWarps;

  // the pair that holds tile x of the line
  const auto locate = [&](int64_t x) {
    int64_t base = 0;
    DecPair p = {0, 0, 0, 1, 0, 0, 0};
    for (int b0 = 0; b0 < a.s.B; b0 += 32) {
      const DecPair q = b0 == 0 ? mine : dec_sequence(a, b0 + lane, G, args.max_rows, false);
      const int64_t n = work_of(q);
      int64_t sum = n;
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const uint32_t in = __ballot_sync(0xffffffffu, x < base + sum);
      if (in != 0) {
        const int src = __ffs(in) - 1;
        p.b = b0 + src;
        p.len = __shfl_sync(0xffffffffu, q.len, src);
        p.tiles = __shfl_sync(0xffffffffu, q.tiles, src);
        p.row0 = __shfl_sync(0xffffffffu, q.row0, src);
        p.n = __shfl_sync(0xffffffffu, q.n, src);
        const int64_t first = base + __shfl_sync(0xffffffffu, sum - n, src);
        const int64_t in_sequence = x - first;
        p.j = in_sequence >> 32 ? static_cast<int>(in_sequence / p.tiles)
                                : static_cast<int>(static_cast<uint32_t>(in_sequence) / static_cast<uint32_t>(p.tiles));
        p.first = first + static_cast<int64_t>(p.j) * p.tiles;
        break;
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
    return p;
  };
  const auto advance = [&](DecPair& p) {  // to the next pair of the line
    const int64_t next = p.first + p.tiles;
    if (++p.j == groups_of(p.n) * a.c.Hkv) {
      int b = p.b;
      do p = dec_sequence(a, ++b, G, args.max_rows, false);
      while (p.tiles == 0 && b < a.s.B);
    }
    p.first = next;
  };

  int n_mine = static_cast<int>(we - ws);
  DecPair cur = locate(n_mine > 0 ? ws : cs), nxt = cur;  // consuming, requesting
  int64_t x_next = ws;
  int blk0 = 0, blk_b = -1;      // the window of the block table that the lanes hold
  int blk = 0;
  const int blocks_per_tile = P < kDecTile ? kDecTile / P : 1;
  const int rows_per_copy = P < kDecTile ? P : kDecTile;

  // requests tile x_next into its stage
  const auto request = [&](int stage) {
    while (x_next >= nxt.first + nxt.tiles) advance(nxt);
    const int tok0 = static_cast<int>(x_next - nxt.first) * kDecTile;
    ++x_next;
    const int n = min(nxt.len - tok0, kDecTile);
    const int b0 = tok0 >> shift;
    if (nxt.b != blk_b || b0 < blk0 || b0 + blocks_per_tile > blk0 + 32) {
      blk_b = nxt.b;
      blk0 = b0;
      const int i = b0 + lane;
      blk = i < a.c.max_blocks && (static_cast<int64_t>(i) << shift) < nxt.len
                ? __ldg(a.c.table + static_cast<int64_t>(nxt.b) * a.c.max_blocks + i) : 0;
      if (blk < 0 || blk >= a.c.num_pages) {
        atomicCAS(a.err, 0, kErrKv8Range);
        blk = 0;
      }
    }
    const int copies = n <= 0 ? 0 : n > rows_per_copy ? 2 : 1;
    const int page0 = __shfl_sync(0xffffffffu, blk, b0 - blk0);
    const int page1 = __shfl_sync(0xffffffffu, blk, min(b0 - blk0 + blocks_per_tile - 1, 31));
    const int kvh = nxt.j / groups_of(nxt.n);
    // lanes 0, 1: the scales of K (first, second half of the tile), 2, 3: of V
    if (lane < 4) {
      const int page = (lane & 1) && copies == 2 ? page1 : page0;
      cp_async_4(meta + stage * 4 + lane,
                 a.c.scales + (static_cast<int64_t>(page) * 2 + (lane >> 1)) * a.c.Hkv + kvh);
      cp_async_arrive(bars + stage);
    }
    if (lane == 0) {
      uint8_t* dst = ring + stage * kDecStageBytes;
      mbar_arrive_expect_tx(bars + stage, 2u * copies * rows_per_copy * kKv8D);
      for (int i = 0; i < copies; ++i) {
        const int page = i == 0 ? page0 : page1;
        const int row = (page * 2 * a.c.Hkv + kvh) * P + (P >= kDecTile ? tok0 & (P - 1) : 0);
        tma_load_2d(dst + i * rows_per_copy * kKv8D, &map, bars + stage, 0, row);
        tma_load_2d(dst + kDecTile * kKv8D + i * rows_per_copy * kKv8D, &map, bars + stage, 0, row + a.c.Hkv * P);
      }
    }
  };

  for (int i = 0; i < kStages && i < n_mine; ++i) request(i);

  uint32_t qf[16];             // this lane's column's query, dimensions 32c ..
  float O[8][4], m[2], l[2];   // columns 2c, 2c + 1
  int limit[2];                // tokens that they see
  bool fresh = true;
  int stage = 0;
  uint32_t phase = 0;
  int64_t x = ws;
  if (lane < 2) s_pairs[2 * warp + lane].b = -1;
  for (int it = 0; it < n_mine; ++it, ++x) {
    while (x >= cur.first + cur.tiles) advance(cur);
    if (fresh) {
      const int groups = groups_of(cur.n), r0 = cur.j % groups * kDecCols;
      const int col = DUP ? g & 3 : g;
      const bool any = r0 + col < cur.n * G;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + dec_row(a, cur, G, cur.j / groups, any ? r0 + col : 0) + 32 * c);
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // (a column without a row: any limit from 1)
        const int r = r0 + (DUP ? (2 * c + k) & 3 : 2 * c + k);
        limit[k] = min(cur.len - cur.n + 1 + r / G, cur.len);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = any ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        qf[4 * i] = v.x;
        qf[4 * i + 1] = v.y;
        qf[4 * i + 2] = v.z;
        qf[4 * i + 3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) O[i][k] = 0.0f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.0f;
      fresh = false;
    }
    const int tok0 = static_cast<int>(x - cur.first) * kDecTile;
    const int n = min(cur.len - tok0, kDecTile);
    if (!kv8_wait(bars + stage, phase, err)) {
      // given up (reported): nothing more is requested, and the copies still
      // under way get their limit before their memory is used for anything else
      for (int i = 1; i < kStages && it + i < n_mine; ++i) {
        const int s2 = (stage + i) % kStages;
        kv8_wait(bars + s2, s2 > stage ? phase : phase ^ 1u, err);
      }
      n_mine = it + 1;
    }
    if (n > 0) {
      const uint8_t* sk = ring + stage * kDecStageBytes;
      const uint8_t* sv = sk + kDecTile * kKv8D;
      // ---- scores: S^T[token, column], two blocks of 16 tokens
      float S[2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t w[2][8];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = mt * 16 + r * 8 + g;  // (row & 7) == g
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 v = *reinterpret_cast<const uint4*>(sk + row * kKv8D + (((2 * c + k) ^ g) << 4));
            w[r][4 * k] = v.x ^ 0x80808080u;
            w[r][4 * k + 1] = v.y ^ 0x80808080u;
            w[r][4 * k + 2] = v.z ^ 0x80808080u;
            w[r][4 * k + 3] = v.w ^ 0x80808080u;
          }
        }
        S[mt][0] = S[mt][1] = S[mt][2] = S[mt][3] = 0.0f;
#pragma unroll
        for (int s = 0; s < 8; ++s)
          mma_16x8x16(S[mt], unbias_pair<0x4140>(w[0][s]), unbias_pair<0x4140>(w[1][s]), unbias_pair<0x4342>(w[0][s]),
                      unbias_pair<0x4342>(w[1][s]), qf[2 * s], qf[2 * s + 1]);
      }
      // ---- weights
      const float4 mv = *reinterpret_cast<const float4*>(meta + stage * 4);
      const float kscale = a.scale * 1.4426950408889634f;
      const float sks[2] = {mv.x * kscale, mv.y * kscale};
      // clamped: smaller scales give values below 2^-50, larger ones are beyond fp16
      const float lsv[2] = {__log2f(fminf(fmaxf(mv.z, 8.673617e-19f), 1.1529215e18f)),
                            __log2f(fminf(fmaxf(mv.w, 8.673617e-19f), 1.1529215e18f))};
      float mx[2] = {m[0], m[1]};
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tok = mt * 16 + (k >> 1) * 8 + g;
          S[mt][k] = tok0 + tok < limit[k & 1] ? S[mt][k] * sks[mt] + lsv[mt] : -INFINITY;
          mx[k & 1] = fmaxf(mx[k & 1], S[mt][k]);
        }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
        const float f[2] = {mx[0] == m[0] ? 1.0f : ex2(m[0] - mx[0]), mx[1] == m[1] ? 1.0f : ex2(m[1] - mx[1])};
        m[0] = mx[0];
        m[1] = mx[1];
        l[0] *= f[0];
        l[1] *= f[1];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) O[i][k] *= f[k & 1];
      }
      // (a column may have seen nothing yet: its tiles before this one are other warps')
      const float up[2] = {m[0] == -INFINITY ? 0.0f : 14.0f - m[0], m[1] == -INFINITY ? 0.0f : 14.0f - m[1]};
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const float isv = ex2(-lsv[mt]);
        float w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[k] = ex2(S[mt][k] + up[k & 1]);
          l[k & 1] += w[k] * isv;
        }
        uint32_t bh[2], bl[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const __half2 hi = __floats2half2_rn(w[2 * r], w[2 * r + 1]);
          const float2 hf = __half22float2(hi);
          const __half2 lo = __floats2half2_rn(w[2 * r] - hf.x, w[2 * r + 1] - hf.y);
          if constexpr (DUP) {
            const __half2 v = c < 2 ? hi : lo;  // columns 4-7 repeat the heads of 0-3
            bh[r] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&v));
          } else {
            bh[r] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&hi));
            bl[r] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&lo));
          }
        }
        // ---- values: O^T[dimension, column] += V^T w^T; row g (g + 8) of
        // block i is dimension 16g + 2i (+ 1)
        uint32_t v[4][4];  // tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = mt * 16 + 2 * c + (r & 1) + (r >> 1) * 8;
          const uint4 q = *reinterpret_cast<const uint4*>(sv + row * kKv8D + ((g ^ (row & 7)) << 4));
          v[r][0] = q.x ^ 0x80808080u;
          v[r][1] = q.y ^ 0x80808080u;
          v[r][2] = q.z ^ 0x80808080u;
          v[r][3] = q.w ^ 0x80808080u;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t sel = i & 1 ? 0x7362u : 0x5140u;
          const uint32_t p0 = __byte_perm(v[0][i >> 1], v[1][i >> 1], sel);
          const uint32_t p1 = __byte_perm(v[2][i >> 1], v[3][i >> 1], sel);
          const uint32_t a0 = unbias_pair<0x4140>(p0), a1 = unbias_pair<0x4342>(p0);
          const uint32_t a2 = unbias_pair<0x4140>(p1), a3 = unbias_pair<0x4342>(p1);
          mma_16x8x16(O[i], a0, a1, a2, a3, bh[0], bh[1]);
          if constexpr (!DUP) mma_16x8x16(O[i], a0, a1, a2, a3, bl[0], bl[1]);
        }
      }
    }
    __syncwarp();  // the stage is read
    if (it + kStages < n_mine) request(stage);
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
    if (x + 1 < cur.first + cur.tiles && it + 1 < n_mine) continue;
    // ---- the pair, or this warp's part of it, is done
    fresh = true;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], o);
    }
    if constexpr (DUP) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) O[i][k] += __shfl_xor_sync(0xffffffffu, O[i][k], 2);
    }
    const bool whole = cur.first >= ws && cur.first + cur.tiles <= we;
    const int slot = cur.first <= ws ? 0 : 1;
    if (whole) {
      const int groups = groups_of(cur.n), r0 = cur.j % groups * kDecCols;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int col = 2 * c + k;
        if (r0 + col < cur.n * G && (!DUP || c < 2)) {
          const int64_t at = dec_row(a, cur, G, cur.j / groups, r0 + col);
          if (!kv8_row_ok(a, at)) continue;
          __half* dst = a.out + at + 16 * g;
          const float r = l[k] > 0.0f ? 1.0f / l[k] : 0.0f;
          uint4 y[2];
          __half2* hv = reinterpret_cast<__half2*>(y);
#pragma unroll
          for (int i = 0; i < 8; ++i) hv[i] = __floats2half2_rn(O[i][k] * r, O[i][k + 2] * r);
          reinterpret_cast<uint4*>(dst)[0] = y[0];
          reinterpret_cast<uint4*>(dst)[1] = y[1];
        }
      }
    } else {
      float* part = part_of(2 * warp + slot);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int col = 2 * c + k;
        if (col >= kCols) continue;
        if (g == 0) {
          part[col] = m[k];
          part[kCols + col] = l[k];
        }
        float4* dst = reinterpret_cast<float4*>(part + 2 * kCols + col * kKv8D + 16 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dst[i] = make_float4(O[2 * i][k], O[2 * i][k + 2], O[2 * i + 1][k], O[2 * i + 1][k + 2]);
      }
      if (lane == 0) s_pairs[2 * warp + slot] = cur;
    }
  }
  __syncthreads();

  // ---- partial results of one pair, joined in the order of the line: thread
  // (column, two dimensions)
  constexpr int kEntries = 2 * kWarps;
  const int64_t my_first = lane < kEntries ? s_pairs[lane].first : 0;
  const uint32_t used = __ballot_sync(0xffffffffu, lane < kEntries && s_pairs[lane].b >= 0);
  const uint32_t before = used & ((1u << lane) - 1u);
  const int64_t prev_first = __shfl_sync(0xffffffffu, my_first, before != 0 ? 31 - __clz(before) : 0);
  uint32_t leaders = __ballot_sync(0xffffffffu, ((used >> lane) & 1u) != 0 && (before == 0 || prev_first != my_first));
  // where a pair that crosses CTAs has its partial result: a CTA has at most
  // two such pairs, one that begins at or before its start and one after
  const auto slot_of = [&](const DecPair& p, int i) {
    return args.part + (2 * i + (p.first <= cta_start(i) ? 0 : 1)) * kDecPart;
  };
  int crossing[2] = {-1, -1};  // their first entries
  while (leaders != 0) {
    const int e = __ffs(leaders) - 1;
    leaders &= leaders - 1u;
    const uint32_t members = used & ~((1u << e) - 1u) & (leaders != 0 ? (leaders & (0u - leaders)) - 1u : 0xffffffffu);
    const DecPair p = s_pairs[e];
    const int groups = groups_of(p.n), r0 = p.j % groups * kDecCols;
    const int nh = min(p.n * G - r0, kDecCols);
    const bool whole = p.first >= cs && p.first + p.tiles <= ce;
    if (!whole) crossing[crossing[0] >= 0 ? 1 : 0] = e;
    for (int i = t; i < nh * (kKv8D / 2); i += kWarps * 32) {
      const int col = i >> 6, d = 2 * (i & 63);
      float m = -INFINITY, l = 0.0f;
      float2 o = make_float2(0.0f, 0.0f);
      for (uint32_t left = members; left != 0; left &= left - 1u)
        m = fmaxf(m, part_of(__ffs(left) - 1)[col]);
      for (uint32_t left = members; left != 0; left &= left - 1u) {
        const float* part = part_of(__ffs(left) - 1);
        const float f = part[col] == -INFINITY ? 0.0f : ex2(part[col] - m);
        const float2 v = *reinterpret_cast<const float2*>(part + 2 * kCols + col * kKv8D + d);
        l = fmaf(part[kCols + col], f, l);
        o.x = fmaf(v.x, f, o.x);
        o.y = fmaf(v.y, f, o.y);
      }
      if (whole) {
        const int64_t at = dec_row(a, p, G, p.j / groups, r0 + col);
        if (kv8_row_ok(a, at)) *reinterpret_cast<__half2*>(a.out + at + d) = dec_pack(o, l);
      } else {
        float* part = slot_of(p, static_cast<int>(blockIdx.x));
        if (d == 0) {
          part[col] = m;
          part[kDecCols + col] = l;
        }
        *reinterpret_cast<float2*>(part + 2 * kDecCols + col * kKv8D + d) = o;
      }
    }
  }
  if (crossing[0] < 0) return;
  // pairs that cross CTAs: the last one to arrive joins them. (Both of a CTA's
  // arrivals together: each step costs a round trip to L2.)
  const auto owner = [&](int64_t x) {
    const int64_t longer = rest * (quot + 1);
    return static_cast<int>(x < longer ? x / (quot + 1) : rest + (x - longer) / quot);
  };
  __threadfence();
  __syncthreads();
  if (t < 2) {
    int last = 0;
    const int e = t == 0 ? crossing[0] : crossing[1];
    if (e >= 0) {
      const int c0 = owner(s_pairs[e].first), c1 = owner(s_pairs[e].first + s_pairs[e].tiles - 1);
      last = in_bounds(c0 >= 0 && c0 <= c1 && c1 < static_cast<int>(gridDim.x) && gridDim.x <= kDecMaxCtas, a.err) &&
                     atom_add_relaxed_gpu(args.count + c0, 1) == c1 - c0
                 ? 1
                 : 0;
    }
    s_last[t] = last;
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (!s_last[k]) continue;
    __threadfence();
    const DecPair p = s_pairs[k == 0 ? crossing[0] : crossing[1]];
    const int groups = groups_of(p.n), r0 = p.j % groups * kDecCols;
    const int nh = min(p.n * G - r0, kDecCols);
    const int c0 = owner(p.first), c1 = owner(p.first + p.tiles - 1);
    for (int i = t; i < nh * (kKv8D / 2); i += kWarps * 32) {
      const int col = i >> 6, d = 2 * (i & 63);
      float m = -INFINITY, l = 0.0f;
      float2 o = make_float2(0.0f, 0.0f);
#pragma unroll 4
      for (int n = c0; n <= c1; ++n) {
        const float* part = slot_of(p, n);
        dec_join(m, l, o, __ldcg(part + col), __ldcg(part + kDecCols + col),
                 __ldcg(reinterpret_cast<const float2*>(part + 2 * kDecCols + col * kKv8D + d)));
      }
      const int64_t at = dec_row(a, p, G, p.j / groups, r0 + col);
      if (kv8_row_ok(a, at)) *reinterpret_cast<__half2*>(a.out + at + d) = dec_pack(o, l);
    }
    if (t == 0) args.count[c0] = 0;
  }
}

}  // namespace w4a8
