// Causal attention of many new tokens per sequence over the paged 8-bit KV
// cache, both contractions on the tensor cores (tcgen05 kind::f16).
#pragma once
#include "kv8_attention.cuh"

namespace w4a8 {

// A CTA takes 256 rows of one (sequence, kv head): row R = i G + h is query
// head h of the group at new token i, so that grouped heads share the cache's
// tiles. Per tile of 128 cached tokens and block t of 128 rows
//   S = Q_t K^T        128 x 128 x 128, Q and K from shared memory
//   P_t = 2^(z - M)    thread = row, the row of S in registers
//   O_t += P_t V       128 x 128 x 128, P from tensor memory, V from shared
// so that the tensor cores need 2 * 2 * 512 cycles a tile and pair of blocks,
// and the exponentials (16 a cycle and SM) as many: the floor of a tile. Tensor
// memory holds O_0, O_1, P_0, P_1 and one S: a softmax reads its row of S at
// once, and the other block's next S is made while it works, so that neither
// block waits for its own products (with S_0 and S_1 in place of the one S, P_t
// over S_t, each block's S, softmax and PV followed one another: 5700 cycles a
// tile and pair of blocks instead of 4500). Measured, replayed graphs over caches
// larger than the L2: 1000 new tokens of 9017 195 us (716 TFLOP/s), 3 prompts of 1500
// to 2100 tokens 181 us (549: some 700 pieces of 1 to 17 tiles, whose first tile and
// last products nothing overlaps). Nothing is full: of the cycles that an SM is
// active the first takes 65 % of the issue slots, 44 % of the tensor pipe, 44 % of the
// exponentials. What is left is the order of a tile: a next S waits until the
// one S is read, a row's two threads exchange their maxima before the first
// exponential. Fewer and longer CTAs that take one piece after another were slower
// (254 and 275 us for 196 and 221), and so were 8 softmax warps with 128 registers
// a thread (222 for 192).
//
// Roles: warps 0-15 the softmax, two threads a row (warps 8 t + 4 h ..: block t,
// columns 64 h ..; with one thread a row and 128 values in its registers nothing
// was left to keep several exponentials under way: 2400 cycles for a tile's, now
// 1700); warps 16-19 turn K's bytes into fp16 integers (exact), 20-23
// V's, from global memory through registers, requested a tile ahead, into double
// buffers; one thread of warp 24 issues the products for S, one of warp 25 those
// for O; warp 26 brings the tiles' scales. The bytes do not pass through shared memory on their way: the products'
// own reads of it (1536 of 2048 cycles a tile) leave room for little more than
// the converted tiles.
//
// Few pieces (a chunk of one long prompt): each piece's tiles are cut into
// `splits` parts on as many CTAs, whose unnormalized outputs, references and sums
// a second kernel joins.
//
// Softmax weights carry their page's value scale, as in the decode kernel: z_j
// = x_j + log2 sV_j, w_j = 2^(z_j - M + 10), rounded once to fp16 for the
// product (relative 2^-11; at most 2^15); the denominator sums w_j / sV_j of
// the unrounded weights in fp32. The reference M only moves when the running
// maximum has passed it by 5, which spares most of the rescales of O.
constexpr int kPreRows = 128;      // rows of a block
constexpr int kPreTile = 128;      // cached tokens of a tile
constexpr int kPreThreads = 28 * 32;  // (warp 27 only fills its group of four)
// Registers a thread: launched with kPreRegs, which the groups then share out.
constexpr int kPreRegs = 72, kPreRegsSoftmax = 88, kPreRegsBytes = 56, kPreRegsIssue = 40;
static_assert(16 * kPreRegsSoftmax + 8 * kPreRegsBytes + 4 * kPreRegsIssue <= 28 * kPreRegs,
              "setmaxnreg draws on the launch's registers");
constexpr int kPreMinTiles = 4;    // of a split
constexpr float kPreShift = 10.0f, kPreSlack = 5.0f;

struct PreSmem {
  static constexpr int kBlock = 128 * 128;     // 64 columns (128 bytes) of a 128-row operand
  static constexpr int kOperand = 2 * kBlock;  // 128 x 128 fp16
  static constexpr int kOffQ = 0;              // [2]
  static constexpr int kOffK = 2 * kOperand;   // [2]
  static constexpr int kOffV = 4 * kOperand;   // [2]
  static constexpr int kOffScale = 6 * kOperand;         // [4][8] (sK', log2 sV, 1 / sV, -)
  static constexpr int kOffMax = kOffScale + 4 * 8 * 16;  // [2 turns][2 blocks][2 halves][128] row maxima
  static constexpr int kOffBars = kOffMax + 8 * 128 * 4;
  static constexpr int kBars = 34;
  static constexpr int kOffMisc = kOffBars + kBars * 8;  // TMEM address, abort flag
  static constexpr int kBytes = kOffMisc + 16 + 1024;    // + alignment slack
  static_assert(kBytes <= 232448, "shared memory of one CTA");
};
enum PreBar { kKFull = 0, kKFree = 2, kVFull = 4, kVFree = 6, kSFull = 8, kSRead = 10, kPFull = 12, kPFree = 14,
              kScale = 16, kDrain = 20, kPair = 22, kScaleFree = 30 };
constexpr int kPreTmemO = 0, kPreTmemP = 256, kPreTmemS = 384, kPreTmemCols = 512;  // O_t: + 128 t, P_t: + 64 t

// Loads 32 consecutive columns of this thread's lane and waits for them (one
// statement: see tmem_ld_16_wait).
__device__ __forceinline__ void tmem_ld_32_wait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// The same for 64 columns.
__device__ __forceinline__ void tmem_ld_64_wait(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64]; "
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, "
      "%44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, "
      "[%65]; "
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
        "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
        "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
        "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
        "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
}
// 16 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void st_shared_16(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// (volatile: loaded where it is used, so that a tile's scales take no registers
// while a row of S is held)
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// mbar_arrive and mbar_wait (bounded, given up when `abort` is set, which it
// sets itself after the limit) on shared addresses and with a 32-bit timer: the
// softmax warps wait with a row of S in their registers.
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// RELAXED: sleeps between polls, for warps that have a tile's time to spare.
template <bool RELAXED>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint32_t abort, int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  uint32_t t0, now;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t0));
#pragma unroll 1
  for (uint32_t it = 1;; ++it) {
    if constexpr (RELAXED) __nanosleep(100);
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 0) {
      uint32_t stop;
      asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(stop) : "r"(abort));
      if (stop) return false;
      asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
      const int32_t ns = static_cast<int32_t>(now - t0);
      if (ns < 0) {  // a backward step of the timer: start again
        t0 = now;
      } else if (ns > static_cast<int32_t>(kWaitLimitNs)) {
        asm volatile("st.volatile.shared.u32 [%0], 1;" ::"r"(abort) : "memory");
        atomicCAS(err, 0, kErrKv8Wait);
        return false;
      }
    }
  }
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
struct Kv8PrefillArgs {
  Kv8AttnArgs a;
  int slots, few_rows, splits;
  // splits > 1: [slots * Hkv][splits][256] rows of 128 outputs, then of (reference, sum)
  float* part;
  float* part_ml;
};
__device__ __forceinline__ int pre_chunk(int tiles, int splits) {
  return max((tiles + splits - 1) / splits, kPreMinTiles);
}

// CUT: pieces are cut (an instantiation of its own: what it keeps in registers
// costs the other 15%).
template <bool CUT>
__global__ void __launch_bounds__(kPreThreads, 1) kv8_prefill_kernel(Kv8PrefillArgs args) {
  const Kv8AttnArgs a = args.a;
  extern __shared__ __align__(1024) uint8_t pre_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pre_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + PreSmem::kOffBars);
  float4* s_scale = reinterpret_cast<float4*>(sm + PreSmem::kOffScale);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + PreSmem::kOffMisc);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const DevErr err{a.err};
  const int P = a.c.P, G = a.Hq / a.c.Hkv;

  grid_dependency_wait();
  grid_launch_dependents();
  // this CTA's rows: slot start_b G / 256 + b + k holds rows 256 k .. of
  // sequence b. Later slots see more of the cache: taken first.
  const int split = CUT ? static_cast<int>(blockIdx.x) % args.splits : 0;
  const int piece = CUT ? static_cast<int>(blockIdx.x) / args.splits : static_cast<int>(blockIdx.x);
  const int kvh = piece % a.c.Hkv;
  const int slot = args.slots - 1 - piece / a.c.Hkv;
  const int b = kv8_find(a.s, slot, G, 2 * kPreRows, 1);
  if (b < 0) return;
  const Kv8Seq sq = kv8_sequence(a.s, b, static_cast<int64_t>(a.c.max_blocks) * P, t == 0 ? a.err : nullptr);
  // (rows times heads of a batch are under 2^31)
  const int first = sq.first, rows = (kv8_row_start(a.s, b + 1) - first) * G;
  const int row0 = (slot - static_cast<int>(static_cast<int64_t>(first) * G / (2 * kPreRows)) - b) * 2 * kPreRows;
  if (row0 >= rows || rows <= args.few_rows) return;  // (few rows: the decode kernel's)
  if (sq.n < 0) {  // a length that does not fit (reported): zeros
    const int r = row0 + t;
    if (split == 0 && t < 2 * kPreRows && r < rows) {
      uint4* dst = reinterpret_cast<uint4*>(a.out + ((static_cast<int64_t>(first) + r / G) * a.Hq + kvh * G + r % G) * kKv8D);
      if (kv8_row_ok(a, (static_cast<int64_t>(first) + r / G) * a.Hq * kKv8D))
        for (int i = 0; i < 16; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  // tiles that each block sees
  int nt[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int last = min(row0 + (k + 1) * kPreRows, rows) - 1;  // its last row
    nt[k] = last < row0 + k * kPreRows ? 0 : (sq.pos0 + last / G + kPreTile) / kPreTile;
  }
  // this CTA's part of them: `tiles` from tile0 on
  int tile0 = 0, tiles = max(nt[0], nt[1]);
  bool whole = true;
  if constexpr (CUT) {
    const int chunk = pre_chunk(tiles, args.splits);
    whole = chunk >= tiles;
    tile0 = split * chunk;
    tiles = min(tiles - tile0, chunk);
    if (tiles <= 0) return;
    nt[0] = max(min(nt[0] - tile0, tiles), 0);
    nt[1] = max(min(nt[1] - tile0, tiles), 0);
  }

  if (t == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + kKFull + i, 4);
      mbar_init(bars + kKFree + i, 1);
      mbar_init(bars + kVFull + i, 4);
      mbar_init(bars + kVFree + i, 1);
      mbar_init(bars + kSFull + i, 1);
      mbar_init(bars + kSRead + i, 8);
      mbar_init(bars + kPFull + i, 8);
      mbar_init(bars + kPFree + i, 1);
      mbar_init(bars + kDrain + i, 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bars + kScale + i, 1);
      mbar_init(bars + kScaleFree + i, 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(bars + kPair + i, 2);
    fence_barrier_init();
    s_tmem[1] = 0u;  // set by the first wait that gives up
  }
  const uint32_t bar0 = smem_u32(bars), abort = smem_u32(s_tmem + 1);
  const auto wait = [&](int bar, int phase) {
    return bar_wait<false>(bar0 + 8 * bar, static_cast<uint32_t>(phase) & 1u, abort, a.err);
  };
  const auto wait_warp_relaxed = [&](int bar, int phase) {
    return __all_sync(0xffffffffu, bar_wait<true>(bar0 + 8 * bar, static_cast<uint32_t>(phase) & 1u, abort, a.err)) != 0;
  };
  const auto wait_warp = [&](int bar, int phase) {  // the same answer in every lane
    return __all_sync(0xffffffffu, wait(bar, phase)) != 0;
  };

  // barriers, queries and the tensor memory's address are there: every role
  // comes here once, after what it can request before
  const auto set_up = [&]() {
    tc_fence_before();
    named_bar_sync(1, kPreThreads);
    tc_fence_after();
    return *s_tmem;
  };

  if (warp < 16) {
    // ------------------------------------------------------------ softmax
    // this thread's row, and its half of the query into shared memory
    const int blk = warp >> 3, half = (warp >> 2) & 1;  // block of rows, half of the columns
    const int lr = (warp & 3) * 32 + lane;              // row of the block, TMEM lane
    const int row = row0 + blk * kPreRows + lr;
    const bool mine = row < rows;
    const int ti = mine ? row / G : 0;
    // where its half row lies in q and out; -1: no row
    const int64_t at =
        mine ? ((static_cast<int64_t>(first) + ti) * a.Hq + kvh * G + (row - ti * G)) * kKv8D + 64 * half : -1;
    const int limit = (mine ? sq.pos0 + ti + 1 : 1) - tile0 * kPreTile;  // tokens that it sees, from tile0 on
    {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = mine ? __ldg(reinterpret_cast<const uint4*>(a.q + at) + i) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t dst = smem_u32(sm) + PreSmem::kOffQ + blk * PreSmem::kOperand + half * PreSmem::kBlock + lr * 128;
      const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;  // scores are taken with |scale|
#pragma unroll
      for (int i = 0; i < 8; ++i)
        st_shared_16(dst + ((i ^ (lr & 7)) << 4), v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip);
    }
    fence_proxy_async_smem();
    const uint32_t tmem = set_up();
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPreRegsSoftmax));
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    // this thread's half of its row of S, P and O
    const uint32_t tS = tmem + kPreTmemS + 64 * half + lane_base, tP = tmem + kPreTmemP + 64 * blk + 32 * half + lane_base;
    const uint32_t tO = tmem + kPreTmemO + 128 * blk + 64 * half + lane_base;
    // a value of the row's other thread, turn by turn (two turns' places: a
    // warp writes turn n + 2 after its partner arrived for n + 1, with n read)
    const uint32_t s_max = smem_u32(sm + PreSmem::kOffMax) + 4 * (blk * 256 + half * 128 + lr);
    const int pair_bar = kPair + blk * 4 + (warp & 3);
    const auto give = [&](int turn, float v) {
      st_shared_f32(s_max + (turn & 1) * 2048, v);
      __syncwarp();
      if (lane == 0) bar_arrive(bar0 + 8 * pair_bar);
    };
    const auto take = [&](int turn, bool& ok) {
      ok = wait_warp(pair_bar, turn);
      return ld_shared_f32(s_max + (turn & 1) * 2048 + (half ? -512 : 512));
    };
    const int mine_nt = nt[blk];
    float ref = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < mine_nt; ++j) {
      if (!(ok = wait_warp(kScale + (j & 3), j >> 2) && wait_warp(kSFull + blk, j))) break;
      tc_fence_after();
      uint32_t r[64];
      tmem_ld_64_wait(tS, r);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(bar0 + 8 * (kSRead + blk));
      const uint32_t sc = smem_u32(s_scale + (j & 3) * 8 + 4 * half);
      const int left = limit - j * kPreTile - 64 * half;  // columns of this half that the row sees
      if (__any_sync(0xffffffffu, left < 64)) {
        __syncwarp();  // (kept a branch: as selects it would cost every tile 128 instructions)
#pragma unroll
        for (int e = 0; e < 64; ++e) r[e] = e < left ? r[e] : 0xFF800000u;  // -inf
      }
      float mx = -INFINITY;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float top = __uint_as_float(r[16 * u]);
#pragma unroll
        for (int e = 1; e < 15; e += 2)
          top = max3(top, __uint_as_float(r[16 * u + e]), __uint_as_float(r[16 * u + e + 1]));
        top = fmaxf(top, __uint_as_float(r[16 * u + 15]));
        const float4 s = ld_shared_f4(sc + 16 * u);
        mx = fmaxf(mx, fmaf(top, s.x, s.y));
      }
      give(j, mx);
      // O and P are this block's again once the last tile's product is done
      if (j > 0) {
        if (!(ok = wait_warp(kPFree + blk, j - 1))) break;
        tc_fence_after();  // of P's stores below too, in tiles that leave O as it is
      }
      mx = fmaxf(mx, take(j, ok));
      if (!ok) break;
      // move the reference where the maximum has passed it
      const bool move = mx > ref + kPreSlack || (ref == -INFINITY && mx > -INFINITY);
      if (__any_sync(0xffffffffu, move)) {
        const float f = move && ref > -INFINITY ? ex2(ref - mx) : 1.0f;
        ref = move ? mx : ref;
        l *= f;
        if (j > 0) {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t o[16];
            tmem_ld_16_wait(tO + 16 * q, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st_16(tO + 16 * q, o);
          }
        }
      }
      const float base = ref > -INFINITY ? kPreShift - ref : 0.0f;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t p[8];
        const float4 s = ld_shared_f4(sc + 16 * u);
        const float off = s.y + base;
        float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = 16 * u + 2 * e;
          const float w0 = ex2(fmaf(__uint_as_float(r[i]), s.x, off)), w1 = ex2(fmaf(__uint_as_float(r[i + 1]), s.x, off));
          sum0 += w0;
          sum1 += w1;
          const __half2 h = __floats2half2_rn(w0, w1);
          p[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        l = fmaf(sum0 + sum1, s.z, l);
        tmem_st_8(tP + 8 * u, p);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(bar0 + 8 * (kPFull + blk));
    }
    if (ok && mine_nt > 0 && wait_warp(kPFree + blk, mine_nt - 1)) {
      tc_fence_after();
      give(mine_nt, l);
      l += take(mine_nt, ok);
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      const int64_t part_row =
          ((static_cast<int64_t>(slot) * a.c.Hkv + kvh) * args.splits + split) * (2 * kPreRows) + blk * kPreRows + lr;
      const bool part_ok = !CUT || whole ||
                           in_bounds(part_row >= 0 && slot >= 0 && slot < args.slots && split < args.splits, a.err);
      const bool out_ok = at < 0 || kv8_row_ok(a, at - 64 * half);
      if (CUT && !whole && part_ok && half == 0) *reinterpret_cast<float2*>(args.part_ml + 2 * part_row) = make_float2(ref, l);
#pragma unroll 1
      for (int q = 0; q < 2; ++q) {
        uint32_t r[32];
        tmem_ld_32_wait(tO + 32 * q, r);
        if (!part_ok || !out_ok) continue;
        if (CUT && !whole) {
          float4* dst = reinterpret_cast<float4*>(args.part + part_row * kKv8D + 64 * half + 32 * q);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]), __uint_as_float(r[4 * i + 2]),
                                 __uint_as_float(r[4 * i + 3]));
        } else if (at >= 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 y;
            __half2* h = reinterpret_cast<__half2*>(&y);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              h[e] = __floats2half2_rn(__uint_as_float(r[8 * i + 2 * e]) * inv,
                                       __uint_as_float(r[8 * i + 2 * e + 1]) * inv);
            reinterpret_cast<uint4*>(a.out + at)[4 * q + i] = y;
          }
        }
      }
    }
  } else if (warp < 24) {
    // ---------------------------------------------------- bytes to operands
    const int kv = warp >= 20 ? 1 : 0;
    // a pass covers 16 tokens: lanes in pairs of rows and quarters of 64 bytes,
    // so that eight lanes' stores meet all banks
    const int ch = (lane & 3) + 4 * ((lane >> 3) & 1);
    const int r0 = (warp & 3) * 4 + ((lane >> 2) & 1) + 2 * (lane >> 4);  // row within a pass
    const int shift = __ffs(P) - 1;
    const int32_t* table = a.c.table + static_cast<int64_t>(b) * a.c.max_blocks;
    // lane i < 8: the page of pass i of tile j, -1 behind the sequence's end;
    // requested two tiles ahead of the codes' use
    const auto page_of = [&](int j) {
      const int tok = (tile0 + j) * kPreTile + 16 * (lane & 7);
      return tok < sq.len && j < tiles ? __ldg(table + (tok >> shift)) : -1;
    };
    // where the pass begins, as a row of 128 bytes of the cache
    const auto place_of = [&](int j, int page) {
      const int tok = (tile0 + j) * kPreTile + 16 * (lane & 7);
      if (tok >= sq.len || j >= tiles) return -1;
      if (page < 0 || page >= a.c.num_pages) {
        atomicCAS(a.err, 0, kErrKv8Range);
        page = 0;
      }
      return (((page * 2 + kv) * a.c.Hkv + kvh) << shift) + (tok & (P - 1));
    };
    uint4 raw[8];
    const int8_t* from = a.c.codes + r0 * kKv8D + 16 * ch;
    const auto load = [&](int i, int places) {
      const int place = __shfl_sync(0xffffffffu, places, i);
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (place >= 0)  // (places behind the end inside its last page: any bytes, weight 0)
        raw[i] = __ldg(reinterpret_cast<const uint4*>(from + static_cast<int64_t>(place) * kKv8D));
    };
    const uint32_t dst0 = smem_u32(sm) + (kv ? PreSmem::kOffV : PreSmem::kOffK) + (ch >> 2) * PreSmem::kBlock + r0 * 128;
    const uint32_t sw0 = ((2 * (ch & 3)) ^ (r0 & 7)) << 4, sw1 = ((2 * (ch & 3) + 1) ^ (r0 & 7)) << 4;
    const int full = kv ? kVFull : kKFull, free = kv ? kVFree : kKFree;
    const int places0 = place_of(0, page_of(0));
#pragma unroll
    for (int i = 0; i < 8; ++i) load(i, places0);
    int page = page_of(1);
    set_up();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPreRegsBytes));
    for (int j = 0; j < tiles; ++j) {
      const int next = place_of(j + 1, page);
      page = page_of(j + 2);
      if (j >= 2 && !wait_warp_relaxed(free + (j & 1), (j >> 1) - 1)) break;
      const uint32_t dst = dst0 + (j & 1) * PreSmem::kOperand;
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // row 16 i + r0
        const uint32_t w[4] = {raw[i].x ^ 0x80808080u, raw[i].y ^ 0x80808080u, raw[i].z ^ 0x80808080u,
                               raw[i].w ^ 0x80808080u};
        st_shared_16(dst + sw0 + i * 2048, unbias_pair<0x4140>(w[0]), unbias_pair<0x4342>(w[0]),
                     unbias_pair<0x4140>(w[1]), unbias_pair<0x4342>(w[1]));
        st_shared_16(dst + sw1 + i * 2048, unbias_pair<0x4140>(w[2]), unbias_pair<0x4342>(w[2]),
                     unbias_pair<0x4140>(w[3]), unbias_pair<0x4342>(w[3]));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(bar0 + 8 * (full + (j & 1)));
      // all of the next tile's requests together: one between two passes would
      // make the next pass wait for it (they share the few counters that a warp
      // waits on), measured 3900 cycles a tile and operand instead of 900
#pragma unroll
      for (int i = 0; i < 8; ++i) load(i, next);
    }
  } else {
    if (warp == 24) {
      tmem_alloc(s_tmem, kPreTmemCols);
      tmem_relinquish();
    }
    const uint32_t tmem = set_up();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPreRegsIssue));
    // ----------------------------------------------------------- products
    // (a descriptor's address is in units of 16 bytes in its low bits)
    if (warp == 24 && lane == 0) {
      constexpr uint32_t idesc = idesc_f16(128, 128);
      const uint64_t dq = smem_desc_k128_sw128(smem_u32(sm + PreSmem::kOffQ));
      const uint64_t dk = smem_desc_k128_sw128(smem_u32(sm + PreSmem::kOffK));
      bool ok = true;
      int last = -1, last_phase = 0;  // whose S is in tensor memory
      for (int j = 0; ok && j < tiles; ++j) {
        if (!(ok = wait(kKFull + (j & 1), j >> 1))) break;
        for (int k = 0; k < 2; ++k) {
          if (j >= nt[k]) continue;
          if (last >= 0 && !(ok = wait(kSRead + last, last_phase))) break;
          tc_fence_after();
          last = k;
          last_phase = j;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int off = ((i >> 2) * PreSmem::kBlock + (i & 3) * 32) >> 4;
            mma_f16_ss(tmem + kPreTmemS, dq + k * (PreSmem::kOperand >> 4) + off, dk + (j & 1) * (PreSmem::kOperand >> 4) + off,
                       idesc, i > 0 ? 1u : 0u);
          }
          mma_commit(bars + kSFull + k);
        }
        if (!ok) break;
        mma_commit(bars + kKFree + (j & 1));
      }
      // nothing in flight when the tensor memory goes back
      mma_commit(bars + kDrain);
      mbar_wait_limit(bars + kDrain, 0, nullptr, err, kErrKv8Wait, kWaitLimitNs);
    } else if (warp == 25 && lane == 0) {
      constexpr uint32_t idesc = idesc_f16(128, 128) | (1u << 16);  // V: N-major
      const uint64_t dv = smem_desc_mn_sw128(smem_u32(sm + PreSmem::kOffV), PreSmem::kBlock, 1024);
      bool ok = true;
      for (int j = 0; ok && j < tiles; ++j) {
        if (!(ok = wait(kVFull + (j & 1), j >> 1))) break;
        for (int k = 0; k < 2; ++k) {
          if (j >= nt[k]) continue;
          if (!(ok = wait(kPFull + k, j))) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            mma_f16_ts(tmem + kPreTmemO + 128 * k, tmem + kPreTmemP + 64 * k + 8 * i,
                       dv + (j & 1) * (PreSmem::kOperand >> 4) + i * (2048 >> 4), idesc, (j > 0 || i > 0) ? 1u : 0u);
          mma_commit(bars + kPFree + k);
        }
        if (!ok) break;
        mma_commit(bars + kVFree + (j & 1));
        bar_arrive(bar0 + 8 * (kScaleFree + (j & 3)));  // both blocks' weights are made
      }
      mma_commit(bars + kDrain + 1);
      mbar_wait_limit(bars + kDrain + 1, 0, nullptr, err, kErrKv8Wait, kWaitLimitNs);
    }
    if (warp == 26) {
      // the scales of a tile's passes of 16 tokens (lane i < 8: of pass i)
      const int32_t* table = a.c.table + static_cast<int64_t>(b) * a.c.max_blocks;
      for (int j = 0; j < tiles; ++j) {
        const int tok = (tile0 + j) * kPreTile + 16 * (lane & 7);
        float sk = 0.0f, sv = 1.0f;
        if (tok < sq.len) {
          const int page = min(max(__ldg(table + tok / P), 0), a.c.num_pages - 1);  // (reported where the codes are read)
          const float* s = a.c.scales + static_cast<int64_t>(page) * 2 * a.c.Hkv + kvh;
          sk = __ldg(s);
          sv = __ldg(s + a.c.Hkv);
        }
        // (K's not 0: a place that a row does not see is -inf times it; V's so
        // that smaller scales give values below 2^-50, larger ones are beyond fp16)
        float4 sc;
        sc.x = fmaxf(sk * fabsf(a.scale) * 1.4426950408889634f, 1e-30f);
        sc.y = __log2f(fminf(fmaxf(sv, 8.673617e-19f), 1.1529215e18f));
        sc.z = ex2(-sc.y);
        sc.w = 0.0f;
        if (j >= 4 && !wait_warp_relaxed(kScaleFree + (j & 3), (j >> 2) - 1)) break;
        if (lane < 8) s_scale[(j & 3) * 8 + lane] = sc;
        __syncwarp();
        if (lane == 0) bar_arrive(bar0 + 8 * (kScale + (j & 3)));
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 24) {
    tc_fence_after();
    tmem_dealloc(*s_tmem, kPreTmemCols);
  }
}

// Joins the parts of cut pieces: a warp for each (row of the batch, query
// head), lane l dimensions 4 l .. 4 l + 3, in the order of the parts.
constexpr int kPreJoinWarps = 8;
__global__ void __launch_bounds__(kPreJoinWarps * 32) kv8_prefill_join_kernel(const __grid_constant__ Kv8PrefillArgs args) {
  const Kv8AttnArgs& a = args.a;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, G = a.Hq / a.c.Hkv;
  const int64_t x = static_cast<int64_t>(blockIdx.x) * kPreJoinWarps + (threadIdx.x >> 5);
  if (x >= static_cast<int64_t>(a.s.T) * a.Hq) return;
  const int batch_row = static_cast<int>(x / a.Hq), h = static_cast<int>(x % a.Hq);
  const int b = kv8_find(a.s, batch_row, 1, 1, 0);
  if (b < 0) return;
  const Kv8Seq sq = kv8_sequence(a.s, b, static_cast<int64_t>(a.c.max_blocks) * a.c.P, nullptr);
  const int n = kv8_row_start(a.s, b + 1) - sq.first, ti = batch_row - sq.first;
  if (ti >= n || sq.n < 0 || n * G <= args.few_rows) return;
  const int kvh = h / G, row = ti * G + h % G, piece_row0 = row / (2 * kPreRows) * (2 * kPreRows);
  const int slot = static_cast<int>(static_cast<int64_t>(sq.first) * G / (2 * kPreRows)) + b + piece_row0 / (2 * kPreRows);
  const int last = min(piece_row0 + 2 * kPreRows, n * G) - 1;  // the piece's last row
  const int tiles = (sq.pos0 + last / G + kPreTile) / kPreTile, chunk = pre_chunk(tiles, args.splits);
  if (chunk >= tiles) return;  // not cut
  const int limit = sq.pos0 + ti + 1;
  if (!in_bounds(slot >= 0 && slot < args.slots && (limit - 1) / (chunk * kPreTile) < args.splits, a.err)) return;
  const int64_t row0 = (static_cast<int64_t>(slot) * a.c.Hkv + kvh) * args.splits * (2 * kPreRows) + row - piece_row0;
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int s = 0; s * chunk * kPreTile < limit; ++s) {  // parts of which the row sees something
    const int64_t at = row0 + static_cast<int64_t>(s) * (2 * kPreRows);
    const float2 ml = *reinterpret_cast<const float2*>(args.part_ml + 2 * at);
    const float4 v = reinterpret_cast<const float4*>(args.part + at * kKv8D)[lane];
    const float mn = fmaxf(m, ml.x);
    const float f = m == -INFINITY ? 0.0f : ex2(m - mn), f2 = ml.x == -INFINITY ? 0.0f : ex2(ml.x - mn);
    m = mn;
    l = l * f + ml.y * f2;
    o.x = o.x * f + v.x * f2;
    o.y = o.y * f + v.y * f2;
    o.z = o.z * f + v.z * f2;
    o.w = o.w * f + v.w * f2;
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  const __half2 y0 = __floats2half2_rn(o.x * inv, o.y * inv), y1 = __floats2half2_rn(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(a.out + x * kKv8D + 4 * lane) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
}

}  // namespace w4a8
