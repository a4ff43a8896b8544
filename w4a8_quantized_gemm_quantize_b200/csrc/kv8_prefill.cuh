// Causal attention of many new tokens per sequence over the paged 8-bit KV
// cache, both contractions on the tensor cores (tcgen05 kind::f16).
#pragma once
#include "kv8_attention.cuh"

namespace w4a8 {

// A CTA takes 256 rows of one (sequence, kv head): row R = i G + h is query
// head h of the group at new token i, so that grouped heads share the cache's
// tiles. Two blocks of 128 rows (t = 0, 1) take turns on the tensor cores:
// while the softmax of one runs, the other's products do. Per tile of 128
// cached tokens
//   S_t = Q_t K^T        128 x 128 x 128, Q and K from shared memory
//   P_t = 2^(z - M)      thread = row, from and to tensor memory (P over S)
//   O_t += P_t V         128 x 128 x 128, P from tensor memory, V from shared
// so that the tensor cores need 2 * 2 * 512 cycles a tile and pair of blocks,
// and the exponentials (16 a cycle and SM) as many: those two bound it.
//
// Roles: warps 0-3 and 4-7 the softmax of block 0 and 1; warps 8-11 turn K's
// bytes into fp16 integers (exact), 12-15 V's, from global memory through
// registers (requested a tile ahead) into the two halves of a double buffer;
// one thread of warp 16 issues every product. The bytes do not pass through
// shared memory on their way: the products' own reads of it (1536 of 2048
// cycles a tile) leave room for little more than the converted tiles.
//
// Softmax weights carry their page's value scale, as in the decode kernel: z_j
// = x_j + log2 sV_j, w_j = 2^(z_j - M + 10), rounded once to fp16 for the
// product (relative 2^-11; at most 2^15); the denominator sums w_j / sV_j of
// the unrounded weights in fp32. The reference M only moves when the running
// maximum has passed it by 5, which spares most of the rescales of O.
constexpr int kPreRows = 128;      // rows of a block
constexpr int kPreTile = 128;      // cached tokens of a tile
constexpr int kPreThreads = 17 * 32;
constexpr float kPreShift = 10.0f, kPreSlack = 5.0f;

struct PreSmem {
  static constexpr int kBlock = 128 * 128;     // 64 columns (128 bytes) of a 128-row operand
  static constexpr int kOperand = 2 * kBlock;  // 128 x 128 fp16
  static constexpr int kOffQ = 0;              // [2]
  static constexpr int kOffK = 2 * kOperand;   // [2]
  static constexpr int kOffV = 4 * kOperand;   // [2]
  static constexpr int kOffScale = 6 * kOperand;         // [4][8] (sK', log2 sV, 1 / sV, -)
  static constexpr int kOffBars = kOffScale + 4 * 8 * 16;
  static constexpr int kBars = 20;
  static constexpr int kOffMisc = kOffBars + kBars * 8;  // TMEM address, abort flag
  static constexpr int kBytes = kOffMisc + 16 + 1024;    // + alignment slack
  static_assert(kBytes <= 232448, "shared memory of one CTA");
};
enum PreBar { kKFull = 0, kKFree = 2, kVFull = 4, kVFree = 6, kSFull = 8, kPFull = 10, kODone = 12, kDrain = 14, kScale = 16 };
constexpr int kPreTmemS = 0, kPreTmemO = 256, kPreTmemCols = 512;  // block t: + 128 t

// Loads 32 consecutive columns of this thread's lane and waits for them.
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
// 16 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__global__ void __launch_bounds__(kPreThreads, 1) kv8_prefill_kernel(Kv8AttnArgs a, int slots, int few_rows) {
  extern __shared__ __align__(1024) uint8_t pre_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pre_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + PreSmem::kOffBars);
  float4* s_scale = reinterpret_cast<float4*>(sm + PreSmem::kOffScale);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + PreSmem::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const DevErr err{a.err};
  const int P = a.c.P, G = a.Hq / a.c.Hkv;

  grid_dependency_wait();
  grid_launch_dependents();
  // this CTA's rows: slot start_b G / 256 + b + k holds rows 256 k .. of
  // sequence b. Later slots see more of the cache: taken first.
  const int kvh = static_cast<int>(blockIdx.x) % a.c.Hkv;
  const int slot = slots - 1 - static_cast<int>(blockIdx.x) / a.c.Hkv;
  const int b = kv8_find(a.s, slot, G, 2 * kPreRows, 1);
  if (b < 0) return;
  const Kv8Seq sq = kv8_sequence(a.s, b, static_cast<int64_t>(a.c.max_blocks) * P, t == 0 ? a.err : nullptr);
  const int first = sq.first, n = kv8_row_start(a.s, b + 1) - first;
  const int64_t row0 = static_cast<int64_t>(slot - (static_cast<int64_t>(first) * G / (2 * kPreRows) + b)) * 2 * kPreRows;
  const int64_t rows = static_cast<int64_t>(n) * G;
  if (row0 >= rows || rows <= few_rows) return;  // (few rows: the decode kernel's)
  if (sq.n < 0) {  // a length that does not fit (reported): zeros
    const int64_t r = row0 + t;
    if (t < 2 * kPreRows && r < rows) {
      uint4* dst = reinterpret_cast<uint4*>(a.out + ((first + r / G) * a.Hq + kvh * G + r % G) * kKv8D);
      for (int i = 0; i < 16; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  // tiles that each block sees
  int nt[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t last = min(row0 + (k + 1) * kPreRows, rows) - 1;  // its last row
    nt[k] = last < row0 + k * kPreRows ? 0 : (sq.pos0 + static_cast<int>(last / G) + kPreTile) / kPreTile;
  }
  const int tiles = max(nt[0], nt[1]);

  if (t == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + kKFull + i, 4);
      mbar_init(bars + kKFree + i, 1);
      mbar_init(bars + kVFull + i, 4);
      mbar_init(bars + kVFree + i, 1);
      mbar_init(bars + kSFull + i, 1);
      mbar_init(bars + kPFull + i, 4);
      mbar_init(bars + kODone + i, 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(bars + kScale + i, 1);
    mbar_init(bars + kDrain, 1);
    fence_barrier_init();
    *s_abort = 0;
  }
  if (warp == 16) {
    tmem_alloc(s_tmem, kPreTmemCols);
    tmem_relinquish();
  }
  const auto wait = [&](int bar, int phase) {
    return mbar_wait(bars + bar, static_cast<uint32_t>(phase) & 1u, s_abort, err, kErrKv8Wait);
  };
  const auto wait_warp = [&](int bar, int phase) {  // the same answer in every lane
    return __all_sync(0xffffffffu, wait(bar, phase)) != 0;
  };

  // this softmax thread's row, and its query into shared memory
  const int blk = warp >> 2;              // block of rows (softmax warps)
  const int lr = (warp & 3) * 32 + lane;  // row of the block, TMEM lane
  const int64_t row = row0 + blk * kPreRows + lr;
  const bool mine = warp < 8 && row < rows;
  const int ti = mine ? static_cast<int>(row / G) : 0;
  const int64_t at = ((static_cast<int64_t>(first) + ti) * a.Hq + kvh * G + (mine ? row % G : 0)) * kKv8D;
  const int limit = mine ? sq.pos0 + ti + 1 : 1;
  const float qsign = a.scale < 0.0f ? -1.0f : 1.0f;
  if (warp < 8) {
    uint8_t* dst = sm + PreSmem::kOffQ + blk * PreSmem::kOperand + lr * 128;
    const uint32_t flip = qsign < 0.0f ? 0x80008000u : 0u;  // scores are taken with |scale|
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (mine) {
        v = __ldg(reinterpret_cast<const uint4*>(a.q + at) + i);
        v.x ^= flip;
        v.y ^= flip;
        v.z ^= flip;
        v.w ^= flip;
      }
      *reinterpret_cast<uint4*>(dst + (i >> 3) * PreSmem::kBlock + (((i & 7) ^ (lr & 7)) << 4)) = v;
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + kPreTmemS + 128 * blk + lane_base, tO = tmem + kPreTmemO + 128 * blk + lane_base;
    const int mine_nt = nt[blk];
    float ref = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < mine_nt; ++j) {
      // (a scale slot is written again only after this block's weights of the tile are done)
      if (!(ok = wait_warp(kSFull + blk, j) && wait_warp(kScale + (j & 3), j >> 2))) break;
      tc_fence_after();
      const float4* sc = s_scale + (j & 3) * 8;
      const int left = limit - j * kPreTile;  // columns that this row sees
      const bool cut = __any_sync(0xffffffffu, left < kPreTile);
      uint32_t r[32];
      float mx = -INFINITY;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        tmem_ld_32_wait(tS + 32 * q, r);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float top = -INFINITY;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float v = __uint_as_float(r[16 * u + e]);
            if (cut) v = 32 * q + 16 * u + e < left ? v : -INFINITY;
            top = fmaxf(top, v);
          }
          const float4 s = sc[2 * q + u];
          mx = fmaxf(mx, fmaf(top, s.x, s.y));
        }
      }
      // move the reference where the maximum has passed it
      const bool move = mx > ref + kPreSlack || (ref == -INFINITY && mx > -INFINITY);
      if (__any_sync(0xffffffffu, move)) {
        const float nr = move ? mx : ref;
        const float f = move && ref > -INFINITY ? ex2(ref - nr) : 1.0f;
        ref = nr;
        l *= f;
        if (j > 0) {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            tmem_ld_32_wait(tO + 32 * q, r);
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
            tmem_st_32(tO + 32 * q, r);
          }
        }
      }
      const float base = ref > -INFINITY ? kPreShift - ref : 0.0f;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        tmem_ld_32_wait(tS + 32 * q, r);
        uint32_t p[16];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float4 s = sc[2 * q + u];
          const float off = s.y + base;
          float sum = 0.0f;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float w0 = ex2(fmaf(__uint_as_float(r[16 * u + e]), s.x, off));
            float w1 = ex2(fmaf(__uint_as_float(r[16 * u + e + 1]), s.x, off));
            if (cut) {
              w0 = 32 * q + 16 * u + e < left ? w0 : 0.0f;
              w1 = 32 * q + 16 * u + e + 1 < left ? w1 : 0.0f;
            }
            sum += w0 + w1;
            const __half2 h = __floats2half2_rn(w0, w1);
            p[8 * u + e / 2] = *reinterpret_cast<const uint32_t*>(&h);
          }
          l = fmaf(sum, s.z, l);
        }
        tmem_st_16(tS + 16 * q, p);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + kPFull + blk);
    }
    if (ok && mine_nt > 0 && wait_warp(kODone + blk, 0)) {
      tc_fence_after();
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t r[32];
        tmem_ld_32_wait(tO + 32 * q, r);
        if (mine) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 y;
            __half2* h = reinterpret_cast<__half2*>(&y);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              h[e] = __floats2half2_rn(__uint_as_float(r[8 * i + 2 * e]) * inv,
                                       __uint_as_float(r[8 * i + 2 * e + 1]) * inv);
            reinterpret_cast<uint4*>(a.out + at + 32 * q)[i] = y;
          }
        }
      }
    }
  } else if (warp < 16) {
    // ---------------------------------------------------- bytes to operands
    const bool is_v = warp >= 12;
    const int full = is_v ? kVFull : kKFull, free = is_v ? kVFree : kKFree;
    // a pass covers 16 tokens: lanes 8 apart in pairs of rows and quarters of
    // 64 bytes, so that eight lanes' stores meet all banks
    const int ch = (lane & 3) + 4 * ((lane >> 3) & 1);
    const int r0 = (warp & 3) * 4 + ((lane >> 2) & 1) + 2 * (lane >> 4);  // row within a pass
    const int32_t* table = a.c.table + static_cast<int64_t>(b) * a.c.max_blocks;
    const auto page_of = [&](int j) {  // lane i < 8: the page of pass i of tile j
      const int tok = j * kPreTile + 16 * (lane & 7);
      int page = tok < sq.len ? __ldg(table + tok / P) : -1;
      if (tok < sq.len && (page < 0 || page >= a.c.num_pages)) {
        atomicCAS(a.err, 0, kErrKv8Range);
        page = 0;
      }
      return page;
    };
    const int64_t head = static_cast<int64_t>(kvh + (is_v ? a.c.Hkv : 0));
    uint4 raw[8];
    const auto load = [&](int j, int pages) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int page = __shfl_sync(0xffffffffu, pages, i);
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (page >= 0) {  // places behind the sequence's end inside its last page: any bytes, weight 0
          const int64_t place = (static_cast<int64_t>(page) * 2 * a.c.Hkv + head) * P + ((j * kPreTile + 16 * i) & (P - 1)) + r0;
          raw[i] = __ldg(reinterpret_cast<const uint4*>(a.c.codes + place * kKv8D) + ch);
        }
      }
    };
    int pages = page_of(0);
    load(0, pages);
    for (int j = 0; j < tiles; ++j) {
      const int next = j + 1 < tiles ? page_of(j + 1) : -1;
      float4 sc = make_float4(0.0f, 0.0f, 1.0f, 0.0f);
      if (warp == 8 && lane < 8 && pages >= 0) {  // the tile's scales
        const float* s = a.c.scales + static_cast<int64_t>(pages) * 2 * a.c.Hkv + kvh;
        const float sv = fminf(fmaxf(__ldg(s + a.c.Hkv), 8.673617e-19f), 1.1529215e18f);
        sc.x = __ldg(s) * fabsf(a.scale) * 1.4426950408889634f;
        sc.y = __log2f(sv);
        sc.z = ex2(-sc.y);
      }
      if (j >= 2 && !wait_warp(free + (j & 1), (j >> 1) - 1)) break;
      if (warp == 8) {
        if (lane < 8) s_scale[(j & 3) * 8 + lane] = sc;
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kScale + (j & 3));
      }
      uint8_t* op = sm + (is_v ? PreSmem::kOffV : PreSmem::kOffK) + (j & 1) * PreSmem::kOperand;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = 16 * i + r0;
        const uint32_t w[4] = {raw[i].x ^ 0x80808080u, raw[i].y ^ 0x80808080u, raw[i].z ^ 0x80808080u,
                               raw[i].w ^ 0x80808080u};
        uint8_t* dst = op + (ch >> 2) * PreSmem::kBlock + row * 128;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<uint4*>(dst + (((2 * (ch & 3) + k) ^ (row & 7)) << 4)) =
              make_uint4(unbias_pair<0x4140>(w[2 * k]), unbias_pair<0x4342>(w[2 * k]),
                         unbias_pair<0x4140>(w[2 * k + 1]), unbias_pair<0x4342>(w[2 * k + 1]));
      }
      if (j + 1 < tiles) load(j + 1, next);
      pages = next;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + full + (j & 1));
    }
  } else {
    if (lane == 0) {
    // ----------------------------------------------------------- products
    constexpr uint32_t idesc_s = idesc_f16(128, 128), idesc_o = idesc_f16(128, 128) | (1u << 16);  // V: N-major
    const auto scores = [&](int k, int j) {
      const uint32_t q = smem_u32(sm + PreSmem::kOffQ + k * PreSmem::kOperand);
      const uint32_t kk = smem_u32(sm + PreSmem::kOffK + (j & 1) * PreSmem::kOperand);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t off = (i >> 2) * PreSmem::kBlock + (i & 3) * 32;
        mma_f16_ss(tmem + kPreTmemS + 128 * k, smem_desc_k128_sw128(q + off), smem_desc_k128_sw128(kk + off), idesc_s,
                   i > 0 ? 1u : 0u);
      }
      mma_commit(bars + kSFull + k);
    };
    const auto values = [&](int k, int j) {
      const uint32_t v = smem_u32(sm + PreSmem::kOffV + (j & 1) * PreSmem::kOperand);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        mma_f16_ts(tmem + kPreTmemO + 128 * k, tmem + kPreTmemS + 128 * k + 8 * i,
                   smem_desc_mn_sw128(v + i * 2048, PreSmem::kBlock, 1024), idesc_o, (j > 0 || i > 0) ? 1u : 0u);
    };
    bool ok = wait(kKFull, 0);
    tc_fence_after();
    if (ok) {
      for (int k = 0; k < 2; ++k)
        if (nt[k] > 0) scores(k, 0);
      mma_commit(bars + kKFree);
    }
    for (int j = 0; ok && j < tiles; ++j) {
      const bool more = j + 1 < tiles;
      ok = wait(kVFull + (j & 1), j >> 1);
      for (int k = 0; ok && k < 2; ++k) {
        if (j >= nt[k]) continue;
        ok = wait(kPFull + k, j);
        if (!ok) break;
        tc_fence_after();
        values(k, j);
        if (j + 1 == nt[k]) {
          mma_commit(bars + kODone + k);
        } else {
          ok = wait(kKFull + ((j + 1) & 1), (j + 1) >> 1);
          if (!ok) break;
          tc_fence_after();
          scores(k, j + 1);
        }
      }
      if (!ok) break;
      mma_commit(bars + kVFree + (j & 1));
      if (more) mma_commit(bars + kKFree + ((j + 1) & 1));
    }
    // nothing in flight when the tensor memory goes back
    mma_commit(bars + kDrain);
    mbar_wait_limit(bars + kDrain, 0, nullptr, err, kErrKv8Wait, kWaitLimitNs);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, kPreTmemCols);
  }
}

}  // namespace w4a8
