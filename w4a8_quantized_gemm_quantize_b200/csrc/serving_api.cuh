// C ABI of the serving operators around the GEMMs: the norm that quantizes,
// and the paged 8-bit KV cache with its append and attention. Declarations
// and contracts in include/w4a8.h; the helpers are w4a8_api.cu's.
#pragma once
#include "kv8_prefill.cuh"
#include "rmsnorm_quantize.cuh"

namespace w4a8 {
namespace {

constexpr int64_t kKv8MaxLen = int64_t(1) << 24;

// Whether [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < static_cast<uintptr_t>(na) : x - y < static_cast<uintptr_t>(nb);
}

template <int THREADS, int VPT>
w4a8_status_t launch_rmsnorm(const __half* X, const __half* R, const __half* W, float eps, int64_t M, int64_t K,
                             __half* H, int8_t* A8, __half* sA, int32_t* rowsum, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(M));
  const int early = M <= kEarlyReleaseRows ? 1 : 0;
  if (R != nullptr)
    return launch_pdl(rmsnorm_quantize_kernel<THREADS, VPT, true>, grid, dim3(THREADS), 0, st, 1, X, R, W, eps, K, H,
                      A8, sA, rowsum, early);
  return launch_pdl(rmsnorm_quantize_kernel<THREADS, VPT, false>, grid, dim3(THREADS), 0, st, 1, X, R, W, eps, K, H,
                    A8, sA, rowsum, early);
}

// Checks of a cache descriptor and of the batch's sizes (each factor bounded
// before the products are formed).
w4a8_status_t check_kv8(const w4a8_kv8_cache_t* c, int64_t B, int64_t T, int64_t Hq) {
  if (c == nullptr) return W4A8_ERR_INVALID_ARG;
  if (c->reserved != 0 || B < 0 || T < 0 || Hq < 0 || c->num_pages < 0 || c->max_blocks < 0 || c->Hkv < 0)
    return W4A8_ERR_INVALID_ARG;
  if (c->D != kKv8D || !(c->page == 16 || c->page == 32 || c->page == 64 || c->page == 128))
    return W4A8_ERR_UNSUPPORTED_SHAPE;
  if (c->Hkv == 0 || Hq == 0 || Hq > 1024 || Hq % c->Hkv != 0 || B > 65535 || T > INT32_MAX / 1024)
    return W4A8_ERR_UNSUPPORTED_SHAPE;
  if (c->num_pages == 0 || c->num_pages > INT32_MAX || c->num_pages * 2 * c->Hkv > INT32_MAX / c->page ||
      c->max_blocks == 0 || c->max_blocks > kKv8MaxLen || c->max_blocks * c->page > kKv8MaxLen)
    return W4A8_ERR_UNSUPPORTED_SHAPE;
  return W4A8_OK;
}

w4a8_status_t check_kv8_pointers(const w4a8_kv8_cache_t* c, const int32_t* seq_lens, const int32_t* q_start) {
  if (c->codes == nullptr || c->scales == nullptr || c->block_table == nullptr || seq_lens == nullptr)
    return W4A8_ERR_INVALID_ARG;
  if (!aligned(c->codes, 128) || !aligned(c->scales, 4) || !aligned(c->block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(q_start, 4))
    return W4A8_ERR_MISALIGNED;
  return W4A8_OK;
}

Kv8Cache kv8_cache_args(const w4a8_kv8_cache_t* c) {
  return {c->codes, c->scales, c->block_table, static_cast<int>(c->num_pages), static_cast<int>(c->max_blocks),
          c->Hkv, c->page};
}

template <Kv8Layout L>
w4a8_status_t launch_kv8_append(int page, dim3 grid, cudaStream_t st, const Kv8AppendArgs& a) {
  const dim3 block(static_cast<unsigned>(kv8_append_threads(page)));
  switch (page) {
    case 0: return launch_pdl(kv8_append_kernel<0, L>, grid, block, 0, st, 1, a);
    case 16: return launch_pdl(kv8_append_kernel<16, L>, grid, block, 0, st, 1, a);
    case 32: return launch_pdl(kv8_append_kernel<32, L>, grid, block, 0, st, 1, a);
    case 64: return launch_pdl(kv8_append_kernel<64, L>, grid, block, 0, st, 1, a);
    default: return launch_pdl(kv8_append_kernel<128, L>, grid, block, 0, st, 1, a);
  }
}

// The cache's codes as rows of 128 bytes, loaded in boxes of a decode tile's
// rows (a page's, where that is smaller) with the 128-byte swizzle.
w4a8_status_t kv8_map(const w4a8_kv8_cache_t* c, int box_rows, CUtensorMap* map) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kKv8D),
                              static_cast<cuuint64_t>(c->num_pages) * 2 * c->Hkv * c->page};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kKv8D)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kKv8D),
                             static_cast<cuuint32_t>(c->page < box_rows ? c->page : box_rows)};
  const cuuint32_t estr[2] = {1u, 1u};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, c->codes, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? W4A8_OK
             : W4A8_ERR_CUDA;
}

template <bool DUP>
w4a8_status_t launch_kv8_decode(const CUtensorMap& map, const Kv8DecodeArgs& d, int grid, cudaStream_t stream) {
  static bool done[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return launch_status();
  if (!done[dev]) {
    if (cudaFuncSetAttribute(kv8_decode_kernel<DUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             DecCfg<DUP>::kBytes) !=
        cudaSuccess)
      return launch_status();
    done[dev] = true;
  }
  return launch_pdl(kv8_decode_kernel<DUP>, dim3(static_cast<unsigned>(grid)), dim3(DecCfg<DUP>::kWarps * 32),
                    DecCfg<DUP>::kBytes, stream, 1, map, d);
}

// Sequences whose rows (new tokens times query heads per kv head) are at most
// this many go to the decode kernel, which reads the cache once for 8 rows,
// others to the prefill kernel, which reads it once for 256. Measured, 8 kv
// heads (decode against prefill kernel): 1 sequence of 32 rows over 1000, 4000,
// 32000 tokens 14, 24, 67 us against 23, 26, 55; of 64 rows 19, 29, 114 against
// 24, 26, 56; 4 sequences of 32 rows over 1000, 4000 tokens 22, 43 against 25,
// 37. Each sequence by its own rows, whatever the batch's. With batches of up to
// 160 rows given to the decode kernel whole, 156 rows over 1000, 8000, 32000
// tokens beside one of 4 over 500 took 24, 78, 262 us, now 40, 53, 110; 8
// sequences of 20 rows over 1500, for which the other kernel has nothing to do, 29,
// now 35.
constexpr int kKv8FewRows = 32;

w4a8_status_t kv8_decode(const Kv8AttnArgs& a, DeviceInfo* dev, const w4a8_kv8_cache_t* c, void* workspace,
                         cudaStream_t stream) {
  CUtensorMap map;
  const w4a8_status_t st = kv8_map(c, kDecTile, &map);
  if (st != W4A8_OK) return st;
  const int G = a.Hq / a.c.Hkv;
  Kv8DecodeArgs d;
  d.a = a;
  d.count = static_cast<int*>(workspace);
  d.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kDecMaxCtas * 4);
  d.max_rows = a.s.q_start == nullptr ? G : kKv8FewRows;
  // one CTA per SM, no more than the longest possible batch has tiles for
  const int64_t tiles = (c->max_blocks * c->page + kDecTile - 1) / kDecTile * a.s.B * a.c.Hkv *
                        ((d.max_rows + kDecCols - 1) / kDecCols);
  int64_t grid = tiles < dev->sms ? tiles : dev->sms;
  if (grid > kDecMaxCtas) grid = kDecMaxCtas;
  if (d.max_rows <= 4) return launch_kv8_decode<true>(map, d, static_cast<int>(grid), stream);
  return launch_kv8_decode<false>(map, d, static_cast<int>(grid), stream);
}

// Pieces of 256 rows of the prefill kernel (sequence b's begin at slot start_b G
// / 256 + b), and into how many parts each is cut: as many as fill a B200's 148
// SMs where the pieces fill half of them at most (a number that the size of a
// workspace follows from, which is asked for without a device).
int64_t kv8_pre_slots(int64_t B, int64_t T, int64_t G) { return T * G / (2 * kPreRows) + B; }
int kv8_pre_splits(int64_t slots, int64_t Hkv) {
  const int64_t n = 148 / (slots * Hkv);
  return static_cast<int>(n < 2 ? 1 : n > 32 ? 32 : n);
}
size_t kv8_part_bytes(int64_t parts) { return static_cast<size_t>(parts) * (2 * kPreRows) * (kKv8D + 2) * 4; }
// What the parts of a call take, and the most that those of any call of at most B
// sequences and T rows do (fewer pieces are cut into more parts).
size_t kv8_pre_part_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hkv) {
  if (T * (Hq / Hkv) <= kKv8FewRows) return 0;
  const int64_t slots = kv8_pre_slots(B, T, Hq / Hkv);
  const int splits = kv8_pre_splits(slots, Hkv);
  return splits > 1 ? kv8_part_bytes(slots * Hkv * splits) : 0;
}
size_t kv8_most_part_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hkv) {
  if (T * (Hq / Hkv) <= kKv8FewRows) return 0;
  const int64_t slots = kv8_pre_slots(B, T, Hq / Hkv);
  int64_t most = 0;
  for (int64_t n = 1; n <= slots; ++n) {  // (148 / 2 at most)
    const int splits = kv8_pre_splits(n, Hkv);
    if (splits == 1) break;
    most = n * Hkv * splits > most ? n * Hkv * splits : most;
  }
  return kv8_part_bytes(most);
}
constexpr size_t kDecWorkspace = kDecMaxCtas * (4 + 2 * kDecPart * sizeof(float));
static_assert(kDecMaxCtas * 4 == W4A8_KV8_COUNTER_BYTES, "the counters come first");
static_assert(kDecWorkspace % 256 == 0, "the prefill parts follow, aligned");

template <bool CUT>
w4a8_status_t launch_kv8_prefill(const Kv8PrefillArgs& p, cudaStream_t stream) {
  static bool done[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return launch_status();
  if (!done[dev]) {
    if (cudaFuncSetAttribute(kv8_prefill_kernel<CUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, PreSmem::kBytes) !=
        cudaSuccess)
      return launch_status();
    done[dev] = true;
  }
  return launch_pdl(kv8_prefill_kernel<CUT>, dim3(static_cast<unsigned>(p.slots * p.a.c.Hkv * p.splits)),
                    dim3(kPreThreads), PreSmem::kBytes, stream, 1, p);
}

w4a8_status_t kv8_prefill(const Kv8AttnArgs& a, int few_rows, void* workspace, cudaStream_t stream) {
  const int64_t slots = kv8_pre_slots(a.s.B, a.s.T, a.Hq / a.c.Hkv);
  if (slots * a.c.Hkv > INT32_MAX) return W4A8_ERR_UNSUPPORTED_SHAPE;
  Kv8PrefillArgs p;
  p.a = a;
  p.slots = static_cast<int>(slots);
  p.few_rows = few_rows;
  p.splits = kv8_pre_splits(slots, a.c.Hkv);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kDecWorkspace);
  p.part_ml = p.part + slots * a.c.Hkv * p.splits * (2 * kPreRows) * kKv8D;
  if (p.splits == 1) return launch_kv8_prefill<false>(p, stream);
  const w4a8_status_t st = launch_kv8_prefill<true>(p, stream);
  if (st != W4A8_OK) return st;
  const int64_t join = (static_cast<int64_t>(a.s.T) * a.Hq + kPreJoinWarps - 1) / kPreJoinWarps;
  return launch_pdl(kv8_prefill_join_kernel, dim3(static_cast<unsigned>(join)), dim3(kPreJoinWarps * 32), 0, stream, 1,
                    p);
}

w4a8_status_t kv8_attention(const void* q, const w4a8_kv8_cache_t* c, const int32_t* seq_lens, const int32_t* q_start,
                            int64_t B, int64_t T, int64_t Hq, float scale, void* out, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream) {
  w4a8_status_t st = check_kv8(c, B, T, Hq);
  if (st != W4A8_OK || B == 0 || T == 0) return st;
  st = check_kv8_pointers(c, seq_lens, q_start);
  if (st != W4A8_OK) return st;
  if (q == nullptr || out == nullptr) return W4A8_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256)) return W4A8_ERR_MISALIGNED;
  if (out != q && overlap(out, T * Hq * 2 * kKv8D, q, T * Hq * 2 * kKv8D)) return W4A8_ERR_INVALID_ARG;
  const size_t parts = q_start == nullptr ? 0 : kv8_pre_part_bytes(B, T, Hq, c->Hkv);
  if (workspace == nullptr || workspace_bytes < kDecWorkspace + parts) return W4A8_ERR_WORKSPACE;
  DeviceInfo* dev = nullptr;
  st = device_info(&dev);
  if (st != W4A8_OK) return st;
  Kv8AttnArgs a;
  a.q = static_cast<const __half*>(q);
  a.c = kv8_cache_args(c);
  a.s = {seq_lens, q_start, static_cast<int>(B), static_cast<int>(T)};
  a.out = static_cast<__half*>(out);
  a.Hq = static_cast<int>(Hq);
  a.scale = scale;
  a.err = dev->err;
  if (q_start == nullptr) return kv8_decode(a, dev, c, workspace, stream);
  // each kernel takes the sequences that suit it; one whose share must be
  // empty is not launched
  const int64_t rows = T * (Hq / c->Hkv);
  if (rows <= kKv8FewRows) return kv8_decode(a, dev, c, workspace, stream);
  if (B == 1) return kv8_prefill(a, 0, workspace, stream);
  st = kv8_decode(a, dev, c, workspace, stream);
  return st != W4A8_OK ? st : kv8_prefill(a, kKv8FewRows, workspace, stream);
}

}  // namespace
}  // namespace w4a8

extern "C" {

w4a8_status_t w4a8_rmsnorm_quantize_act(const void* X, const void* residual, const void* weight, float eps, int64_t M,
                                        int64_t K, void* H, int8_t* A8, void* sA, int32_t* rowsum,
                                        w4a8_stream_t stream) {
  const w4a8_status_t st = check_quantize_args(X, M, K, A8, sA, rowsum);
  if (st != W4A8_OK || M == 0) return st;
  if (weight == nullptr || (residual == nullptr) != (H == nullptr) || !(eps >= 0.0f)) return W4A8_ERR_INVALID_ARG;
  if (!aligned(weight, 16) || !aligned(residual, 16) || !aligned(H, 16)) return W4A8_ERR_MISALIGNED;
  if (H != nullptr && ((H != X && overlap(H, 2 * M * K, X, 2 * M * K)) ||
                       (H != residual && overlap(H, 2 * M * K, residual, 2 * M * K))))
    return W4A8_ERR_INVALID_ARG;
  const __half* x = static_cast<const __half*>(X);
  const __half* r = static_cast<const __half*>(residual);
  const __half* w = static_cast<const __half*>(weight);
  __half* h = static_cast<__half*>(H);
  __half* s = static_cast<__half*>(sA);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const int64_t nvec = K / 8;
  if (nvec <= 128) return launch_rmsnorm<128, 1>(x, r, w, eps, M, K, h, A8, s, rowsum, cs);
  if (nvec <= 256) return launch_rmsnorm<256, 1>(x, r, w, eps, M, K, h, A8, s, rowsum, cs);
  if (nvec <= 512) return launch_rmsnorm<256, 2>(x, r, w, eps, M, K, h, A8, s, rowsum, cs);
  if (nvec <= 1024) return launch_rmsnorm<256, 4>(x, r, w, eps, M, K, h, A8, s, rowsum, cs);
  if (nvec <= 2048) return launch_rmsnorm<256, 8>(x, r, w, eps, M, K, h, A8, s, rowsum, cs);
  if (nvec <= 4096) return launch_rmsnorm<1024, 4>(x, r, w, eps, M, K, h, A8, s, rowsum, cs);
  return launch_rmsnorm<1024, 8>(x, r, w, eps, M, K, h, A8, s, rowsum, cs);
}

w4a8_status_t w4a8_kv8_rope_append(const void* qkv, const w4a8_kv8_cache_t* cache, const int32_t* seq_lens,
                                   const int32_t* q_start, int64_t B, int64_t T, int64_t Hq, const float* inv_freq,
                                   int32_t rotary_dim, int32_t interleaved, float rope_scale, void* q_out,
                                   w4a8_stream_t stream) {
  w4a8_status_t st = check_kv8(cache, B, T, Hq);
  if (st != W4A8_OK) return st;
  if (interleaved != 0 && interleaved != 1) return W4A8_ERR_INVALID_ARG;
  if (rotary_dim < 0 || rotary_dim > kKv8D || rotary_dim % 2 != 0) return W4A8_ERR_UNSUPPORTED_SHAPE;
  if (B == 0 || T == 0) return W4A8_OK;
  if (q_start == nullptr && B != T) return W4A8_ERR_INVALID_ARG;
  st = check_kv8_pointers(cache, seq_lens, q_start);
  if (st != W4A8_OK) return st;
  if (qkv == nullptr || q_out == nullptr || (rotary_dim > 0 && inv_freq == nullptr)) return W4A8_ERR_INVALID_ARG;
  if (!aligned(qkv, 16) || !aligned(q_out, 16) || !aligned(inv_freq, 4)) return W4A8_ERR_MISALIGNED;
  if (overlap(q_out, T * Hq * 2 * kKv8D, qkv, T * (Hq + 2 * cache->Hkv) * 2 * kKv8D)) return W4A8_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  st = device_info(&dev);
  if (st != W4A8_OK) return st;
  Kv8AppendArgs a;
  a.qkv = static_cast<const __half*>(qkv);
  a.c = kv8_cache_args(cache);
  a.s = {seq_lens, q_start, static_cast<int>(B), static_cast<int>(T)};
  a.inv_freq = inv_freq;
  a.q_out = static_cast<__half*>(q_out);
  a.Hq = static_cast<int>(Hq);
  a.rotary = rotary_dim;
  a.rope_scale = rope_scale;
  a.err = dev->err;
  a.q_rows = T > 8 * dev->sms ? 4 : 1;
  a.q_blocks = static_cast<int>((T + a.q_rows - 1) / a.q_rows);
  const int64_t items = q_start == nullptr ? B : T / cache->page + 2 * B;
  const int64_t grid = a.q_blocks + items * 2 * cache->Hkv;
  if (grid > INT32_MAX) return W4A8_ERR_UNSUPPORTED_SHAPE;
  const dim3 g(static_cast<unsigned>(grid));
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const int page = q_start == nullptr ? 0 : cache->page;
  if (interleaved) return launch_kv8_append<kPairs>(page, g, cs, a);
  if (rotary_dim % 8 == 0) return launch_kv8_append<kSplit>(page, g, cs, a);
  return launch_kv8_append<kSingle>(page, g, cs, a);
}

size_t w4a8_kv8_attention_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hkv) {
  if (B <= 0 || T <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || B > 65535 || T > INT32_MAX / 1024 || Hq > 1024)
    return 0;
  return kDecWorkspace + kv8_most_part_bytes(B, T, Hq, Hkv);
}

size_t w4a8_kv8_decode_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv) {
  return w4a8_kv8_attention_workspace_bytes(B, B, Hq, Hkv) != 0 ? kDecWorkspace : 0;
}

w4a8_status_t w4a8_kv8_attention_decode(const void* q, const w4a8_kv8_cache_t* cache, const int32_t* seq_lens,
                                        int64_t B, int64_t Hq, float scale, void* out, void* workspace,
                                        size_t workspace_bytes, w4a8_stream_t stream) {
  return kv8_attention(q, cache, seq_lens, nullptr, B, B, Hq, scale, out, workspace, workspace_bytes,
                       reinterpret_cast<cudaStream_t>(stream));
}

w4a8_status_t w4a8_kv8_attention_prefill(const void* q, const w4a8_kv8_cache_t* cache, const int32_t* seq_lens,
                                         const int32_t* q_start, int64_t B, int64_t T, int64_t Hq, float scale,
                                         void* out, void* workspace, size_t workspace_bytes, w4a8_stream_t stream) {
  if (q_start == nullptr && B > 0 && T > 0) return W4A8_ERR_INVALID_ARG;
  return kv8_attention(q, cache, seq_lens, q_start, B, T, Hq, scale, out, workspace, workspace_bytes,
                       reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
