// Host side of the 8-bit-cache decoding entry points declared in include/attn.h: argument
// checks, TMA tensor maps over the code pools, the decoding launch and (with more than one
// split) the merge launch, all on the caller's stream.
#include "attn.h"

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "attn_decode8_kernel.cuh"

using namespace attn_sm100_dec8;

namespace attn_sm100_dec8 {
// Device error word of the 8-bit decoding kernel (read and cleared by attn_decode_kv8_debug_error).
__device__ int g_attn_dec8_error;
}  // namespace attn_sm100_dec8

namespace {

constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;  // 2 s per wait
constexpr int kMaxDevices = 64;
constexpr int64_t kMaxSplits = 4096;
constexpr int64_t kMaxRows = 32;  // query rows of a work item

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

struct Dec8Device {
  bool probed = false;
  bool supported = false;
  int sm_count = 0;
  int* err_word = nullptr;
};
std::mutex g_dec8_mutex;
Dec8Device g_dec8_dev[kMaxDevices];

template <int D, int NR>
bool set_smem() {
  return cudaFuncSetAttribute(attn_decode8_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Smem8<D, NR>::kAlloc) == cudaSuccess;
}

int dec8_device_setup(Dec8Device& out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_dec8_mutex);
  Dec8Device& info = g_dec8_dev[dev];
  if (!info.probed) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return ATTN_ERR_CUDA;
    info.supported = (major == 10 && minor == 0);
    info.sm_count = sms;
    if (info.supported) {
      void* addr = nullptr;
      if (cudaGetSymbolAddress(&addr, g_attn_dec8_error) != cudaSuccess) return ATTN_ERR_CUDA;
      info.err_word = static_cast<int*>(addr);
      if (!set_smem<64, 16>() || !set_smem<64, 32>() || !set_smem<128, 16>() || !set_smem<128, 32>())
        return ATTN_ERR_CUDA;
    }
    info.probed = true;
  }
  out = info;
  return info.supported ? ATTN_OK : ATTN_ERR_UNSUPPORTED;
}

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (na == 0 || nb == 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + nb && pb < pa + na;
}
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int log2_of(int64_t x) {
  int n = 0;
  while ((int64_t(1) << n) < x) ++n;
  return n;
}

// Workspace: 256 bytes of work-item counters (zero between calls), then with more than one
// split the partial log-sum-exps and the partial outputs.
constexpr size_t kSchedBytes = 256;
size_t workspace_bytes(int64_t rows, int64_t d, int64_t splits) {
  if (splits <= 1) return kSchedBytes;
  return kSchedBytes + align_up(static_cast<size_t>(rows) * splits * 4, 256) +
         static_cast<size_t>(rows) * splits * d * 4;
}

template <int D, int NR>
cudaError_t launch(const Dec8Params& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem8<D, NR>::kAlloc;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, attn_decode8_kernel<D, NR>, p);
}
template <int D>
cudaError_t launch_rows(const Dec8Params& p, int grid, cudaStream_t stream) {
  // The narrower product that holds an item's rows.
  return p.rows_chunk <= 16 ? launch<D, 16>(p, grid, stream) : launch<D, 32>(p, grid, stream);
}

}  // namespace

extern "C" size_t attn_decode_kv8_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t d,
                                                  int64_t num_splits) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Nq < 1 || (d != 64 && d != 128) || num_splits < 1 ||
      num_splits > kMaxSplits)
    return 0;
  if (B > (int64_t(1) << 30) || Hq > (int64_t(1) << 30) || Nq > (int64_t(1) << 30) || B * Hq > 0x7fffffff) return 0;
  const int64_t rows = B * Hq * Nq;
  if (rows > 0x7fffffff) return 0;
  return workspace_bytes(rows, d, num_splits);
}

extern "C" int64_t attn_decode_kv8_num_splits(int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t max_seq_len,
                                              int mask_kind, int64_t window, int64_t sinks) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1 || max_seq_len < Nq || Hq % Hkv != 0) return -1;
  if (mask_kind < ATTN_MASK_FULL || mask_kind > ATTN_MASK_SLIDING_WINDOW || sinks < 0) return -1;
  if (mask_kind == ATTN_MASK_SLIDING_WINDOW ? window < 1 : sinks != 0) return -1;
  if (B > (int64_t(1) << 30) || Hq > (int64_t(1) << 30) || Nq > (int64_t(1) << 30)) return -1;
  int sms = 148, dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) {
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && v > 0) sms = v;
  }
  const int64_t rows_total = (Hq / Hkv) * Nq;
  const int64_t chunks = (rows_total + kMaxRows - 1) / kMaxRows;
  const int64_t units = B * Hkv * chunks;
  int64_t tiles = (max_seq_len + kKeys - 1) / kKeys + 1;
  const bool windowed = mask_kind == ATTN_MASK_SLIDING_WINDOW && window < max_seq_len;
  if (windowed)
    tiles = std::min(tiles, (window + Nq - 1 + kKeys - 1) / kKeys + 1 + (std::min(sinks, max_seq_len) + kKeys - 1) / kKeys);
  // One sequence, or windows (equal lengths): one wave of items.  Sequences of several lengths: items
  // from the shared counter, about three for each CTA and of at most 48 tiles, so that the longest
  // sequence does not end alone: 441 us in one wave and 304 in three for 12 sequences of
  // 30k-60k positions (16 heads), 79 and 61 for 30 of 1k-8k (8 heads), 88 and 90 for 8 of equal
  // lengths.  Items of under 16 tiles are not made for that, of under four not at all.  (16
  // sequences of 8k-32k positions with 32 heads: 450 us at 64 tiles, 434 at 43, 442 at 32.)
  constexpr int64_t kMaxItemTiles = 48, kMinItemTiles = 16, kWaves = 3;
  const int64_t ctas = kCtasPerSm * static_cast<int64_t>(sms);
  int64_t s = ctas / units;
  if (units >= ctas || (B > 1 && !windowed))
    s = std::max(s, std::min(tiles / kMinItemTiles,
                             std::max(units < ctas ? kWaves * ctas / units : 1, (tiles + kMaxItemTiles - 1) / kMaxItemTiles)));
  return std::max<int64_t>(1, std::min<int64_t>({s, std::max<int64_t>(1, tiles / 4), kMaxSplits}));
}

extern "C" int attn_decode_kv8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                               const float* v_scale, const int32_t* block_table, const int32_t* seq_lens, void* out,
                               float* lse, void* workspace, size_t workspace_bytes_given, int64_t B, int64_t Hq,
                               int64_t Hkv, int64_t Nq, int64_t d, int64_t num_pages, int64_t page_size,
                               int64_t max_pages_per_seq, int64_t scale_block, int64_t num_splits, float scale,
                               int mask_kind, int64_t window, int64_t sinks, cudaStream_t stream,
                               const attn_fwd_options* opts) {
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !out || !lse)
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1 || Hq % Hkv != 0 || num_pages < 1 || max_pages_per_seq < 1)
    return ATTN_ERR_INVALID_ARG;
  if (num_splits < 1 || num_splits > kMaxSplits) return ATTN_ERR_INVALID_ARG;
  if (mask_kind < ATTN_MASK_FULL || mask_kind > ATTN_MASK_SLIDING_WINDOW) return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_SLIDING_WINDOW && window < 1) return ATTN_ERR_INVALID_ARG;
  if (sinks < 0 || (sinks > 0 && mask_kind != ATTN_MASK_SLIDING_WINDOW)) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256)
    return ATTN_ERR_UNSUPPORTED;
  if (scale_block < 1 || scale_block > page_size || (scale_block & (scale_block - 1)) != 0)
    return ATTN_ERR_INVALID_ARG;
  const int64_t lim = 0x7fffffff;
  if (B > (int64_t(1) << 30) || Hq > (int64_t(1) << 30) || Nq > (int64_t(1) << 30) || B * Hq > lim ||
      B * Hq * Nq > lim || num_pages > lim / Hkv || max_pages_per_seq > lim / page_size ||
      B > lim / max_pages_per_seq)
    return ATTN_ERR_INVALID_ARG;
  const int64_t rows = B * Hq * Nq;
  const int64_t rows_total = (Hq / Hkv) * Nq;
  const int64_t rows_chunk = std::min(rows_total, kMaxRows);
  const int64_t row_chunks = (rows_total + rows_chunk - 1) / rows_chunk;
  if (B * Hkv > lim / row_chunks || B * Hkv * row_chunks > lim / num_splits) return ATTN_ERR_INVALID_ARG;
  const int64_t items = B * Hkv * row_chunks * num_splits;
  const size_t ws_need = workspace_bytes(rows, d, num_splits);
  if (!workspace || workspace_bytes_given < ws_need) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(workspace, 16))
    return ATTN_ERR_MISALIGNED;

  const size_t q_bytes = static_cast<size_t>(rows) * d * 2;
  const size_t cache_bytes = static_cast<size_t>(num_pages) * Hkv * page_size * d;
  const size_t scale_bytes = static_cast<size_t>(num_pages) * Hkv * (page_size / scale_block) * 4;
  const void* ins[7] = {q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens};
  const size_t in_sz[7] = {q_bytes, cache_bytes, cache_bytes, scale_bytes, scale_bytes,
                           static_cast<size_t>(B) * max_pages_per_seq * 4, static_cast<size_t>(B) * 4};
  const void* outs[3] = {out, lse, workspace};
  const size_t out_sz[3] = {q_bytes, static_cast<size_t>(rows) * 4, ws_need};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 7; ++i)
      if (overlaps(outs[o], out_sz[o], ins[i], in_sz[i])) return ATTN_ERR_INVALID_ARG;
    for (int o2 = o + 1; o2 < 3; ++o2)
      if (overlaps(outs[o], out_sz[o], outs[o2], out_sz[o2])) return ATTN_ERR_INVALID_ARG;
  }

  Dec8Device dev;
  const int st = dec8_device_setup(dev);
  if (st != ATTN_OK) return st;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return ATTN_ERR_CUDA;

  Dec8Params p;
  std::memset(&p, 0, sizeof(p));
  const int rows_per_load = static_cast<int>(std::min<int64_t>(page_size, kKeys));
  for (int kv = 0; kv < 2; ++kv) {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page_size),
                          static_cast<cuuint64_t>(num_pages * Hkv)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page_size * d)};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(rows_per_load), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    if (enc(kv ? &p.tm_v : &p.tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(kv ? v_cache : k_cache), dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return ATTN_ERR_CUDA;
  }
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.sched = static_cast<unsigned int*>(workspace);
  if (num_splits > 1) {
    uint8_t* ws = static_cast<uint8_t*>(workspace) + kSchedBytes;
    p.part_lse = reinterpret_cast<float*>(ws);
    p.part_o = reinterpret_cast<float*>(ws + align_up(static_cast<size_t>(rows) * num_splits * 4, 256));
  }
  p.err = dev.err_word;
  p.B = static_cast<int>(B);
  p.Hq = static_cast<int>(Hq);
  p.Hkv = static_cast<int>(Hkv);
  p.Nq = static_cast<int>(Nq);
  p.group = static_cast<int>(Hq / Hkv);
  p.rows_total = static_cast<int>(rows_total);
  p.rows_chunk = static_cast<int>(rows_chunk);
  p.row_chunks = static_cast<int>(row_chunks);
  p.page_size = static_cast<int>(page_size);
  p.page_shift = log2_of(page_size);
  p.rows_per_load = rows_per_load;
  p.loads_per_tile = kKeys / rows_per_load;
  p.max_pages = static_cast<int>(max_pages_per_seq);
  p.num_pages = static_cast<int>(num_pages);
  p.block_shift = log2_of(scale_block);
  p.mask_kind = mask_kind;
  p.window = static_cast<int>(std::min<int64_t>(window, int64_t(1) << 30));
  p.sinks = static_cast<int>(std::min<int64_t>(sinks, int64_t(1) << 30));
  p.num_splits = static_cast<int>(num_splits);
  p.num_items = static_cast<int>(items);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.timeout_ns = (opts && opts->wait_timeout_ns) ? opts->wait_timeout_ns : kDefaultTimeoutNs;
  p.stall = (opts && opts->inject_stall > 0) ? static_cast<unsigned>(opts->inject_stall) - 1u : 0xffffffffu;

  int grid = static_cast<int>(std::min<int64_t>(items, kCtasPerSm * dev.sm_count));
  if (opts && opts->grid_ctas > 0) grid = std::min(grid, opts->grid_ctas);
  if ((d == 64 ? launch_rows<64>(p, grid, stream) : launch_rows<128>(p, grid, stream)) != cudaSuccess)
    return ATTN_ERR_CUDA;
  if (num_splits > 1) {
    Merge8Params mp;
    mp.part_o = p.part_o;
    mp.part_lse = p.part_lse;
    mp.out = p.out;
    mp.lse = lse;
    mp.num_splits = static_cast<int>(num_splits);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows));
    // Eight warps where there are splits for them and room beside the other rows: 49.3 us instead of
    // 50.6 for 64 rows of 37 splits, 119 instead of 117 for 2048 rows of 20.
    const bool wide = num_splits > 16 && rows <= 4 * dev.sm_count;
    cfg.blockDim = dim3(wide ? 256 : 128);
    cfg.dynamicSmemBytes = static_cast<size_t>(num_splits) * sizeof(float);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = d == 64 ? (wide ? cudaLaunchKernelEx(&cfg, attn_decode8_merge_kernel<64, 8>, mp)
                                          : cudaLaunchKernelEx(&cfg, attn_decode8_merge_kernel<64, 4>, mp))
                                  : (wide ? cudaLaunchKernelEx(&cfg, attn_decode8_merge_kernel<128, 8>, mp)
                                          : cudaLaunchKernelEx(&cfg, attn_decode8_merge_kernel<128, 4>, mp));
    if (e != cudaSuccess) return ATTN_ERR_CUDA;
  }
  return ATTN_OK;
}

extern "C" int attn_decode_kv8_debug_error(cudaStream_t stream, int* device_code) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ATTN_ERR_CUDA;
  Dec8Device dev;
  const int st = dec8_device_setup(dev);
  if (st != ATTN_OK) return st;
  int code = 0;
  if (cudaMemcpy(&code, dev.err_word, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return ATTN_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpy(dev.err_word, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return ATTN_ERR_CUDA;
  if (device_code) *device_code = code;
  if (code == 0) return ATTN_OK;
  return (code & (kDErrSeqLen | kDErrPage)) ? ATTN_ERR_INVALID_ARG : ATTN_ERR_TIMEOUT;
}
