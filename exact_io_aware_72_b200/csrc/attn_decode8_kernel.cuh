// Attention decoding against a paged KV cache held in 8 bits, for sm_100a.
//
// Cached keys and values are E4M3 codes with one fp32 scale for each block of tokens and
// head: K_j = ks[block(j)] code, V_j likewise.  The step is the exact masked softmax
// attention of those values for the new tokens' bf16 queries, as in the bf16 decoding
// kernel.  It reads half the bytes per position, so the work per byte doubles and the
// design differs: the codes go to the tensor core as they are (nothing is converted to 16
// bits), and the products are laid out with keys as the M dimension.
//
// Mathematics.  With codes k_j, v_j, scales a_j, c_j, score x_j = scale log2(e) a_j (q . k_j)
// and y_j = x_j + log2 c_j,
//   out = sum_j 2^(y_j - m) v_j / sum_j 2^(y_j - m) / c_j,   lse = ln sum_j 2^x_j,
// so the value scale is folded into the weight that the P V product takes, and the running
// maximum m is that of y.
//
// * S^T = K Q^T (128 keys x NR query rows, NR in {16, 32, 64}): an SS product with the K
//   tile as A and Q as B.  bf16 q has 8 significant bits and E4M3 holds 4, so each q row,
//   scaled by a power of two to a maximum in [128, 256), is the sum of two E4M3 numbers:
//   the rounded value and the rest, which fits 4 bits exactly (elements below 2^-10 of the
//   row's largest keep an absolute error of 2^-18 of it).  Both terms accumulate into S.
// * A softmax thread owns one key (TMEM lane) and its NR scores, so its scales and mask are
//   scalars, and no thread computes an exponential that no row needs.
// * O^T = V^T P^T (d x NR): A is the V tile read MN-major, B is P written to shared memory by
//   the softmax threads, 16 rows (16 bytes) per key.  E4M3 V needs an 8-bit P: the weight is
//   held as a sum of three E5M2 numbers (3 significant bits each, 9 together: off by at most
//   2^-9, half of a bf16 weight's rounding), three products into one accumulator.  Weights are
//   scaled so that m sits at 2^9: they reach 2^15 before m must move (E5M2 ends at 57344),
//   and a weight is lost only below 2^-26 of the largest.
// * Sums l and all statistics are fp32; out is rounded once to bf16.
//
// Work items, splits and the item counter are the bf16 decoding kernel's.  Two softmax
// warpgroups take the tiles of an item in turn, each with its own m, l and O, merged at the
// item's end.  m is per row and warpgroup: a vote over the warpgroup (one hardware barrier
// with a reduction) finds the rare tiles where some row's maximum grew by more than 2^6.
//
// The splits of one (sequence, KV head, row chunk) count themselves in the workspace as they
// finish, and the CTA that finishes the last one merges their partial results, in the order
// of the splits (a merge launch of its own took 9 us behind a 70 us step).
//
// Warps: 0-3 and 4-7 softmax, 8 loads K (and fetches items), 9 loads V, 10 issues the P V
// products, 11 prepares Q and issues the S products up to four tiles ahead.  (One issuing
// warp spent 1500 cycles per tile on waits and issue latencies of both products, whose
// execution takes 340; HBM delivers a tile per 1400.)  TMEM: four S buffers, then the two
// O.  All mbarrier waits are bounded; the warpgroup barriers are reached by every warp
// whether or not a wait gave up, and carry that news, so the roles leave together.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cmath>
#include <cstdint>

#include "attn_decode_kernel.cuh"
#include "sm100_ptx.cuh"

namespace attn_sm100_dec8 {
using namespace attn_sm100;
using attn_sm100_dec::DecWaiter;
using attn_sm100_dec::dec_exp2;
using attn_sm100_dec::kDErrPage;
using attn_sm100_dec::kDErrSeqLen;
using attn_sm100_dec::kDMaskCausal;
using attn_sm100_dec::kDMaskFull;
using attn_sm100_dec::kDMaskWindow;
using attn_sm100_dec::kDRoleLoader;
using attn_sm100_dec::kDRoleMma;
using attn_sm100_dec::kDRoleSoftmax;
constexpr int kDRoleS = 4;

constexpr int kKeys = 128;  // keys per tile
constexpr int kThreads = 384;
constexpr int kWg = 128;    // threads of a softmax warpgroup
constexpr int kKWarp = 8, kVWarp = 9, kPvWarp = 10, kSWarp = 11;
constexpr int kItemSlots = 4;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTop = 9.f;      // weights at the running maximum are 2^kTop
constexpr float kGrow = 6.f;     // the running maximum moves when a row's grows by more
constexpr float kNoMax = -1e30f; // running maximum of a row that has seen no key
constexpr float kScaleMin = 9.094947017729282e-13f, kScaleMax = 1099511627776.f;  // 2^-40, 2^40

struct Dec8Params {
  CUtensorMap tm_k;        // [num_pages * Hkv][page_size][d] codes, box d x rows_per_load
  CUtensorMap tm_v;
  const __nv_bfloat16* q;  // [B * Hq * Nq, d]
  const float* k_scale;    // [num_pages, Hkv, page_size / block]
  const float* v_scale;
  const int* block_table;  // [B, max_pages]
  const int* seq_lens;     // [B]
  __nv_bfloat16* out;      // [B * Hq * Nq, d]
  float* lse;              // [B * Hq * Nq]
  float* part_o;           // [B * Hq * Nq, num_splits, d] (num_splits > 1)
  float* part_lse;         // [B * Hq * Nq, num_splits], base-2 units
  int* err;
  int B, Hq, Hkv, Nq, group;
  int rows_total, rows_chunk, row_chunks;
  int page_size, page_shift, rows_per_load, loads_per_tile, max_pages, num_pages;
  int block_shift, blocks_per_page;
  int mask_kind, window, sinks;
  int num_splits, num_items;
  float scale_log2;
  unsigned long long timeout_ns;
  unsigned int* sched;     // [0] next work item, [1] CTAs finished; zero between launches
  unsigned int* done;      // splits finished, per (b, KV head, row chunk); zero between launches (null: no merge here)
};

template <int D, int NR>
struct Smem8 {
  static_assert(D == 64 || D == 128, "head dim");
  static_assert(NR == 16 || NR == 32 || NR == 64, "query rows");
  static constexpr uint32_t kTileBytes = kKeys * D;
  static constexpr uint32_t kQTerm = NR * D, kQBuf = 2 * kQTerm;     // two E4M3 terms
  static constexpr uint32_t kPTerm = NR * kKeys, kPBuf = 3 * kPTerm; // three E5M2 terms
  static constexpr uint32_t kSmall = 8192;                            // arrays and barriers below
  static constexpr uint32_t kRoom = 232448 - 1024 - kSmall - 2 * kQBuf - 2 * kPBuf;
  static constexpr int kStages = static_cast<int>(kRoom / kTileBytes) / 2 * 2 < 20
                                     ? static_cast<int>(kRoom / kTileBytes) / 2 * 2
                                     : 20;
  static constexpr uint32_t kRingOff = 0;
  static constexpr uint32_t kQOff = kStages * kTileBytes;
  static constexpr uint32_t kPOff = kQOff + 2 * kQBuf;
  static constexpr uint32_t kFrOff = kPOff + 2 * kPBuf;         // [2 Q buffers][NR] row factors
  static constexpr uint32_t kNegMOff = kFrOff + 2 * NR * 4;     // [2 warpgroups][NR] kTop - m
  static constexpr uint32_t kHiOff = kNegMOff + 2 * NR * 4;     // [2][NR] last visible position
  static constexpr uint32_t kLoOff = kHiOff + 2 * NR * 4;       // [2][NR] first position of the window
  static constexpr uint32_t kWmaxOff = kLoOff + 2 * NR * 4;     // [2][4 warps][NR]
  static constexpr uint32_t kLsumOff = kWmaxOff + 8 * NR * 4;   // [2][4 warps][NR]
  static constexpr uint32_t kCoefOff = kLsumOff + 8 * NR * 4;   // [2][NR] weight of a warpgroup's O
  static constexpr uint32_t kBarOff = kCoefOff + 2 * NR * 4;
  static constexpr int kQFull = 0;                     // x2
  static constexpr int kQEmpty = 2;                    // x2
  static constexpr int kKVFull = 4;
  static constexpr int kKVEmpty = kKVFull + kStages;
  static constexpr int kSFull = kKVEmpty + kStages;    // x4
  static constexpr int kSFree = kSFull + 4;            // x4
  static constexpr int kPFull = kSFree + 4;            // x2, one per warpgroup
  static constexpr int kPVDone = kPFull + 2;           // x2
  static constexpr int kOFree = kPVDone + 2;
  static constexpr int kFin = kOFree + 1;              // x2, one per issuing warp
  static constexpr int kItemFull = kFin + 2;
  static constexpr int kItemEmpty = kItemFull + kItemSlots;
  static constexpr int kNumBars = kItemEmpty + kItemSlots;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kItemOff = kMiscOff + 16;
  static constexpr uint32_t kBytes = kItemOff + 4 * kItemSlots;
  static constexpr uint32_t kAlloc = 232448;
  static_assert(kBytes - kFrOff <= kSmall && kBytes + 1024 <= kAlloc, "shared memory per CTA");
  // The terms of Q and of P are side by side in one product's N where TMEM has room for
  // their separate sums (a product of few rows takes the time of reading its A operand, 128
  // rows, whatever N is), and further products into the same sums otherwise.
  static constexpr bool kWide = NR <= 32;
  static constexpr uint32_t kSCols = kWide ? 2 * NR : NR, kOCols = kWide ? 3 * NR : NR;
  static constexpr uint32_t kSCol = 0, kOCol = 4 * kSCols;      // + kSCols per buffer, kOCols per warpgroup
  static constexpr uint32_t kTmemCols = NR == 16 ? 256 : 512;
  static_assert(4 * kSCols + 2 * kOCols <= kTmemCols, "TMEM columns");
};

// ------------------------------------------------------------ work items
// Tiles of a sequence are numbered u = 0, 1, ... over what the step can see: the ns tiles
// that hold sinks before the window's first tile, then the window's.  tile(u) is the
// position range's tile.
struct Item8 {
  int b, hkv, s;
  int L, lo_pos, sinks;  // cached positions; oldest position in any row's window; sinks
  int ns, first;         // tile(u) = u < ns ? u : u - ns + first
  int t0, t1;            // range of u of this split (empty when t1 < t0)
  int row0, rows;
  bool bad;
  __device__ __forceinline__ int tile(int u) const { return u < ns ? u : u - ns + first; }
  __device__ __forceinline__ bool seen(int pos) const { return pos < L && (pos >= lo_pos || pos < sinks); }
};

__device__ __forceinline__ Item8 item8(const Dec8Params& p, int idx) {
  Item8 it;
  it.s = idx % p.num_splits;
  idx /= p.num_splits;
  const int rc = idx % p.row_chunks;
  idx /= p.row_chunks;
  it.hkv = idx % p.Hkv;
  it.b = idx / p.Hkv;
  it.L = __ldg(p.seq_lens + it.b);
  it.bad = (it.L != 0 && it.L < p.Nq) || it.L > p.max_pages * p.page_size;
  it.row0 = rc * p.rows_chunk;
  it.rows = min(p.rows_chunk, p.rows_total - it.row0);
  it.lo_pos = it.ns = it.first = it.t0 = 0;
  it.sinks = 0;
  it.t1 = -1;
  if (!it.bad && it.L > 0) {
    if (p.mask_kind == kDMaskWindow) {
      it.lo_pos = max(0, it.L - p.Nq - p.window + 1);
      it.sinks = min(p.sinks, it.L);
      it.first = it.lo_pos / kKeys;
      it.ns = min((it.sinks + kKeys - 1) / kKeys, it.first);
    }
    const int tiles = (it.L - 1) / kKeys - it.first + 1 + it.ns;
    const int chunk = (tiles + p.num_splits - 1) / p.num_splits;
    it.t0 = it.s * chunk;
    it.t1 = min(tiles, it.t0 + chunk) - 1;
  }
  return it;
}

template <class L>
__device__ __forceinline__ int take_item8(uint32_t sbase, const uint8_t* smem, const DecWaiter& w, uint32_t& k,
                                          int code) {
  const uint32_t slot = k % kItemSlots;
  const uint32_t full = sbase + L::kBarOff + 8u * (L::kItemFull + slot);
  if (!w.wait_warp(full, (k / kItemSlots) & 1, code | (L::kItemFull + slot))) return -1;
  const int idx = *reinterpret_cast<const volatile int*>(smem + L::kItemOff + 4 * slot);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(sbase + L::kBarOff + 8u * (L::kItemEmpty + slot));
  ++k;
  return idx;
}

// ------------------------------------------------------------ small pieces
// Barrier of `n` threads that also ors a predicate over them.
__device__ __forceinline__ bool bar_or(int id, int n, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.aligned.pred p, %2, %3, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(pred ? 1u : 0u), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tmem_load_16cols(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_load_2x16cols(uint32_t ta, uint32_t tb, uint32_t (&a)[16], uint32_t (&b)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]),
        "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]), "=r"(b[0]),
        "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]), "=r"(b[8]), "=r"(b[9]),
        "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15])
      : "r"(ta), "r"(tb)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_first(uint32_t dst, const CUtensorMap* map, uint32_t bar, int y, int z,
                                                  uint64_t policy) {
  tma_load_3d(dst, map, bar, 0, y, z, policy);
}
// Shared-memory descriptors: swizzle by the row's bytes (128: layout 2, 64: layout 4), or none.
__device__ __forceinline__ uint64_t desc8(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
         static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32 | static_cast<uint64_t>(1u) << 46 |
         static_cast<uint64_t>(layout) << 61;
}
// kind::f8f6f4, fp32 accumulator: formats 0 = E4M3, 1 = E5M2; majorness 1 = MN.
__host__ __device__ constexpr uint32_t idesc8(int N, uint32_t a_fmt, uint32_t b_fmt, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_fmt << 7) | (b_fmt << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(kKeys >> 4) << 24);
}
__device__ __forceinline__ uint32_t half2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ int ordered(float x) {  // order-preserving, its own inverse on the bits
  const int b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int b) { return __int_as_float(b ^ ((b >> 31) & 0x7fffffff)); }

// ------------------------------------------------------------ loaders
// As in the bf16 kernel: K of the CTA's g-th tile goes to ring index 2g, V to 2g + 1; lane i
// copies the i-th box of the tile; page-table entries are read two tiles ahead.
template <int D, int NR, bool kV>
__device__ __forceinline__ uint32_t loader8(const Dec8Params& p, uint32_t sbase, uint8_t* smem, const DecWaiter& w) {
  using L = Smem8<D, NR>;
  auto bar = [&](int i) { return sbase + L::kBarOff + 8u * i; };
  const int lane = threadIdx.x & 31;
  const uint64_t pol = l2_policy_evict_first();
  const CUtensorMap* map = kV ? &p.tm_v : &p.tm_k;
  if (lane == 0) tma_prefetch_map(map);
  const int code = kDRoleLoader << 8;
  uint32_t gt = 0, k_item = 0;
  int next = 0;
  if (!kV && lane == 0) next = static_cast<int>(atomicAdd(p.sched, 1u));
  bool ok = true;
  while (ok) {
    int idx;
    if constexpr (kV) {
      idx = take_item8<L>(sbase, smem, w, k_item, code);
      if (idx < 0) break;
    } else {
      const uint32_t slot_i = k_item % kItemSlots;
      if (k_item >= (uint32_t)kItemSlots &&
          !w.wait_warp(bar(L::kItemEmpty + slot_i), ((k_item / kItemSlots) - 1) & 1, code | (L::kItemEmpty + slot_i)))
        break;
      idx = __shfl_sync(0xffffffffu, next, 0);
      if (lane == 0) {
        *reinterpret_cast<volatile int*>(smem + L::kItemOff + 4 * slot_i) = idx < p.num_items ? idx : -2;
        mbar_arrive(bar(L::kItemFull + slot_i));
      }
      ++k_item;
      if (idx >= p.num_items) break;
      if (lane == 0) next = static_cast<int>(atomicAdd(p.sched, 1u));
    }
    const Item8 it = item8(p, idx);
    if (it.t1 < it.t0) continue;
    const int* trow = p.block_table + static_cast<size_t>(it.b) * p.max_pages;
    // First position of this lane's box in tile u, or -1 when the box holds nothing the step sees.
    auto box_pos = [&](int u) -> int {
      if (u > it.t1 || lane >= p.loads_per_tile) return -1;
      const int pos0 = it.tile(u) * kKeys + lane * p.rows_per_load;
      return (pos0 >= it.L || (pos0 + p.rows_per_load <= it.lo_pos && pos0 >= it.sinks)) ? -1 : pos0;
    };
    auto entry = [&](int pos0) -> int { return pos0 < 0 ? 0 : __ldg(trow + (pos0 >> p.page_shift)); };
    int p0 = box_pos(it.t0), p1 = box_pos(it.t0 + 1);
    int e0 = entry(p0), e1 = entry(p1);
    for (int u = it.t0; u <= it.t1; ++u) {
      const int p2 = box_pos(u + 2), e2 = entry(p2);
      int page = e0;
      if (p0 >= 0 && (page < 0 || page >= p.num_pages)) {
        atomicCAS(p.err, 0, kDErrPage | (it.b & 0xFFFFF));
        page = 0;  // a stand-in inside the pool; the step's result is then undefined
      }
      const uint32_t ring_idx = 2 * gt + (kV ? 1 : 0), slot = ring_idx % L::kStages;
      if (ring_idx >= (uint32_t)L::kStages &&
          !w.wait_warp(bar(L::kKVEmpty + slot), ((ring_idx / L::kStages) - 1) & 1, code | (L::kKVEmpty + slot))) {
        ok = false;
        break;
      }
      const unsigned boxes = __ballot_sync(0xffffffffu, p0 >= 0);
      if (lane == 0)
        mbar_arrive_expect_tx(bar(L::kKVFull + slot), __popc(boxes) * static_cast<uint32_t>(p.rows_per_load) * D);
      __syncwarp();
      if (p0 >= 0)
        tma_load_3d_first(sbase + L::kRingOff + slot * L::kTileBytes + lane * p.rows_per_load * D, map,
                          bar(L::kKVFull + slot), p0 & (p.page_size - 1), page * p.Hkv + it.hkv, pol);
      ++gt;
      p0 = p1;
      e0 = e1;
      p1 = p2;
      e1 = e2;
    }
  }
  return gt;
}

template <class L>
__device__ __forceinline__ void drain_ring8(uint32_t sbase, const DecWaiter& w, uint32_t gt_k, uint32_t gt_v) {
  for (uint32_t s = 0; s < (uint32_t)L::kStages; ++s) {
    // an even ring: even slots hold K, odd slots V
    const uint32_t gt = (s & 1) ? gt_v : gt_k, lead = s >> 1, half = L::kStages / 2;
    if (gt > lead) {
      const uint32_t fills = (gt - 1 - lead) / half;  // completed refills of the slot's last load
      w.drain(sbase + L::kBarOff + 8u * (L::kKVFull + s), fills & 1, (kDRoleLoader << 8) | (L::kKVFull + s));
    }
  }
}

// ------------------------------------------------------------ Q
// One warp: each row of an item becomes two E4M3 terms in shared memory (K-major, in the
// swizzle of a D-byte row), with its factor scale log2(e) / (the row's power of two).
template <int D, int NR>
__device__ __forceinline__ void prepare_q8(const Dec8Params& p, const Item8& it, uint8_t* smem, uint32_t buf) {
  using L = Smem8<D, NR>;
  const int lane = threadIdx.x & 31;
  const size_t row = (static_cast<size_t>(it.b) * p.Hq + static_cast<size_t>(it.hkv) * p.group) * p.Nq + it.row0;
  const __nv_bfloat16* src = p.q + row * D;
  float* fr = reinterpret_cast<float*>(smem + L::kFrOff) + buf * NR;
  uint8_t* q1 = smem + L::kQOff + buf * L::kQBuf;
  constexpr int E = D / 32;  // elements of a lane
#pragma unroll 8
  for (int r = 0; r < NR; ++r) {
    float x[E];
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = 0.f;
    if (r < it.rows) {
      const uint32_t* s32 = reinterpret_cast<const uint32_t*>(src + static_cast<size_t>(r) * D) + lane * (E / 2);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const uint32_t v = __ldg(s32 + i);
        x[2 * i] = __uint_as_float(v << 16);
        x[2 * i + 1] = __uint_as_float(v & 0xffff0000u);
      }
    }
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) big = max(big, __float_as_uint(x[i]) & 0x7fffffffu);
    big = __reduce_max_sync(0xffffffffu, big);
    // Multiplier 2^(7 - exponent): the row's largest lands in [128, 256).
    const int e = static_cast<int>(big >> 23) - 127;
    const int mul_e = min(max(7 - e, -126), 126);
    float mul = big ? __uint_as_float(static_cast<uint32_t>(mul_e + 127) << 23) : 1.f;
    if (big >= 0x7f800000u) mul = __int_as_float(0x7fffffff);  // E4M3 has no infinities: the row becomes NaN
    float hi[4] = {0.f, 0.f, 0.f, 0.f}, lo[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) hi[i] = x[i] * mul;
    const uint32_t c1 = pack_e4m3x4(hi[0], hi[1], hi[2], hi[3]);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      uint32_t h2;
      float f;
      asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}"
          : "=r"(h2)
          : "r"((c1 >> (8 * i)) & 0xffu));
      asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h2));
      lo[i] = hi[i] - f;
    }
    const uint32_t c2 = pack_e4m3x4(lo[0], lo[1], lo[2], lo[3]);
    if constexpr (D == 128) {
      const uint32_t at = r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
      *reinterpret_cast<uint32_t*>(q1 + at) = c1;
      *reinterpret_cast<uint32_t*>(q1 + L::kQTerm + at) = c2;
    } else {
      const uint32_t at = r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2;
      *reinterpret_cast<uint16_t*>(q1 + at) = static_cast<uint16_t>(c1);
      *reinterpret_cast<uint16_t*>(q1 + L::kQTerm + at) = static_cast<uint16_t>(c2);
    }
    if (lane == 0) fr[r] = p.scale_log2 / mul;
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// ------------------------------------------------------------ products
// S^T_j = K_j (Q1 + Q2)^T for every tile of every item, as far ahead as K, the four S buffers
// and the two Q buffers allow.
template <int D, int NR>
__device__ __forceinline__ void s_role8(const Dec8Params& p, uint32_t sbase, uint8_t* smem, uint32_t tmem,
                                        const DecWaiter& w) {
  using L = Smem8<D, NR>;
  auto bar = [&](int i) { return sbase + L::kBarOff + 8u * i; };
  constexpr uint32_t kLayout = D == 128 ? 2 : 4;   // 128- or 64-byte swizzle: one row per line
  constexpr uint32_t kAtom = 8 * D;                // eight rows
  constexpr uint32_t idesc_s = idesc8(L::kSCols, 0, 0, false, false);
  constexpr int kProducts = L::kWide ? 1 : 2;
  const uint64_t k_desc0 = desc8(sbase + L::kRingOff, 16, kAtom, kLayout);
  const uint64_t q_desc0 = desc8(sbase + L::kQOff, 16, kAtom, kLayout);
  const bool leader = elect_one();  // issues the products, so that the commits track them
  const int code = kDRoleS << 8;
  uint32_t g = 0, items = 0, k_item = 0;
  bool ok = true;
  while (ok) {
    const int idx = take_item8<L>(sbase, smem, w, k_item, code);
    if (idx < 0) break;
    const Item8 it = item8(p, idx);
    if (it.t1 < it.t0) continue;
    const int n = it.t1 - it.t0 + 1;
    const uint32_t qbuf = items & 1;
    if (items >= 2 && !w.wait_warp(bar(L::kQEmpty + qbuf), ((items >> 1) - 1) & 1, code | (L::kQEmpty + qbuf))) break;
    prepare_q8<D, NR>(p, it, smem, qbuf);
    if (leader) mbar_arrive(bar(L::kQFull + qbuf));
    const uint64_t qd = q_desc0 + ((qbuf * L::kQBuf) >> 4);
    for (int j = 0; j < n; ++j) {
      const uint32_t gi = g + j, ki = 2 * gi, slot = ki % L::kStages;
      if ((gi >= 4 && !w.wait_warp(bar(L::kSFree + (gi & 3)), ((gi >> 2) - 1) & 1, code | (L::kSFree + (gi & 3)))) ||
          !w.wait_warp(bar(L::kKVFull + slot), (ki / L::kStages) & 1, code | (L::kKVFull + slot))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t s_tmem = tmem + L::kSCol + (gi & 3) * L::kSCols;
      const uint64_t kd = k_desc0 + ((slot * L::kTileBytes) >> 4);
      if (leader) {
#pragma unroll
        for (int term = 0; term < kProducts; ++term)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            mma_f8f6f4_ss(s_tmem, kd + ((kk * 32) >> 4), qd + ((term * L::kQTerm + kk * 32) >> 4), idesc_s,
                          (term | kk) ? 1u : 0u);
        tc_commit(bar(L::kSFull + (gi & 3)));
        tc_commit(bar(L::kKVEmpty + slot));
        if (j == n - 1) tc_commit(bar(L::kQEmpty + qbuf));
      }
      __syncwarp();
    }
    g += n;
    ++items;
  }
  // Every product this warp issued must complete before TMEM is freed.
  if (leader) tc_commit(bar(L::kFin));
  __syncwarp();
  w.drain(bar(L::kFin), 0, code | L::kFin);
}

// O_w += V_j^T (P1 + P2 + P3), w the tile's warpgroup.
template <int D, int NR>
__device__ __forceinline__ void pv_role8(const Dec8Params& p, uint32_t sbase, const uint8_t* smem, uint32_t tmem,
                                         const DecWaiter& w) {
  using L = Smem8<D, NR>;
  auto bar = [&](int i) { return sbase + L::kBarOff + 8u * i; };
  constexpr uint32_t kLayout = D == 128 ? 2 : 4;
  constexpr uint32_t idesc_o = idesc8(L::kOCols, 0, 1, true, true);
  constexpr int kProducts = L::kWide ? 1 : 3;
  // V^T: M runs along a row.  With d = 64 the rows end after 64, and a stride of 0 to the
  // next 64 lets lanes 64 .. 127 repeat lanes 0 .. 63.
  const uint64_t v_desc0 = desc8(sbase + L::kRingOff, 0, 8 * D, kLayout);
  // P: units of 16 rows, 16 bytes per key; eight keys are a core matrix.
  const uint64_t p_desc0 = desc8(sbase + L::kPOff, 128, kKeys * 16, 0);
  const bool leader = elect_one();
  const int code = kDRoleMma << 8;
  uint32_t g = 0, items = 0, k_item = 0;
  bool ok = true;
  while (ok) {
    const int idx = take_item8<L>(sbase, smem, w, k_item, code);
    if (idx < 0) break;
    const Item8 it = item8(p, idx);
    if (it.t1 < it.t0) continue;
    const int n = it.t1 - it.t0 + 1;
    for (int j = 0; j < n; ++j) {
      const uint32_t gi = g + j, wg = gi & 1, vi = 2 * gi + 1, slot = vi % L::kStages;
      if (!w.wait_warp(bar(L::kPFull + wg), (gi >> 1) & 1, code | (L::kPFull + wg)) ||
          !w.wait_warp(bar(L::kKVFull + slot), (vi / L::kStages) & 1, code | (L::kKVFull + slot)) ||
          (j == 0 && items > 0 && !w.wait_warp(bar(L::kOFree), (items - 1) & 1, code | L::kOFree))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t o_tmem = tmem + L::kOCol + wg * L::kOCols;
      const uint64_t vd = v_desc0 + ((slot * L::kTileBytes) >> 4);
      const uint64_t pd = p_desc0 + ((wg * L::kPBuf) >> 4);
      const uint32_t more = j >= 2 ? 1u : 0u;  // each warpgroup's first tile of the item starts its O
      if (leader) {
#pragma unroll
        for (int term = 0; term < kProducts; ++term)
#pragma unroll
          for (int kk = 0; kk < kKeys / 32; ++kk)
            mma_f8f6f4_ss(o_tmem, vd + ((kk * 32 * D) >> 4), pd + ((term * L::kPTerm + kk * 32 * 16) >> 4), idesc_o,
                          (term | kk) ? 1u : more);
        tc_commit(bar(L::kPVDone + wg));
        tc_commit(bar(L::kKVEmpty + slot));
      }
      __syncwarp();
    }
    g += n;
    ++items;
  }
  if (leader) tc_commit(bar(L::kFin + 1));
  __syncwarp();
  w.drain(bar(L::kFin + 1), 0, code | (L::kFin + 1));
}

// ------------------------------------------------------------ softmax
template <int D, int NR>
__device__ __forceinline__ void softmax_role8(const Dec8Params& p, uint32_t sbase, uint8_t* smem, uint32_t tmem,
                                              const DecWaiter& w) {
  using L = Smem8<D, NR>;
  auto bar = [&](int i) { return sbase + L::kBarOff + 8u * i; };
  constexpr int CH = NR / 16;
  const int tid = threadIdx.x, lane = tid & 31;
  const int wg = tid >> 7, key = tid & 127, warp = key >> 5;  // key: this thread's key of a tile
  const uint32_t lane_addr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  float* fr_all = reinterpret_cast<float*>(smem + L::kFrOff);
  float* negm = reinterpret_cast<float*>(smem + L::kNegMOff) + wg * NR;
  int* row_hi = reinterpret_cast<int*>(smem + L::kHiOff) + wg * NR;
  int* row_lo = reinterpret_cast<int*>(smem + L::kLoOff) + wg * NR;
  float* wmax = reinterpret_cast<float*>(smem + L::kWmaxOff) + wg * 4 * NR;
  float* lsum_all = reinterpret_cast<float*>(smem + L::kLsumOff);
  float* coef = reinterpret_cast<float*>(smem + L::kCoefOff);
  const float* negm_all = reinterpret_cast<float*>(smem + L::kNegMOff);
  const int wg_bar = 1 + wg;         // barrier of the warpgroup; 3: of both
  const int code = kDRoleSoftmax << 8;
  const int S = p.num_splits;
  uint32_t g = 0, items = 0, k_item = 0;
  bool ok = true;

  while (ok) {
    const int idx = take_item8<L>(sbase, smem, w, k_item, code);
    // An item that could not be taken is the end, or an abort that every warp will see: the
    // barriers below are reached by all warps or by none, as a wait that gives up is
    // agreed on at each barrier and an item is taken by all or missed for good.
    if (bar_or(3, 2 * kWg, idx == -1)) break;
    if (idx < 0) break;
    const Item8 it = item8(p, idx);
    const size_t grow0 = (static_cast<size_t>(it.b) * p.Hq + static_cast<size_t>(it.hkv) * p.group) * p.Nq + it.row0;
    // This item's partial result is written: the CTA whose item is the last of its rows to get
    // here merges all S of them (out = sum_s w_s O_s / sum_s w_s, w_s = 2^(lse2_s - max)), four
    // columns of a row per thread.
    auto merge_if_last = [&]() {
      if (!p.done) return;
      __threadfence();
      bool last = false;
      bar_or(3, 2 * kWg, false);
      if (tid == 0) {
        unsigned int* count = p.done + idx / S;
        last = atomicAdd(count, 1u) == static_cast<unsigned>(S - 1);
        if (last) atomicExch(count, 0u);
        __threadfence();
      }
      if (!bar_or(3, 2 * kWg, last)) return;
      constexpr int Q = D / 4;
      for (int t = tid; t < it.rows * Q; t += 2 * kWg) {
        const size_t row = grow0 + t / Q;
        const int c = t % Q * 4;
        const float* pl = p.part_lse + row * S;
        const float* po = p.part_o + row * S * D + c;
        float top = -INFINITY;
        for (int k = 0; k < S; ++k) top = fmaxf(top, __ldcg(pl + k));
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        float wsum = 0.f;
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll 4
        for (int k = 0; k < S; ++k) {
          const float l2 = __ldcg(pl + k), wgt = dec_exp2(l2 - base);
          if (l2 != -INFINITY) {   // a split that saw nothing wrote no O
            const float4 o = __ldcg(reinterpret_cast<const float4*>(po + static_cast<size_t>(k) * D));
            wsum += wgt;
            sum.x = fmaf(wgt, o.x, sum.x);
            sum.y = fmaf(wgt, o.y, sum.y);
            sum.z = fmaf(wgt, o.z, sum.z);
            sum.w = fmaf(wgt, o.w, sum.w);
          }
        }
        const float inv = wsum != 0.f ? 1.f / wsum : 0.f;
        uint2 h;
        h.x = attn_sm100_dec::dec_pack_bf16x2(sum.x * inv, sum.y * inv);
        h.y = attn_sm100_dec::dec_pack_bf16x2(sum.z * inv, sum.w * inv);
        *reinterpret_cast<uint2*>(p.out + row * D + c) = h;
        if (c == 0) p.lse[row] = wsum != 0.f ? (top + __log2f(wsum)) * kLn2 : -INFINITY;
      }
    };
    if (it.t1 < it.t0) {
      if (it.bad && tid == 0) atomicCAS(p.err, 0, kDErrSeqLen | (it.b & 0xFFFFF));
      for (int e = tid; e < it.rows; e += 2 * kWg) {
        if (S > 1) {
          p.part_lse[(grow0 + e) * S + it.s] = -INFINITY;
        } else {
          p.lse[grow0 + e] = -INFINITY;
          for (int c = 0; c < D; ++c) p.out[(grow0 + e) * D + c] = __float2bfloat16_rn(0.f);
        }
      }
      if (S > 1) merge_if_last();
      continue;
    }
    const int n = it.t1 - it.t0 + 1;
    const uint32_t qbuf = items & 1;
    const float* fr = fr_all + qbuf * NR;
    bool failed = !w.wait_warp(bar(L::kQFull + qbuf), (items >> 1) & 1, code | (L::kQFull + qbuf));
    for (int r = key; r < NR; r += kWg) {
      const int qpos = it.L - p.Nq + (it.row0 + r) % p.Nq;
      const bool live = r < it.rows;
      negm[r] = live ? kTop - kNoMax : -1e30f;   // rows that are not there keep weights of zero
      row_hi[r] = live ? (p.mask_kind == kDMaskFull ? it.L - 1 : qpos) : -1;
      row_lo[r] = p.mask_kind == kDMaskWindow ? qpos - p.window + 1 : 0;
    }
    if (bar_or(wg_bar, kWg, failed)) ok = false;  // both warpgroups leave at the item's end
    // Positions that every row sees: [all_lo, all_hi], and the sinks up to all_hi.
    const int all_hi = p.mask_kind == kDMaskFull ? it.L - 1 : it.L - p.Nq;
    const int all_lo = p.mask_kind == kDMaskWindow ? it.L - p.window : 0;

    float l[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) l[r] = 0.f;
    // Scales of this thread's key, loaded a tile ahead, their page-table entry two ahead.
    const int* trow = p.block_table + static_cast<size_t>(it.b) * p.max_pages;
    auto pos_of = [&](int j) -> int {
      if (j >= n) return -1;
      const int pos = it.tile(it.t0 + j) * kKeys + key;
      return it.seen(pos) ? pos : -1;
    };
    auto entry_of = [&](int pos) -> int { return pos < 0 ? 0 : __ldg(trow + (pos >> p.page_shift)); };
    auto scales_of = [&](int pos, int entry, float& ks, float& vs) {
      ks = 0.f;
      vs = 1.f;
      if (pos < 0) return;
      const int page = (entry < 0 || entry >= p.num_pages) ? 0 : entry;
      const size_t at = (static_cast<size_t>(page) * p.Hkv + it.hkv) * p.blocks_per_page +
                        ((pos & (p.page_size - 1)) >> p.block_shift);
      ks = __ldg(p.k_scale + at);
      vs = __ldg(p.v_scale + at);
    };
    const int j0 = static_cast<int>((wg - g) & 1u);
    float ks, vs;
    int pos_next = pos_of(j0 + 2), entry_next = entry_of(pos_next);
    {
      const int pos = pos_of(j0);
      scales_of(pos, entry_of(pos), ks, vs);
    }
    bool any_pv = false;
    for (int j = j0; ok && j < n; j += 2) {
      const uint32_t gi = g + j;
      float ks_next, vs_next;
      scales_of(pos_next, entry_next, ks_next, vs_next);
      const int pos_2 = pos_of(j + 4), entry_2 = entry_of(pos_2);
      const int base = it.tile(it.t0 + j) * kKeys, pos = base + key;
      const bool whole = base + kKeys - 1 <= all_hi && (base >= all_lo || base + kKeys <= it.sinks);
      const float vsc = fminf(fmaxf(vs, kScaleMin), kScaleMax);
      const float lv = __log2f(vsc), ivs = __frcp_rn(vsc);
      if (!failed) failed = !w.wait_warp(bar(L::kSFull + (gi & 3)), (gi >> 2) & 1, code | (L::kSFull + (gi & 3)));
      // The previous P V of this warpgroup is done: its P may be overwritten and O rescaled.
      if (!failed && (gi >> 1) > 0)
        failed = !w.wait_warp(bar(L::kPVDone + wg), ((gi >> 1) - 1) & 1, code | (L::kPVDone + wg));
      tc_fence_after_sync();
      const uint32_t s_addr = lane_addr + L::kSCol + (gi & 3) * L::kSCols;
      // e[i] = y - m + kTop of rows 16 ch + i (the exponent of the weight), -inf where masked.
      auto exponents = [&](int ch, float add, bool with_m, float (&e)[16]) {
        uint32_t sr[16];
        if constexpr (L::kWide) {
          uint32_t s2[16];
          tmem_load_2x16cols(s_addr + ch * 16, s_addr + NR + ch * 16, sr, s2);
#pragma unroll
          for (int i = 0; i < 16; ++i) sr[i] = __float_as_uint(__uint_as_float(sr[i]) + __uint_as_float(s2[i]));
        } else {
          tmem_load_16cols(s_addr + ch * 16, sr);
        }
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 f4 = *reinterpret_cast<const float4*>(fr + ch * 16 + i);
          const float4 m4 = *reinterpret_cast<const float4*>(negm + ch * 16 + i);
          const float ff[4] = {f4.x, f4.y, f4.z, f4.w}, mm[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            e[i + k] = fmaf(__uint_as_float(sr[i + k]) * ks, ff[k], with_m ? add + mm[k] : add);
        }
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r = ch * 16 + i;
            if (pos > row_hi[r] || (pos < row_lo[r] && pos >= it.sinks)) e[i] = -INFINITY;
          }
        }
      };
      // Up to 32 rows' exponents stay in registers; of 64 rows the first 16's do, and the
      // others' are formed again below.
      constexpr int kKeep = CH <= 2 ? CH : 1;
      float e[kKeep][16];
      float top = -INFINITY;
      if (!failed) {
#pragma unroll
        for (int ch = CH - 1; ch >= 0; --ch) {
          exponents(ch, lv, true, e[ch % kKeep]);
#pragma unroll
          for (int i = 0; i < 16; i += 2) top = max3f(top, e[ch % kKeep][i], e[ch % kKeep][i + 1]);
        }
      }
      if (bar_or(wg_bar, kWg, failed || top > kTop + kGrow)) {
        // Some row's maximum grew (or some warp gives up): every warp's row maxima.
        if (!failed) {
#pragma unroll 1
          for (int ch = 0; ch < CH; ++ch) {
            float y[16];
            exponents(ch, lv, false, y);
            int mine = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int m = __reduce_max_sync(0xffffffffu, ordered(y[i]));
              if (lane == i) mine = m;
            }
            if (lane < 16) wmax[warp * NR + ch * 16 + lane] = unordered(mine);
          }
        }
        if (bar_or(wg_bar, kWg, failed)) {
          ok = false;
          break;
        }
        float mine_new = 0.f;
        // negm' and factor of every row; a row's m moves to its maximum when that is kGrow above it.
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
          float f[16];
          bool any = false;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r = ch * 16 + i;
            const float mx = fmaxf(fmaxf(wmax[r], wmax[NR + r]), fmaxf(wmax[2 * NR + r], wmax[3 * NR + r]));
            const float old = negm[r];
            const bool move = mx + old > kTop + kGrow && mx < INFINITY;
            const float now = move ? kTop - mx : old;
            f[i] = move ? dec_exp2(now - old) : 1.f;
            any |= move;
            if (key == r) mine_new = now;
            l[r] *= f[i];
          }
          if (any && any_pv) {
#pragma unroll
            for (int term = 0; term < (L::kWide ? 3 : 1); ++term) {
              uint32_t o[16];
              const uint32_t at = lane_addr + L::kOCol + wg * L::kOCols + term * NR + ch * 16;
              tmem_load_16cols(at, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f[i]);
              tmem_store_16cols(at, o);
            }
          }
        }
        tmem_store_wait();
        bar_or(wg_bar, kWg, false);   // every thread has read the old maxima
        if (key < NR) negm[key] = mine_new;
        bar_or(wg_bar, kWg, false);
#pragma unroll
        for (int ch = kKeep - 1; ch >= 0; --ch) exponents(ch, lv, true, e[ch]);
      }
      // Weights, their sum, and their three E5M2 terms: a weight in fp16 (11 significant
      // bits), whose upper byte is an E5M2 number; what that leaves, likewise; the last
      // remainder rounded to nearest.
      const uint32_t p_addr = sbase + L::kPOff + wg * L::kPBuf + key * 16;
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        if (ch >= kKeep) exponents(ch, lv, true, e[ch % kKeep]);
        const float(&e0)[16] = e[ch % kKeep];
        uint32_t t1[8], t2[8], t3[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = dec_exp2(e0[2 * i]), b = dec_exp2(e0[2 * i + 1]);
          l[ch * 16 + 2 * i] = fmaf(a, ivs, l[ch * 16 + 2 * i]);
          l[ch * 16 + 2 * i + 1] = fmaf(b, ivs, l[ch * 16 + 2 * i + 1]);
          const uint32_t h = pack_f16x2(a, b);
          t1[i] = h & 0xff00ff00u;
          const uint32_t r1 = half2_sub(h, t1[i]);
          t2[i] = r1 & 0xff00ff00u;
          t3[i] = half2_sub(r1, t2[i]) + 0x00800080u;
        }
        const uint32_t at = p_addr + ch * (kKeys * 16);
        auto put = [&](uint32_t a, const uint32_t (&t)[8]) {
          st_shared_v4(a, __byte_perm(t[0], t[1], 0x7531), __byte_perm(t[2], t[3], 0x7531),
                       __byte_perm(t[4], t[5], 0x7531), __byte_perm(t[6], t[7], 0x7531));
        };
        put(at, t1);
        put(at + L::kPTerm, t2);
        put(at + 2 * L::kPTerm, t3);
      }
      if (base + kKeys > it.L || (base < it.lo_pos && base + kKeys > it.sinks)) {
        // Rows of V that the step does not see were not loaded, or hold anything: zero them.
        const uint32_t vi = 2 * gi + 1, slot = vi % L::kStages;
        failed = !w.wait_warp(bar(L::kKVFull + slot), (vi / L::kStages) & 1, code | (L::kKVFull + slot));
        if (!failed && !it.seen(pos)) {
          const uint32_t at = sbase + L::kRingOff + slot * L::kTileBytes + key * D;
#pragma unroll
          for (int c = 0; c < D; c += 16) st_shared_v4(at + c, 0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(L::kPFull + wg));
        mbar_arrive(bar(L::kSFree + (gi & 3)));
      }
      any_pv = true;
      ks = ks_next;
      vs = vs_next;
      pos_next = pos_2;
      entry_next = entry_2;
    }
    // ---- epilogue: this warpgroup's O is complete; sums over its keys.
    failed |= !ok;
    if (!failed && any_pv) {
      const uint32_t last = (g + n - 1 - ((g + n - 1 - wg) & 1u)) >> 1;
      failed = !w.wait_warp(bar(L::kPVDone + wg), last & 1, code | (L::kPVDone + wg));
    }
    if (!failed) {
      // Sixteen sums over 32 lanes: each step halves the rows a lane carries.
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = l[ch * 16 + i];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
          const bool up = lane & o;
#pragma unroll
          for (int i = 0; i < o; ++i) {
            const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
          }
        }
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
        if (lane < 16) lsum_all[(wg * 4 + warp) * NR + ch * 16 + lane] = v[0];
      }
    }
    if (lane == 0) mbar_arrive(bar(L::kQEmpty + qbuf));  // this warp has read the row factors
    if (bar_or(3, 2 * kWg, failed)) {
      ok = false;
      break;
    }
    tc_fence_after_sync();
    for (int r = tid; r < NR; r += 2 * kWg) {
      const float n0 = negm_all[r], n1 = negm_all[NR + r];
      const float top = fminf(n0, n1);   // kTop - the larger maximum
      const float f0 = dec_exp2(top - n0), f1 = dec_exp2(top - n1);
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s0 += lsum_all[k * NR + r];
        s1 += lsum_all[(4 + k) * NR + r];
      }
      const float sum = f0 * s0 + f1 * s1;
      const float inv = sum != 0.f ? 1.f / sum : 0.f;   // (a NaN sum stays NaN)
      coef[r] = f0 * inv;
      coef[NR + r] = f1 * inv;
      if (r < it.rows) {
        const float l2 = sum != 0.f ? __log2f(sum) - top : -INFINITY;
        if (S > 1) p.part_lse[(grow0 + r) * S + it.s] = l2;
        else p.lse[grow0 + r] = l2 * kLn2;
      }
    }
    bar_or(3, 2 * kWg, false);
    // Rows are dealt to the two warpgroups in halves; thread = column of d.
    const bool has0 = n > 1 || (g & 1) == 0, has1 = n > 1 || (g & 1) == 1;
    constexpr int kHalf = NR / 2 < 16 ? NR / 2 : 16;
#pragma unroll 1
    for (int c0 = wg * (NR / 2); c0 < (wg + 1) * (NR / 2); c0 += kHalf) {
      if (c0 >= it.rows) break;
      uint32_t a[16], b[16];
      // 16 columns even where 8 are used: the columns behind belong to the other half.
      const int col = NR == 16 ? 0 : c0;
      auto load_o = [&](int g2, uint32_t (&o)[16]) {
        const uint32_t at = lane_addr + L::kOCol + g2 * L::kOCols + col;
        tmem_load_16cols(at, o);
        if constexpr (L::kWide) {
          uint32_t o2[16], o3[16];
          tmem_load_2x16cols(at + NR, at + 2 * NR, o2, o3);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o[i] = __float_as_uint(__uint_as_float(o[i]) + (__uint_as_float(o2[i]) + __uint_as_float(o3[i])));
        }
      };
      if (has0) load_o(0, a);
      if (has1) load_o(1, b);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = col + i;
        if (r >= c0 && r < c0 + kHalf && r < it.rows && key < D) {
          float v = 0.f;
          if (has0) v = __uint_as_float(a[i]) * coef[r];
          if (has1) v = fmaf(__uint_as_float(b[i]), coef[NR + r], v);
          if (S > 1) p.part_o[((grow0 + r) * S + it.s) * D + key] = v;
          else p.out[(grow0 + r) * D + key] = __float2bfloat16_rn(v);
        }
      }
    }
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(L::kOFree));
    if (S > 1) merge_if_last();
    g += n;
    ++items;
  }
}

template <int D, int NR>
__global__ void __launch_bounds__(kThreads, 1) attn_decode8_kernel(const __grid_constant__ Dec8Params p) {
  using L = Smem8<D, NR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const int warp = threadIdx.x >> 5;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  volatile uint32_t* loaded = reinterpret_cast<volatile uint32_t*>(smem + L::kMiscOff + 8);
  if (threadIdx.x == 0) {
    auto bar = [&](int i) { return sbase + L::kBarOff + 8u * i; };
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::kQFull + i), 1);
      mbar_init(bar(L::kQEmpty + i), 9);  // the last S product and the eight softmax warps
      mbar_init(bar(L::kPFull + i), 4);
      mbar_init(bar(L::kPVDone + i), 1);
    }
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar(L::kKVFull + s), 1);
      mbar_init(bar(L::kKVEmpty + s), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(L::kSFull + i), 1);
      mbar_init(bar(L::kSFree + i), 4);
    }
    mbar_init(bar(L::kOFree), 8);
    mbar_init(bar(L::kFin), 1);
    mbar_init(bar(L::kFin + 1), 1);
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(bar(L::kItemFull + i), 1);
      mbar_init(bar(L::kItemEmpty + i), 11);  // every warp but the K loader
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kPvWarp) {
    tmem_alloc(smem_addr(const_cast<uint32_t*>(tmem_slot)), L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const DecWaiter w{p.timeout_ns, abort_flag, p.err};

  if (warp < 8) {
    softmax_role8<D, NR>(p, sbase, smem, tmem, w);
  } else if (warp == kKWarp) {
    const uint32_t gt = loader8<D, NR, false>(p, sbase, smem, w);
    if ((threadIdx.x & 31) == 0) loaded[0] = gt;
  } else if (warp == kVWarp) {
    const uint32_t gt = loader8<D, NR, true>(p, sbase, smem, w);
    if ((threadIdx.x & 31) == 0) loaded[1] = gt;
  } else if (warp == kPvWarp) {
    pv_role8<D, NR>(p, sbase, smem, tmem, w);
  } else {
    s_role8<D, NR>(p, sbase, smem, tmem, w);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (threadIdx.x == kKWarp * 32) drain_ring8<L>(sbase, w, loaded[0], loaded[1]);
  if (warp == kPvWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, L::kTmemCols);
  }
  // The last CTA to finish puts the work counter back to zero for the next launch.
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(p.sched + 1, 1u) == gridDim.x - 1) {
      atomicExch(p.sched, 0u);
      atomicExch(p.sched + 1, 0u);
    }
  }
}

}  // namespace attn_sm100_dec8
