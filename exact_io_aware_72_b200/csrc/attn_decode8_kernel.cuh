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
// * S^T = K Q^T (128 keys x NR query rows, NR = 16 or 32): an SS product with the K
//   tile as A and Q as B.  bf16 q has 8 significant bits and E4M3 holds 4, so each q row,
//   scaled by a power of two to a maximum in [128, 256), is the sum of two E4M3 numbers:
//   the rounded value and the rest, which fits 4 bits exactly (elements below 2^-9 of the
//   row's largest keep an absolute error of up to 2^-17 of it).  Both terms accumulate into S.
// * A softmax thread owns one key (TMEM lane) and its NR scores, so its scales and mask are
//   scalars, and no thread computes an exponential that no row needs.
// * O^T = V^T P^T (d x NR): A is the V tile read MN-major, B is P written to shared memory by
//   the softmax threads, 16 rows (16 bytes) per key.  E4M3 V needs an 8-bit P: the weight is
//   rounded to fp16 and held as a sum of three E5M2 numbers (3 significant bits each, 9
//   together: off by at most 2^-9 + 2^-11, a bf16 weight by 2^-8), three products into one
//   accumulator.  Weights are scaled so that m sits at 2^12: they reach 2^15 before m must move
//   (E5M2 ends at 57344), and E5M2's smallest step, 2^-16, rounds them to 2^-28 of the largest: nine
//   bits are kept down to about 2^-20 of it, none below 2^-29.  (With m at 2^9 and room for a
//   growth of 2^6 a long context's many small weights beside one large were lost from 2^-26 on.)
//   What is held is softmax weight times V scale, so "the largest" is the largest of these.
// * Sums l and all statistics are fp32; out is rounded once to bf16.
//
// Work items and splits are the bf16 decoding kernel's.  Two CTAs share an
// SM, each with its own items, ring and softmax warpgroup: at an item's ends (its first page
// entries and scales, the last product, the merge) one CTA's chain of latencies, some 5 us,
// runs under the other's tiles.  (One CTA whose two warpgroups took the tiles of an item in
// turn stopped for it: 9 us for each item, 70 us instead of 58 for a batch of windows.)
// m is per row: a vote over the warpgroup (one hardware barrier with a reduction) finds the
// rare tiles where some row's maximum grew by more than 2^3 (32 rows: 115 us, 114 with room for 2^6).
//
// The partial results of splits are merged by a second, small kernel whose launch overlaps the
// first one's end (programmatic dependent launch).  Merged by the CTA that finished last, they
// kept one SM reading for 9 us behind the other 147 (37 splits of 8 rows) and cost each item a
// fence and an atomic.
//
// Warps: 0-3 softmax, 4 loads K (and fetches items), 5 loads V, 6 issues the P V products, 7
// prepares Q and issues the S products ahead.  (One issuing warp spent 1500 cycles per tile
// on waits and issue latencies of both products, whose execution takes 340; HBM delivers a
// tile per 1400.)  TMEM: the S buffers, then O.  All mbarrier waits are bounded; the
// warpgroup's barriers are reached by every warp whether or not a wait gave up, and carry
// that news, so the roles leave together.
//
// The code is kept small: what is not in the tile loop is a call or a rolled loop, items are
// decoded once (by the K loader) and read from shared memory.  With everything inlined the
// kernel was 130 KB, and each item's start and end ran at the speed of instruction fetches,
// 10 us an item.
//
// Measured, with the bytes of the visible codes and scales over 6544 GB/s (a copy) as 100 %: one
// sequence of 131072 positions, 64/8 heads, 49.5 us (83 %: the start and the end of the one wave
// of items, the merge and the launches, 8 us, are not overlapped); 16 of 8k-32k with 32 heads 415 to
// 438 us (99 to 94 %); 32 windows of 4096 with
// 4 sinks 52 us (79 %); 8 of 16k-32k with 32 rows (four new tokens, groups of 8) 116 us (53 %: the
// softmax warps' 3300 cycles a tile, two tiles at a time on an SM, against the 1400 in
// which HBM delivers one).
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
constexpr int kThreads = 256;
constexpr int kCtasPerSm = 2;
constexpr int kWg = 128;    // threads of the softmax warpgroup
constexpr int kKWarp = 4, kVWarp = 5, kPvWarp = 6, kSWarp = 7;
constexpr int kItemSlots = 4;
constexpr int kFetchTiles = 2;  // tiles before an item's last at which the next item is fetched
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTop = 12.f;     // weights at the running maximum are 2^kTop
constexpr float kGrow = 3.f;     // the running maximum moves when a row's grows by more
constexpr float kNoMax = -3e38f; // running maximum of a row that has seen no key
// V scales c are taken within [2^-40, 2^60]; the append writes none below.  The sum of softmax weights
// is formed from w / c, and w ends at fp32's 2^-126: with 100 powers of two between scales it
// loses a key's softmax weight only below 2^-38 of that of the key that sets the maximum.
constexpr float kScaleMin = 9.094947017729282e-13f, kScaleMax = 1152921504606846976.f;  // 2^-40, 2^60

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
  int block_shift;
  int mask_kind, window, sinks;
  int num_splits, num_items;
  float scale_log2;
  unsigned long long timeout_ns;
  unsigned int stall;      // test hook: loads before a CTA's loaders stop (0xffffffff: they do not)
  unsigned int* sched;     // [0] next work item, [1] CTAs finished; zero between launches
};

template <int D, int NR>
struct Smem8 {
  static_assert(D == 64 || D == 128, "head dim");
  static_assert(NR == 16 || NR == 32, "query rows");
  static constexpr uint32_t kTileBytes = kKeys * D;
  static constexpr uint32_t kQTerm = NR * D, kQBuf = 2 * kQTerm;     // two E4M3 terms
  static constexpr uint32_t kPTerm = NR * kKeys, kPBuf = 3 * kPTerm; // three E5M2 terms
  static constexpr uint32_t kAlloc = 115712;                         // half of an SM's shared memory
  static constexpr uint32_t kSmall = 2304;                           // arrays and barriers below
  static constexpr int kSlots = static_cast<int>((kAlloc - 1024 - kSmall - 2 * kQBuf - kPBuf) / kTileBytes);
  // Separate rings for K and V: each is waited on by one loader, in order, so a slot's phases
  // cannot be mistaken (on one ring of odd length, K and V would take turns on a slot and a
  // parity wait could pass two phases early).  V slots are held longer.
  static constexpr int kKSlots = kSlots / 2 < 6 ? kSlots / 2 : 6;
  static constexpr int kVSlots = (kSlots + 1) / 2 < 6 ? (kSlots + 1) / 2 : 6;
  static constexpr int kSBufs = NR == 16 ? 4 : 2;
  static constexpr uint32_t kKOff = 0;
  static constexpr uint32_t kVOff = kKSlots * kTileBytes;
  static constexpr uint32_t kQOff = kVOff + kVSlots * kTileBytes;
  static constexpr uint32_t kPOff = kQOff + 2 * kQBuf;
  static constexpr uint32_t kFrOff = kPOff + kPBuf;             // [2 Q buffers][NR] row factors
  static constexpr uint32_t kNegMOff = kFrOff + 2 * NR * 4;     // [2][NR] kTop - m, the buffers in turn
  static constexpr uint32_t kHiOff = kNegMOff + 2 * NR * 4;     // [NR] last visible position
  static constexpr uint32_t kLoOff = kHiOff + NR * 4;           // [NR] first position of the window
  static constexpr uint32_t kWmaxOff = kLoOff + NR * 4;         // [4 warps][NR]; at an item's end its sums
  static constexpr uint32_t kCoefOff = kWmaxOff + 4 * NR * 4;   // [NR] 1 / sum
  static constexpr uint32_t kBarOff = kCoefOff + NR * 4;
  static constexpr int kQFull = 0;                     // x2
  static constexpr int kQEmpty = 2;                    // x2
  static constexpr int kKFull = 4;                     // x kKSlots
  static constexpr int kKEmpty = kKFull + kKSlots;
  static constexpr int kVFull = kKEmpty + kKSlots;     // x kVSlots
  static constexpr int kVEmpty = kVFull + kVSlots;
  static constexpr int kSFull = kVEmpty + kVSlots;     // x kSBufs
  static constexpr int kSFree = kSFull + kSBufs;       // x kSBufs
  static constexpr int kPFull = kSFree + kSBufs;
  static constexpr int kPVDone = kPFull + 1;
  static constexpr int kOFree = kPVDone + 1;
  static constexpr int kFin = kOFree + 1;              // x2, one per issuing warp
  static constexpr int kItemFull = kFin + 2;
  static constexpr int kItemEmpty = kItemFull + kItemSlots;
  static constexpr int kNumBars = kItemEmpty + kItemSlots;
  static constexpr uint32_t kItemOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;  // kItemSlots items of 64 bytes
  static constexpr uint32_t kMiscOff = kItemOff + 64 * kItemSlots;
  static constexpr uint32_t kBytes = kMiscOff + 16;
  static_assert(kKSlots >= 2 && kBytes - kFrOff <= kSmall && kBytes + 1024 <= kAlloc, "shared memory per CTA");
  // The terms of Q and of P lie side by side in one product's N, with separate sums: a product
  // of few rows takes the time of reading its A operand, 128 rows, whatever N is.
  static constexpr uint32_t kSCols = 2 * NR, kOCols = 3 * NR;
  static constexpr uint32_t kSCol = 0, kOCol = kSBufs * kSCols;
  static constexpr uint32_t kTmemCols = 256;                    // two CTAs share 512
  static_assert(kOCol + kOCols <= kTmemCols, "TMEM columns");
};

// ------------------------------------------------------------ work items
// Tiles of a sequence are numbered u = 0, 1, ... over what the step can see: the ns tiles
// that hold sinks before the window's first tile, then the window's.  tile(u) is the
// position range's tile.
struct __align__(16) Item8 {
  int idx;               // its number; -2: no more items
  int b, hkv, s;
  int L, lo_pos, sinks;  // cached positions; oldest position in any row's window; sinks
  int ns, first;         // tile(u) = u < ns ? u : u - ns + first
  int t0, t1;            // range of u of this split (empty when t1 < t0)
  int row0, rows;
  int bad, pad[2];
  __device__ __forceinline__ int tile(int u) const { return u < ns ? u : u - ns + first; }
  __device__ __forceinline__ bool seen(int pos) const { return pos < L && (pos >= lo_pos || pos < sinks); }
};

__device__ __forceinline__ Item8 item8(const Dec8Params& p, int idx) {
  Item8 it;
  it.idx = idx;
  // Row chunks of one split are neighbours: they run together and share its keys in L2.
  const int rc = idx % p.row_chunks;
  idx /= p.row_chunks;
  it.s = idx % p.num_splits;
  idx /= p.num_splits;
  it.hkv = idx % p.Hkv;
  it.b = idx / p.Hkv;
  it.L = __ldg(p.seq_lens + it.b);
  it.bad = (it.L != 0 && it.L < p.Nq) || it.L > p.max_pages * p.page_size;
  if (it.bad) it.L = 0;  // nothing of it is looked up
  it.row0 = rc * p.rows_chunk;
  it.rows = min(p.rows_chunk, p.rows_total - it.row0);
  it.lo_pos = it.ns = it.first = it.t0 = 0;
  it.sinks = 0;
  it.t1 = -1;
  it.pad[0] = it.pad[1] = 0;
  if (it.L > 0) {
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

// A bounded wait whose rarely needed part is a call.
__device__ __noinline__ bool wait_long8(uint32_t bar, uint32_t parity, int code, const DecWaiter* w) {
  return w->wait(bar, parity, code);
}
struct Waiter8 {
  const DecWaiter* w;
  // This lane's answer, for the softmax warps, which agree on it at their next barrier (called
  // by the whole warp, whatever its lanes have seen before).
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, int code) const {
    bool got = mbar_try_wait(bar, parity);
    if (!got) got = wait_long8(bar, parity, code, w);
    __syncwarp();
    return got;
  }
  __device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, int code) const {
    bool got = mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, got)) got = got || wait_long8(bar, parity, code, w);
    return __all_sync(0xffffffffu, got);
  }
};

// The next item for a consuming warp; idx -2: no more, -1: the wait gave up.
template <class L>
__device__ __forceinline__ Item8 take_item8(uint32_t sbase, const uint8_t* smem, const Waiter8& w, uint32_t& k,
                                            int code) {
  const uint32_t slot = k % kItemSlots;
  const uint32_t full = sbase + L::kBarOff + 8u * (L::kItemFull + slot);
  Item8 it;
  if (w.wait_warp(full, (k / kItemSlots) & 1, code | (L::kItemFull + slot))) {
    it = *reinterpret_cast<const Item8*>(smem + L::kItemOff + sizeof(Item8) * slot);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(sbase + L::kBarOff + 8u * (L::kItemEmpty + slot));
    ++k;
  } else {
    it = Item8{};
    it.idx = -1;
    it.t1 = -1;
  }
  return it;
}

// ------------------------------------------------------------ small pieces
__device__ __forceinline__ float log2_approx(float x) {  // x normal
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
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
// *at, or 0 without a read.  (As a branch it cost the 32-row kernel 100 bytes of spills.)
__device__ __forceinline__ int load_if(bool read, const int* at) {
  int v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.nc.b32 %0, [%1];\n\t}"
      : "=&r"(v)
      : "l"(at), "r"(read ? 1u : 0u));
  return v;
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
// One warp for K and one for V, on rings of their own; lane i copies the i-th box of a tile.
// Page-table entries are read two tiles ahead.  The K warp also fetches the items and
// publishes them.
template <int D, int NR>
__device__ __forceinline__ uint32_t loader8(const Dec8Params& p, uint32_t sbase, uint8_t* smem, const Waiter8& w,
                                            bool kv) {
  using L = Smem8<D, NR>;
  auto bar = [&](int i) { return sbase + L::kBarOff + 8u * i; };
  const int lane = threadIdx.x & 31;
  // Every cached byte is read once per step, or once per row chunk.
  const uint64_t pol = p.row_chunks == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
  const CUtensorMap* map = kv ? &p.tm_v : &p.tm_k;
  const uint32_t slots = kv ? L::kVSlots : L::kKSlots;
  const uint32_t ring = sbase + (kv ? L::kVOff : L::kKOff) + lane * p.rows_per_load * D;
  const int full = kv ? L::kVFull : L::kKFull, empty = kv ? L::kVEmpty : L::kKEmpty;
  if (lane == 0) tma_prefetch_map(map);
  const int code = kDRoleLoader << 8;
  uint32_t gt = 0, k_item = 0, slot = 0, round = 0;  // tile gt goes to `slot`, filled `round` times before
  // A CTA's first item is its own number, the others come from the counter, fetched while the
  // current item's last tiles are asked for: a CTA that holds an item it has not begun leaves
  // others idle at the end.
  int next = blockIdx.x;
  auto fetch = [&]() {
    if (lane == 0) next = static_cast<int>(gridDim.x + atomicAdd(p.sched, 1u));
  };
  // Decodes and publishes the fetched item (or the end).
  auto publish = [&](Item8& it) -> bool {
    const uint32_t s = k_item % kItemSlots;
    if (k_item >= kItemSlots &&
        !w.wait_warp(bar(L::kItemEmpty + s), (k_item / kItemSlots - 1) & 1, code | (L::kItemEmpty + s)))
      return false;
    const int idx = __shfl_sync(0xffffffffu, next, 0);
    if (idx < p.num_items) {
      it = item8(p, idx);
    } else {
      it = Item8{};
      it.idx = -2;
      it.t1 = -1;
    }
    if (lane == 0) {
      *reinterpret_cast<Item8*>(smem + L::kItemOff + sizeof(Item8) * s) = it;
      mbar_arrive(bar(L::kItemFull + s));
    }
    __syncwarp();
    ++k_item;
    return true;
  };
  Item8 it;
  while (true) {
    if (kv) {
      it = take_item8<L>(sbase, smem, w, k_item, code);
    } else if (!publish(it)) {
      break;
    }
    if (it.idx < 0) break;
    if (!kv && it.t1 - it.t0 < kFetchTiles) fetch();
    // First position of this lane's box in tile u, or -1 when the box holds nothing the step sees.
    auto box_pos = [&](int u) -> int {
      if (u > it.t1 || lane >= p.loads_per_tile) return -1;
      const int pos0 = it.tile(u) * kKeys + lane * p.rows_per_load;
      return (pos0 >= it.L || (pos0 + p.rows_per_load <= it.lo_pos && pos0 >= it.sinks)) ? -1 : pos0;
    };
    const int* trow = p.block_table + static_cast<size_t>(it.b) * p.max_pages;
    auto entry = [&](int pos0) -> int { return pos0 < 0 ? 0 : __ldg(trow + (pos0 >> p.page_shift)); };
    bool ok = true;
    int p0 = -1, p1 = -1, e0 = 0, e1 = 0;
#pragma unroll 1
    for (int u = it.t0 - 2; u <= it.t1; ++u) {   // two rounds ahead to fill the entries
      int page = e0;
      if (p0 >= 0 && (page < 0 || page >= p.num_pages)) {
        atomicCAS(p.err, 0, kDErrPage | (it.b & 0xFFFFF));
        page = 0;  // a stand-in inside the pool; the step's result is then undefined
      }
      const int z = page * p.Hkv + it.hkv, at = p0;
      asm volatile("" ::"r"(z) : "memory");  // this entry is used before a later one is asked for
      p0 = p1;
      e0 = e1;
      p1 = box_pos(u + 2);
      e1 = entry(p1);
      if (u < it.t0) continue;
      if (gt == p.stall) {
        ok = false;
        break;
      }
      if (!kv && u == it.t1 - kFetchTiles) fetch();
      if (round > 0 && !w.wait_warp(bar(empty + slot), (round - 1) & 1, code | (empty + slot))) {
        ok = false;
        break;
      }
      const unsigned boxes = __ballot_sync(0xffffffffu, at >= 0);
      if (lane == 0)
        mbar_arrive_expect_tx(bar(full + slot), __popc(boxes) * static_cast<uint32_t>(p.rows_per_load) * D);
      __syncwarp();
      if (at >= 0) tma_load_3d(ring + slot * L::kTileBytes, map, bar(full + slot), 0, at & (p.page_size - 1), z, pol);
      ++gt;
      if (++slot == slots) {
        slot = 0;
        ++round;
      }
    }
    if (!ok) break;
  }
  return gt;
}

// Every copy must land before the CTA exits: a slot is loaded again only after its load
// landed and was read, so each slot's last load is waited for.
__device__ __forceinline__ void drain_ring8(uint32_t full, int slots, const DecWaiter& w, uint32_t gt) {
  for (uint32_t s = 0; s < static_cast<uint32_t>(slots) && s < gt; ++s)
    w.drain(full + 8u * s, ((gt - 1 - s) / slots) & 1, (kDRoleLoader << 8) | s);
}

// ------------------------------------------------------------ Q
// One warp: each of the rows b0 .. b1 - 1 of an item becomes two E4M3 terms in shared memory (K-major, in the
// swizzle of a D-byte row), with its factor 1 / (the row's power of two).
template <int D, int NR>
__device__ __noinline__ void prepare_q8(const Dec8Params& p, int b, int hkv, int item_row0, int rows, uint8_t* smem,
                                        uint32_t buf, int b0, int b1) {
  using L = Smem8<D, NR>;
  constexpr int G = D / 16;          // lanes of a row, 16 elements each
  constexpr int kRows = 32 / G;      // rows of a pass
  const int lane = threadIdx.x & 31, c = lane % G;
  const size_t row0 = (static_cast<size_t>(b) * p.Hq + static_cast<size_t>(hkv) * p.group) * p.Nq + item_row0;
  const uint4* src = reinterpret_cast<const uint4*>(p.q + row0 * D) + 2 * c;
  float* fr = reinterpret_cast<float*>(smem + L::kFrOff) + buf * NR;
  uint8_t* q1 = smem + L::kQOff + buf * L::kQBuf;
#pragma unroll 1
  for (int r0 = b0; r0 < b1; r0 += kRows) {
    const int r = r0 + lane / G;
    const bool live = r < rows && r < b1;
    const uint4 lo = live ? __ldg(src + static_cast<size_t>(r) * (D / 8)) : make_uint4(0u, 0u, 0u, 0u);
    const uint4 hi = live ? __ldg(src + static_cast<size_t>(r) * (D / 8) + 1) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t big = 0;  // largest magnitude, bf16 bits in each half
#pragma unroll
    for (int i = 0; i < 8; ++i) big = max_u16x2(big, w[i] & 0x7fff7fffu);
    big = max(big >> 16, big & 0xffffu);
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
    // Multiplier 2^(7 - exponent): the row's largest lands in [128, 256).  E4M3 has no
    // infinities: a row that holds one (or a NaN) becomes NaN.
    const int e = min(max(134 - static_cast<int>(big >> 7), -126), 126);
    const float mul = big >= 0x7f80u ? __int_as_float(0x7fffffff)
                                     : (big ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : 1.f);
    uint32_t c1[4], c2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = __uint_as_float(w[2 * i] << 16) * mul, x1 = __uint_as_float(w[2 * i] & 0xffff0000u) * mul;
      const float x2 = __uint_as_float(w[2 * i + 1] << 16) * mul;
      const float x3 = __uint_as_float(w[2 * i + 1] & 0xffff0000u) * mul;
      c1[i] = pack_e4m3x4(x0, x1, x2, x3);
      float y0, y1, y2, y3;
      e4m3x4_values(c1[i], y0, y1, y2, y3);
      c2[i] = pack_e4m3x4(x0 - y0, x1 - y1, x2 - y2, x3 - y3);
    }
    // 16-byte chunk c of the row, where the swizzle of D-byte rows puts it.
    const uint32_t at = D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    if (r < b1) {
      *reinterpret_cast<uint4*>(q1 + at) = make_uint4(c1[0], c1[1], c1[2], c1[3]);
      *reinterpret_cast<uint4*>(q1 + L::kQTerm + at) = make_uint4(c2[0], c2[1], c2[2], c2[3]);
      if (c == 0) fr[r] = 1.f / mul;
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// ------------------------------------------------------------ products
// S^T_j = K_j (Q1, Q2)^T for every tile of every item, as far ahead as K, the S buffers and
// the two Q buffers allow.
template <int D, int NR>
__device__ __forceinline__ void s_role8(const Dec8Params& p, uint32_t sbase, uint8_t* smem, uint32_t tmem,
                                        const Waiter8& w) {
  using L = Smem8<D, NR>;
  auto bar = [&](int i) { return sbase + L::kBarOff + 8u * i; };
  constexpr uint32_t kLayout = D == 128 ? 2 : 4;   // 128- or 64-byte swizzle: one row per line
  constexpr uint32_t kAtom = 8 * D;                // eight rows
  constexpr uint32_t idesc_s = idesc8(L::kSCols, 0, 0, false, false);
  const uint64_t k_desc0 = desc8(sbase + L::kKOff, 16, kAtom, kLayout);
  const uint64_t q_desc0 = desc8(sbase + L::kQOff, 16, kAtom, kLayout);
  const bool leader = elect_one();  // issues the products, so that the commits track them
  const int code = kDRoleS << 8;
  uint32_t g = 0, items = 0, k_item = 0;
  bool ok = true;
  while (ok) {
    const Item8 it = take_item8<L>(sbase, smem, w, k_item, code);
    if (it.idx < 0) break;
    if (it.t1 < it.t0) continue;
    const int n = it.t1 - it.t0 + 1;
    const uint32_t qbuf = items & 1;
    if (items >= 2 && !w.wait_warp(bar(L::kQEmpty + qbuf), ((items >> 1) - 1) & 1, code | (L::kQEmpty + qbuf))) break;
    if (items == 0) {  // the softmax warps prepare the first item's, while they have nothing else to do
      if (!w.wait_warp(bar(L::kQFull), 0, code | L::kQFull)) break;
      tc_fence_after_sync();
    } else {
      prepare_q8<D, NR>(p, it.b, it.hkv, it.row0, it.rows, smem, qbuf, 0, NR);
      if (leader) mbar_arrive(bar(L::kQFull + qbuf));
    }
    const uint64_t qd = q_desc0 + ((qbuf * L::kQBuf) >> 4);
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const uint32_t gi = g + j, slot = gi % L::kKSlots;
      const uint32_t sb = gi % L::kSBufs;
      if ((gi >= L::kSBufs && !w.wait_warp(bar(L::kSFree + sb), (gi / L::kSBufs - 1) & 1, code | (L::kSFree + sb))) ||
          !w.wait_warp(bar(L::kKFull + slot), (gi / L::kKSlots) & 1, code | (L::kKFull + slot))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t s_tmem = tmem + L::kSCol + sb * L::kSCols;
      const uint64_t kd = k_desc0 + ((slot * L::kTileBytes) >> 4);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          mma_f8f6f4_ss(s_tmem, kd + ((kk * 32) >> 4), qd + ((kk * 32) >> 4), idesc_s, kk > 0 ? 1u : 0u);
        tc_commit(bar(L::kSFull + sb));
        tc_commit(bar(L::kKEmpty + slot));
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
  w.w->drain(bar(L::kFin), 0, code | L::kFin);
}

// O += V_j^T (P1, P2, P3).
template <int D, int NR>
__device__ __forceinline__ void pv_role8(const Dec8Params& p, uint32_t sbase, const uint8_t* smem, uint32_t tmem,
                                         const Waiter8& w) {
  using L = Smem8<D, NR>;
  auto bar = [&](int i) { return sbase + L::kBarOff + 8u * i; };
  constexpr uint32_t kLayout = D == 128 ? 2 : 4;
  constexpr uint32_t idesc_o = idesc8(L::kOCols, 0, 1, true, true);
  // V^T: M runs along a row.  With d = 64 the rows end after 64, and a stride of 0 to the
  // next 64 lets lanes 64 .. 127 repeat lanes 0 .. 63.
  const uint64_t v_desc0 = desc8(sbase + L::kVOff, 0, 8 * D, kLayout);
  // P: units of 16 rows, 16 bytes per key; eight keys are a core matrix.
  const uint64_t p_desc0 = desc8(sbase + L::kPOff, 128, kKeys * 16, 0);
  const bool leader = elect_one();
  const int code = kDRoleMma << 8;
  uint32_t g = 0, items = 0, k_item = 0;
  bool ok = true;
  while (ok) {
    const Item8 it = take_item8<L>(sbase, smem, w, k_item, code);
    if (it.idx < 0) break;
    if (it.t1 < it.t0) continue;
    const int n = it.t1 - it.t0 + 1;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const uint32_t gi = g + j, slot = gi % L::kVSlots;
      if (!w.wait_warp(bar(L::kPFull), gi & 1, code | L::kPFull) ||
          !w.wait_warp(bar(L::kVFull + slot), (gi / L::kVSlots) & 1, code | (L::kVFull + slot)) ||
          (j == 0 && items > 0 && !w.wait_warp(bar(L::kOFree), (items - 1) & 1, code | L::kOFree))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint64_t vd = v_desc0 + ((slot * L::kTileBytes) >> 4);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < kKeys / 32; ++kk)
          mma_f8f6f4_ss(tmem + L::kOCol, vd + ((kk * 32 * D) >> 4), p_desc0 + ((kk * 32 * 16) >> 4), idesc_o,
                        (j | kk) ? 1u : 0u);
        tc_commit(bar(L::kPVDone));
        tc_commit(bar(L::kVEmpty + slot));
      }
      __syncwarp();
    }
    g += n;
    ++items;
  }
  if (leader) tc_commit(bar(L::kFin + 1));
  __syncwarp();
  w.w->drain(bar(L::kFin + 1), 0, code | (L::kFin + 1));
}

// ------------------------------------------------------------ softmax
template <int D, int NR>
__device__ __forceinline__ void softmax_role8(const Dec8Params& p, uint32_t sbase, uint8_t* smem, uint32_t tmem,
                                              const Waiter8& w) {
  using L = Smem8<D, NR>;
  auto bar = [&](int i) { return sbase + L::kBarOff + 8u * i; };
  constexpr int CH = NR / 16;
  const int key = threadIdx.x, lane = key & 31, warp = key >> 5;  // key: this thread's key of a tile
  const uint32_t lane_addr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  const float* fr_all = reinterpret_cast<const float*>(smem + L::kFrOff);
  float* negm_all = reinterpret_cast<float*>(smem + L::kNegMOff);
  int* row_hi = reinterpret_cast<int*>(smem + L::kHiOff);
  int* row_lo = reinterpret_cast<int*>(smem + L::kLoOff);
  float* wmax = reinterpret_cast<float*>(smem + L::kWmaxOff);
  float* coef = reinterpret_cast<float*>(smem + L::kCoefOff);
  constexpr int kBar = 1;
  const int code = kDRoleSoftmax << 8;
  const int S = p.num_splits;
  uint32_t g = 0, items = 0, k_item = 0;
  bool failed = false;

  // What the threads of an item ask for ahead: the scales of this thread's key, loaded a tile
  // ahead, and their page-table entry two tiles ahead.  Where there is no such tile, or the
  // step does not see the key, the sequence's last position, which it always sees, stands in (the
  // weight is zero whatever is read): other pages may be another's by now.  Without a length (an
  // idle slot, no more items) that is -1, and nothing is read.
  const int hkv_block = p.page_shift - p.block_shift;
  auto pos_of = [&](const Item8& it, int j) -> int {
    const int pos = it.tile(it.t0 + j) * kKeys + key;
    return it.t0 + j <= it.t1 && it.seen(pos) ? pos : it.L - 1;
  };
  auto entry_of = [&](const Item8& it, int pos) -> int {
    return load_if(pos >= 0, p.block_table + static_cast<size_t>(it.b) * p.max_pages + (pos >> p.page_shift));
  };
  auto scales_of = [&](const Item8& it, int pos, int entry, float& ks, float& vs) {
    const int page = static_cast<unsigned>(entry) < static_cast<unsigned>(p.num_pages) ? entry : 0;
    const size_t at = (static_cast<size_t>(page * p.Hkv + it.hkv) << hkv_block) +
                      ((pos & (p.page_size - 1)) >> p.block_shift);
    ks = __int_as_float(load_if(pos >= 0, reinterpret_cast<const int*>(p.k_scale + at)));
    vs = __int_as_float(load_if(pos >= 0, reinterpret_cast<const int*>(p.v_scale + at)));
  };

  Item8 it = take_item8<L>(sbase, smem, w, k_item, code);
  float ks, vs;
  int pos_next, entry_next;
  {
    const int pos = pos_of(it, 0), entry = entry_of(it, pos);
    pos_next = pos_of(it, 1);
    entry_next = entry_of(it, pos_next);
    scales_of(it, pos, entry, ks, vs);
  }
#pragma unroll 1
  while (true) {
    // -1: this warp's wait gave up.  Every warp gets here with the same item otherwise.
    if (bar_or(kBar, kWg, failed || it.idx == -1) || it.idx < 0) break;
    const size_t grow0 = (static_cast<size_t>(it.b) * p.Hq + static_cast<size_t>(it.hkv) * p.group) * p.Nq + it.row0;
    const int n = it.t1 - it.t0 + 1;
    const uint32_t qbuf = items & 1;
    const float* fr = fr_all + qbuf * NR;
    if (n > 0 && items == 0) {
      prepare_q8<D, NR>(p, it.b, it.hkv, it.row0, it.rows, smem, 0, warp * (NR / 4), (warp + 1) * (NR / 4));
      bar_or(kBar, kWg, false);
      if (key == 0) mbar_arrive(bar(L::kQFull));
    }
    if (n > 0) failed = !w.wait(bar(L::kQFull + qbuf), (items >> 1) & 1, code | (L::kQFull + qbuf));
    else if (it.bad && key == 0) atomicCAS(p.err, 0, kDErrSeqLen | (it.b & 0xFFFFF));
    uint32_t mbuf = 0;  // which negm is current
    if (key < NR) {
      const int qpos = it.L - p.Nq + (it.row0 + key) % p.Nq;
      const bool live = key < it.rows;
      negm_all[key] = live ? kTop - kNoMax : -1e30f;   // rows that are not there keep weights of zero
      row_hi[key] = live ? (p.mask_kind == kDMaskFull ? it.L - 1 : qpos) : -1;
      row_lo[key] = p.mask_kind == kDMaskWindow ? qpos - p.window + 1 : 0;
    }
    bool ok = !bar_or(kBar, kWg, failed);
    // Positions that every row sees: [all_lo, all_hi], and the sinks up to all_hi.
    const int all_hi = p.mask_kind == kDMaskFull ? it.L - 1 : it.L - p.Nq;
    const int all_lo = p.mask_kind == kDMaskWindow ? it.L - p.window : 0;

    // Pairs of rows share a 64-bit register: packed fp32 arithmetic halves the instructions of
    // the tile loop, which bound it at 32 rows.
    uint64_t l2[NR / 2];
#pragma unroll
    for (int r = 0; r < NR / 2; ++r) l2[r] = 0;  // (+0.f, +0.f)
#pragma unroll 1
    for (int j = 0; ok && j < n; ++j) {
      const uint32_t gi = g + j, sb = gi % L::kSBufs;
      // This tile's scales are used before the next tile's are asked for: the loads share a
      // scoreboard, and a use behind the newer loads waited for those too (850 cycles a tile).
      const float vsc = fminf(fmaxf(vs, kScaleMin), kScaleMax);
      const float lv = log2_approx(vsc), ivs = dec_exp2(-lv), ksl = ks * p.scale_log2;
      asm volatile("" ::"f"(lv), "f"(ivs), "f"(ksl) : "memory");
      scales_of(it, pos_next, entry_next, ks, vs);
      pos_next = pos_of(it, j + 2);
      entry_next = entry_of(it, pos_next);
      const int base = it.tile(it.t0 + j) * kKeys, pos = base + key;
      failed |= !w.wait(bar(L::kSFull + sb), (gi / L::kSBufs) & 1, code | (L::kSFull + sb));
      tc_fence_after_sync();
      // y_r = x_r + log2 c of this key and every row, -inf where the row does not see the key.
      const uint64_t ksl2 = f32x2_pack(ksl, ksl), lv2 = f32x2_pack(lv, lv);
      uint64_t y2[NR / 2];
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        const uint32_t s_addr = lane_addr + L::kSCol + sb * L::kSCols + ch * 16;
        uint32_t s1[16], s2[16];
        tmem_load_2x16cols(s_addr, s_addr + NR, s1, s2);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const ulonglong2 f4 = *reinterpret_cast<const ulonglong2*>(fr + ch * 16 + i);
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const uint64_t a = f32x2_pack(__uint_as_float(s1[i + k]), __uint_as_float(s1[i + k + 1]));
            const uint64_t b = f32x2_pack(__uint_as_float(s2[i + k]), __uint_as_float(s2[i + k + 1]));
            y2[(ch * 16 + i + k) / 2] = f32x2_fma(f32x2_mul(f32x2_add(a, b), ksl2), k ? f4.y : f4.x, lv2);
          }
        }
      }
      if (!(base + kKeys - 1 <= all_hi && (base >= all_lo || base + kKeys <= it.sinks))) {
        uint32_t hidden = 0;
#pragma unroll 1
        for (int r = 0; r < NR; ++r)
          hidden |= ((pos > row_hi[r]) | ((pos < row_lo[r]) & (pos >= it.sinks)) ? 1u : 0u) << r;
#pragma unroll
        for (int r = 0; r < NR / 2; ++r) {
          float a, b;
          f32x2_unpack(y2[r], a, b);
          y2[r] = f32x2_pack(hidden & (1u << (2 * r)) ? -INFINITY : a, hidden & (2u << (2 * r)) ? -INFINITY : b);
        }
      }
      // y - m + kTop are the exponents of the weights, unless some row's maximum has grown.
      const float* negm = negm_all + mbuf * NR;
      bool grown = j == 0;  // an item's first tile sets the maxima
      if (j > 0) {
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < NR; r += 4) {
          const ulonglong2 m4 = *reinterpret_cast<const ulonglong2*>(negm + r);
          float a, b, c, d;
          f32x2_unpack(f32x2_add(y2[r / 2], m4.x), a, b);
          f32x2_unpack(f32x2_add(y2[r / 2 + 1], m4.y), c, d);
          top = max3f(top, a, b);
          top = max3f(top, c, d);
        }
        grown = bar_or(kBar, kWg, failed || top > kTop + kGrow);
      }
      // The last product has read P, and O may be changed.
      if (gi > 0) failed |= !w.wait(bar(L::kPVDone), (gi - 1) & 1, code | L::kPVDone);
      if (grown) {
        // Every warp's row maxima, then m and factor of every row: m moves to the maximum of each
        // row that grew at all (moving only those that grew by more than kGrow, the others did it in
        // later tiles: 120 us instead of 115 for 8 x 16k-32k positions and 32 rows).
        tc_fence_after_sync();
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
          int mine = 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            f32x2_unpack(y2[(ch * 16 + i) / 2], a, b);
            const int m = __reduce_max_sync(0xffffffffu, ordered(i & 1 ? b : a));
            if (lane == i) mine = m;
          }
          if (lane < 16) wmax[warp * NR + ch * 16 + lane] = unordered(mine);
        }
        if (bar_or(kBar, kWg, failed)) {
          ok = false;
          break;
        }
        // Thread r < NR moves row r; every thread then applies the factors.
        if (key < NR) {
          const float mx = fmaxf(fmaxf(wmax[key], wmax[NR + key]), fmaxf(wmax[2 * NR + key], wmax[3 * NR + key]));
          const float old = negm[key];
          const bool move = mx + old > kTop && mx < INFINITY;
          const float now = move ? kTop - mx : old;
          negm_all[(mbuf ^ 1) * NR + key] = now;
          coef[key] = move ? dec_exp2(now - old) : 1.f;
        }
        bar_or(kBar, kWg, false);
        mbuf ^= 1;
        negm = negm_all + mbuf * NR;
        if (j > 0) {
#pragma unroll
          for (int r = 0; r < NR / 2; ++r) l2[r] = f32x2_mul(l2[r], *reinterpret_cast<const uint64_t*>(coef + 2 * r));
#pragma unroll 1
          for (int c = 0; c < 3 * NR; c += 16) {
            uint32_t o[16];
            const uint32_t at = lane_addr + L::kOCol + c;
            const float* f = coef + c % NR;
            tmem_load_16cols(at, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f[i]);
            tmem_store_16cols(at, o);
          }
          tmem_store_wait();
        }
      }
      // Weights, their sum, and their three E5M2 terms: a weight in fp16 (11 significant
      // bits), whose upper byte is an E5M2 number; what that leaves, likewise; the last
      // remainder rounded to nearest.
      const uint32_t p_addr = sbase + L::kPOff + key * 16;
      const uint64_t ivs2 = f32x2_pack(ivs, ivs);
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        uint32_t t1[8], t2[8], t3[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = ch * 8 + i;
          float a, b;
          f32x2_unpack(f32x2_add(y2[r], *reinterpret_cast<const uint64_t*>(negm + 2 * r)), a, b);
          a = dec_exp2(a);
          b = dec_exp2(b);
          l2[r] = f32x2_fma(f32x2_pack(a, b), ivs2, l2[r]);
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
        const uint32_t slot = gi % L::kVSlots;
        failed |= !w.wait(bar(L::kVFull + slot), (gi / L::kVSlots) & 1, code | (L::kVFull + slot));
        if (!failed && !it.seen(pos)) {
          const uint32_t at = sbase + L::kVOff + slot * L::kTileBytes + key * D;
#pragma unroll
          for (int c = 0; c < D; c += 16) st_shared_v4(at + c, 0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(L::kPFull));
        mbar_arrive(bar(L::kSFree + sb));
      }
    }
    // ---- the item's end: the last product, the sums over the keys, the rows.  In between,
    // the next item's page entries and scales are asked for.
    failed |= !ok;
    const Item8 nx = take_item8<L>(sbase, smem, w, k_item, code);
    const int npos = pos_of(nx, 0), nentry = entry_of(nx, npos);
    pos_next = pos_of(nx, 1);
    entry_next = entry_of(nx, pos_next);
    // Sixteen sums over 32 lanes: each step halves the rows a lane carries.
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) f32x2_unpack(l2[ch * 8 + i], v[2 * i], v[2 * i + 1]);
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
      if (lane < 16) wmax[warp * NR + ch * 16 + lane] = v[0];
    }
    if (n > 0) {
      failed |= !w.wait(bar(L::kPVDone), (g + n - 1) & 1, code | L::kPVDone);
      if (lane == 0) mbar_arrive(bar(L::kQEmpty + qbuf));  // this warp has read the row factors
    }
    if (bar_or(kBar, kWg, failed)) break;
    tc_fence_after_sync();
    if (key < it.rows) {
      const float top = negm_all[mbuf * NR + key];   // kTop - m
      const float sum = (wmax[key] + wmax[NR + key]) + (wmax[2 * NR + key] + wmax[3 * NR + key]);
      coef[key] = sum != 0.f ? 1.f / sum : 0.f;      // (a NaN sum stays NaN; nothing seen: zero)
      const float l2 = sum != 0.f ? __log2f(sum) - top : -INFINITY;
      if (S > 1) p.part_lse[(grow0 + key) * S + it.s] = l2;
      else p.lse[grow0 + key] = l2 * kLn2;
    }
    scales_of(nx, npos, nentry, ks, vs);
    bar_or(kBar, kWg, false);
    // Thread = column of d.  An item without tiles has no O: its rows are zero (one split), or
    // carry no weight in the merge.
    float* po = S > 1 ? p.part_o + (grow0 * S + it.s) * D + key : nullptr;
    __nv_bfloat16* ob = p.out + grow0 * D + key;
    const size_t po_step = static_cast<size_t>(S) * D;
#pragma unroll 1
    for (int r0 = 0; r0 < it.rows; r0 += 16) {
      uint32_t o[16], o2[16], o3[16];
      const uint32_t at = lane_addr + L::kOCol + r0;
      tmem_load_16cols(at, o);
      tmem_load_2x16cols(at + NR, at + 2 * NR, o2, o3);
      const int left = key < D ? it.rows - r0 : 0;
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 c4 = *reinterpret_cast<const float4*>(coef + r0 + i);
        const float cc[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[i + k] = n <= 0 ? 0.f
                            : (__uint_as_float(o[i + k]) + (__uint_as_float(o2[i + k]) + __uint_as_float(o3[i + k]))) *
                                  cc[k];
      }
      if (po) {
#pragma unroll
        for (int i = 0; i < 16; ++i, po += po_step)
          if (i < left) *po = v[i];
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i, ob += D)
          if (i < left) *ob = __float2bfloat16_rn(v[i]);
      }
    }
    if (n > 0) {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kOFree));
      g += n;
      ++items;
    }
    it = nx;
  }
}

template <int D, int NR>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) attn_decode8_kernel(const __grid_constant__ Dec8Params p) {
  using L = Smem8<D, NR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const int warp = threadIdx.x >> 5;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  volatile uint32_t* loaded = reinterpret_cast<volatile uint32_t*>(smem + L::kMiscOff + 8);
  // The merge may be set up; it waits for this grid's end.  (Without splits the next kernel is not
  // this library's: it might take tensor memory before this CTA has.)
  if (p.num_splits > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    auto bar = [&](int i) { return sbase + L::kBarOff + 8u * i; };
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::kQFull + i), 1);
      mbar_init(bar(L::kQEmpty + i), 5);  // the last S product and the softmax warps
      mbar_init(bar(L::kFin + i), 1);
    }
    mbar_init(bar(L::kPFull), 4);
    mbar_init(bar(L::kPVDone), 1);
    mbar_init(bar(L::kOFree), 4);
    for (int s = 0; s < 2 * L::kKSlots; ++s) mbar_init(bar(L::kKFull + s), 1);  // full and empty
    for (int s = 0; s < 2 * L::kVSlots; ++s) mbar_init(bar(L::kVFull + s), 1);
    for (int i = 0; i < L::kSBufs; ++i) {
      mbar_init(bar(L::kSFull + i), 1);
      mbar_init(bar(L::kSFree + i), 4);
    }
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(bar(L::kItemFull + i), 1);
      mbar_init(bar(L::kItemEmpty + i), 7);  // every warp but the K loader
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
  const DecWaiter bounded{p.timeout_ns, abort_flag, p.err};
  const Waiter8 w{&bounded};

  if (warp < 4) {
    softmax_role8<D, NR>(p, sbase, smem, tmem, w);
  } else if (warp == kKWarp || warp == kVWarp) {
    const uint32_t gt = loader8<D, NR>(p, sbase, smem, w, warp == kVWarp);
    if ((threadIdx.x & 31) == 0) loaded[warp - kKWarp] = gt;
  } else if (warp == kPvWarp) {
    pv_role8<D, NR>(p, sbase, smem, tmem, w);
  } else {
    s_role8<D, NR>(p, sbase, smem, tmem, w);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (threadIdx.x == kKWarp * 32) {
    drain_ring8(sbase + L::kBarOff + 8u * L::kKFull, L::kKSlots, bounded, loaded[0]);
    drain_ring8(sbase + L::kBarOff + 8u * L::kVFull, L::kVSlots, bounded, loaded[1]);
  }
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

// ------------------------------------------------------------ split merge
// One CTA per query row: out = sum_s w_s O_s / sum_s w_s, w_s = 2^(lse2_s - max lse2), lse = ln
// sum_s 2^lse2_s.  Warp g of W takes splits g, g + W, ..., a lane D / 32 columns; its first loads of O
// are under way while the weights are formed.  Sums in a fixed order.
struct Merge8Params {
  const float* part_o;
  const float* part_lse;
  __nv_bfloat16* out;
  float* lse;
  int num_splits;
};
constexpr int kMergeBatch = 8;  // splits of a warp whose loads are in flight together

template <int D, int W>
__global__ void __launch_bounds__(32 * W) attn_decode8_merge_kernel(const Merge8Params p) {
  constexpr int V = D / 32;
  extern __shared__ float s_w[];  // [num_splits]
  __shared__ float s_red[2][W], s_acc[W - 1][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = p.num_splits;
  const float* po = p.part_o + static_cast<size_t>(row) * S * D + lane * V;
  float o[kMergeBatch][V];
  auto load = [&](int first) {
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const int k = first + W * u;
#pragma unroll
      for (int v = 0; v < V; ++v) o[u][v] = 0.f;
      if (k < S) {
        const float* src = po + static_cast<size_t>(k) * D;
        if constexpr (V == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
          o[u][0] = x.x;
          o[u][1] = x.y;
          o[u][2] = x.z;
          o[u][3] = x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
          o[u][0] = x.x;
          o[u][1] = x.y;
        }
      }
    }
  };
  load(warp);
  float top = -INFINITY;
  for (int k = tid; k < S; k += 32 * W) {
    const float l2 = __ldcg(p.part_lse + static_cast<size_t>(row) * S + k);
    s_w[k] = l2;
    top = fmaxf(top, l2);
  }
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
  if (lane == 0) s_red[0][warp] = top;
  __syncthreads();
#pragma unroll
  for (int g = 0; g < W; ++g) top = fmaxf(top, s_red[0][g]);
  const float base = top == -INFINITY ? 0.f : top;
  float acc[V], wsum = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  for (int k0 = warp;; ) {
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const int k = k0 + W * u;
      const float w = k < S ? attn_sm100_dec::dec_exp2(s_w[k] - base) : 0.f;
      wsum += w;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(w, o[u][v], acc[v]);
    }
    k0 += W * kMergeBatch;
    if (k0 >= S) break;
    load(k0);
  }
  if (lane == 0) s_red[1][warp] = wsum;
  if (warp > 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) s_acc[warp - 1][lane * V + v] = acc[v];
  }
  __syncthreads();
  if (warp > 0) return;
  wsum = 0.f;
#pragma unroll
  for (int g = 0; g < W; ++g) wsum += s_red[1][g];
#pragma unroll
  for (int g = 0; g < W - 1; ++g) {
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] += s_acc[g][lane * V + v];
  }
  const float inv = wsum != 0.f ? 1.f / wsum : 0.f;
  __nv_bfloat16* dst = p.out + static_cast<size_t>(row) * D + lane * V;
#pragma unroll
  for (int v = 0; v < V; v += 2) {
    const float a = acc[v] * inv, b = acc[v + 1] * inv;
    *reinterpret_cast<uint32_t*>(dst + v) = attn_sm100_dec::dec_pack_bf16x2(a, b);
  }
  if (lane == 0) p.lse[row] = wsum != 0.f ? (top + __log2f(wsum)) * kLn2 : -INFINITY;
}

}  // namespace attn_sm100_dec8
