// The write side of the paged KV cache declared in include/attn.h: new tokens' keys and
// values go into their sequences' pages, the keys (and the queries of the same tokens)
// rotated by their positions on the way; the cache holds bf16 values or E4M3 codes with a
// power-of-two scale for each block of tokens and head.
//
// Rotation of a pair (a, b) at position x with frequency f: (a c - b s, b c + a s) with
// c = cos(x f), s = sin(x f).  An angle of a far position (2^17 and more) needs more bits
// than fp32 has: x f is formed in fp64 as turns, x f / 2 pi, whose distance from the
// nearest whole turn (at most a half) goes to fp32, and what that rounding loses turns the result
// once more, so cos and sin are good to about one fp32 rounding at every position.  The rotation itself is fp32, rounded once (to bf16, or
// to the E4M3 code).
//
// Scales are powers of two (the smallest s >= 2^-40 with amax <= 448 s): E4M3 is a floating
// format, so a finer scale would only shift its exponent window, while with powers of two
// the division x / s is exact and raising a block's scale only moves its older codes'
// exponents (a code is rounded again only where it turns subnormal).
//
// What bounds it: HBM for prefill chunks (every row is read once and written once), the
// latency of the chain length -> page -> store for a decoding step's few rows.  One CTA
// takes one unit: the new tokens of one sequence that fall into one aligned run of `unit`
// slots (a block, or 16 or 32 slots), so a block's largest magnitude is found inside one CTA, in
// a fixed order, without atomics.  The unit's cos / sin table is computed once into shared
// memory; a group of D / 16 lanes takes a token's 16-element pieces of one head after another
// with that token's cosines in registers, four heads' loads in flight.  (Rows dealt to the
// groups head by head read the table anew for each, four lanes on a bank: 137 us instead of
// 112 us for 16384 tokens of 64/8 heads.)  The heads are dealt over gridDim.y when there are
// few units.  Measured: that chunk at 6000 GB/s, 92 % of a copy's; 8191 tokens of 32/8 heads
// into E4M3 blocks of 16 in 44.2 us, 63 % (queries alone run at 80 %; a block's codes wait for
// the maximum of 16 rows, a barrier a head).
#include "attn.h"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "sm100_ptx.cuh"

namespace attn_sm100_app {
using namespace attn_sm100;

constexpr int kAppThreads = 256;
constexpr int kErrSeq = 1 << 20;   // a sequence's length or token range is unusable
constexpr int kErrPage = 2 << 20;  // a page-table entry the call needs is out of range

// Device error word (read and cleared by attn_kv_append_debug_error).
__device__ int g_attn_app_error;

struct AppParams {
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements from token to token
  __nv_bfloat16* q_out;
  void *k_cache, *v_cache;               // bf16 values or E4M3 codes
  float *k_scale, *v_scale;
  const int *block_table, *seq_lens, *cu_tokens, *positions;
  const float* inv_freq;
  int* err;
  int64_t T;
  int B, Hq, Hkv, half;                  // half = rotated pairs
  int interleaved;
  int page_size, num_pages, max_pages;
  int unit;                              // slots of a unit (a multiple of block)
  int block;                             // slots that share a scale
  int per_seq;                           // equal sequences: tokens of each (0: cu_tokens)
  int units_per_seq;                     // equal sequences: upper bound
};

struct Unit {
  int b;
  int t0, n;     // first token row of the unit, number of new tokens in it (-1 - j: unit j of an idle slot)
  int slot0;     // slot of the first new token inside the unit
  int pos0;      // position of the first new token
  int64_t page;  // physical page, -1 if unusable
  int in_page;   // first slot of the unit inside its page
  int first;     // the sequence's first token row
};

// Which tokens CTA `idx` takes; n = 0 when there are none.  Called by the whole CTA, every
// thread of which gets the answer.
__device__ __forceinline__ Unit find_unit(const AppParams& p, int idx) {
  Unit u{0, 0, 0, 0, 0, -1, 0, 0};
  const int tid = threadIdx.x;
  int len = 0, n = 0, first = 0, j = 0;
  if (p.per_seq) {
    u.b = idx / p.units_per_seq;
    j = idx - u.b * p.units_per_seq;
    n = p.per_seq;
    first = u.b * n;
    len = __ldg(p.seq_lens + u.b);
    if (len == 0) {
      u.n = -1 - j;
      return u;
    }
    if (len < n || len > p.max_pages * p.page_size) {
      if (tid == 0) atomicCAS(p.err, 0, kErrSeq | (u.b & 0xFFFFF));
      return u;
    }
    if (j > (len - 1) / p.unit - (len - n) / p.unit) return u;
  } else {
    // Units are numbered sequence by sequence: a running count, a thread a sequence.  (A warp's
    // count, 32 sequences at a time, took 82 us for 1024 sequences of one token, this 26.)
    __shared__ int s_cnt[kAppThreads / 32], s_found[5];
    const int lane = tid & 31, warp = tid >> 5;
    int before = 0;
    bool found = false;
    for (int b0 = 0; b0 < p.B && !found; b0 += kAppThreads) {
      const int b = b0 + tid;
      int l = 0, c0 = 0, m = 0, cnt = 0;
      if (b < p.B) {
        c0 = __ldg(p.cu_tokens + b);
        const int c1 = __ldg(p.cu_tokens + b + 1);
        l = __ldg(p.seq_lens + b);
        m = c1 - c0;
        if (c0 < 0 || m < 0 || c1 > p.T || (m > 0 && (l < m || l > p.max_pages * p.page_size))) {
          atomicCAS(p.err, 0, kErrSeq | (b & 0xFFFFF));
        } else if (m > 0) {
          cnt = (l - 1) / p.unit - (l - m) / p.unit + 1;
        }
      }
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) s_cnt[warp] = incl;
      __syncthreads();
      int total = 0;
#pragma unroll
      for (int w = 0; w < kAppThreads / 32; ++w) {
        if (w == warp) incl += total;
        total += s_cnt[w];
      }
      const int at = idx - before - (incl - cnt);  // the unit's number in this sequence
      if (at >= 0 && at < cnt) {
        s_found[0] = b;
        s_found[1] = l;
        s_found[2] = m;
        s_found[3] = c0;
        s_found[4] = at;
      }
      __syncthreads();
      found = idx < before + total;
      before += total;
    }
    if (!found) return u;
    u.b = s_found[0];
    len = s_found[1];
    n = s_found[2];
    first = s_found[3];
    j = s_found[4];
  }
  const int p0 = len - n;                            // position of the sequence's first new token
  const int run = (p0 / p.unit + j) * p.unit;        // first position of the unit
  u.pos0 = max(run, p0);
  u.n = min(run + p.unit, len) - u.pos0;
  u.slot0 = u.pos0 - run;
  u.first = first;
  u.t0 = first + (u.pos0 - p0);
  u.in_page = run % p.page_size;
  const int entry = __ldg(p.block_table + static_cast<int64_t>(u.b) * p.max_pages + run / p.page_size);
  if (entry >= 0 && entry < p.num_pages) {
    u.page = entry;
  } else if (tid == 0) {
    atomicCAS(p.err, 0, kErrPage | (u.b & 0xFFFFF));
  }
  return u;
}

__device__ __forceinline__ void widen8(const uint4& w, float (&x)[8]) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(r[i] << 16);
    x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
  return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}

// Element offsets of the two 8-element chunks of lane c of a row (D / 16 lanes): chunk
// pairs (8c, half + 8c) in the rotated part of the half-split form; elsewhere, and in the
// interleaved form, 16 consecutive elements.
__device__ __forceinline__ void chunk_at(const AppParams& p, int c, int& lo, int& hi) {
  if (!p.interleaved && 8 * c < p.half) {
    lo = 8 * c;
    hi = p.half + 8 * c;
  } else {
    lo = 16 * c;
    hi = 16 * c + 8;
  }
}

// The table's entry of token t and pair f: the pairs 8c + i of lanes c = 0, 1, ... are
// neighbours, and tokens lie 64 bytes apart in the banks, so that the lanes of a warp read
// without conflicts.
__device__ __forceinline__ int cs_at(const AppParams& p, int t, int f) {
  return t * (p.half + 8) + (f & 7) * (p.half / 8) + (f >> 3);
}
__device__ __forceinline__ void read_cs(const AppParams& p, const float2* table, int t, int c, float2 (&cs)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = table[cs_at(p, t, 8 * c + i)];
}
// Rotates a lane's 16 elements in place; cs = the token's (cos, sin) of pairs 8c .. 8c + 7.
__device__ __forceinline__ void rotate16(bool interleaved, const float2 (&cs)[8], float (&a)[8], float (&b)[8]) {
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i];
      a[i] = x * cs[i].x - y * cs[i].y;
      b[i] = y * cs[i].x + x * cs[i].y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float x = a[i], y = a[i + 1], z = b[i], w = b[i + 1];
      const float2 c0 = cs[i / 2], c1 = cs[4 + i / 2];
      a[i] = x * c0.x - y * c0.y;
      a[i + 1] = y * c0.x + x * c0.y;
      b[i] = z * c1.x - w * c1.y;
      b[i + 1] = w * c1.x + z * c1.y;
    }
  }
}

// The smallest power of two s >= 2^-40 with amax <= 448 s (amax finite): 448 = 1.75 * 2^8.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 127 - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return __uint_as_float(static_cast<uint32_t>(max(e, -40) + 127) << 23);
}
// Largest finite magnitude of a lane's 16 values: NaN and infinities do not set a scale.  (NaN
// loses against any number; an infinity, rare, is taken out in a second look.)
__device__ __forceinline__ float largest16(const float (&a)[8], const float (&b)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max3f(m, fabsf(a[i]), fabsf(b[i]));
  if (m > 3.402823466e38f) {
    m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = fabsf(a[i]), y = fabsf(b[i]);
      m = max3f(m, x <= 3.402823466e38f ? x : 0.f, y <= 3.402823466e38f ? y : 0.f);
    }
  }
  return m;
}
// The division by a kept scale that is no power of two, which only a caller brings: out of line
// (sixteen divisions in the row loop made it too large for the instruction cache).
__device__ __noinline__ float quotient(float x, float s) { return __fdiv_rn(x, s); }
// A lane's 16 values to E4M3 codes of x / s at two places; s is nearly always a power of two,
// and x (1 / s) the quotient.
__device__ __forceinline__ void encode16(float (&a)[8], float (&b)[8], float s, uint8_t* at_a, uint8_t* at_b) {
  if ((__float_as_uint(s) & 0x7fffffu) == 0) {
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] *= inv;
      b[i] *= inv;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = quotient(a[i], s);
      b[i] = quotient(b[i], s);
    }
  }
  *reinterpret_cast<uint2*>(at_a) =
      make_uint2(pack_e4m3x4(a[0], a[1], a[2], a[3]), pack_e4m3x4(a[4], a[5], a[6], a[7]));
  *reinterpret_cast<uint2*>(at_b) =
      make_uint2(pack_e4m3x4(b[0], b[1], b[2], b[3]), pack_e4m3x4(b[4], b[5], b[6], b[7]));
}
// Sixteen codes in place, under a scale that is 1 / ratio times theirs.
__device__ __forceinline__ void recode16(uint8_t* codes, float ratio) {
  uint4* at = reinterpret_cast<uint4*>(codes);
  const uint4 w = *at;
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x0, x1, x2, x3;
    e4m3x4_values(in[i], x0, x1, x2, x3);
    out[i] = pack_e4m3x4(x0 * ratio, x1 * ratio, x2 * ratio, x3 * ratio);
  }
  *at = make_uint4(out[0], out[1], out[2], out[3]);
}

// What a CTA's unit is, and how it goes through the heads.  kBf16: 16 slots, no scales.  kSmall,
// kSmall2: 16 or 32 slots in blocks of up to 16; kBlock2, kBlock4: one block of 32 or 64; their
// rows stay in registers between the block's maximum and its codes.  kBlock8: one block of 128
// or 256, read twice.
enum Mode { kBf16, kSmall, kSmall2, kBlock2, kBlock4, kBlock8 };

// CTAs of an SM.  Most of these kernels' time is latency, so their registers are kept to what lets
// several CTAs in, as measured: 8191 tokens of 8 heads into blocks of 16 took 31 us at two
// CTAs, 28 at three, 33 at four (spilling).
constexpr int ctas_per_sm(int mode) {
  return mode == kSmall ? 3 : mode == kSmall2 || mode == kBlock2 || mode == kBlock4 ? 2 : 1;
}

// An idle slot's queries are zeros, its CTAs sharing the rows: the decoding step does not read them,
// but what the caller is handed is defined.
template <int D>
__device__ __noinline__ void zero_queries(const AppParams& p, int b, int unit) {
  const int64_t pieces = static_cast<int64_t>(p.Hq) * p.per_seq * (D / 8);
  uint4* dst = reinterpret_cast<uint4*>(p.q_out) + b * pieces;
  const int64_t cta = static_cast<int64_t>(unit) * gridDim.y + blockIdx.y;
  const int64_t ctas = static_cast<int64_t>(p.units_per_seq) * gridDim.y;
  for (int64_t i = cta * kAppThreads + threadIdx.x; i < pieces; i += ctas * kAppThreads) dst[i] = make_uint4(0u, 0u, 0u, 0u);
}

template <int D, int MODE>
__global__ void __launch_bounds__(kAppThreads, ctas_per_sm(MODE))
    attn_append_kernel(const __grid_constant__ AppParams p) {
  constexpr int G = D / 16;                  // lanes of a row
  constexpr int kRows = kAppThreads / G;     // rows a pass of the CTA takes
  extern __shared__ float2 s_cs[];           // (cos, sin) of the unit's tokens and pairs, see cs_at
  __shared__ float s_amax[2][kAppThreads / 32];
  __shared__ float s_row[2][2][kRows];       // largest magnitudes of a head's rows, in turn
  const int tid = threadIdx.x, lane = tid & 31;
  const Unit u = find_unit(p, blockIdx.x);
  if (u.n <= 0) {
    if (u.n < 0 && p.q) zero_queries<D>(p, u.b, -1 - u.n);
    return;
  }
  for (int i = tid; i < u.n * p.half; i += kAppThreads) {
    const int t = i / p.half, f = i - t * p.half;
    const int pos = p.positions ? __ldg(p.positions + u.t0 + t) : u.pos0 + t;
    const double turns = static_cast<double>(pos) * static_cast<double>(__ldg(p.inv_freq + f)) * 0.15915494309189535;
    const double part = turns - rint(turns);
    const float r = static_cast<float>(part);
    const float rest = static_cast<float>((part - r) * 6.283185307179586);  // radians that r lost
    float sn, cn;
    sincospif(2.f * r, &sn, &cn);
    s_cs[cs_at(p, t, f)] = make_float2(fmaf(-sn, rest, cn), fmaf(cn, rest, sn));
  }
  __syncthreads();
  const int c = tid % G, g = tid / G;
  int at_lo, at_hi;
  chunk_at(p, c, at_lo, at_hi);
  const bool turn = 8 * c < p.half;
  const int parts = gridDim.y, part = blockIdx.y;

  // Groups of lanes: `nt` tokens at a time (a power of two), kRows / nt groups for each.
  int nt = 1;
  while (nt < kRows && nt < u.n) nt *= 2;
  const int tg = g % nt, hg = g / nt, hstep = kRows / nt;
  // Rows (t, h), h0 <= h < h1, of one tensor: src_of and dst_of give a row's place.
  auto sweep = [&](int h0, int h1, bool rotate, auto src_of, auto dst_of) {
    for (int t = tg; t < u.n; t += nt) {
      float2 cs[8];
      if (rotate) read_cs(p, s_cs, t, c, cs);
      for (int h = h0 + hg; h < h1; h += 4 * hstep) {
        uint4 lo[4], hi[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (h + k * hstep < h1) {
            const __nv_bfloat16* src = src_of(t, h + k * hstep);
            lo[k] = __ldg(reinterpret_cast<const uint4*>(src + at_lo));
            hi[k] = __ldg(reinterpret_cast<const uint4*>(src + at_hi));
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (h + k * hstep < h1) {
            if (rotate) {
              float a[8], b[8];
              widen8(lo[k], a);
              widen8(hi[k], b);
              rotate16(p.interleaved, cs, a, b);
              lo[k] = narrow8(a);
              hi[k] = narrow8(b);
            }
            __nv_bfloat16* dst = dst_of(t, h + k * hstep);
            *reinterpret_cast<uint4*>(dst + at_lo) = lo[k];
            *reinterpret_cast<uint4*>(dst + at_hi) = hi[k];
          }
        }
      }
    }
  };

  // Queries: rotated into the decoding step's layout [B, Hq, Nq, d] (equal sequences) or
  // left token-major.
  if (p.q) {
    const int h0 = static_cast<int>(static_cast<int64_t>(p.Hq) * part / parts);
    const int h1 = static_cast<int>(static_cast<int64_t>(p.Hq) * (part + 1) / parts);
    const int64_t row0 = p.per_seq ? static_cast<int64_t>(u.b) * p.Hq * p.per_seq + (u.t0 - u.first)
                                   : static_cast<int64_t>(u.t0) * p.Hq;
    const int64_t row_t = p.per_seq ? 1 : p.Hq, row_h = p.per_seq ? p.per_seq : 1;
    sweep(h0, h1, turn, [&](int t, int h) { return p.q + (u.t0 + t) * p.q_stride + h * D; },
          [&](int t, int h) { return p.q_out + (row0 + t * row_t + h * row_h) * D; });
  }
  if (u.page < 0) return;
  const int h0 = static_cast<int>(static_cast<int64_t>(p.Hkv) * part / parts);
  const int h1 = static_cast<int>(static_cast<int64_t>(p.Hkv) * (part + 1) / parts);
  if constexpr (MODE == kBf16) {
    for (int kv = 0; kv < 2; ++kv) {
      const __nv_bfloat16* base = kv ? p.v : p.k;
      const int64_t stride = kv ? p.v_stride : p.k_stride;
      __nv_bfloat16* cache = static_cast<__nv_bfloat16*>(kv ? p.v_cache : p.k_cache) +
                             (u.page * p.Hkv * p.page_size + u.in_page + u.slot0) * D;
      sweep(h0, h1, !kv && turn, [&](int t, int h) { return base + (u.t0 + t) * stride + h * D; },
            [&](int t, int h) { return cache + (static_cast<int64_t>(h) * p.page_size + t) * D; });
    }
  } else if constexpr (MODE != kBlock8) {
    // Half of the CTA takes K and half V; a group of lanes takes slots slot, slot + 16, ... of
    // the unit, one head after another (with d = 64, every other head), the next head's rows
    // and scales asked for ahead.  The largest magnitudes of a head's rows go to shared
    // memory, and a block's is the largest of its rows': one barrier a head.
    constexpr int kPass = kRows / 2, kHeads = kPass / 16;
    constexpr int kR = MODE == kSmall ? 1 : MODE == kBlock4 ? 4 : 2;  // rows of a thread
    constexpr bool kOne = MODE == kBlock2 || MODE == kBlock4;         // ... of one block, or each of its own
    constexpr int kB = kOne ? 1 : kR;
    constexpr bool kAhead = MODE != kBlock4;                          // (64 registers more)
    const int kv = g / kPass, slot = g % kPass % 16, hs = g % kPass / 16;
    const __nv_bfloat16* base = (kv ? p.v : p.k);
    const int64_t stride = kv ? p.v_stride : p.k_stride;
    float* scales = kv ? p.v_scale : p.k_scale;
    const int blocks_per_page = p.page_size / p.block;
    const int in16 = kOne ? 0 : slot & ~(p.block - 1);
    auto b0 = [&](int k) { return 16 * k + in16; };                   // block k of this thread: its first slot,
    auto first = [&](int k) { return max(b0(k), u.slot0); };          // its first new one,
    auto has_new = [&](int k) { return b0(k) + p.block > u.slot0 && b0(k) < u.slot0 + u.n; };
    auto held = [&](int k) { return has_new(k) && u.slot0 > b0(k); }; // and whether it held tokens before
    auto scale_at = [&](int h, int k) {
      return scales + (u.page * p.Hkv + h) * blocks_per_page + (u.in_page + b0(k)) / p.block;
    };
    auto fresh = [&](int r) { return slot + 16 * r >= u.slot0 && slot + 16 * r < u.slot0 + u.n; };
    const bool rotate = !kv && turn;
    float2 cs[8];
    if (kR == 1 && rotate && fresh(0)) read_cs(p, s_cs, slot - u.slot0, c, cs);
    const __nv_bfloat16* src = base + (u.t0 + slot - u.slot0) * stride;
    uint8_t* rows = static_cast<uint8_t*>(kv ? p.v_cache : p.k_cache) +
                    (u.page * p.Hkv * p.page_size + u.in_page + slot) * D;
    struct Rows {
      uint4 lo[kR], hi[kR];
      float old[kB];
    };
    auto ask = [&](int h, Rows& x) {
#pragma unroll
      for (int k = 0; k < kB; ++k) x.old[k] = h < h1 && held(k) ? *scale_at(h, k) : 0.f;
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (h < h1 && fresh(r)) {
          x.lo[r] = __ldg(reinterpret_cast<const uint4*>(src + 16 * r * stride + h * D + at_lo));
          x.hi[r] = __ldg(reinterpret_cast<const uint4*>(src + 16 * r * stride + h * D + at_hi));
        }
      }
    };
    auto values = [&](const Rows& x, int r, float (&a)[8], float (&b)[8]) {
      widen8(x.lo[r], a);
      widen8(x.hi[r], b);
      if (rotate) {
        if (kR > 1) read_cs(p, s_cs, slot + 16 * r - u.slot0, c, cs);
        rotate16(p.interleaved, cs, a, b);
      }
    };
    int par = 0;
    Rows x, next;
    if (kAhead) ask(h0 + hs, next);
#pragma unroll 1
    for (int h = h0 + hs; h - hs < h1; h += kHeads, par ^= 1) {
      if (kAhead) {
        x = next;
        ask(h + kHeads, next);
      } else {
        ask(h, x);
      }
      float amax[kB] = {};
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (h < h1 && fresh(r)) {
          float a[8], b[8];
          values(x, r, a, b);
          amax[r % kB] = fmaxf(amax[r % kB], largest16(a, b));
        }
      }
#pragma unroll
      for (int k = 0; k < kB; ++k) {
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) amax[k] = fmaxf(amax[k], __shfl_xor_sync(0xffffffffu, amax[k], o));
        if (c == 0) s_row[par][k][g] = amax[k];
      }
      __syncthreads();  // (also: every thread has read this head's old scales)
#pragma unroll
      for (int k = 0; k < kB; ++k) {
        if (!has_new(k) || h >= h1) continue;
        float top = 0.f;
        const float* rowmax = &s_row[par][k][g - slot + in16];
        if (kOne || p.block == 16) {
#pragma unroll
          for (int r = 0; r < 16; ++r) top = fmaxf(top, rowmax[r]);
        } else {
          for (int r = 0; r < p.block; ++r) top = fmaxf(top, rowmax[r]);
        }
        const float old = x.old[k];
        const bool keep = held(k) && old >= 1.17549435e-38f && top <= 448.f * old;
        const float s = keep ? old : block_scale(top);
        uint8_t* dst = rows + static_cast<int64_t>(h) * p.page_size * D;
#pragma unroll
        for (int r = k; r < kR; r += kB) {
          if (fresh(r)) {
            float a[8], b[8];
            values(x, r, a, b);
            encode16(a, b, s, dst + 16 * r * D + at_lo, dst + 16 * r * D + at_hi);
          } else if (!keep && slot + 16 * r < u.slot0) {
            recode16(dst + 16 * r * D + 16 * c, old / s);
          }
          if (!keep && c == 0 && slot + 16 * r == first(k)) *scale_at(h, k) = s;
        }
      }
    }
  } else {
    // One block; half of the CTA takes K and half V, and each head's rows are read twice, for the
    // largest magnitude and for the codes.
    constexpr int kPass = kRows / 2;
    const int kv = g / kPass, r0 = g - kv * kPass;
    const __nv_bfloat16* base = kv ? p.v : p.k;
    const int64_t stride = kv ? p.v_stride : p.k_stride;
    uint8_t* cache = static_cast<uint8_t*>(kv ? p.v_cache : p.k_cache);
    float* scales = kv ? p.v_scale : p.k_scale;
    const int blocks_per_page = p.page_size / p.block;
    auto load = [&](int t, int h, float (&a)[8], float (&b)[8]) {
      const __nv_bfloat16* src = base + (u.t0 + t) * stride + h * D;
      widen8(__ldg(reinterpret_cast<const uint4*>(src + at_lo)), a);
      widen8(__ldg(reinterpret_cast<const uint4*>(src + at_hi)), b);
      if (!kv && turn) {
        float2 cs[8];
        read_cs(p, s_cs, t, c, cs);
        rotate16(p.interleaved, cs, a, b);
      }
    };
    for (int h = h0; h < h1; ++h) {
      for (int s0 = u.slot0 / p.block * p.block; s0 < u.slot0 + u.n; s0 += p.block) {
        const int ta = max(s0 - u.slot0, 0), tb = min(s0 + p.block - u.slot0, u.n);  // its new tokens [ta, tb)
        const int held = max(u.slot0 - s0, 0);                                      // slots filled before
        float amax = 0.f;
        for (int t = ta + r0; t < tb; t += kPass) {
          float a[8], b[8];
          load(t, h, a, b);
          amax = fmaxf(amax, largest16(a, b));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        __syncthreads();  // the previous block's maxima have been read
        if (lane == 0) s_amax[kv][tid / 32] = amax;
        __syncthreads();
        constexpr int kHalfWarps = kAppThreads / 64;
        amax = 0.f;
#pragma unroll
        for (int w = 0; w < kHalfWarps; ++w) amax = fmaxf(amax, s_amax[kv][kv * kHalfWarps + w]);
        const int64_t head = u.page * p.Hkv + h;
        float* sc = scales + head * blocks_per_page + (u.in_page + s0) / p.block;
        const float old = held ? *sc : 0.f;
        const bool keep = held && old >= 1.17549435e-38f && amax <= 448.f * old;
        const float s = keep ? old : block_scale(amax);
        uint8_t* rows = cache + (head * p.page_size + u.in_page) * D;
        for (int t = ta + r0; t < tb; t += kPass) {
          float a[8], b[8];
          load(t, h, a, b);
          uint8_t* dst = rows + (u.slot0 + t) * D;
          encode16(a, b, s, dst + at_lo, dst + at_hi);
        }
        if (held && !keep) {
          // Codes that were here before, under the new scale.
          const float ratio = old / s;
          for (int r = r0; r < held; r += kPass) recode16(rows + (s0 + r) * D + 16 * c, ratio);
        }
        if (held) __syncthreads();  // every thread has read the old scale
        if (!keep && r0 == 0 && c == 0) *sc = s;
      }
    }
  }
}

}  // namespace attn_sm100_app

using namespace attn_sm100_app;

namespace {

constexpr int kMaxDevices = 64;
struct AppDevice {
  bool probed = false;
  bool supported = false;
  int sm_count = 0;
  int* err_word = nullptr;
};
std::mutex g_app_mutex;
AppDevice g_app_dev[kMaxDevices];

template <int D, int MODE>
bool allow_smem(int bytes) {
  return cudaFuncSetAttribute(attn_append_kernel<D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) ==
         cudaSuccess;
}

template <int D>
cudaError_t launch_append(const AppParams& p, int mode, dim3 grid, size_t smem, cudaStream_t stream) {
  switch (mode) {
    case kBf16: attn_append_kernel<D, kBf16><<<grid, kAppThreads, smem, stream>>>(p); break;
    case kSmall: attn_append_kernel<D, kSmall><<<grid, kAppThreads, smem, stream>>>(p); break;
    case kSmall2: attn_append_kernel<D, kSmall2><<<grid, kAppThreads, smem, stream>>>(p); break;
    case kBlock2: attn_append_kernel<D, kBlock2><<<grid, kAppThreads, smem, stream>>>(p); break;
    case kBlock4: attn_append_kernel<D, kBlock4><<<grid, kAppThreads, smem, stream>>>(p); break;
    default: attn_append_kernel<D, kBlock8><<<grid, kAppThreads, smem, stream>>>(p); break;
  }
  return cudaGetLastError();
}

int app_device_setup(AppDevice& out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_app_mutex);
  AppDevice& info = g_app_dev[dev];
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
      if (cudaGetSymbolAddress(&addr, g_attn_app_error) != cudaSuccess) return ATTN_ERR_CUDA;
      info.err_word = static_cast<int*>(addr);
      // a unit of 256 slots: 256 x (d/2 + 8) entries of 8 bytes
      if (!allow_smem<64, kBlock8>(256 * 40 * 8) || !allow_smem<128, kBlock8>(256 * 72 * 8)) return ATTN_ERR_CUDA;
    }
    info.probed = true;
  }
  out = info;
  return info.supported ? ATTN_OK : ATTN_ERR_UNSUPPORTED;
}

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + nb && pb < pa + na;
}
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

extern "C" int attn_kv_append(const attn_kv_append_args* a, cudaStream_t stream) {
  if (!a) return ATTN_ERR_INVALID_ARG;
  const bool fp8 = a->scale_block != 0;
  if ((a->T > 0 && (!a->k || !a->v)) || !a->k_cache || !a->v_cache || !a->block_table || !a->seq_lens)
    return ATTN_ERR_INVALID_ARG;
  if (fp8 != (a->k_scale != nullptr) || fp8 != (a->v_scale != nullptr)) return ATTN_ERR_INVALID_ARG;
  if (a->T > 0 && (a->q != nullptr) != (a->q_out != nullptr)) return ATTN_ERR_INVALID_ARG;
  if (a->B < 1 || a->T < 0 || a->Hkv < 1 || (a->q && a->Hq < 1) || a->num_pages < 1 || a->max_pages_per_seq < 1)
    return ATTN_ERR_INVALID_ARG;
  if (!a->cu_tokens && a->T % a->B != 0) return ATTN_ERR_INVALID_ARG;
  if (a->d != 64 && a->d != 128) return ATTN_ERR_UNSUPPORTED;
  const int64_t ps = a->page_size;
  if (ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256) return ATTN_ERR_UNSUPPORTED;
  if (a->rot_dim < 0 || a->rot_dim > a->d || (a->rot_dim > 0) != (a->inv_freq != nullptr)) return ATTN_ERR_INVALID_ARG;
  if (a->rot_dim % 16 != 0) return ATTN_ERR_UNSUPPORTED;
  if (fp8 && (a->scale_block < 1 || a->scale_block > ps || (a->scale_block & (a->scale_block - 1)) != 0))
    return ATTN_ERR_INVALID_ARG;
  const int64_t Hq = a->q ? a->Hq : 0, lim = 0x7fffffff;
  if (a->T > lim || a->B > (int64_t(1) << 30) || Hq > (int64_t(1) << 20) || a->Hkv > (int64_t(1) << 20) ||
      a->num_pages > lim / a->Hkv || a->max_pages_per_seq > lim / ps || a->B > lim / a->max_pages_per_seq)
    return ATTN_ERR_INVALID_ARG;
  if (a->k_stride < a->Hkv * a->d || a->v_stride < a->Hkv * a->d || (a->q && a->q_stride < Hq * a->d) ||
      a->k_stride > (int64_t(1) << 31) || a->v_stride > (int64_t(1) << 31) ||
      (a->q && a->q_stride > (int64_t(1) << 31)))
    return ATTN_ERR_INVALID_ARG;
  if (a->k_stride % 8 != 0 || a->v_stride % 8 != 0 || (a->q && a->q_stride % 8 != 0)) return ATTN_ERR_MISALIGNED;
  if (!aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->q, 16) || !aligned(a->q_out, 16) ||
      !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) || !aligned(a->k_scale, 4) || !aligned(a->v_scale, 4) ||
      !aligned(a->block_table, 4) || !aligned(a->seq_lens, 4) || !aligned(a->cu_tokens, 4) ||
      !aligned(a->positions, 4) || !aligned(a->inv_freq, 4))
    return ATTN_ERR_MISALIGNED;
  // Everything written must lie apart from everything else.
  const size_t cache = static_cast<size_t>(a->num_pages) * a->Hkv * ps * a->d * (fp8 ? 1 : 2);
  const size_t scale = fp8 ? static_cast<size_t>(a->num_pages) * a->Hkv * (ps / a->scale_block) * 4 : 0;
  auto span = [&](int64_t stride, int64_t heads) -> size_t {
    return a->T ? static_cast<size_t>((a->T - 1) * stride + heads * a->d) * 2 : 0;
  };
  const void* outs[5] = {a->k_cache, a->v_cache, a->k_scale, a->v_scale, a->q_out};
  const size_t out_sz[5] = {cache, cache, scale, scale, static_cast<size_t>(a->T) * Hq * a->d * 2};
  const void* ins[8] = {a->k, a->v, a->q, a->block_table, a->seq_lens, a->cu_tokens, a->positions, a->inv_freq};
  const size_t in_sz[8] = {span(a->k_stride, a->Hkv), span(a->v_stride, a->Hkv), a->q ? span(a->q_stride, Hq) : 0,
                           static_cast<size_t>(a->B) * a->max_pages_per_seq * 4, static_cast<size_t>(a->B) * 4,
                           static_cast<size_t>(a->B + 1) * 4, static_cast<size_t>(a->T) * 4,
                           static_cast<size_t>(a->rot_dim) * 2};
  for (int o = 0; o < 5; ++o) {
    for (int i = 0; i < 8; ++i)
      if (overlaps(outs[o], out_sz[o], ins[i], in_sz[i])) return ATTN_ERR_INVALID_ARG;
    for (int o2 = o + 1; o2 < 5; ++o2)
      if (overlaps(outs[o], out_sz[o], outs[o2], out_sz[o2])) return ATTN_ERR_INVALID_ARG;
  }

  AppDevice dev;
  const int st = app_device_setup(dev);
  if (st != ATTN_OK) return st;
  if (a->T == 0) return ATTN_OK;

  AppParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.k = static_cast<const __nv_bfloat16*>(a->k);
  p.v = static_cast<const __nv_bfloat16*>(a->v);
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.v_stride = a->v_stride;
  p.q_out = static_cast<__nv_bfloat16*>(a->q_out);
  p.k_cache = a->k_cache;
  p.v_cache = a->v_cache;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.block_table = a->block_table;
  p.seq_lens = a->seq_lens;
  p.cu_tokens = a->cu_tokens;
  p.positions = a->positions;
  p.inv_freq = a->inv_freq;
  p.err = dev.err_word;
  p.T = a->T;
  p.B = static_cast<int>(a->B);
  p.Hq = static_cast<int>(Hq);
  p.Hkv = static_cast<int>(a->Hkv);
  p.half = static_cast<int>(a->rot_dim / 2);
  p.interleaved = a->interleaved ? 1 : 0;
  p.page_size = static_cast<int>(ps);
  p.num_pages = static_cast<int>(a->num_pages);
  p.max_pages = static_cast<int>(a->max_pages_per_seq);
  p.block = static_cast<int>(fp8 ? a->scale_block : 16);
  p.per_seq = a->cu_tokens ? 0 : static_cast<int>(a->T / a->B);
  // Small blocks go two runs of 16 at a time where pages allow it, there are tokens enough for every
  // SM and no more heads than keep the CTAs short: half the look-ups and cosine tables (8191 tokens
  // into blocks of 16: 24.7 us instead of 28.0 with 8 heads, 44 and 44 with 16, 79 and 70 with 32).
  const bool two = fp8 && p.block <= 16 && ps >= 32 && a->Hkv <= 16 && a->T / 32 >= dev.sm_count;
  p.unit = two ? 32 : std::max(p.block, 16);
  // A run of n positions touches at most (n - 2 + unit) / unit + 1 units.
  int64_t units;
  if (p.per_seq) {
    p.units_per_seq = (p.per_seq - 2 + p.unit) / p.unit + 1;
    units = a->B * p.units_per_seq;
  } else {
    units = (a->T + p.unit - 1) / p.unit + std::min<int64_t>(a->B, a->T) * 2;
  }
  if (units > lim) return ATTN_ERR_INVALID_ARG;
  // Few units: the heads are dealt evenly over several CTAs of a unit, up to about two CTAs per
  // SM.  (Four per SM: 15.5 us instead of 10.4 for 2048 tokens of 32/8 heads; each CTA computes its
  // unit's cosines.)  Units of 16 slots of codes are split in two up to four units per SM, whose
  // second wave would be nearly empty: 68 us instead of 78 for 8191 tokens of 32 KV heads.
  const int64_t want = std::max<int64_t>(fp8 && p.unit == 16 && units < 4 * dev.sm_count ? 2 : 1,
                                         2 * dev.sm_count / units);
  const int64_t part_heads = std::max<int64_t>(1, a->Hkv / want);
  const int64_t parts = std::min<int64_t>((a->Hkv + part_heads - 1) / part_heads, 65535);
  const dim3 grid(static_cast<unsigned>(units), static_cast<unsigned>(parts));
  const size_t smem = static_cast<size_t>(p.unit) * (p.half + 8) * sizeof(float2);
  const int mode = !fp8              ? kBf16
                   : two             ? kSmall2
                   : p.unit == 16    ? kSmall
                   : p.unit == 32    ? kBlock2
                   : p.unit == 64    ? kBlock4
                                     : kBlock8;
  return (a->d == 64 ? launch_append<64>(p, mode, grid, smem, stream)
                     : launch_append<128>(p, mode, grid, smem, stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

extern "C" int attn_kv_append_debug_error(cudaStream_t stream, int* device_code) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ATTN_ERR_CUDA;
  AppDevice dev;
  const int st = app_device_setup(dev);
  if (st != ATTN_OK) return st;
  int code = 0;
  if (cudaMemcpy(&code, dev.err_word, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return ATTN_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpy(dev.err_word, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return ATTN_ERR_CUDA;
  if (device_code) *device_code = code;
  return code ? ATTN_ERR_INVALID_ARG : ATTN_OK;
}
