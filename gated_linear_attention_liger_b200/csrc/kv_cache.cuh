// kv_cache.cuh -- the paged 8-bit key/value cache of the hybrid's standard attention layer:
// block assignment (block tables and slot maps from request lengths) and the quantising append.
//
//   cache  [n_blocks, Hkv, 2, bs, d]  e4m3 or int8: keys, then values, of bs tokens
//   scales [n_blocks, Hkv, 2]         fp32: value = code * scale
//   slot = block * bs + offset        where a token's key and value stand
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "common.cuh"

namespace liger {
namespace kvc {

constexpr int kMaxSeqs = 8192;   // sequences of one call (their prefix sums stand in shared memory)

__device__ __forceinline__ void pdl_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ============================================================== block assignment

struct AssignArgs {
  const int32_t* new_lens;   // [B] tokens to add; negative: the sequence ends
  const int32_t* seq_lens;   // [B]
  int32_t* table;            // [B, width]
  int32_t* ring;             // [n_blocks] free blocks, first at span[0], span[1] of them
  const int32_t* span;       // [2]
  int32_t* slots;            // [N]
  int32_t* cu;               // [B + 1]
  int32_t* lens_out;         // [B] (may be seq_lens)
  int32_t* span_out;         // [2] (may be span)
  int B, width, n_blocks, lbs, N;   // blocks of 2^lbs tokens
};

// Exclusive prefix sums over the block of K values; the block's totals in total[].
template <int THREADS, int K>
__device__ __forceinline__ void block_scan(long long (&v)[K], long long (&total)[K], long long (*part)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int W = THREADS / 32;
  long long x[K];
#pragma unroll
  for (int k = 0; k < K; ++k) x[k] = v[k];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const long long u = __shfl_up_sync(0xffffffffu, x[k], o);
      if (lane >= o) x[k] += u;
    }
  __syncthreads();   // part is free again
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (lane == 31) part[warp][k] = x[k];
  __syncthreads();
  // every warp scans the warps' sums for itself
#pragma unroll
  for (int k = 0; k < K; ++k) {
    long long p = lane < W ? part[lane][k] : 0;
#pragma unroll
    for (int o = 1; o < W; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, p, o);
      if (lane >= o) p += u;
    }
    const long long before = __shfl_sync(0xffffffffu, p, warp ? warp - 1 : 0);
    v[k] = x[k] - v[k] + (warp ? before : 0);
    total[k] = __shfl_sync(0xffffffffu, p, W - 1);
  }
}

constexpr int kAssignThreads = 512;
constexpr int kTokenEach = 4;   // up to that many tokens a thread are taken one by one
constexpr int kUnserved = -1;   // pre[] of a sequence that gets no slots

inline size_t assign_smem_bytes(int B) { return sizeof(int32_t) * (4 * (size_t)B + 1); }

// Every CTA scans all sequences (one block scan of tokens, blocks taken and blocks given back; a second one only
// where the slot map is too short) and takes its share of the rest: the slots of its threads' tokens, and a
// warp per sequence for its table row and the blocks it gives back.  With SLOTS, it reads the tables and
// the ring and writes slots, table and ring: blocks are taken from [head, head + taken) of the
// ring and given back at [head + count, ...), which never overlap while the free blocks and
// those in use are n_blocks in all, and only columns >= ceil(len / bs) of a table row are
// written, which no slot reads (a new block's number is read from the ring).  So no CTA
// depends on another.  With STATE (the first CTA), it writes the offsets, lengths and span; where they stand in the
// inputs' place, that is one CTA's work, in the same launch or in a later one.
// What bounds it: latency.  The lengths, a scan and one dependent table or ring read; for millions of slots also their
// write.  Measured on a B200: 64 sequences, a token each: 4.6 us; 512 prompts, 4.4 million slots (17.6 MB): 14.1 us (a
// grid of four CTAs an SM, which scanned in waves, took 31.7; sixteen tokens a lane written by that lane 21).
template <bool SLOTS, bool STATE>
__global__ void __launch_bounds__(kAssignThreads, 2) assign_kernel(AssignArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ long long part[kAssignThreads / 32][3];
  __shared__ int s_taken;
  int32_t* cu = sm;                  // [B + 1] token offsets, saturated
  int32_t* pre = cu + a.B + 1;       // [B] blocks taken before this sequence, or kUnserved
  int32_t* len = pre + a.B;          // [B]
  int32_t* back = len + a.B;         // [B] blocks given back before this sequence, or -1 (it goes on)
  pdl_launch_next();
  pdl_wait_previous();
  const int n = a.n_blocks, lbs = a.lbs, bs = 1 << lbs;
  int head = a.span[0], count = a.span[1];
  head = head < 0 || head >= n ? 0 : head;
  count = count < 0 ? 0 : (count > n ? n : count);
  const long long cap = (long long)a.width << lbs;
  long long tok0 = 0, need0 = 0, back0 = 0;   // running totals
  if (threadIdx.x == 0) s_taken = 0;   // (the scans below synchronise)
  for (int s0 = 0; s0 < a.B; s0 += kAssignThreads) {
    const int s = s0 + threadIdx.x;
    const bool in = s < a.B;
    long long L = in ? a.seq_lens[s] : 0;
    const int nw = in ? a.new_lens[s] : 0;
    L = L < 0 ? 0 : (L > cap ? cap : L);
    const long long add = nw > 0 ? nw : 0;
    const long long have = (L + bs - 1) >> lbs;
    const bool ends = in && nw < 0;
    bool fits = in && nw >= 0 && L + add <= cap;
    long long want = fits ? ((L + add + bs - 1) >> lbs) - have : 0;
    long long v[3] = {add, ends ? have : 0, want}, total[3];
    block_scan<kAssignThreads, 3>(v, total, part);
    const long long c0 = tok0 + v[0], c1 = c0 + add;
    if (tok0 + total[0] > a.N) {   // the slot map is too short for some
      fits = fits && c1 <= a.N;
      want = fits ? want : 0;
      long long again[1] = {want}, sum[1];
      block_scan<kAssignThreads, 1>(again, sum, part);
      v[2] = again[0];
      total[2] = sum[0];
    }
    const long long gone = v[1], need = need0 + v[2];
    const bool served = fits && (want == 0 || need + want <= count);
    // once one does not fit, none behind it that needs a block does: the served ones' blocks are the first
    if (served && want > 0) atomicMax(&s_taken, (int)(need + want));
    if (in) {
      cu[s + 1] = (int32_t)(c1 > 0x7fffffffLL ? 0x7fffffffLL : c1);
      pre[s] = served ? (int32_t)(need > n ? n : need) : kUnserved;   // above n only where no block is needed
      len[s] = (int32_t)L;
      back[s] = nw < 0 ? (int32_t)((back0 + gone) % n) : -1;
      if (STATE && blockIdx.x == 0) a.lens_out[s] = nw < 0 ? 0 : (int32_t)(L + (served ? add : 0));
    }
    tok0 += total[0];
    back0 += total[1];
    need0 += total[2];
  }
  if (threadIdx.x == 0) cu[0] = 0;
  __syncthreads();
  const int taken = s_taken;
  if (STATE && blockIdx.x == 0) {
    for (int i = threadIdx.x; i <= a.B; i += kAssignThreads) a.cu[i] = cu[i];
    if (threadIdx.x == 0) {
      const long long left = (long long)count - taken + back0;
      a.span_out[0] = (int32_t)(((long long)head + taken) % n);
      a.span_out[1] = (int32_t)(left > n ? n : left);
    }
  }
  if (!SLOTS) return;

  // place i of the ring (n and the blocks of a row are below 2^27)
  auto wrap = [&](int i) { return i < n ? i : (i < 2 * n ? i - n : i % n); };
  // a sequence's new blocks into its row, an ended one's blocks back to the ring, eight a lane in flight
  const int warps = gridDim.x * (kAssignThreads / 32);
  for (int s = (threadIdx.x >> 5) * gridDim.x + blockIdx.x; s < a.B; s += warps) {
    const int lane = threadIdx.x & 31, have = (int)(((long long)len[s] + bs - 1) >> lbs);
    int32_t* row = a.table + (size_t)s * a.width;
    const bool ended = back[s] >= 0;
    if (!ended && pre[s] == kUnserved) continue;
    const int upto = ended ? have : (int)(((long long)len[s] + (cu[s + 1] - cu[s]) + bs - 1) >> lbs);
    const int at = ended ? wrap(wrap(head + count) + back[s]) : wrap(head + pre[s]);   // of the first one in the ring
    const int from = ended ? 0 : have;
    for (int j0 = from + lane; j0 < upto; j0 += 32 * 8) {
      int32_t x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = j0 + 32 * e;
        if (j < upto) x[e] = ended ? row[j] : a.ring[wrap(at + j - from)];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = j0 + 32 * e;
        if (j < upto) {
          if (ended) a.ring[wrap(at + j - from)] = x[e];
          else row[j] = x[e];
        }
      }
    }
  }

  const int total = cu[a.B] < a.N ? cu[a.B] : a.N;
  // the last sequence whose tokens begin at or before i
  auto sequence_of = [&](int i) {
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= i) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  // where the number of block b of sequence s stands
  auto place_of = [&](int s, int b) -> const int32_t* {
    const int have = (int)(((long long)len[s] + bs - 1) >> lbs);
    return b < have ? a.table + (size_t)s * a.width + b : a.ring + wrap(head + pre[s] + b - have);
  };
  auto slot_of = [&](int id, int p) { return id < 0 || id >= n ? -1 : (id << lbs) + (p & (bs - 1)); };
  const int step = gridDim.x * kAssignThreads;
  if (a.N <= kTokenEach * step) {   // few: a token a thread
    for (int i = blockIdx.x * kAssignThreads + threadIdx.x; i < a.N; i += step) {
      int slot = -1;
      if (i < total) {
        const int s = sequence_of(i);
        if (pre[s] != kUnserved) {
          const int p = len[s] + (i - cu[s]);
          slot = slot_of(*place_of(s, p >> lbs), p);
        }
      }
      a.slots[i] = slot;
    }
    return;
  }
  // Many: 512 consecutive tokens a warp.  Each lane looks up sixteen, which lie in one or two blocks of one sequence
  // but at a sequence's end; then all lanes write them four by four, side by side.
  const int lane = threadIdx.x & 31;
  for (int c = blockIdx.x * (kAssignThreads / 32) + (threadIdx.x >> 5); c < (a.N + 511LL) / 512; c += step / 32) {
    const int i0 = 512 * c + 16 * lane;
    const int s0 = i0 < total ? sequence_of(i0) : 0;
    const bool one = i0 < total && min(cu[s0 + 1], total) - i0 >= 16;
    int id0 = -1, id1 = -1, p0 = 0;
    if (one && pre[s0] != kUnserved) {
      p0 = len[s0] + (i0 - cu[s0]);
      id0 = *place_of(s0, p0 >> lbs);
      id1 = *place_of(s0, (p0 + 15) >> lbs);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int from = 8 * q + (lane >> 2), iq = 512 * c + 128 * q + 4 * lane;
      const bool f_one = __shfl_sync(0xffffffffu, (int)one, from);
      const int f_id0 = __shfl_sync(0xffffffffu, id0, from), f_id1 = __shfl_sync(0xffffffffu, id1, from);
      const int f_p0 = __shfl_sync(0xffffffffu, p0, from);
      int s = __shfl_sync(0xffffffffu, s0, from);
      int out[4] = {-1, -1, -1, -1};
      if (f_one) {
        const int p = f_p0 + 4 * (lane & 3);
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = slot_of((p + e) >> lbs == f_p0 >> lbs ? f_id0 : f_id1, p + e);
      } else if (iq < total) {
#pragma unroll 1
        for (int e = 0; e < 4 && iq + e < total; ++e) {
          while (cu[s + 1] <= iq + e) ++s;
          if (pre[s] != kUnserved) {
            const int p = len[s] + (iq + e - cu[s]), slot = slot_of(*place_of(s, p >> lbs), p);
#pragma unroll
            for (int x = 0; x < 4; ++x) out[x] = x == e ? slot : out[x];
          }
        }
      }
      if (a.N - iq >= 4) {
        *reinterpret_cast<int4*>(a.slots + iq) = make_int4(out[0], out[1], out[2], out[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (e < a.N - iq) a.slots[iq + e] = out[e];
      }
    }
  }
}

// ============================================================== codes

enum KvType { kE4m3 = 0, kInt8 = 1 };

// Largest code value, and the exponent of the smallest scale.
template <KvType T> struct Format;
template <> struct Format<kE4m3> {
  static constexpr int kTopExp = 8;              // 448 = 1.75 * 2^8
  static constexpr uint32_t kTopFrac = 0x600000u;
};
template <> struct Format<kInt8> {
  static constexpr int kTopExp = 6;              // 127 = 1.984375 * 2^6
  static constexpr uint32_t kTopFrac = 0x7E0000u;
};
constexpr int kMinScaleExp = -64;

// The smallest power of two s >= 2^-64 with amax <= s * (largest code), from the bits of
// amax = f * 2^k.  A power of two makes the division by s exact, so a value is rounded once, to
// its code; for e4m3 it costs no precision (a floating format), for int8 at most one bit.
template <KvType T>
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  int e = (int)(bits >> 23) - 127 - Format<T>::kTopExp + ((bits & 0x7FFFFFu) > Format<T>::kTopFrac ? 1 : 0);
  e = e < kMinScaleExp ? kMinScaleExp : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two scaled values to their codes: nearest, ties to even, saturated; NaN stays NaN (e4m3) or
// becomes 0 (int8).  The first value in the low byte.
template <KvType T>
__device__ __forceinline__ uint32_t code2(float lo, float hi) {
  if (T == kE4m3) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  }
  int a, b;
  const float l = fminf(fmaxf(lo, -127.f), 127.f), h = fminf(fmaxf(hi, -127.f), 127.f);
  a = __float2int_rn(lo != lo ? 0.f : l);
  b = __float2int_rn(hi != hi ? 0.f : h);
  return ((uint32_t)a & 0xFFu) | (((uint32_t)b & 0xFFu) << 8);
}
template <KvType T>
__device__ __forceinline__ float value_of(uint32_t code) {   // low 8 bits
  if (T == kInt8) return (float)(int)(int8_t)(code & 0xFFu);
  uint32_t h2;
  const uint16_t c = (uint16_t)(code & 0xFFu);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
  return __half2float(__ushort_as_half((unsigned short)(h2 & 0xFFFFu)));
}

// ============================================================== append

struct AppendArgs {
  const void* k;            // [N, Hkv, d], tokens kstride / vstride elements apart
  const void* v;
  const int32_t* slots;     // [N]
  uint8_t* cache;
  float* scales;
  long kstride, vstride;
  int N, Hkv, n_slots;      // n_slots = n_blocks * bs
};

// Eight elements of a row.  add_max gathers the largest magnitude's bits (magnitudes order like their bits), max_bits
// gives them as fp32's.
template <typename Tin> struct Eight;
template <> struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void add_max(uint32_t& m) const {   // two 16-bit maxima
    m = __vmaxu2(m, u.x & 0x7FFF7FFFu);
    m = __vmaxu2(m, u.y & 0x7FFF7FFFu);
    m = __vmaxu2(m, u.z & 0x7FFF7FFFu);
    m = __vmaxu2(m, u.w & 0x7FFF7FFFu);
  }
  static __device__ __forceinline__ uint32_t max_bits(uint32_t m) { return max(m & 0xFFFF0000u, m << 16); }
};
template <> struct Eight<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const uint4*>(p));
    b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
  __device__ __forceinline__ void add_max(uint32_t& m) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
  }
  static __device__ __forceinline__ uint32_t max_bits(uint32_t m) { return m; }
};
constexpr uint32_t kInfBits = 0x7F800000u;

// Largest finite magnitude, as bits.
__device__ __forceinline__ uint32_t finite_max8(const float* x) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    m = max(m, b < kInfBits ? b : 0u);
  }
  return m;
}

// Codes of eight elements.  `plain`: the scale is a power of two (`inv` its reciprocal) and, for int8, all elements are
// finite, so that |x / scale| <= 127 and adding 1.5 * 2^23 leaves the code, rounded to even, in the low byte.
template <KvType T>
__device__ __forceinline__ uint2 quantise8(const float* x, float scale, float inv, bool plain) {
  uint32_t c[2];
  if (plain && T == kInt8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = __float_as_uint(fmaf(x[4 * i + e], inv, 12582912.f));
      c[i] = __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float y[4];
      // a scale that is no power of two (a cache from elsewhere) takes the exact division
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = plain ? x[4 * i + e] * inv : __fdiv_rn(x[4 * i + e], scale);
      c[i] = code2<T>(y[0], y[1]) | (code2<T>(y[2], y[3]) << 16);
    }
  }
  return make_uint2(c[0], c[1]);
}

// Rows [0, rows) of one block half held under `old` again under `after` (after > old).
template <KvType T, int D>
__device__ __forceinline__ void requantise(uint8_t* half, int rows, float old, float after, int tid, int nthr) {
  const float f = __fdiv_rn(old, after);
  for (int i = tid; i < rows * D / 8; i += nthr) {
    uint2* p = reinterpret_cast<uint2*>(half) + i;
    const uint2 w = *p;
    const uint32_t in[2] = {w.x, w.y};
    uint32_t out[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      out[j] = code2<T>(value_of<T>(in[j]) * f, value_of<T>(in[j] >> 8) * f) |
               (code2<T>(value_of<T>(in[j] >> 16) * f, value_of<T>(in[j] >> 24) * f) << 16);
    *p = make_uint2(out[0], out[1]);
  }
}

// A run is a stretch of consecutive tokens with consecutive slots in one block: with the tokens of a
// sequence in order, all the tokens that a call brings to that block.  Its first token leads
// it.  CTA (x, y) finds the runs that start in its `range` tokens and takes them for a few kv heads: the keys, or
// the values, of a run and head go to a team of as many warps as hold a whole block's rows in registers between the
// maximum and the codes (128 bytes a lane), so that they are read once; where a team has several warps, runs of a
// few tokens go to single warps.
// A run that starts at offset 0 gives the block its scale; another one raises the scale if it has to, and
// the rows before it are then requantised under the new one.
// What bounds it: HBM for prompts (one read, one write); latency for single tokens.
// Measured on a B200 against the 6570 GB/s of a copy: two prompts of 8192 tokens (Hkv 8, d 128, bf16, blocks of 64)
// 20.2 us, 0.76 of it; nine ragged ones into blocks of 32 that have begun, int8: 37.3 us, 0.93; fp32, d 64, blocks of 16,
// four of up to 2048: 10.1 us, 0.55 (two short waves of CTAs, and 64 registers are too few for fp32: 88 to 144 bytes of
// stack); a token each for 64 sequences: 2.7 us.  A CTA for each
// run's keys and values whatever their size, with the finite test at each element, took 37.5, 69.1 and 14.0 us.
template <typename Tin, int D, int BS>
struct AppendShape {
  static constexpr int kRowLanes = D / 8;                                       // lanes of a row, eight elements each
  static constexpr int kTeam = BS * D * (int)sizeof(Tin) <= 4096 ? 1 : BS * D * (int)sizeof(Tin) / 4096;   // warps
  static constexpr int kThreads = 2 * kTeam * 32 < 256 ? 256 : 2 * kTeam * 32;
  static constexpr int kHeads = kThreads / (2 * kTeam * 32);                    // of a CTA
  static constexpr int kPieces = BS * kRowLanes / (32 * kTeam);                 // eight elements each, of a thread
  static constexpr int kRange = BS < 64 ? (BS < 32 ? 16 : 32) : 64;             // tokens of a CTA, when there are many
};
constexpr int kShortRun = 4;

template <typename Tin, KvType T, int D, int BS>
__global__ void __launch_bounds__(AppendShape<Tin, D, BS>::kThreads, 1024 / AppendShape<Tin, D, BS>::kThreads)
    append_kernel(AppendArgs a, int range) {
  using S = AppendShape<Tin, D, BS>;
  constexpr int kWindow = 256, kWords = kWindow / 32, kWarps = S::kThreads / 32;
  static_assert(S::kRange + BS <= kWindow, "a run that starts in the CTA's tokens ends in its window");
  __shared__ uint32_t s_cont[kWords], s_valid[kWords];    // bit i: token r0 + i continues a run / has a slot
  __shared__ int s_slot[kWindow];
  __shared__ uint32_t s_max[2][kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = blockIdx.x * range;
  pdl_launch_next();
  pdl_wait_previous();
  if (tid < kWindow) {
    const int i = r0 + tid;
    int slot = -1, prev = -1;
    if (tid < range + BS && i < a.N) {
      slot = a.slots[i];
      prev = i > 0 ? a.slots[i - 1] : -1;
    }
    const bool valid = slot >= 0 && slot < a.n_slots;
    const bool cont = valid && prev >= 0 && slot == prev + 1 && slot % BS != 0;
    const uint32_t bv = __ballot_sync(0xffffffffu, valid), bc = __ballot_sync(0xffffffffu, cont);
    if (lane == 0) { s_valid[warp] = bv; s_cont[warp] = bc; }
    s_slot[tid] = slot;
  }
  __syncthreads();
  // tokens of the run that token i leads (at most BS: a run ends with its block)
  auto run_length = [&](int i) {
    int n = 1;
    while (n < BS) {
      const int at = i + n, w = at >> 5, b = at & 31;
      if (w >= kWords) break;
      const uint32_t gaps = ~s_cont[w] >> b;
      if (gaps) { n += __ffs(gaps) - 1; break; }
      n += 32 - b;
    }
    return n < BS ? n : BS;
  };
  // The keys (half 0) or values of tokens i .. i + n - 1 and head h, by `kTeamWarps` warps of which the calling thread is
  // number t: kLoads pieces a thread.  `top` reduces a warp's maximum over the team.
  auto take = [&](auto loads, auto team_warps, int i, int n, int h, int half, int t, auto top) {
    constexpr int kLoads = decltype(loads)::value, kTeamWarps = decltype(team_warps)::value;
    const int slot = s_slot[i], off = slot % BS;
    const size_t unit = ((size_t)(slot / BS) * a.Hkv + h) * 2 + half;
    const long stride = half ? a.vstride : a.kstride;
    const Tin* src = static_cast<const Tin*>(half ? a.v : a.k) + (size_t)(r0 + i) * stride + (size_t)h * D + (t % S::kRowLanes) * 8;
    const int row0 = t / S::kRowLanes;
    constexpr int kStep = 32 * kTeamWarps / S::kRowLanes;   // rows from a thread's piece to its next
    Eight<Tin> e[kLoads];
    const float old = off ? a.scales[unit] : 0.f;
#pragma unroll
    for (int p = 0; p < kLoads; ++p) {
      e[p].zero();
      if (row0 + p * kStep < n) e[p].load(src + (size_t)(row0 + p * kStep) * stride);
    }
    uint32_t m = 0u;
#pragma unroll
    for (int p = 0; p < kLoads; ++p) e[p].add_max(m);
    m = top(__reduce_max_sync(0xffffffffu, Eight<Tin>::max_bits(m)));   // (and every thread has read the old scale)
    const bool finite = m < kInfBits;
    if (!finite) {
      m = 0u;
#pragma unroll
      for (int p = 0; p < kLoads; ++p) {
        float x[8];
        e[p].get(x);
        m = max(m, finite_max8(x));
      }
      m = top(__reduce_max_sync(0xffffffffu, m));
    }
    float after = scale_for<T>(__uint_as_float(m));
    if (off) after = fmaxf(after, old);
    uint8_t* dst = a.cache + unit * (size_t)(BS * D);
    if (off && after > old) requantise<T, D>(dst, off, old, after, t, 32 * kTeamWarps);
    if (t == 0 && (!off || after > old)) a.scales[unit] = after;
    const bool pow2 = (__float_as_uint(after) & 0x7FFFFFu) == 0u, plain = pow2 && (T == kE4m3 || finite);
    const float inv = 1.f / after;
    dst += (size_t)(off + row0) * D + (t % S::kRowLanes) * 8;
    auto write = [&](bool as_plain) {
#pragma unroll
      for (int p = 0; p < kLoads; ++p) {
        float x[8];
        e[p].get(x);
        if (row0 + p * kStep < n) *reinterpret_cast<uint2*>(dst + p * kStep * D) = quantise8<T>(x, after, inv, as_plain);
      }
    };
    if (plain) write(true);
    else write(false);
  };
  using std::integral_constant;
  auto in_warp = [](uint32_t m) { return m; };
  const int team = warp / S::kTeam, half = team & 1, h = blockIdx.y * S::kHeads + (team >> 1), t = tid - team * S::kTeam * 32;
  int n_short = 0, n_long = 0;
  for (int w = 0; w * 32 < range; ++w) {
    uint32_t lead = s_valid[w] & ~s_cont[w];
    if (range - w * 32 < 32) lead &= (1u << (range - w * 32)) - 1u;
    while (lead) {
      const int i = w * 32 + __ffs(lead) - 1;
      lead &= lead - 1u;
      const int n = run_length(i);
      if (S::kTeam > 1 && n <= kShortRun) {
#pragma unroll 1
        for (int j = 0; j < 2 * S::kHeads; ++j, ++n_short) {
          const int hj = blockIdx.y * S::kHeads + (j >> 1);
          if ((n_short & (kWarps - 1)) == warp && hj < a.Hkv)
            take(integral_constant<int, (kShortRun * S::kRowLanes + 31) / 32>{}, integral_constant<int, 1>{}, i, n, hj, j & 1, lane, in_warp);
        }
      } else if (S::kTeam == 1) {
        if (h < a.Hkv) take(integral_constant<int, S::kPieces>{}, integral_constant<int, 1>{}, i, n, h, half, t, in_warp);
      } else if (h < a.Hkv) {
        take(integral_constant<int, S::kPieces>{}, integral_constant<int, S::kTeam>{}, i, n, h, half, t, [&](uint32_t m) {
          uint32_t* mine = s_max[n_long++ & 1];   // (two in turn: one barrier for each)
          if (lane == 0) mine[warp] = m;
          asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(S::kTeam * 32) : "memory");
          m = 0u;
#pragma unroll
          for (int x = 0; x < S::kTeam; ++x) m = max(m, mine[team * S::kTeam + x]);
          return m;
        });
      }
    }
  }
}

}  // namespace kvc
}  // namespace liger
