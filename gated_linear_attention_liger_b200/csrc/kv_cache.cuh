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

// Exclusive prefix sums over the block of two values; returns the block's totals in *ta, *tb.
template <int THREADS>
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long* ta, long long* tb,
                                            long long (*part)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int W = THREADS / 32;
  long long x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) { x += u; y += v; }
  }
  __syncthreads();   // part is free again
  if (lane == 31) { part[warp][0] = x; part[warp][1] = y; }
  __syncthreads();
  if (warp == 0) {
    long long u = lane < W ? part[lane][0] : 0, v = lane < W ? part[lane][1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long p = __shfl_up_sync(0xffffffffu, u, o), q = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) { u += p; v += q; }
    }
    if (lane < W) { part[lane][0] = u; part[lane][1] = v; }
  }
  __syncthreads();
  a = x - a + (warp ? part[warp - 1][0] : 0);
  b = y - b + (warp ? part[warp - 1][1] : 0);
  *ta = part[W - 1][0];
  *tb = part[W - 1][1];
}

constexpr int kAssignThreads = 512;
constexpr int kUnserved = -1;   // pre[] of a sequence that gets no slots

inline size_t assign_smem_bytes(int B) { return sizeof(int32_t) * (4 * (size_t)B + 1); }

// Every CTA scans all sequences (two block scans: tokens, then blocks taken and given back) and
// takes its share of the rest: the slots of four consecutive tokens per thread, and a warp per
// sequence for its table row and the blocks it gives back.  With SLOTS, it reads the tables and
// the ring and writes slots, table and ring: blocks are taken from [head, head + taken) of the
// ring and given back at [head + count, ...), which never overlap while the free blocks and
// those in use are n_blocks in all, and only columns >= ceil(len / bs) of a table row are
// written, which no slot reads (a new block's number is read from the ring).  So no CTA
// depends on another.  With STATE (one CTA, the same launch or a later one), it writes the
// offsets, lengths and span, which may stand where the inputs stand.
// What bounds it: latency.  One CTA takes the lengths, two scans and one dependent table read in
// a single launch; more tokens than kOneCtaSlots go to many CTAs and a second launch.
template <bool SLOTS, bool STATE>
__global__ void __launch_bounds__(kAssignThreads) assign_kernel(AssignArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ long long part[kAssignThreads / 32][2];
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
    long long toks = add, gone = in && nw < 0 ? have : 0, t1, t2;
    block_scan2<kAssignThreads>(toks, gone, &t1, &t2, part);
    const long long c0 = tok0 + toks, c1 = c0 + add;
    const bool fits = in && nw >= 0 && L + add <= cap && c1 <= a.N;
    const long long want = fits ? ((L + add + bs - 1) >> lbs) - have : 0;
    long long need = want, unused = 0, t3, t4;
    block_scan2<kAssignThreads>(need, unused, &t3, &t4, part);
    need += need0;
    const bool served = fits && (want == 0 || need + want <= count);
    // once one does not fit, none behind it that needs a block does: the served ones' blocks are the first
    if (served && want > 0) atomicMax(&s_taken, (int)(need + want));
    if (in) {
      cu[s + 1] = (int32_t)(c1 > 0x7fffffffLL ? 0x7fffffffLL : c1);
      pre[s] = served ? (int32_t)(need > n ? n : need) : kUnserved;   // above n only where no block is needed
      len[s] = (int32_t)L;
      back[s] = nw < 0 ? (int32_t)((back0 + gone) % n) : -1;
      if (STATE) a.lens_out[s] = nw < 0 ? 0 : (int32_t)(L + (served ? add : 0));
    }
    tok0 += t1;
    back0 += t2;
    need0 += t3;
  }
  if (threadIdx.x == 0) cu[0] = 0;
  __syncthreads();
  const int taken = s_taken;
  if (STATE) {
    for (int i = threadIdx.x; i <= a.B; i += kAssignThreads) a.cu[i] = cu[i];
    if (threadIdx.x == 0) {
      const long long left = (long long)count - taken + back0;
      a.span_out[0] = (int32_t)(((long long)head + taken) % n);
      a.span_out[1] = (int32_t)(left > n ? n : left);
    }
  }
  if (!SLOTS) return;

  // a sequence's new blocks into its row, an ended one's blocks back to the ring
  const int warps = gridDim.x * (kAssignThreads / 32);
  for (int s = blockIdx.x * (kAssignThreads / 32) + (threadIdx.x >> 5); s < a.B; s += warps) {
    const int lane = threadIdx.x & 31, have = (int)(((long long)len[s] + bs - 1) >> lbs);
    int32_t* row = a.table + (size_t)s * a.width;
    if (back[s] >= 0) {
      for (int j = lane; j < have; j += 32) a.ring[((long long)head + count + back[s] + j) % n] = row[j];
    } else if (pre[s] != kUnserved) {
      const long long end = (long long)len[s] + (cu[s + 1] - cu[s]);
      const int upto = (int)((end + bs - 1) >> lbs);
      for (int j = have + lane; j < upto; j += 32) row[j] = a.ring[((long long)head + pre[s] + j - have) % n];
    }
  }

  // slots, four tokens a thread
  const int total = cu[a.B];
  const long long quads = ((long long)a.N + 3) / 4;
  const long long step = (long long)gridDim.x * kAssignThreads;
  for (long long g = (long long)blockIdx.x * kAssignThreads + threadIdx.x; g < quads; g += step) {
    const int i0 = (int)(4 * g);
    int32_t out[4] = {-1, -1, -1, -1};
    if (i0 < total) {
      int lo = 0, hi = a.B;   // the last s with cu[s] <= i0
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= i0) lo = mid;
        else hi = mid;
      }
      int s = lo, blk = -1, id = -1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + e;
        if (i >= total || i >= a.N) break;
        while (cu[s + 1] <= i) { ++s; blk = -1; }
        if (pre[s] == kUnserved) continue;
        const int p = len[s] + (i - cu[s]);
        const int b = p >> lbs;
        if (b != blk) {
          const int have = (int)(((long long)len[s] + bs - 1) >> lbs);
          blk = b;
          id = b < have ? a.table[(size_t)s * a.width + b] : a.ring[((long long)head + pre[s] + b - have) % n];
          if (id < 0 || id >= n) id = -1;
        }
        out[e] = id < 0 ? -1 : (id << lbs) + (p & (bs - 1));
      }
    }
    if (a.N - i0 >= 4) {
      *reinterpret_cast<int4*>(a.slots + i0) = make_int4(out[0], out[1], out[2], out[3]);
    } else {
      for (int e = 0; i0 + e < a.N; ++e) a.slots[i0 + e] = out[e];
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

// Eight elements of a row in fp32.
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
};
template <> struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};

// Largest finite magnitude, as bits (magnitudes order like their bits; infinities and NaN are left out).
__device__ __forceinline__ uint32_t amax8(const float* x) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    m = max(m, b < 0x7F800000u ? b : 0u);
  }
  return m;
}

template <KvType T>
__device__ __forceinline__ uint2 quantise8(const float* x, float scale, float inv, bool pow2) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // a scale that is no power of two (a cache from elsewhere) takes the exact division
    const float lo = pow2 ? x[2 * i] * inv : __fdiv_rn(x[2 * i], scale);
    const float hi = pow2 ? x[2 * i + 1] * inv : __fdiv_rn(x[2 * i + 1], scale);
    c[i] = code2<T>(lo, hi);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
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

constexpr int kAppendThreads = 256;
constexpr int kShortRun = 4;   // runs up to this many tokens are taken by one warp each

// A run is a stretch of consecutive tokens with consecutive slots in one block: with the tokens of a
// sequence in order, all the tokens that a call brings to that block.  Its first token leads
// it.  CTA (x, h) finds the runs that start in its `range` tokens, for kv head h: a long run is taken by the
// whole CTA (half of it the keys, half the values, every element held in registers between the maximum
// and the codes, so that it is read once), short runs by one warp for each of keys and values.
// A run that starts at offset 0 gives the block its scale; another one raises the scale if it has to, and
// the rows before it are then requantised under the new one.
// What bounds it: HBM for prompts (one read, one write); latency for single tokens.
template <typename Tin, KvType T, int D, int BS>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendArgs a, int range) {
  constexpr int kVecRow = D / 8;                          // 8-element pieces of a row
  constexpr int kHalf = kAppendThreads / 2;
  constexpr int kPieces = (BS * kVecRow + kHalf - 1) / kHalf;   // of a thread, in a long run
  constexpr int kWords = kAppendThreads / 32;
  __shared__ uint32_t s_cont[kWords], s_valid[kWords];    // bit i: token r0 + i continues a run / has a slot
  __shared__ uint32_t s_max[kWords];
  const int h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = blockIdx.x * range;
  pdl_launch_next();
  pdl_wait_previous();
  {
    const int i = r0 + tid;
    int slot = -1, prev = -1;
    if (i < a.N && tid < range + BS) {
      slot = a.slots[i];
      prev = i > 0 ? a.slots[i - 1] : -1;
    }
    const bool valid = slot >= 0 && slot < a.n_slots;
    const bool cont = valid && prev >= 0 && slot == prev + 1 && slot % BS != 0;
    const uint32_t bv = __ballot_sync(0xffffffffu, valid), bc = __ballot_sync(0xffffffffu, cont);
    if (lane == 0) { s_valid[warp] = bv; s_cont[warp] = bc; }
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
  int n_short = 0;
  for (int w = 0; w * 32 < range; ++w) {
    uint32_t lead = s_valid[w] & ~s_cont[w];
    if (range - w * 32 < 32) lead &= (1u << (range - w * 32)) - 1u;
    while (lead) {
      const int i = w * 32 + __ffs(lead) - 1;
      lead &= lead - 1u;
      const int n = run_length(i);
      if (n <= kShortRun) {   // one warp for the keys, one for the values, in turn
#pragma unroll 1
        for (int half = 0; half < 2; ++half, ++n_short) {
          if ((n_short & (kWords - 1)) != warp) continue;
          const int slot = a.slots[r0 + i], off = slot % BS;
          const size_t unit = ((size_t)(slot / BS) * a.Hkv + h) * 2 + half;
          const Tin* src = static_cast<const Tin*>(half ? a.v : a.k) + (size_t)(r0 + i) * (half ? a.vstride : a.kstride) +
                           (size_t)h * D;
          const long stride = half ? a.vstride : a.kstride;
          constexpr int kRows = 32 / kVecRow;                       // rows of one warp load
          constexpr int kLoads = (kShortRun + kRows - 1) / kRows;
          Eight<Tin> e[kLoads];
          const float old = off ? a.scales[unit] : 0.f;
          uint32_t m = 0u;
#pragma unroll
          for (int l = 0; l < kLoads; ++l) {
            const int row = l * kRows + lane / kVecRow;
            e[l].zero();
            if (row < n) e[l].load(src + (size_t)row * stride + (lane % kVecRow) * 8);
          }
#pragma unroll
          for (int l = 0; l < kLoads; ++l) {
            float x[8];
            e[l].get(x);
            m = max(m, amax8(x));
          }
          m = __reduce_max_sync(0xffffffffu, m);
          float after = scale_for<T>(__uint_as_float(m));
          if (off) after = fmaxf(after, old);
          uint8_t* dst = a.cache + unit * (size_t)(BS * D);
          if (off && after > old) requantise<T, D>(dst, off, old, after, lane, 32);
          if (lane == 0 && (!off || after > old)) a.scales[unit] = after;
          const bool pow2 = (__float_as_uint(after) & 0x7FFFFFu) == 0u;
          const float inv = 1.f / after;
#pragma unroll
          for (int l = 0; l < kLoads; ++l) {
            const int row = l * kRows + lane / kVecRow;
            float x[8];
            e[l].get(x);
            if (row < n)
              *reinterpret_cast<uint2*>(dst + (size_t)(off + row) * D + (lane % kVecRow) * 8) =
                  quantise8<T>(x, after, inv, pow2);
          }
        }
        continue;
      }
      // the whole CTA
      const int half = tid / kHalf, t = tid % kHalf;
      const int slot = a.slots[r0 + i], off = slot % BS;
      const size_t unit = ((size_t)(slot / BS) * a.Hkv + h) * 2 + half;
      const long stride = half ? a.vstride : a.kstride;
      const Tin* src = static_cast<const Tin*>(half ? a.v : a.k) + (size_t)(r0 + i) * stride + (size_t)h * D;
      Eight<Tin> e[kPieces];
      const float old = off ? a.scales[unit] : 0.f;
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int idx = p * kHalf + t, row = idx / kVecRow;
        e[p].zero();
        if (row < n) e[p].load(src + (size_t)row * stride + (idx % kVecRow) * 8);
      }
      uint32_t m = 0u;
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        float x[8];
        e[p].get(x);
        m = max(m, amax8(x));
      }
      m = __reduce_max_sync(0xffffffffu, m);
      __syncthreads();   // s_max is free again
      if (lane == 0) s_max[warp] = m;
      __syncthreads();   // (and every thread has read the old scale)
      m = 0u;
#pragma unroll
      for (int x = 0; x < kWords / 2; ++x) m = max(m, s_max[half * (kWords / 2) + x]);
      float after = scale_for<T>(__uint_as_float(m));
      if (off) after = fmaxf(after, old);
      uint8_t* dst = a.cache + unit * (size_t)(BS * D);
      if (off && after > old) requantise<T, D>(dst, off, old, after, t, kHalf);
      if (t == 0 && (!off || after > old)) a.scales[unit] = after;
      const bool pow2 = (__float_as_uint(after) & 0x7FFFFFu) == 0u;
      const float inv = 1.f / after;
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int idx = p * kHalf + t, row = idx / kVecRow;
        float x[8];
        e[p].get(x);
        if (row < n)
          *reinterpret_cast<uint2*>(dst + (size_t)(off + row) * D + (idx % kVecRow) * 8) =
              quantise8<T>(x, after, inv, pow2);
      }
    }
  }
}

}  // namespace kvc
}  // namespace liger
