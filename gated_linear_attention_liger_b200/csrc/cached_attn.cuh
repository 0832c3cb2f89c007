// cached_attn.cuh -- softmax attention of a few new tokens over the paged 8-bit cache (the
// hybrid's standard attention layer, one decode step).
//
//   o_i = sum_j softmax_j(q_i . k_j / sqrt(d)) v_j,   j <= len - n_q + i,   i = 0 .. n_q - 1
//
// with k_j = ks * code, v_j = vs * code, the scales ks, vs those of token j's block.
//
// What bounds it: HBM, and for short calls the chain of latencies before the first copy and after the last one.  A
// cached byte is used for 2 G n_q multiply-adds (G = Hq / Hkv), 8 to 64 flops, so it is read once for up to 16 query rows
// and all else has to fit under that stream.
//
// The work is cut into tiles of 16 KB of keys and values (64 tokens at d = 128, 128 at d = 64) of one unit (sequence, kv
// head, up to 16 query rows); the units stand in one line, and each CTA (two an SM) takes an equal stretch of it, however
// ragged the lengths.  A unit that lies in several stretches is joined by a second small kernel, in the order of the
// stretches, so results do not depend on timing.  (A join by the last CTA to arrive would want counters that are zero
// before the call; the workspace's contents are the caller's.)
//
// In a CTA a producer warp finds each tile's blocks (a lane per block, the next batch's table entries and scales in
// flight) and brings a block's keys and values in with one TMA copy (swizzled, a ring of stages); four consumer warps
// take a quarter of the tokens of every tile each; an output warp adds up their four parts of a unit while they go on with
// the next one.  The products run on mma.sync m16n8k16 in fp16: the codes of
// e4m3 and int8 are exact in fp16, the query row is scaled by a power of two into fp16's range
// (an fp32 row is split into two fp16 terms, as is the probability), and sums are fp32.  Tokens are the rows of both
// products,
//   S^T [tokens x rows] = K Q^T,       O^T [d x rows] += V^T P^T,
// so that a product is 8 query rows wide (the G heads of a group), not 16, and P^T becomes the second product's operand
// by one 8 x 8 transpose in registers (movmatrix).  The tensor pipe is a fifth busy; mma.sync
// is enough, and its operands come straight from the codes' registers, where tcgen05 would need
// the fp16 values written back to shared memory.  (The e4m3 form of mma.sync, with q in two e4m3 terms, saves the
// keys' conversion and yet was slower: 64 sequences of 2048 to 8192 tokens 123 us instead of 116, 4 new tokens each at
// d = 64 44 us instead of 36.)
// The order of d inside the first product and of tokens inside the second is free, so each
// thread reads 16 consecutive bytes of a row and converts them in place: for the keys, the four
// bytes of a word are one k-step's elements of a thread; for the values, bytes of the same d
// from two tokens are paired by a byte permute.
//
// Softmax: with the score s in log2 units, the row sum takes t = 2^(s - m) and the value codes p = t vs, one running
// reference m for both.  m is raised only when some s + log2(vs) exceeds it by 15 (a warp vote per tile; the accumulators
// are then rescaled); p stays below 2^15, inside fp16, and keeps full fp16 precision 2^29 below that.  t needs fp32's
// range: a token's s is up to 64 above s + log2(vs) (append writes no scale below 2^-64; below that one the reference
// takes log2(vs) as -64), so t is at most 2^79 and a sum of 2^31 of them finite, and in a sequence whose largest value scale is
// 2^e a weight counts down to 2^(e - 133) of the largest (2^-33 at 2^100).  Rescaling and joining take a sum's factor in two
// halves, since the references of a zero block (scale 2^-64) and its neighbour may lie more than 2^126 apart.
// Roundings to fewer bits: p to fp16 (2^-11 of itself; fp32 outputs: two terms, 2^-22; either way up to 2^-25, which is 2^-32
// of the row's largest p or less), the output to its type.
//
// Measured on a B200 (calls back to back in a CUDA graph; bytes of the cache, queries and outputs over the 6570 GB/s of a
// copy): 64 sequences of 2048 to 8192 tokens, Hq 32, Hkv 8, d 128, e4m3: 115.0 us, 0.89 of it (the copies without the
// products took as long: the stream bounds it); one of 131072 tokens: 49.8 us, 0.82; 256 of up to 1500 tokens in blocks of 16,
// int8: 83.5 us, 0.73; 4 new tokens each for 32 sequences of up to 6000, d 64: 34.6 us, 0.44 (16 rows a unit: the consumers'
// latencies bound it, two warps a scheduler at 157 registers; 32 rows a unit spilled and took 117 us where two units of 16
// take 72), and for 32 of 2000 to 6000, d 128: 73.7 us, 0.55 (the same, and 16 rows at d 128 spill: bf16 96 bytes of stack,
// fp32 up to 248); one of 1000 tokens: 8.3 us, of latencies (the first tile comes after 2.5, its products take 1, its output 1.5,
// the join 3).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "kv_cache.cuh"
#include "sm100.cuh"

namespace liger {
namespace ca {

using namespace liger::sm100;
using kvc::KvType;
using kvc::kE4m3;
using kvc::kInt8;

constexpr int kWarps = 4;              // consumer warps
constexpr int kThreads = 32 * (kWarps + 2);   // and the producer's and the output's warp
constexpr int kEarly = 2;              // tiles that a stretch starts with before their scales have come
constexpr int kJoinThreads = 256;
constexpr int kJoinLanes = 8;         // at most, for a piece of a joined unit (16 took 0.7 us more on one short sequence)
constexpr float kNoRef = -3e38f;       // reference of a row that has seen nothing: below every finite score
constexpr float kRefBelow = 7.f;       // the reference is set this far below the maximum,
constexpr float kRaiseAt = 15.f;       // and raised when a score exceeds it by this much

// Division of 0 .. 2^31 - 1 by a number known on the host: n m / 2^(31 + s), m the next integer above 2^(31 + s) / d, with
// 2^s >= d.  (A division on the device takes some 300 cycles, and several stood one behind the other before the first copy.)
struct Divisor {
  uint32_t m;
  int s, d;
  static Divisor of(int d) {
    Divisor x{0u, 0, d};
    while ((1LL << x.s) < d) ++x.s;
    x.m = (uint32_t)((1ULL << (31 + x.s)) / d + 1);
    return x;
  }
  __device__ __forceinline__ int operator()(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> (31 + s)); }
};
// A unit that several CTAs have parts of, as each of them but the last notes it down for the join.
struct Split {
  int seq, head, row0, n_rows;         // seq -1: none
  int c0, parts;                       // the unit's first CTA, and how many it has
  int share, log_lanes;                // 16-byte pieces of the output for each of those CTAs; lanes for each piece, as a power of two
};
struct Args {
  const void* q;            // [B, n_q, Hq, d], tokens qstride elements apart
  const float* scales;      // [n_blocks, Hkv, 2]
  const int32_t* table;     // [B, width]
  const int32_t* lens;      // [B]
  void* out;                // [B, n_q, Hq, d]
  float* part_ml;           // [2 ctas][2][kMaxRows] references and sums of the parts
  float* part_o;            // [2 ctas][kMaxRows][d]
  Split* split;             // [ctas] the unit that goes on behind a CTA's stretch
  uint32_t* err;
  uint64_t wait_ns;
  long qstride;
  float scale_log2;         // log2(e) / sqrt(d)
  int B, n_q, Hq, Hkv, G, width, n_blocks, lbs;   // blocks of 2^lbs tokens
  int rows, row_tiles;                            // rows = n_q * G
  int inject_stall;         // test switch: the first CTA's first tile is never announced, so that waits run out
  Divisor by_ctas, by_units, by_row_tiles, by_G;  // units = Hkv * row_tiles
};
constexpr int kMaxRows = 16;           // query rows of a unit

struct StageInfo {
  int seq, head, row0, tok0;           // kv head, first query row, first cached token
  int len, flags;                      // tokens of the sequence; kFirst | kLast | kBegins | kEnds
  int pad0, pad1;
  float4 scale[8];                     // per 16 tokens: key scale (0: no such block), log2 of the value scale (at least -64), value scale
};
// the first, last tile of this CTA's stretch of the unit / of the unit itself; the stretch's last tile; no tile at all
enum { kFirst = 1, kLast = 2, kBegins = 4, kEnds = 8, kFinal = 16, kNone = 32 };

// Cached tokens of a tile: 16 KB of keys and values, whatever d, since a tile costs the producer and each consumer warp
// about 1000 cycles besides its bytes.
constexpr int tile_tokens(int d) { return 8192 / d; }

// What the consumer warps tell the output's warp about the unit that they have just ended.
struct UnitInfo {
  int seq, head, row0, flags;
};

// Shared memory.  NT: query rows in eights (1 or 2).
template <typename Tin, int D, int NT>
struct Smem {
  static constexpr uint32_t KV = 16384;                           // keys and values of a tile
  static constexpr uint32_t Q = 8 * NT * D * sizeof(Tin);
  static constexpr uint32_t STAGE = KV + Q;                       // a multiple of 1024
  static constexpr int MAX_STAGES = 12;
  static constexpr uint32_t FIXED = MAX_STAGES * (sizeof(StageInfo) + 16) + sizeof(UnitInfo) + 16 + 80;
  static __host__ __device__ int part_rows(int rows) { return rows < 8 * NT ? rows : 8 * NT; }
  // the four warps' parts of a unit: sums, then references and sums of weights; then the parts' weights
  static __host__ __device__ uint32_t red(int rows) { return kWarps * part_rows(rows) * (D * 4 + 8 + 4); }
  static uint32_t bytes(int stages, int rows, int B) { return 1024 + stages * STAGE + FIXED + (red(rows) + 15) / 16 * 16 + 4 * (3 * B + 2); }
};

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t x) {
  return __half22float2(*reinterpret_cast<__half2*>(&x));
}

// The four codes of a word as two fp16 pairs (bytes 0, 1 and bytes 2, 3): exact.
template <KvType T>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (T == kE4m3) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // code + 128 in the low bits of 1024 (fp16 0x6400), then minus 1152
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), off), y = __hsub2(*reinterpret_cast<__half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// Place of row n (0..7) of an operand in its group of eight tokens: 0 1 3 2 4 5 7 6.  With this order
// the rows that the lanes of one shared-memory wavefront read, both as key rows (two rows
// by eight 16-byte columns) and as value rows (four rows by two columns), fall into different
// banks under the TMA swizzle.
__device__ __forceinline__ int token_of(int n) { return n ^ ((n >> 1) & 1); }

// Byte offset of column `byte` of row `row` of a swizzled tile of D-byte rows.
template <int D>
__device__ __forceinline__ uint32_t swz(int row, int byte) {
  if (D == 128) return (uint32_t)(row * 128 + (byte ^ ((row & 7) << 4)));
  return (uint32_t)(row * 64 + (byte ^ (((row >> 1) & 3) << 4)));
}

__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// The line of work: sequence by sequence, unit by unit, a place for each tile and unit_cost more behind a unit's last one
// (its query operands and its output cost that much; with 16 rows a place more or less took 5 to 10% longer on short
// units, with 8 rows 1%), cut into equal stretches of `per` places, one for each CTA.  The tiles of one unit lie in
// consecutive stretches.
constexpr int unit_cost(int nt) { return nt + 1; }   // nt: query rows in eights, at most 2

template <typename Tin, int D, KvType T, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    cached_attn_kernel(const __grid_constant__ CUtensorMap tm, Args a, int stages) {
  using S = Smem<Tin, D, NT>;
  constexpr bool kSplit = sizeof(Tin) == 4;                 // fp32: two fp16 terms of q and of p
  constexpr int kRows = 8 * NT, kTile = tile_tokens(D), kUnitCost = unit_cost(NT);
  extern __shared__ __align__(1024) char smem_raw[];
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  StageInfo* info = reinterpret_cast<StageInfo*>(smem + stages * S::STAGE);
  UnitInfo* unit_info = reinterpret_cast<UnitInfo*>(info + S::MAX_STAGES);
  uint64_t* full = reinterpret_cast<uint64_t*>(unit_info + 1);
  uint64_t* empty = full + S::MAX_STAGES;
  uint64_t* parts_full = empty + S::MAX_STAGES;                       // the warps' parts are written
  uint64_t* parts_empty = parts_full + 1;                             // and read
  int* part = reinterpret_cast<int*>(parts_empty + 1);                // [2][8] warp sums of the scan
  volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(part + 16);
  volatile uint32_t* never = abort_flag + 1;
  const int part_rows = S::part_rows(a.rows);
  float* red = reinterpret_cast<float*>(part + 20);                   // [kWarps][part_rows][D]
  float* red_ml = red + kWarps * part_rows * D;                       // [kWarps][part_rows][2]
  float* wgt = red_ml + kWarps * part_rows * 2;                       // [part_rows][kWarps]
  int* first = reinterpret_cast<int*>(part + 20) + (S::red(a.rows) + 15) / 16 * 4;   // [B + 1] tiles before each sequence
  int* line = first + a.B + 1;                                        // [B + 1] places before each sequence, for one unit
  int* lens = line + a.B + 1;                                         // [B]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < stages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], kWarps); }
    mbar_init(parts_full, kWarps);
    mbar_init(parts_empty, 1);
    *abort_flag = 0u;
    *never = 0u;
    fence_mbar_init();
    prefetch_tensormap(&tm);
  }
  kvc::pdl_launch_next();
  __syncthreads();
  kvc::pdl_wait_previous();

  const int cap = a.width << a.lbs;
  auto length = [&](int s) { return min(max(a.lens[s], 0), cap); };
  auto tiles_of = [&](int len) { return (int)(((long long)len + kTile - 1) / kTile); };
  // tiles before each sequence, for the producer: its own scan if a warp holds them, else a block's, each thread over
  // consecutive sequences
  if (a.B <= 32) {
    if (warp == kWarps) {
      const int len = lane < a.B ? length(lane) : 0, n = tiles_of(len);
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += u;
      }
      const int seqs = __popc(__ballot_sync(0xffffffffu, n > 0) & ((2u << lane) - 1u));
      if (lane < a.B) {
        lens[lane] = len;
        first[lane + 1] = x;
        line[lane + 1] = x + kUnitCost * seqs;
      }
      if (lane == 0) first[0] = line[0] = 0;
      __syncwarp();
    }
  } else {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int s0 = tid * per, s1 = min(a.B, s0 + per);
    int sum = 0, some = 0;
    for (int s = s0; s < s1; ++s) {
      lens[s] = length(s);
      const int n = tiles_of(lens[s]);
      sum += n;
      some += n > 0;
    }
    int x = sum, y = some;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) { x += u; y += v; }
    }
    if (lane == 31) { part[warp] = x; part[8 + warp] = y; }
    __syncthreads();
    int run = x - sum, seqs = y - some;
    for (int w = 0; w < warp; ++w) { run += part[w]; seqs += part[8 + w]; }
    for (int s = s0; s < s1; ++s) {
      const int n = tiles_of(lens[s]);
      first[s] = run;
      line[s] = run + kUnitCost * seqs;
      run += n;
      seqs += n > 0;
    }
    if (s1 == a.B && s0 < a.B) { first[a.B] = run; line[a.B] = run + kUnitCost * seqs; }
    __syncthreads();
  }
  const int units = a.Hkv * a.row_tiles;                     // of one sequence
  const int cta = blockIdx.x;
  const WaitCtx wc{abort_flag, a.err, a.wait_ns};

  const int bs = 1 << a.lbs, kLog = D == 128 ? 6 : 7, lbox = a.lbs < kLog ? a.lbs : kLog, box = 1 << lbox;   // rows of keys, and of values, of one copy

  if (warp == kWarps) {   // ---------------- producer
    const int lppt = kLog - lbox;                       // 2^lppt blocks of a tile
    const int batch = 32 >> lppt;                    // tiles looked up at once, a lane per block
    const int in_tile = lane & ((1 << lppt) - 1), lane_tile = lane >> lppt;
    // this CTA's stretch of the line
    const int W = line[a.B] * units, per = a.by_ctas(W + (int)gridDim.x - 1);   // (the whole line fits 31 bits)
    const int p0 = min(W, per * cta), p1 = min(W, p0 + per);
    // the last sequence whose places begin at or before p0, 32 probes at a time
    int seq0 = 0;
    for (int n = a.B, f = a.by_units(p0); n > 1;) {
      const int step = (n + 31) >> 5;
      const uint32_t below = __ballot_sync(0xffffffffu, lane * step < n && line[min(seq0 + lane * step, a.B)] <= f);
      const int hit = 31 - __clz(below);   // (the first probe always is)
      n = min(step, n - hit * step);
      seq0 += hit * step;
    }
    struct Item { int seq, head, row0, tile, tiles, id; float ks, vs; };   // tile < tiles where there is one
    // The lane's block of the batch of places that starts at p: where it belongs, then its number (`id`, as the table
    // has it), then its scales.  Each step's load is used a batch later, so none is waited for but the first.
    auto locate = [&](int p, int lo) {
      Item it{lo, 0, 0, 0, 0, -1, 0.f, 1.f};
      p += lane_tile;
      if (p < p1) {
        for (int near = 0; near < 4 && line[lo + 1] * units <= p; ++near) ++lo;
        if (line[lo + 1] * units <= p) {
          int hi = a.B;   // line[lo] * units <= p < line[hi] * units
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (line[mid] * units <= p) lo = mid;
            else hi = mid;
          }
        }
        const uint32_t r = p - line[lo] * units;
        it.seq = lo;
        it.tiles = first[lo + 1] - first[lo];
        const int unit = (int)(r / (uint32_t)(it.tiles + kUnitCost));
        it.tile = (int)r - unit * (it.tiles + kUnitCost);
        it.head = unit;
        if (a.row_tiles > 1) {
          it.head = a.by_row_tiles(unit);
          it.row0 = (unit - it.head * a.row_tiles) * kMaxRows;
        }
        const int tok = it.tile * kTile + in_tile * box;   // (a row's tokens fit 31 bits, with a tile to spare)
        if (it.tile < it.tiles && tok < lens[lo]) it.id = a.table[(size_t)lo * a.width + (tok >> a.lbs)];
      }
      return it;
    };
    auto fetch_scales = [&](Item& it) {
      if (it.id < 0 || it.id >= a.n_blocks) it.id = -1;
      if (it.id >= 0) {
        const float2 s = *reinterpret_cast<const float2*>(a.scales + ((size_t)it.id * a.Hkv + it.head) * 2);
        it.ks = s.x;
        it.vs = s.y;
      }
    };
    Item cur = locate(p0, seq0), next = locate(p0 + batch, cur.seq);
    fetch_scales(cur);
    int st = 0, issued = 0, turn = 0;   // the next stage, tiles issued (up to `stages`), uses of the stages
    bool ok = true, any = false;
    if (lane == 0) a.split[cta].seq = -1;   // (written again by the lane that finds a unit that goes on)
    __syncwarp();
    for (int pb = p0; pb < p1 && ok; pb += batch) {
      const int p = pb + lane_tile;
      const bool real = cur.tile < cur.tiles;
      const bool opens = cur.tile == 0 || p == p0, ends = cur.tile == cur.tiles - 1;
      const bool final = p + 1 + (ends ? kUnitCost : 0) >= p1;
      const int flags = (opens ? kFirst : 0) | (ends || final ? kLast : 0) | (cur.tile == 0 ? kBegins : 0) | (ends ? kEnds : 0) |
                        (final ? kFinal : 0);
      const uint32_t live = __ballot_sync(0xffffffffu, cur.id >= 0), opening = __ballot_sync(0xffffffffu, opens);
      uint32_t todo = __ballot_sync(0xffffffffu, real && in_tile == 0);   // a bit for each tile, at its first lane
      any = any || todo;
      const uint32_t blocks = (live >> (lane & ~((1 << lppt) - 1))) & ((1u << (1 << lppt)) - 1u);   // of the lane's tile
      const uint32_t bytes = __popc(blocks) * 2 * box * D + (opens ? min(kRows, a.rows - cur.row0) * D * (int)sizeof(Tin) : 0);
      // Tiles are issued a few at a time, each by its own lanes: `sel` has a bit for each at its first lane, and they go to
      // the stages from `base` on.
      const int owner = lane & ~((1 << lppt) - 1);
      auto stage_of = [&](uint32_t sel, int base, int first_lane) {
        const int at = base + __popc(sel & ((1u << first_lane) - 1u));
        return at >= stages ? at - stages : at;
      };
      // the copies: keys and values of each block in one, and the query rows where a unit starts
      auto issue = [&](uint32_t sel, int base) {
        const bool mine = (sel >> owner) & 1u;
        const int at = stage_of(sel, base, owner);
        if (mine && in_tile == 0) mbar_expect_tx(&full[at], bytes);
        __syncwarp();
        if (mine && cur.id >= 0)
          tma_load_4d(smem + at * S::STAGE + in_tile * 2 * box * D, &tm, &full[at], 0, (cur.tile * kTile) & (bs - 1), 0,
                      cur.id * a.Hkv + cur.head);
        for (uint32_t open = sel & opening; open; open &= open - 1u) {   // rows are (token, head) pairs: one copy for each token's heads
          const int from = __ffs(open) - 1;
          const int seq = __shfl_sync(0xffffffffu, cur.seq, from), head = __shfl_sync(0xffffffffu, cur.head, from);
          const int q_at = __shfl_sync(0xffffffffu, at, from);
          const int r0 = __shfl_sync(0xffffffffu, cur.row0, from), r1 = min(r0 + kRows, a.rows);
          const int i = a.by_G(r0) + lane, lo = max(r0, i * a.G), hi = min(r1, (i + 1) * a.G);
          if (lo < hi)
            bulk_load(smem + q_at * S::STAGE + S::KV + (lo - r0) * D * sizeof(Tin),
                      static_cast<const Tin*>(a.q) + ((size_t)seq * a.n_q + i) * a.qstride + (size_t)(head * a.G + lo - i * a.G) * D,
                      (hi - lo) * D * sizeof(Tin), &full[q_at]);
        }
      };
      float ks, lv, vs;   // of the lane's block
      // the tiles' descriptions for the consumers; the scales once for each 16 tokens
      auto publish = [&](uint32_t sel, int base) {
        const bool mine = (sel >> owner) & 1u;
        const int at = stage_of(sel, base, owner);
        if (mine) {
          StageInfo& si = info[at];
          for (int e = 0; e < box / 16; ++e) si.scale[in_tile * (box / 16) + e] = make_float4(ks, lv, vs, 0.f);
          if (in_tile == 0) {
            *reinterpret_cast<int4*>(&si.seq) = make_int4(cur.seq, cur.head, cur.row0, cur.tile * kTile);
            *reinterpret_cast<int2*>(&si.len) = make_int2(lens[cur.seq], flags);
          }
        }
        __syncwarp();
        if (mine && in_tile == 0 && !(a.inject_stall && cta == 0 && pb == p0 && at == 0)) mbar_arrive(&full[at]);
      };
      // up to n of the tiles to do
      auto take = [&](int n) {
        uint32_t rest = todo;
        for (int i = 0; i < n; ++i) rest &= rest - 1u;
        const uint32_t sel = todo & ~rest;
        todo = rest;
        return sel;
      };
      uint32_t early = 0u;
      if (pb == p0) {   // the first tiles' copies do not wait for their scales
        early = take(1);
        issue(early, 0);
        const uint32_t more = take(min(stages, kEarly) - 1);
        issue(more, 1);
        early |= more;
      }
      ks = cur.id >= 0 ? cur.ks : 0.f;
      vs = cur.vs;
      lv = fmaxf(__log2f(vs), (float)kvc::kMinScaleExp);   // (decides when the reference is raised, no weight)
      if (pb == p0) {
        publish(early, 0);
        issued = __popc(early);
        st = issued == stages ? 0 : issued;
        turn = issued == stages ? 1 : 0;
      }
      fetch_scales(next);
      const Item later = locate(pb + 2 * batch, next.seq);
      while (todo) {
        // wait for one stage; a second tile goes along if its stage is free by now
        if (turn > 0) ok = warp_all(mbar_wait(&empty[st], (turn - 1) & 1, wc, wsite(1, st, turn)));
        if (!ok) break;
        const int base = st;
        if (++st == stages) { st = 0; ++turn; }
        const bool two = (todo & (todo - 1u)) && (turn == 0 || warp_all(mbar_test(&empty[st], (turn - 1) & 1)));
        if (two && ++st == stages) { st = 0; ++turn; }
        const uint32_t sel = take(two ? 2 : 1);
        issue(sel, base);
        publish(sel, base);
        issued = min(issued + __popc(sel), stages);
      }
      // the unit that goes on behind this stretch, for the join
      if (real && final && !ends && in_tile == 0) {
        const int c0 = (p - cur.tile) / per, parts = (p - cur.tile + cur.tiles - 1) / per - c0 + 1;
        const int n_rows = min(kRows, a.rows - cur.row0), share = (n_rows * (D / 4) + parts - 2) / (parts - 1);
        int log_lanes = 0;
        while ((2 << log_lanes) <= min(kJoinLanes, parts) && (share << (log_lanes + 1)) <= kJoinThreads) ++log_lanes;
        a.split[cta] = Split{cur.seq, cur.head, cur.row0, n_rows, c0, parts, share, log_lanes};
      }
      cur = next;
      next = later;
    }
    if (!any) {   // an empty stretch, or two places behind a unit
      if (lane == 0) {
        info[0].flags = kNone;
        mbar_arrive(&full[0]);
      }
      __syncwarp();
    }
    // never leave with copies in flight
    const WaitCtx dw{never, nullptr, a.wait_ns};
    for (int i = 0; i < issued; ++i) {
      if (--st < 0) { st = stages - 1; --turn; }
      mbar_wait(&full[st], turn & 1, dw);
    }
    return;
  }

  if (warp == kWarps + 1) {   // ---------------- output
    // sequences without tokens: zero rows
    for (int s = cta; s < a.B; s += gridDim.x)
      if (length(s) == 0) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<Tin*>(a.out) + (size_t)s * a.n_q * a.Hq * D);
        const int n16 = a.n_q * a.Hq * D * (int)sizeof(Tin) / 16;
        for (int i = lane; i < n16; i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    // joins the four warps' parts of each unit's stretch
    for (int use = 0;; ++use) {
      if (!warp_all(mbar_wait(parts_full, use & 1, wc, wsite(4, 0, use)))) return;
      const UnitInfo u = *unit_info;
      if (u.flags & kNone) return;
      const int n_rows = min(kRows, a.rows - u.row0);
      const bool begins = u.flags & kBegins, whole = begins && (u.flags & kEnds);
      const int place = 2 * cta + (begins ? 1 : 0);   // of a part of a unit that goes on, or that an earlier CTA began
      // the parts' weights, a lane for each warp's part of a row
      for (int at = 0; at < 4 * n_rows; at += 32) {
        const int r = min((at + lane) >> 2, n_rows - 1), w = lane & 3;
        const float2 ml = *reinterpret_cast<const float2*>(red_ml + (w * part_rows + r) * 2);
        float m = fmaxf(ml.x, __shfl_xor_sync(0xffffffffu, ml.x, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const float half = ex2(0.5f * (ml.x - m)), f = half * half;
        float l = (half * ml.y) * half;
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (at + lane < 4 * n_rows) {
          wgt[4 * r + w] = !whole ? f : (l == 0.f ? 0.f : f / l);   // (a row that sees nothing is zero)
          if (!whole && w == 0) {
            a.part_ml[(size_t)place * 2 * kMaxRows + r] = m;
            a.part_ml[(size_t)place * 2 * kMaxRows + kMaxRows + r] = l;
          }
        }
      }
      __syncwarp();
#pragma unroll 4
      for (int v = lane; v < n_rows * (D / 4); v += 32) {
        const int r = v / (D / 4), c = v % (D / 4);
        const float4 f = *reinterpret_cast<const float4*>(wgt + 4 * r);
        const float* x = red + r * D + 4 * c;
        const float4 x0 = *reinterpret_cast<const float4*>(x), x1 = *reinterpret_cast<const float4*>(x + part_rows * D);
        const float4 x2 = *reinterpret_cast<const float4*>(x + 2 * part_rows * D), x3 = *reinterpret_cast<const float4*>(x + 3 * part_rows * D);
        float4 y;
        y.x = f.x * x0.x + f.y * x1.x + f.z * x2.x + f.w * x3.x;
        y.y = f.x * x0.y + f.y * x1.y + f.z * x2.y + f.w * x3.y;
        y.z = f.x * x0.z + f.y * x1.z + f.z * x2.z + f.w * x3.z;
        y.w = f.x * x0.w + f.y * x1.w + f.z * x2.w + f.w * x3.w;
        if (whole) {
          const int row = u.row0 + r, i = a.by_G(row), h = u.head * a.G + row - i * a.G;
          Tin* dst = static_cast<Tin*>(a.out) + (((size_t)u.seq * a.n_q + i) * a.Hq + h) * D + 4 * c;
          if (sizeof(Tin) == 2)
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
          else
            *reinterpret_cast<float4*>(dst) = y;
        } else {
          *reinterpret_cast<float4*>(a.part_o + ((size_t)place * kMaxRows + r) * D + 4 * c) = y;
        }
      }
      if (u.flags & kFinal) return;
      __syncwarp();
      if (lane == 0) mbar_arrive(parts_empty);
    }
  }

  // ---------------- consumers: a warp takes kSlices times 16 tokens of each tile
  constexpr int kSlices = kTile / 16 / kWarps;
  const int g = lane >> 2, t4 = lane & 3;
  const int slot = kSlices * warp;      // the warp's first 16 tokens of a tile
  const int krow = ((16 * slot) >> lbox) * 2 * box + ((16 * slot) & (box - 1)), kslice = box == 16 ? 32 : 16;   // their key rows in a stage, and from there to the next 16's
  constexpr int KS = D / 16;            // k-steps of the first product
  constexpr int MT = D / 16;            // 16-row tiles of O^T
  uint32_t qf[NT][KS][2], ql[kSplit ? NT : 1][kSplit ? KS : 1][2];   // Q^T operands (and the rows' low terms)
  float o[NT][MT][4];
  float ref[NT][2], sum[NT][2], rs[NT][2];
  int lim[NT][2];                       // tokens that a row sees
  int row0 = 0;
  bool begins = false;                  // the CTA's stretch of the unit starts with its first tile
  uint32_t units_done = 0;
  bool ready = false;                   // the next tile had come when the last one was begun (a test's answer takes 100 cycles)
  for (int k = 0, st = 0, phase = 0;; ++k) {
    if (!warp_all(ready) && !warp_all(mbar_wait(&full[st], phase, wc, wsite(2, st, k)))) return;
    const StageInfo& si = info[st];
    const char* sk = smem + st * S::STAGE;
    const int4 where = *reinterpret_cast<const int4*>(&si.seq);   // sequence, head, first row, first token
    const int2 what = *reinterpret_cast<const int2*>(&si.len);    // length, flags
    const int flags = what.y;
    if (flags & kNone) {
      if (tid == 0) unit_info->flags = kNone;
      __syncwarp();
      if (lane == 0) mbar_arrive(parts_full);
      return;
    }
    const int len = what.x, tok = where.w + 16 * slot;
    if (flags & kFirst) {
      row0 = where.z;
      begins = (flags & kBegins) != 0;
      const char* sq = sk + S::KV;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // row g of this eight: the thread's d are those whose key bytes it reads (16-byte column c = word j / 4)
        const int row = row0 + 8 * n + g;
        const bool in = row < a.rows;
        float x[KS][4];
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          const int at = D == 128 ? (2 * t4 + j / 4) * 16 + (j % 4) * 4 : t4 * 16 + j * 4;
          if (sizeof(Tin) == 2) {
            const uint2 u = *reinterpret_cast<const uint2*>(sq + ((8 * n + g) * D + at) * 2);
            x[j][0] = bf16_lo(u.x); x[j][1] = bf16_hi(u.x); x[j][2] = bf16_lo(u.y); x[j][3] = bf16_hi(u.y);
          } else {
            const float4 u = *reinterpret_cast<const float4*>(sq + ((8 * n + g) * D + at) * 4);
            x[j][0] = u.x; x[j][1] = u.y; x[j][2] = u.z; x[j][3] = u.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[j][e] = in ? x[j][e] : 0.f;
            top = fmaxf(top, fabsf(x[j][e]));
          }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the row times 2^-e, its maximum in [2^7, 2^8): exact, and elements 2^-21 of it are still normal in fp16
        int e = (int)(__float_as_uint(top) >> 23) - 127 - 7;
        e = min(max(e, -119), 119);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          const float y0 = x[j][0] * down, y1 = x[j][1] * down, y2 = x[j][2] * down, y3 = x[j][3] * down;
          qf[n][j][0] = pack_f16(y0, y1);
          qf[n][j][1] = pack_f16(y2, y3);
          if (kSplit) {
            const float2 h0 = unpack_f16(qf[n][j][0]), h1 = unpack_f16(qf[n][j][1]);
            ql[kSplit ? n : 0][kSplit ? j : 0][0] = pack_f16(y0 - h0.x, y1 - h0.y);
            ql[kSplit ? n : 0][kSplit ? j : 0][1] = pack_f16(y2 - h1.x, y3 - h1.y);
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {   // the thread's score columns are rows 2 t4 + c
          const int r = row0 + 8 * n + 2 * t4 + c;
          rs[n][c] = __shfl_sync(0xffffffffu, up, (2 * t4 + c) * 4) * a.scale_log2;
          lim[n][c] = len - a.n_q + a.by_G(r) + 1;
          ref[n][c] = kNoRef;
          sum[n][c] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[n][i][c] = 0.f;
      }
    }
    const int st_next = st + 1 == stages ? 0 : st + 1, phase_next = st_next ? phase : phase ^ 1;
    ready = mbar_test(&full[st_next], phase_next);
    {
      const float4* sc = si.scale + slot;
      // One or two slices of 16 tokens: `u` the first, its first token `at`.  At the sequence's end (at_end), or where a
      // slice has no block, they are taken one by one and masked.
      auto slices = [&](auto count, auto at_end, int u, int at) {
        constexpr int NS = decltype(count)::value;
        constexpr bool kEdge = decltype(at_end)::value;
        constexpr int NA = NS * NT >= 4 ? 1 : 4 / (NS * NT);   // sums side by side: a product waits 30 cycles for the last one
        float s[NS][NT][4], sa[NA][NS][NT][4];
#pragma unroll
        for (int x = 0; x < NA; ++x)
#pragma unroll
          for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 4; ++c) sa[x][i][n][c] = 0.f;
        {
          uint32_t kw[NS][2][KS];   // keys: rows g and g + 8 of the 16 tokens
#pragma unroll
          for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int c = 0; c < KS / 4; ++c) {
                const int row = krow + (u + i) * kslice + token_of(g) + 8 * r;
                const uint4 x = *reinterpret_cast<const uint4*>(sk + swz<D>(row, (D == 128 ? 2 * t4 + c : t4) * 16));
                kw[i][r][4 * c] = x.x; kw[i][r][4 * c + 1] = x.y; kw[i][r][4 * c + 2] = x.z; kw[i][r][4 * c + 3] = x.w;
              }
#pragma unroll
          for (int j = 0; j < KS; ++j)
#pragma unroll
            for (int i = 0; i < NS; ++i) {
              uint32_t a0, a1, a2, a3;
              codes_to_f16<T>(kw[i][0][j], a0, a2);
              codes_to_f16<T>(kw[i][1][j], a1, a3);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma16816(sa[j % NA][i][n], a0, a1, a2, a3, qf[n][j][0], qf[n][j][1]);
                if (kSplit)
                  mma16816(sa[j % NA][i][n], a0, a1, a2, a3, ql[kSplit ? n : 0][kSplit ? j : 0][0], ql[kSplit ? n : 0][kSplit ? j : 0][1]);
              }
            }
        }
        uint32_t vw[NS][4][D / 32];   // values: the thread's four tokens of a slice, D / 8 bytes at column g
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = krow + (u + i) * kslice + box + 8 * (r >> 1) + token_of(2 * t4 + (r & 1));
            if (D == 128) {
              const uint4 x = *reinterpret_cast<const uint4*>(sk + swz<D>(row, g * 16));
              vw[i][r][0] = x.x; vw[i][r][1] = x.y; vw[i][r][D / 32 - 2] = x.z; vw[i][r][D / 32 - 1] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(sk + swz<D>(row, g * 8));
              vw[i][r][0] = x.x; vw[i][r][1] = x.y;
            }
          }
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              s[i][n][c] = sa[0][i][n][c];
#pragma unroll
              for (int x = 1; x < NA; ++x) s[i][n][c] += sa[x][i][n][c];
            }
        // to log2 units, from the row's reference; tokens that a row does not see
        auto hidden = [&](int n, int c) { return kEdge && at + 8 * (c >> 1) + token_of(g) >= lim[n][c & 1]; };
        float p[NS][NT][4];
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const float ks = sc[u + i].x;
          float most = -INFINITY;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              p[i][n][c] = hidden(n, c) ? -INFINITY : fmaf(s[i][n][c], ks * rs[n][c & 1], -ref[n][c & 1]);
              most = fmaxf(most, p[i][n][c]);
            }
          top = fmaxf(top, most + sc[u + i].y);
        }
        if (__any_sync(0xffffffffu, top > kRaiseAt)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float f[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float m = -INFINITY;
#pragma unroll
              for (int i = 0; i < NS; ++i)
#pragma unroll
                for (int e = c; e < 4; e += 2) {
                  p[i][n][e] = hidden(n, e) ? -INFINITY : s[i][n][e] * (sc[u + i].x * rs[n][c]);
                  m = fmaxf(m, p[i][n][e] + sc[u + i].y);
                }
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
              const float to = fmaxf(ref[n][c], m - kRefBelow);
              const float half = ex2(0.5f * (ref[n][c] - to));
              f[c] = half * half;
              ref[n][c] = to;
              sum[n][c] = (sum[n][c] * half) * half;
#pragma unroll
              for (int i = 0; i < NS; ++i)
#pragma unroll
                for (int e = c; e < 4; e += 2) {   // (no NaN is dropped; scores so large that `to` rounds away log2(vs) stay in fp16's range)
                  const float x = p[i][n][e] - to, limit = kRaiseAt - sc[u + i].y;
                  p[i][n][e] = x > limit ? limit : x;
                }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[n][i][0] *= f[0]; o[n][i][1] *= f[1];
              o[n][i][2] *= f[0]; o[n][i][3] *= f[1];
            }
          }
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const float vs = sc[u + i].z;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int c = 0; c < 4; ++c) p[i][n][c] = ex2(p[i][n][c]);
            sum[n][0] += p[i][n][0] + p[i][n][2];
            sum[n][1] += p[i][n][1] + p[i][n][3];
#pragma unroll
            for (int c = 0; c < 4; ++c) p[i][n][c] *= vs;
          }
        }
        // O^T += V^T P^T.  At the end there is one pass for each new token, over the value codes that it sees, and only its
        // rows take the sums: with weights of zero alone, a NaN code behind a row's last visible token would reach it.
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          uint32_t pb[NT][2], pl[kSplit ? NT : 1][2];   // P^T operands (and their low terms)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float* x = p[i][n];
            const uint32_t h0 = pack_f16(x[0], x[1]), h1 = pack_f16(x[2], x[3]);
            pb[n][0] = transpose8x8(h0);
            pb[n][1] = transpose8x8(h1);
            if (kSplit) {
              const float2 y0 = unpack_f16(h0), y1 = unpack_f16(h1);
              pl[kSplit ? n : 0][0] = transpose8x8(pack_f16(x[0] - y0.x, x[1] - y0.y));
              pl[kSplit ? n : 0][1] = transpose8x8(pack_f16(x[2] - y1.x, x[3] - y1.y));
            }
          }
          auto weigh = [&](int sees) {
            bool seen[4];   // of the thread's four tokens
#pragma unroll
            for (int r = 0; r < 4; ++r) seen[r] = !kEdge || at + 8 * (r >> 1) + token_of(2 * t4 + (r & 1)) < sees;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              const uint32_t v0 = seen[0] ? vw[i][0][c] : 0u, v1 = seen[1] ? vw[i][1][c] : 0u;
              const uint32_t v2 = seen[2] ? vw[i][2][c] : 0u, v3 = seen[3] ? vw[i][3][c] : 0u;
              // bytes of the same d from the tokens of a pair, side by side
              const uint32_t lo01 = __byte_perm(v0, v1, 0x5140), hi01 = __byte_perm(v0, v1, 0x7362);
              const uint32_t lo23 = __byte_perm(v2, v3, 0x5140), hi23 = __byte_perm(v2, v3, 0x7362);
              uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
              codes_to_f16<T>(lo01, a0, a1);
              codes_to_f16<T>(lo23, a2, a3);
              codes_to_f16<T>(hi01, b0, b1);
              codes_to_f16<T>(hi23, b2, b3);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float x[2][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) { x[0][e] = o[n][2 * c][e]; x[1][e] = o[n][2 * c + 1][e]; }
                mma16816(x[0], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                mma16816(x[1], b0, b1, b2, b3, pb[n][0], pb[n][1]);
                if (kSplit) {
                  mma16816(x[0], a0, a1, a2, a3, pl[kSplit ? n : 0][0], pl[kSplit ? n : 0][1]);
                  mma16816(x[1], b0, b1, b2, b3, pl[kSplit ? n : 0][0], pl[kSplit ? n : 0][1]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (!kEdge || lim[n][e & 1] == sees) { o[n][2 * c][e] = x[0][e]; o[n][2 * c + 1][e] = x[1][e]; }
              }
            }
          };
          if (!kEdge) {
            weigh(0);
          } else {
#pragma unroll 1
            for (int sees = max(len - a.n_q + 1, at + 1); sees <= len; ++sees) weigh(sees);
          }
        }
      };
      using One = std::integral_constant<int, 1>;
      // two slices side by side where there are two and their operands fit the registers
      constexpr int kSide = kSlices > 1 && NT * D <= 128 ? 2 : 1;
      bool whole = tok + 16 * kSlices <= len - a.n_q + 1;
#pragma unroll
      for (int u = 0; u < kSlices; ++u) whole = whole && sc[u].x != 0.f;
      if (whole) {
#pragma unroll 1
        for (int u = 0; u < kSlices; u += kSide) slices(std::integral_constant<int, kSide>{}, std::false_type{}, u, 0);
      } else {
#pragma unroll 1
        for (int u = 0; u < kSlices; ++u)
          if (tok + 16 * u < len && sc[u].x != 0.f) slices(One{}, std::true_type{}, u, tok + 16 * u);
      }
    }
    const UnitInfo u{where.x, where.y, row0, (flags & (kEnds | kFinal)) | (begins ? kBegins : 0)};
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
    st = st_next;
    phase = phase_next;

    if (flags & kLast) {   // this stretch of the unit ends: the warp's part to the output's warp
      if (units_done > 0 && !warp_all(mbar_wait(parts_empty, (units_done - 1) & 1, wc, wsite(3, 0, k)))) return;
      ++units_done;
      if (tid == 0) *unit_info = u;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float l = sum[n][c];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          const int r = 8 * n + 2 * t4 + c;
          if (r < part_rows) {   // (rows behind the unit's last one are written and not read)
            if (g == 0) *reinterpret_cast<float2*>(red_ml + (warp * part_rows + r) * 2) = make_float2(ref[n][c], l);
            // O^T: the thread holds d = 2 MT g .. 2 MT g + 2 MT - 1 of the row
            float* dst = red + (warp * part_rows + r) * D + 2 * MT * g;
#pragma unroll
            for (int i = 0; i < MT; i += 2)
              *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(o[n][i][c], o[n][i][c + 2], o[n][i + 1][c], o[n][i + 1][c + 2]);
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(parts_full);
    }
    if (flags & kFinal) return;
  }
}

// Joins the units that lie in several stretches: the parts stand in the begin slot of the unit's first CTA and in the
// continue slots of the others, and are added in a fixed order.  Each CTA whose stretch a unit goes on behind (all of the
// unit's but the last) takes a share of the unit's output; 16 bytes of it and a power of two of neighbouring lanes, which
// share the parts.
template <typename Tin, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(Args a) {
  const int tid = threadIdx.x;
  kvc::pdl_launch_next();
  kvc::pdl_wait_previous();
  const Split u = a.split[blockIdx.x];
  if (u.seq < 0) return;
  const int v0 = ((int)blockIdx.x - u.c0) * u.share, v1 = min(u.n_rows * (D / 4), v0 + u.share);
  const int lanes = 1 << u.log_lanes, e = tid & (lanes - 1);
  for (int vb = v0; vb < v1; vb += kJoinThreads >> u.log_lanes) {
    const int v = vb + (tid >> u.log_lanes), r = v / (D / 4), c = v % (D / 4);
    const bool in = v < v1;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = kNoRef, l = 0.f;
    auto add = [&](float om, float ol, float4 y) {
      const float top = fmaxf(m, om), fh = ex2(0.5f * (m - top)), gh = ex2(0.5f * (om - top)), f = fh * fh, g = gh * gh;
      m = top;
      l = (l * fh) * fh + (ol * gh) * gh;
      x.x = x.x * f + y.x * g; x.y = x.y * f + y.y * g;
      x.z = x.z * f + y.z * g; x.w = x.w * f + y.w * g;
    };
    if (in)
#pragma unroll 2
      for (int p = e; p < u.parts; p += lanes) {
        const int slot = p == 0 ? 2 * u.c0 + 1 : 2 * (u.c0 + p);
        const float* ml = a.part_ml + (size_t)slot * 2 * kMaxRows + r;
        const float4 y = *reinterpret_cast<const float4*>(a.part_o + ((size_t)slot * kMaxRows + r) * D + 4 * c);
        add(ml[0], ml[kMaxRows], y);
      }
    for (int o = 1; o < lanes; o <<= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m, o), ol = __shfl_xor_sync(0xffffffffu, l, o);
      float4 y;
      y.x = __shfl_xor_sync(0xffffffffu, x.x, o);
      y.y = __shfl_xor_sync(0xffffffffu, x.y, o);
      y.z = __shfl_xor_sync(0xffffffffu, x.z, o);
      y.w = __shfl_xor_sync(0xffffffffu, x.w, o);
      add(om, ol, y);
    }
    if (in && e == 0) {
      const float il = l == 0.f ? 0.f : 1.f / l;
      const int row = u.row0 + r, i = a.by_G(row), h = u.head * a.G + row - i * a.G;
      Tin* dst = static_cast<Tin*>(a.out) + (((size_t)u.seq * a.n_q + i) * a.Hq + h) * D + 4 * c;
      if (sizeof(Tin) == 2)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(x.x * il, x.y * il), pack_bf16(x.z * il, x.w * il));
      else
        *reinterpret_cast<float4*>(dst) = make_float4(x.x * il, x.y * il, x.z * il, x.w * il);
    }
  }
}

}  // namespace ca
}  // namespace liger
