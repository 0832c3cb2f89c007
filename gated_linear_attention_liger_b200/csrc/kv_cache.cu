// kv_cache.cu -- C ABI of the paged 8-bit key/value cache (include/liger_attn.h): block
// assignment, the quantising append and attention over the cache.  Argument checks and
// launches on the caller's stream; no allocation, no host synchronisation.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <utility>

#include "cached_attn.cuh"
#include "hooks.cuh"
#include "kv_cache.cuh"
#include "liger_attn.h"

namespace {

using liger::kvc::KvType;
using liger::kvc::kE4m3;
using liger::kvc::kInt8;

// Error word of the cached attention (bit 0: a bounded wait gave up; word 1: the first
// site), one per device; read and cleared by liger_attn_cached_status().
__device__ uint32_t g_cached_attn_err[2];

struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
  Range(const Range&) = delete;
  Range& operator=(const Range&) = delete;
};

liger_status fail(liger_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  liger::set_last_error(s, buf);
  return s;
}
liger_status cuda_fail(cudaError_t e, const char* where) {
  cudaGetLastError();   // reported here: not left for the next call
  return fail(LIGER_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorString(e), cudaGetErrorName(e));
}
bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int log2_block(int bs) {
  switch (bs) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    default: return -1;
  }
}

// What the three entry points share: the cache's shape.
liger_status check_cache(int n_blocks, int block_size) {
  if (n_blocks < 1) return fail(LIGER_ERR_INVALID_ARG, "need n_blocks >= 1 (n_blocks=%d)", n_blocks);
  if (block_size < 1) return fail(LIGER_ERR_INVALID_ARG, "need block_size >= 1 (block_size=%d)", block_size);
  if (log2_block(block_size) < 0)
    return fail(LIGER_ERR_UNSUPPORTED, "block_size=%d (supported: 16, 32, 64, 128)", block_size);
  if ((long long)n_blocks * block_size > 0x7fffffffLL)
    return fail(LIGER_ERR_UNSUPPORTED, "n_blocks * block_size must fit 31 bits (slots are int32)");
  return LIGER_OK;
}
liger_status check_sequences(int B, int width, int block_size) {
  if (B < 1 || width < 1)
    return fail(LIGER_ERR_INVALID_ARG, "need B >= 1 and table_width >= 1 (B=%d table_width=%d)", B, width);
  if (B > liger::kvc::kMaxSeqs)
    return fail(LIGER_ERR_UNSUPPORTED, "B=%d sequences (at most %d)", B, liger::kvc::kMaxSeqs);
  if ((long long)width * block_size > 0x7fffffffLL - 128)
    return fail(LIGER_ERR_UNSUPPORTED, "table_width * block_size must fit 31 bits");
  return LIGER_OK;
}
liger_status check_types(int Hkv, int d, liger_dtype dt, liger_kv_dtype kv) {
  if (Hkv < 1) return fail(LIGER_ERR_INVALID_ARG, "need Hkv >= 1 (Hkv=%d)", Hkv);
  if (dt != LIGER_BF16 && dt != LIGER_FP32) return fail(LIGER_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
  if (kv != LIGER_KV_E4M3 && kv != LIGER_KV_INT8) return fail(LIGER_ERR_INVALID_ARG, "unknown cache dtype %d", (int)kv);
  if (d != 64 && d != 128) return fail(LIGER_ERR_UNSUPPORTED, "head dim d=%d (supported: 64, 128)", d);
  return LIGER_OK;
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
  if (e == cudaSuccess) liger::count_kernel_launches(1);
  return e;
}

// ------------------------------------------------------------------ assign

// Slots that one CTA writes along with everything else.  More go to many CTAs.
constexpr int kOneCtaSlots = 16384;

template <bool SLOTS, bool STATE>
cudaError_t launch_assign(const liger::kvc::AssignArgs& a, int ctas, cudaStream_t s) {
  auto kern = liger::kvc::assign_kernel<SLOTS, STATE>;
  const size_t smem = liger::kvc::assign_smem_bytes(a.B);
  if (smem > 40 * 1024) {   // (static shared memory counts toward the default 48 KB)
    // the limit belongs to the kernel, not to the call: the most that any call takes, since another thread's call may
    // set it between this one's setting and launch
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)liger::kvc::assign_smem_bytes(liger::kvc::kMaxSeqs));
    if (e != cudaSuccess) return e;
  }
  return launch(kern, dim3((unsigned)ctas), liger::kvc::kAssignThreads, smem, s, a);
}

// ------------------------------------------------------------------ append

template <typename Tin, KvType T, int D, int BS>
cudaError_t launch_append(const liger::kvc::AppendArgs& a, cudaStream_t s) {
  using S = liger::kvc::AppendShape<Tin, D, BS>;
  // One token a CTA while that is a few CTAs an SM (each run then has its own); else a block's worth, so that a prompt's
  // tokens that lead no run do not cost a CTA each.
  const int heads = (a.Hkv + S::kHeads - 1) / S::kHeads;
  const int range = (long long)a.N * heads <= 32LL * liger::device_sm_count() ? 1 : S::kRange;
  const dim3 grid((unsigned)((a.N + range - 1) / range), (unsigned)heads);
  return launch(liger::kvc::append_kernel<Tin, T, D, BS>, grid, S::kThreads, 0, s, a, range);
}
template <typename Tin, KvType T, int D>
cudaError_t append_bs(const liger::kvc::AppendArgs& a, int bs, cudaStream_t s) {
  switch (bs) {
    case 16: return launch_append<Tin, T, D, 16>(a, s);
    case 32: return launch_append<Tin, T, D, 32>(a, s);
    case 64: return launch_append<Tin, T, D, 64>(a, s);
    default: return launch_append<Tin, T, D, 128>(a, s);
  }
}
template <typename Tin>
cudaError_t append_t(const liger::kvc::AppendArgs& a, int d, int bs, liger_kv_dtype kv, cudaStream_t s) {
  if (kv == LIGER_KV_E4M3) return d == 64 ? append_bs<Tin, kE4m3, 64>(a, bs, s) : append_bs<Tin, kE4m3, 128>(a, bs, s);
  return d == 64 ? append_bs<Tin, kInt8, 64>(a, bs, s) : append_bs<Tin, kInt8, 128>(a, bs, s);
}

// ------------------------------------------------------------------ attention

constexpr int kCtasPerSm = 2;
constexpr int kMaxCtas = 4096;

struct AttnLayout {
  int ctas;
  size_t off_ml, off_o, off_split, total;
};
AttnLayout attn_layout(int d) {
  AttnLayout L;
  L.ctas = liger::device_sm_count() * kCtasPerSm;
  if (L.ctas > kMaxCtas) L.ctas = kMaxCtas;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  L.off_ml = 0;
  L.off_o = up(L.off_ml + (size_t)L.ctas * 2 * 2 * liger::ca::kMaxRows * 4);
  L.off_split = up(L.off_o + (size_t)L.ctas * 2 * liger::ca::kMaxRows * d * 4);
  L.total = up(L.off_split + (size_t)L.ctas * sizeof(liger::ca::Split));
  return L;
}

template <typename Tin, int D, KvType T, int NT>
liger_status launch_attn(const CUtensorMap& tm, liger::ca::Args a, int ctas, cudaStream_t s) {
  using S = liger::ca::Smem<Tin, D, NT>;
  // shared memory of one CTA with two on an SM (228 KB, 1 KB of it the system's, each), else alone
  constexpr int kShare = (228 * 1024) / kCtasPerSm - 1024, kAlone = 227 * 1024;
  const int fixed = (int)S::bytes(0, a.rows, a.B);
  int stages = (kShare - fixed) / (int)S::STAGE;
  if (stages < 3) {   // thousands of sequences: their prefix sums take the second CTA's place
    stages = (kAlone - fixed) / (int)S::STAGE;
    ctas = (ctas + kCtasPerSm - 1) / kCtasPerSm;
  }
  if (stages > S::MAX_STAGES) stages = S::MAX_STAGES;
  a.by_ctas = liger::ca::Divisor::of(ctas);
  const int smem = (int)S::bytes(stages, a.rows, a.B);
  auto kern = liger::ca::cached_attn_kernel<Tin, D, T, NT>;
  // (whatever this call takes: the limit is the kernel's, and calls from other threads set it too)
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kAlone);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(cached attention)");
  liger::mark_dominant_start(s);
  e = launch(kern, dim3((unsigned)ctas), liger::ca::kThreads, (size_t)smem, s, tm, a, stages);
  if (e != cudaSuccess) return cuda_fail(e, "cached attention launch");
  liger::mark_dominant_stop(s);
  e = launch(liger::ca::join_kernel<Tin, D>, dim3((unsigned)ctas), liger::ca::kJoinThreads, 0, s, a);
  if (e != cudaSuccess) return cuda_fail(e, "cached attention join launch");
  return LIGER_OK;
}
template <typename Tin, int D, KvType T>
liger_status attn_nt(const CUtensorMap& tm, const liger::ca::Args& a, int ctas, cudaStream_t s) {
  return a.rows <= 8 ? launch_attn<Tin, D, T, 1>(tm, a, ctas, s) : launch_attn<Tin, D, T, 2>(tm, a, ctas, s);
}
template <typename Tin>
liger_status attn_t(const CUtensorMap& tm, const liger::ca::Args& a, int d, liger_kv_dtype kv, int ctas, cudaStream_t s) {
  if (kv == LIGER_KV_E4M3) return d == 64 ? attn_nt<Tin, 64, kE4m3>(tm, a, ctas, s) : attn_nt<Tin, 128, kE4m3>(tm, a, ctas, s);
  return d == 64 ? attn_nt<Tin, 64, kInt8>(tm, a, ctas, s) : attn_nt<Tin, 128, kInt8>(tm, a, ctas, s);
}

}  // namespace

extern "C" {

liger_status liger_kv_cache_assign(const int32_t* new_lens, const int32_t* seq_lens, int32_t* block_table,
                                   int32_t* free_blocks, const int32_t* free_span, int32_t* slot_map, int32_t* cu_new,
                                   int32_t* seq_lens_out, int32_t* free_span_out, int B, int table_width, int n_blocks,
                                   int block_size, int n_slots, void* stream) {
  const Range range("liger_kv_cache_assign");
  liger::clear_last_error();
  liger_status st = check_cache(n_blocks, block_size);
  if (st == LIGER_OK) st = check_sequences(B, table_width, block_size);
  if (st != LIGER_OK) return st;
  if (n_slots < 0) return fail(LIGER_ERR_INVALID_ARG, "need n_slots >= 0 (n_slots=%d)", n_slots);
  if (n_slots > 0x7fffffff - 1024) return fail(LIGER_ERR_UNSUPPORTED, "too many slots (n_slots=%d)", n_slots);
  if (!new_lens || !seq_lens || !block_table || !free_blocks || !free_span || (n_slots && !slot_map) || !cu_new ||
      !seq_lens_out || !free_span_out)
    return fail(LIGER_ERR_INVALID_ARG, "all pointers must be non-null");
  const void* ptrs[] = {new_lens, seq_lens, block_table, free_blocks, free_span, cu_new, seq_lens_out, free_span_out};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return fail(LIGER_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
  if (!aligned(slot_map, 16)) return fail(LIGER_ERR_INVALID_ARG, "slot_map must be 16-byte aligned");
  const liger::kvc::AssignArgs a{new_lens, seq_lens, block_table, free_blocks, free_span, slot_map, cu_new, seq_lens_out,
                                 free_span_out, B, table_width, n_blocks, log2_block(block_size), n_slots};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (n_slots <= kOneCtaSlots) {
    liger::mark_dominant_start(s);
    e = launch_assign<true, true>(a, 1, s);
  } else {
    const long long ctas = ((long long)n_slots + 4 * liger::kvc::kAssignThreads - 1) / (4 * liger::kvc::kAssignThreads);
    const long long most = 2LL * liger::device_sm_count();   // (each scans all sequences; all resident up to 7000 of them, above
                                                             // that their sums leave room for one CTA an SM, and half run later)
    const int n = (int)(ctas < most ? ctas : most);
    liger::mark_dominant_start(s);
    if (seq_lens_out != seq_lens && free_span_out != free_span) {
      e = launch_assign<true, true>(a, n, s);
    } else {   // every CTA reads the lengths and the span: they change when all have
      e = launch_assign<true, false>(a, n, s);
      if (e == cudaSuccess) e = launch_assign<false, true>(a, 1, s);
    }
  }
  liger::mark_dominant_stop(s);
  return e == cudaSuccess ? LIGER_OK : cuda_fail(e, "cache assignment launch");
}

liger_status liger_kv_cache_append(const void* k, const void* v, const int32_t* slot_map, void* cache, float* scales,
                                   int n_tokens, int Hkv, int d, int n_blocks, int block_size, long long k_stride,
                                   long long v_stride, liger_dtype dt, liger_kv_dtype kv_dt, void* stream) {
  const Range range("liger_kv_cache_append");
  liger::clear_last_error();
  liger_status st = check_types(Hkv, d, dt, kv_dt);
  if (st == LIGER_OK) st = check_cache(n_blocks, block_size);
  if (st != LIGER_OK) return st;
  if (n_tokens < 0) return fail(LIGER_ERR_INVALID_ARG, "need n_tokens >= 0 (n_tokens=%d)", n_tokens);
  if (n_tokens > 0x7fffffff - 1024) return fail(LIGER_ERR_UNSUPPORTED, "too many tokens (n_tokens=%d)", n_tokens);
  if (Hkv > 65535) return fail(LIGER_ERR_UNSUPPORTED, "too many kv heads (Hkv=%d)", Hkv);
  const int per16 = dt == LIGER_BF16 ? 8 : 4;
  if (k_stride < (long long)Hkv * d || v_stride < (long long)Hkv * d || k_stride % per16 || v_stride % per16)
    return fail(LIGER_ERR_INVALID_ARG, "token strides must be at least Hkv * d elements and a multiple of 16 bytes");
  if (n_tokens == 0) return LIGER_OK;
  if (!k || !v || !slot_map || !cache || !scales) return fail(LIGER_ERR_INVALID_ARG, "all pointers must be non-null");
  const void* ptrs[] = {k, v, cache};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return fail(LIGER_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  if (!aligned(slot_map, 4) || !aligned(scales, 8))
    return fail(LIGER_ERR_INVALID_ARG, "slot_map must be 4-byte and scales 8-byte aligned");
  const liger::kvc::AppendArgs a{k, v, slot_map, static_cast<uint8_t*>(cache), scales, (long)k_stride, (long)v_stride,
                                 n_tokens, Hkv, n_blocks * block_size};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  liger::mark_dominant_start(s);
  const cudaError_t e = dt == LIGER_BF16 ? append_t<__nv_bfloat16>(a, d, block_size, kv_dt, s)
                                         : append_t<float>(a, d, block_size, kv_dt, s);
  liger::mark_dominant_stop(s);
  return e == cudaSuccess ? LIGER_OK : cuda_fail(e, "cache append launch");
}

size_t liger_attn_cached_workspace_size(int d) { return d == 64 || d == 128 ? attn_layout(d).total : 0; }

liger_status liger_attn_cached(const void* q, const void* cache, const float* scales, const int32_t* block_table,
                               const int32_t* seq_lens, void* out, int B, int n_q, int Hq, int Hkv, int d,
                               int table_width, int n_blocks, int block_size, long long q_stride, liger_dtype dt,
                               liger_kv_dtype kv_dt, void* workspace, size_t workspace_bytes, void* stream) {
  const Range range("liger_attn_cached");
  liger::clear_last_error();
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0)
    return fail(LIGER_ERR_INVALID_ARG, "need Hq >= 1, Hkv >= 1 and Hq %% Hkv == 0 (Hq=%d Hkv=%d)", Hq, Hkv);
  liger_status st = check_types(Hkv, d, dt, kv_dt);
  if (st == LIGER_OK) st = check_cache(n_blocks, block_size);
  if (st == LIGER_OK) st = check_sequences(B, table_width, block_size);
  if (st != LIGER_OK) return st;
  if (n_q < 1) return fail(LIGER_ERR_INVALID_ARG, "need n_q >= 1 (n_q=%d)", n_q);
  const long long rows = (long long)n_q * (Hq / Hkv);
  if (n_q > LIGER_CACHED_MAX_NEW || rows > 65536 || Hkv > 65536 || (long long)n_q * Hq > 1 << 20)
    return fail(LIGER_ERR_UNSUPPORTED, "n_q=%d new tokens a sequence (at most %d), Hq=%d", n_q, LIGER_CACHED_MAX_NEW, Hq);
  const int per16 = dt == LIGER_BF16 ? 8 : 4;
  if (q_stride < (long long)Hq * d || q_stride % per16)
    return fail(LIGER_ERR_INVALID_ARG, "the query's token stride must be at least Hq * d elements and a multiple of 16 bytes");
  const int tile = liger::ca::tile_tokens(d), row_tiles = (int)((rows + liger::ca::kMaxRows - 1) / liger::ca::kMaxRows);
  // the kernel's line of work, were all sequences as long as their rows of the table
  const long long places = (((long long)table_width * block_size + tile - 1) / tile + liger::ca::unit_cost(2)) * B;
  if ((long long)n_blocks * Hkv > 0x7fffffffLL || places > (0x7fffffffLL - (1 << 20)) / ((long long)Hkv * row_tiles))
    return fail(LIGER_ERR_UNSUPPORTED, "too large: n_blocks * Hkv and B * table_width * block_size / %d * Hkv must fit 31 bits", tile);
  if (!q || !cache || !scales || !block_table || !seq_lens || !out)
    return fail(LIGER_ERR_INVALID_ARG, "all pointers must be non-null");
  const void* ptrs[] = {q, cache, out, workspace};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return fail(LIGER_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  if (!aligned(scales, 8)) return fail(LIGER_ERR_INVALID_ARG, "scales must be 8-byte aligned");
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4))
    return fail(LIGER_ERR_INVALID_ARG, "block_table and seq_lens must be 4-byte aligned");
  const AttnLayout L = attn_layout(d);
  if (!workspace || workspace_bytes < L.total)
    return fail(LIGER_ERR_INVALID_ARG, "workspace too small: need %zu bytes, got %zu", L.total, workspace_bytes);

  // the cache as (d, tokens of a block, keys then values, (block, kv head)) bytes; a copy brings the keys and values of up to 64 tokens
  CUtensorMap tm;
  const auto enc = liger::tensor_map_encoder();
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)block_size, 2, (cuuint64_t)n_blocks * Hkv};
  const cuuint64_t strides[3] = {(cuuint64_t)d, (cuuint64_t)block_size * d, (cuuint64_t)2 * block_size * d};
  const cuuint32_t box[4] = {(cuuint32_t)d, (cuuint32_t)(block_size < tile ? block_size : tile), 2, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  if (!enc || enc(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(cache), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return fail(LIGER_ERR_CUDA, "cuTensorMapEncodeTiled failed for the cache");
  void* err = nullptr;
  const cudaError_t ge = cudaGetSymbolAddress(&err, g_cached_attn_err);
  if (ge != cudaSuccess) return cuda_fail(ge, "cudaGetSymbolAddress");

  char* ws = static_cast<char*>(workspace);
  liger::ca::Args a{};
  a.q = q;
  a.scales = scales;
  a.table = block_table;
  a.lens = seq_lens;
  a.out = out;
  a.part_ml = reinterpret_cast<float*>(ws + L.off_ml);
  a.part_o = reinterpret_cast<float*>(ws + L.off_o);
  a.split = reinterpret_cast<liger::ca::Split*>(ws + L.off_split);
  a.err = static_cast<uint32_t*>(err);
  a.wait_ns = liger::bounded_wait_ns();
  a.inject_stall = liger::take_injected_stall() ? 1 : 0;
  a.qstride = (long)q_stride;
  a.scale_log2 = 1.4426950408889634f / std::sqrt((float)d);
  a.B = B;
  a.n_q = n_q;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.width = table_width;
  a.n_blocks = n_blocks;
  a.lbs = log2_block(block_size);
  a.rows = (int)rows;
  a.row_tiles = row_tiles;
  a.by_units = liger::ca::Divisor::of(Hkv * a.row_tiles);
  a.by_row_tiles = liger::ca::Divisor::of(a.row_tiles);
  a.by_G = liger::ca::Divisor::of(a.G);
  // no more CTAs than the line can have places (short tables)
  const long long most = places * Hkv * row_tiles;
  const int ctas = most < L.ctas ? (int)most : L.ctas;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dt == LIGER_BF16 ? attn_t<__nv_bfloat16>(tm, a, d, kv_dt, ctas, s) : attn_t<float>(tm, a, d, kv_dt, ctas, s);
}

liger_status liger_attn_cached_status(void) {
  liger::clear_last_error();
  uint32_t hdr[2] = {0u, 0u};
  cudaError_t e = cudaMemcpyFromSymbol(hdr, g_cached_attn_err, sizeof hdr);
  if (e != cudaSuccess) return cuda_fail(e, "reading the cached attention's error word");
  const uint32_t zero[2] = {0u, 0u};
  e = cudaMemcpyToSymbol(g_cached_attn_err, zero, sizeof zero);
  if (e != cudaSuccess) return cuda_fail(e, "clearing the cached attention's error word");
  if (hdr[0] & 1u)
    return fail(LIGER_ERR_TIMEOUT, "a cached attention kernel gave up waiting (site 0x%08x: role %u, barrier %u, tile %u)",
                hdr[1], hdr[1] >> 28, (hdr[1] >> 20) & 0xFFu, hdr[1] & 0xFFFFFu);
  return LIGER_OK;
}

}  // extern "C"
