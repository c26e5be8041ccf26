// Entry points of the 8-bit KV cache (declared in include/lwm_blockattn.h):
// host-side validation, then one launcher each.
#include <initializer_list>

#include "api_checks.cuh"
#include "kv8.cuh"

namespace lwm {
namespace {

constexpr size_t kAlign = 256;

bool aligned_to(std::initializer_list<const void*> ps, uintptr_t bytes) {
  for (const void* p : ps)
    if (!p || (reinterpret_cast<uintptr_t>(p) & (bytes - 1))) return false;
  return true;
}
// Tensors that the kernels read or write 16 bytes at a time.
bool wide_ok(std::initializer_list<const void*> ps) {
  return aligned_to(ps, 16);
}
// Vectors of 4-byte words that they take one at a time: a slice of a longer
// one (the step's positions, a row's lengths) starts anywhere.
bool words_ok(std::initializer_list<const void*> ps) {
  return aligned_to(ps, 4);
}

int cuda_status(cudaError_t e) {
  return e == cudaSuccess ? LWM_OK : LWM_ERR_CUDA;
}

// Slots or tokens of all rows are counted in 32 bits, rounded up to blocks.
constexpr int64_t kMostSlots = (int64_t(1) << 31) - kKv8Block;

// Sizes that every call shares. Slots, blocks and (row, head) pairs are
// counted in 32 bits; bytes in 64.
int cache_status(int B, int L, int H, int D, int cache_type) {
  if (B < 0 || L < 0 || H < 0 || int64_t(B) * L > kMostSlots ||
      L > kMostSlots ||
      int64_t(B) * H >= (int64_t(1) << 28))
    return LWM_ERR_INVALID_ARG;
  if (cache_type != LWM_KV8_E4M3 && cache_type != LWM_KV8_INT8)
    return LWM_ERR_INVALID_ARG;
  if (D != kHeadDim) return LWM_ERR_UNSUPPORTED;
  return LWM_OK;
}

// Blocks of 128 slots that T tokens per row can touch, all heads, K and V.
int64_t tiles_of(int B, int T, int H) {
  return int64_t(B) * H * 2 * ((int64_t(T) + kKv8Block - 1) / kKv8Block + 1);
}

int query_status(int Hq, int H, int max_pos, int rope_layout) {
  if (Hq < 0 || max_pos < 0 ||
      (rope_layout != LWM_ROPE_INTERLEAVED && rope_layout != LWM_ROPE_HALF))
    return LWM_ERR_INVALID_ARG;
  if (H == 0 ? Hq > 0 : Hq % H != 0) return LWM_ERR_INVALID_ARG;
  if (H > 0 && Hq / H > kKv8MaxGroup) return LWM_ERR_UNSUPPORTED;
  return LWM_OK;
}

}  // namespace
}  // namespace lwm

using namespace lwm;

extern "C" {

int lwm_kv8_write(const void* k, const void* v, const int32_t* positions,
                  const int32_t* start, const int32_t* n_new,
                  const float* rope_table, int max_pos, int B, int T, int L,
                  int H, int D, int dtype, int cache_type, int rope_layout,
                  void* k_cache, void* v_cache, float* k_scale,
                  float* v_scale, int8_t* k_bounds, void* stream) {
  int s = cache_status(B, L, H, D, cache_type);
  if (s != LWM_OK) return s;
  if (T < 0 || max_pos < 0 || int64_t(B) * T > kMostSlots ||
      (rope_layout != LWM_ROPE_INTERLEAVED && rope_layout != LWM_ROPE_HALF))
    return LWM_ERR_INVALID_ARG;
  if (dtype != LWM_DTYPE_BF16) return LWM_ERR_UNSUPPORTED;
  if (int64_t(B) * H == 0 || T == 0 || L == 0) return LWM_OK;
  // blocks of all heads, K and V, are counted in 32 bits
  if (tiles_of(B, T, H) >= (int64_t(1) << 31)) return LWM_ERR_UNSUPPORTED;
  if (!wide_ok({k, v, rope_table, k_cache, v_cache, k_bounds}) ||
      !words_ok({positions, start, k_scale, v_scale}) ||
      (n_new && !words_ok({n_new})) || max_pos < 1)
    return LWM_ERR_INVALID_ARG;
  Kv8WriteArgs a{};
  a.x[0] = k;
  a.x[1] = v;
  a.codes[0] = k_cache;
  a.codes[1] = v_cache;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.k_bounds = k_bounds;
  a.positions = positions;
  a.start = start;
  a.n_new = n_new;
  a.table = rope_table;
  a.max_pos = max_pos;
  a.B = B;
  a.T = T;
  a.H = H;
  a.L = L;
  a.int8 = cache_type == LWM_KV8_INT8;
  a.half = rope_layout == LWM_ROPE_HALF;
  int* status = status_word();
  if (!status) return LWM_ERR_CUDA;
  return cuda_status(
      launch_kv8_write(a, status, static_cast<cudaStream_t>(stream)));
}

int lwm_kv8_read(const void* k_cache, const void* v_cache,
                 const float* k_scale, const float* v_scale,
                 const int32_t* start, const int32_t* kv_len, int B, int T,
                 int L, int H, int D, int dtype, int cache_type, void* k_rot,
                 void* v, void* stream) {
  int s = cache_status(B, L, H, D, cache_type);
  if (s != LWM_OK) return s;
  if (T < 0 || int64_t(B) * T > kMostSlots)
    return LWM_ERR_INVALID_ARG;
  if (dtype != LWM_DTYPE_BF16) return LWM_ERR_UNSUPPORTED;
  if (int64_t(B) * H == 0 || T == 0) return LWM_OK;
  // a CTA per 32 tokens, head and tensor
  if (tiles_of(B, T, H) >= (int64_t(1) << 29)) return LWM_ERR_UNSUPPORTED;
  if (!wide_ok({k_rot, v}) || !words_ok({start}) ||
      (L > 0 && !(wide_ok({k_cache, v_cache}) &&
                  words_ok({k_scale, v_scale}))) ||
      (kv_len && !words_ok({kv_len})))
    return LWM_ERR_INVALID_ARG;
  Kv8ReadArgs a{};
  a.codes[0] = k_cache;
  a.codes[1] = v_cache;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.start = start;
  a.kv_len = kv_len;
  a.out[0] = k_rot;
  a.out[1] = v;
  a.B = B;
  a.T = T;
  a.H = H;
  a.L = L;
  a.int8 = cache_type == LWM_KV8_INT8;
  return cuda_status(launch_kv8_read(a, static_cast<cudaStream_t>(stream)));
}

int lwm_kv8_select(const void* q, const int8_t* k_bounds,
                   const float* k_scale, const int32_t* kv_start,
                   const int32_t* kv_len, const int32_t* q_pos,
                   const float* rope_table, int max_pos, int B, int L, int Hq,
                   int H, int D, int dtype, int rope_layout, int n_select,
                   int n_sink, int n_recent, int32_t* blocks, float* scores,
                   void* stream) {
  int s = cache_status(B, L, H, D, LWM_KV8_E4M3);
  if (s != LWM_OK) return s;
  s = query_status(Hq, H, max_pos, rope_layout);
  if (s != LWM_OK) return s;
  if (n_select < 1 || n_sink < 0 || n_recent < 0 ||
      int64_t(n_sink) + n_recent > n_select)
    return LWM_ERR_INVALID_ARG;
  if (dtype != LWM_DTYPE_BF16 || L > kKv8SelectMaxLen)
    return LWM_ERR_UNSUPPORTED;
  if (int64_t(B) * Hq == 0) return LWM_OK;
  if (!wide_ok({q, rope_table}) ||
      !words_ok({kv_start, kv_len, q_pos, blocks, scores}) ||
      (L > 0 && !(wide_ok({k_bounds}) && words_ok({k_scale}))) ||
      max_pos < 1)
    return LWM_ERR_INVALID_ARG;
  Kv8SelectArgs a{};
  a.q = q;
  a.k_bounds = k_bounds;
  a.k_scale = k_scale;
  a.kv_start = kv_start;
  a.kv_len = kv_len;
  a.q_pos = q_pos;
  a.table = rope_table;
  a.blocks = blocks;
  a.scores = scores;
  a.max_pos = max_pos;
  a.B = B;
  a.L = L;
  a.H = H;
  a.G = Hq / H;
  a.K = n_select;
  a.n_sink = n_sink;
  a.n_recent = n_recent;
  a.half = rope_layout == LWM_ROPE_HALF;
  return cuda_status(launch_kv8_select(a, static_cast<cudaStream_t>(stream)));
}

size_t lwm_kv8_decode_workspace_size(int B, int L, int Hq, int H, int D,
                                     int n_blocks) {
  if (cache_status(B, L, H, D, LWM_KV8_E4M3) != LWM_OK ||
      query_status(Hq, H, 0, LWM_ROPE_HALF) != LWM_OK ||
      int64_t(B) * Hq == 0)
    return 0;
  const size_t n =
      kv8_part_floats(B, L, H, Hq / H, n_blocks < 0 ? -1 : n_blocks) *
      sizeof(float);
  return (n + kAlign - 1) / kAlign * kAlign;
}

int lwm_kv8_decode(const void* q, const void* k_cache, const void* v_cache,
                   const float* k_scale, const float* v_scale,
                   const int32_t* kv_start, const int32_t* kv_len,
                   const int32_t* q_pos, const int32_t* blocks, int n_blocks,
                   const float* rope_table, int max_pos, int B, int L, int Hq,
                   int H, int D, int dtype, int cache_type, int rope_layout,
                   void* out, float* lse, void* workspace,
                   size_t workspace_bytes, void* stream) {
  int s = cache_status(B, L, H, D, cache_type);
  if (s != LWM_OK) return s;
  s = query_status(Hq, H, max_pos, rope_layout);
  if (s != LWM_OK) return s;
  const bool listed = n_blocks >= 0;
  // tiles (blocks of all rows and heads) are counted in 32 bits
  const int64_t per =
      listed ? n_blocks : (int64_t(L) + kKv8Block - 1) / kKv8Block;
  if (int64_t(B) * H * per >= (int64_t(1) << 31) - 4096)
    return LWM_ERR_UNSUPPORTED;
  if (dtype != LWM_DTYPE_BF16) return LWM_ERR_UNSUPPORTED;
  if (int64_t(B) * Hq == 0) return LWM_OK;
  if (!wide_ok({q, rope_table, out, workspace}) ||
      !words_ok({kv_start, kv_len, q_pos, lse}) ||
      (L > 0 && !(wide_ok({k_cache, v_cache}) &&
                  words_ok({k_scale, v_scale}))) ||
      (n_blocks > 0 && !words_ok({blocks})) || max_pos < 1)
    return LWM_ERR_INVALID_ARG;
  if (workspace_bytes < lwm_kv8_decode_workspace_size(
                            B, L, Hq, H, D, n_blocks))
    return LWM_ERR_WORKSPACE;
  Kv8DecodeArgs a{};
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.kv_start = kv_start;
  a.kv_len = kv_len;
  a.q_pos = q_pos;
  a.blocks = blocks;
  a.table = rope_table;
  a.out = out;
  a.lse = lse;
  a.part = static_cast<float*>(workspace);
  a.max_pos = max_pos;
  a.B = B;
  a.L = L;
  a.H = H;
  a.G = Hq / H;
  a.K = listed ? n_blocks : 0;
  a.listed = listed;
  a.int8 = cache_type == LWM_KV8_INT8;
  a.half = rope_layout == LWM_ROPE_HALF;
  a.status = status_word();
  if (!a.status) return LWM_ERR_CUDA;
  return cuda_status(launch_kv8_decode(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
