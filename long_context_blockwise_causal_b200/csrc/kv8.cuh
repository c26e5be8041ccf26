// 8-bit KV cache: launchers and the pieces its kernels share.
//
// Cache of H heads and L slots per batch row: codes k, v [B][H][L][128]
// (e4m3 or int8), one fp32 scale per block of 128 slots and head
// (k_scale, v_scale [B][H][ceil(L/128)]) and per block the channel-wise
// bounds of its keys, int8 [B][H][ceil(L/128)][2][128] (smallest, largest)
// in units of scale * Q / 127. A code c stands for c * scale.
#pragma once

#include "common.cuh"

namespace lwm {

constexpr int kKv8Block = 128;      // slots per scale
constexpr int kKv8MaxGroup = 16;    // query heads per cache head
constexpr float kE4m3Max = 448.f;
constexpr float kInt8Max = 127.f;
constexpr float kTinyScale = 1.17549435e-38f;  // smaller scales become 0

// Reads what the kernel before may have written (a cache's scales, bounds and
// codes, a row's length). That kernel can still run when this one begins, so
// the read-only path, whose data must hold from a kernel's start to its end,
// is not for it: these are plain loads behind pdl_wait().
template <typename T>
__device__ __forceinline__ T ld_now(const T* p) {
  return *p;
}

struct Kv8WriteArgs {
  const void* x[2];            // k, v: bf16 [B][T][H][128], un-rotated
  void* codes[2];
  float* scale[2];
  int8_t* k_bounds;
  const int32_t* positions;    // [B][T]
  const int32_t* start;        // [B]
  const int32_t* n_new;        // [B] or null (T tokens in every row)
  const float* table;
  int max_pos, B, T, H, L;
  bool int8, half;
};
cudaError_t launch_kv8_write(const Kv8WriteArgs& a, int* status,
                             cudaStream_t st);

struct Kv8ReadArgs {
  const void* codes[2];
  const float* scale[2];
  const int32_t* start;        // [B]
  const int32_t* kv_len;       // [B] or null (L)
  void* out[2];                // bf16 [B][T][H][128]
  int B, T, H, L;
  bool int8;
};
cudaError_t launch_kv8_read(const Kv8ReadArgs& a, cudaStream_t st);

struct Kv8SelectArgs {
  const void* q;               // bf16 [B][Hq][128]
  const int8_t* k_bounds;
  const float* k_scale;
  const int32_t* kv_start;
  const int32_t* kv_len;
  const int32_t* q_pos;
  const float* table;
  int32_t* blocks;             // [B][H][K]
  float* scores;               // [B][H][K]
  int max_pos, B, L, H, G, K, n_sink, n_recent;
  bool half;
};
// Largest L: the scores of a row's blocks stay in one CTA's shared memory.
constexpr int kKv8SelectMaxLen = 1 << 22;
cudaError_t launch_kv8_select(const Kv8SelectArgs& a, cudaStream_t st);

struct Kv8DecodeArgs {
  const void* q;               // bf16 [B][H*G][128]
  const void* k;
  const void* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* kv_start;
  const int32_t* kv_len;
  const int32_t* q_pos;
  const int32_t* blocks;       // [B][H][K], read only when listed
  const float* table;
  void* out;                   // bf16 [B][H*G][128]
  float* lse;                  // [B][H*G]
  float* part;                 // kv8_part_floats(...) floats
  int max_pos, B, L, H, G, K;
  bool int8, half, listed;
  int* status;
};
// CTAs of the decode kernel, and the floats of its partial results (K < 0:
// no block list).
int kv8_decode_grid(int B, int L, int H, int K);
size_t kv8_part_floats(int B, int L, int H, int G, int K);
cudaError_t launch_kv8_decode(const Kv8DecodeArgs& a, cudaStream_t st);

#ifdef __CUDACC__
// Two floats to two e4m3 codes (nearest even, saturating; NaN stays NaN),
// lo in bits 0-7.
__device__ __forceinline__ uint32_t enc2_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 dec2_e4m3(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(w)));
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
// The same for int8 codes: nearest even, clamped to +-127.
__device__ __forceinline__ uint32_t enc2_int8(float lo, float hi) {
  const int a = __float2int_rn(fminf(fmaxf(lo, -kInt8Max), kInt8Max));
  const int b = __float2int_rn(fminf(fmaxf(hi, -kInt8Max), kInt8Max));
  return uint32_t(a & 255) | (uint32_t(b & 255) << 8);
}
__device__ __forceinline__ float2 dec2_int8(uint32_t w) {
  return make_float2(float(int8_t(w & 255)), float(int8_t((w >> 8) & 255)));
}
template <bool kInt8>
__device__ __forceinline__ uint32_t enc2(float lo, float hi) {
  return kInt8 ? enc2_int8(lo, hi) : enc2_e4m3(lo, hi);
}
template <bool kInt8>
__device__ __forceinline__ float2 dec2(uint32_t w) {
  return kInt8 ? dec2_int8(w) : dec2_e4m3(w);
}
// Four values to codes in one word. int8: |v| is at most 127 but for the
// last bit of a product, so adding 1.5 * 2^23 rounds it to nearest even and
// leaves the code in the low byte, with nothing to clamp.
template <bool kInt8>
__device__ __forceinline__ uint32_t enc4(float a, float b, float c, float d) {
  if constexpr (kInt8) {
    constexpr float kMagic = 12582912.f;
    const uint32_t ua = __float_as_uint(__fadd_rn(a, kMagic));
    const uint32_t ub = __float_as_uint(__fadd_rn(b, kMagic));
    const uint32_t uc = __float_as_uint(__fadd_rn(c, kMagic));
    const uint32_t ud = __float_as_uint(__fadd_rn(d, kMagic));
    return __byte_perm(__byte_perm(ua, ub, 0x0040),
                       __byte_perm(uc, ud, 0x0040), 0x5410);
  } else {
    return enc2_e4m3(a, b) | (enc2_e4m3(c, d) << 16);
  }
}
// max that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Largest of a warp's magnitudes (no sign bit); as unsigned words their
// order is the numbers', with NaN on top.
__device__ __forceinline__ float warp_max_abs(float x) {
  return __uint_as_float(
      __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(x))));
}
#endif

}  // namespace lwm
