// Writing and reading the 8-bit KV cache.
//
// Write: x = R(pos) k (or v) of the new tokens in fp32, then per block of
// 128 slots and head
//   s = max(s_old if the block keeps older tokens, max |x| * (1 / Q)),
//   code = enc(x * (1 / s)),  older codes c -> enc(c * (s_old / s)) if s
//   grew, and for keys the channel bounds floor(min c * u), ceil(max c * u)
// with u = 127 / Q. The rotation's products and sums are rounded one by
// one, so that equal inputs give equal codes wherever the definition is
// evaluated. A scale below the smallest normal number becomes 0 (its codes
// too); a NaN or an infinity among the new values makes the scale NaN.
#include <algorithm>

#include "kv8.cuh"
#include "tc_kernels.cuh"

namespace lwm {
namespace {

constexpr float kMaxFinite = 3.402823466e38f;

// New slots of row b: tokens t in [lo - start, hi - start) go to slots
// [lo, hi); older tokens lie below lo.
struct NewSlots {
  int64_t start, lo, hi;
};
__device__ __forceinline__ NewSlots new_slots(const Kv8WriteArgs& a, int b) {
  NewSlots n;
  n.start = __ldg(a.start + b);
  const int count = a.n_new ? max(0, min(__ldg(a.n_new + b), a.T)) : a.T;
  n.lo = n.start > 0 ? n.start : 0;
  n.hi = min(n.start + count, int64_t(a.L));
  return n;
}

// Scale of a block that had s_old and meets amax.
template <bool kInt8>
__device__ __forceinline__ float block_scale(float s_old, float amax) {
  constexpr float kRq = kInt8 ? 1.f / kInt8Max : 1.f / kE4m3Max;
  float s = max_nan(s_old, __fmul_rn(amax, kRq));
  if (s < kTinyScale) s = 0.f;
  return s <= kMaxFinite ? s : __int_as_float(0x7fffffff);  // NaN
}

// Two new values to codes; inv = 1 / s, or 0 for codes of 0 whatever x is.
template <bool kInt8>
__device__ __forceinline__ uint32_t code2(float x, float y, float inv) {
  return inv > 0.f ? enc2<kInt8>(__fmul_rn(x, inv), __fmul_rn(y, inv)) : 0u;
}

__device__ __forceinline__ float2 scaled(float2 v, float f) {
  return make_float2(__fmul_rn(v.x, f), __fmul_rn(v.y, f));
}

// Four codes of a block whose scale grew.
template <bool kInt8>
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
  const float2 f = dec2<kInt8>(w & 0xffffu), g = dec2<kInt8>(w >> 16);
  return enc4<kInt8>(__fmul_rn(f.x, ratio), __fmul_rn(f.y, ratio),
                     __fmul_rn(g.x, ratio), __fmul_rn(g.y, ratio));
}

// Bounds of a channel whose codes lie in [lo, hi], in units of s Q / 127.
template <bool kInt8>
__device__ __forceinline__ int bound_lo(float lo) {
  constexpr float kUnit = kInt8 ? 1.f : kInt8Max / kE4m3Max;
  return max(-127, min(127, __float2int_rd(__fmul_rn(lo, kUnit))));
}
template <bool kInt8>
__device__ __forceinline__ int bound_hi(float hi) {
  constexpr float kUnit = kInt8 ? 1.f : kInt8Max / kE4m3Max;
  return max(-127, min(127, __float2int_ru(__fmul_rn(hi, kUnit))));
}

__device__ __forceinline__ void rotate(float& x, float& y, float c, float s) {
  const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(x, s), __fmul_rn(y, c));
  x = u;
}

// ------------------------------------------------------------ few tokens
//
// A warp per (row, head, K or V, block touched), four channels per lane
// (two pairs of the rotation: adjacent channels, or channels 64 apart). The
// tokens are taken twice, for the maximum and for the codes; the usual
// append of a token that leaves the scale alone reads the token, the scale
// and 256 bounds and writes 128 codes. Bound by latency.
constexpr int kFewThreads = 128;
constexpr int kFewTokens = 16;

template <bool kInt8, bool kHalf>
__global__ void __launch_bounds__(kFewThreads)
kv8_write_few_kernel(const __grid_constant__ Kv8WriteArgs a, int64_t items) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  int64_t e = blockIdx.x * int64_t(kFewThreads / 32) + (threadIdx.x >> 5);
  if (e >= items) return;
  // the second block of a row's tokens comes after all the first ones
  const int64_t per = int64_t(a.B) * a.H * 2;
  const int blk_i = int(e / per);
  e -= blk_i * per;
  const bool key = (e & 1) == 0;
  const int64_t bh = e >> 1;
  const int b = int(bh / a.H), h = int(bh - int64_t(b) * a.H);

  const NewSlots ns = new_slots(a, b);
  const int64_t base = (ns.lo / kKv8Block + blk_i) * kKv8Block;
  if (ns.lo >= ns.hi || base >= ns.hi) return;
  const int lo = int(max(ns.lo - base, int64_t(0)));
  const int hi = int(min(ns.hi - base, int64_t(kKv8Block)));
  const int nblk = (a.L + kKv8Block - 1) / kKv8Block;
  const int64_t at = bh * nblk + base / kKv8Block;
  float* scale = (key ? a.scale[0] : a.scale[1]) + at;
  uint8_t* codes = static_cast<uint8_t*>(key ? a.codes[0] : a.codes[1]) +
                   (bh * a.L + base) * kHeadDim;
  const char* x_all = static_cast<const char*>(key ? a.x[0] : a.x[1]);
  const float s_old = lo > 0 ? *scale : 0.f;
  const int c0 = kHalf ? 2 * lane : 4 * lane;        // channels c0, c0 + 1,
  const int c1 = kHalf ? 64 + 2 * lane : c0 + 2;     // c1, c1 + 1

  float x[4];
  auto load = [&](int r) {
    const int64_t tok = int64_t(b) * a.T + (base + r - ns.start);
    const char* row = x_all + (tok * a.H + h) * (kHeadDim * 2);
    const uint32_t w0 = __ldg(reinterpret_cast<const uint32_t*>(row + 2 * c0));
    const uint32_t w1 = __ldg(reinterpret_cast<const uint32_t*>(row + 2 * c1));
    x[0] = bf16lo_to_f32(w0);
    x[1] = bf16hi_to_f32(w0);
    x[2] = bf16lo_to_f32(w1);
    x[3] = bf16hi_to_f32(w1);
    if (key) {
      const int p = max(0, min(__ldg(a.positions + tok), a.max_pos - 1));
      // pairs 2 lane and 2 lane + 1
      const float4 cs = __ldg(reinterpret_cast<const float4*>(
                                  a.table + int64_t(p) * kHeadDim) + lane);
      if (kHalf) {
        rotate(x[0], x[2], cs.x, cs.y);
        rotate(x[1], x[3], cs.z, cs.w);
      } else {
        rotate(x[0], x[1], cs.x, cs.y);
        rotate(x[2], x[3], cs.z, cs.w);
      }
    }
  };
  float mn[4], mx[4], amax = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    mn[k] = INFINITY;
    mx[k] = -INFINITY;
  }
  for (int r = lo; r < hi; ++r) {
    load(r);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      mn[k] = min_nan(mn[k], x[k]);
      mx[k] = max_nan(mx[k], x[k]);
      amax = max_nan(amax, fabsf(x[k]));
    }
  }
  amax = warp_max_abs(amax);
  const float s = block_scale<kInt8>(s_old, amax);
  const float inv = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
  const bool grew = lo > 0 && s > s_old;
  for (int r = lo; r < hi; ++r) {
    if (hi - lo > 1) load(r);
    uint8_t* row = codes + r * kHeadDim;
    const uint32_t w0 = code2<kInt8>(x[0], x[1], inv);
    const uint32_t w1 = code2<kInt8>(x[2], x[3], inv);
    if (kHalf) {
      *reinterpret_cast<uint16_t*>(row + c0) = uint16_t(w0);
      *reinterpret_cast<uint16_t*>(row + c1) = uint16_t(w1);
    } else {
      *reinterpret_cast<uint32_t*>(row + c0) = w0 | (w1 << 16);
    }
  }
  if (lane == 0) *scale = s;
  // the new codes' range: encoding keeps the order
  float cl[4], ch[4];
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    const float2 f = dec2<kInt8>(code2<kInt8>(mn[k], mn[k + 1], inv));
    const float2 g = dec2<kInt8>(code2<kInt8>(mx[k], mx[k + 1], inv));
    cl[k] = f.x; cl[k + 1] = f.y;
    ch[k] = g.x; ch[k + 1] = g.y;
  }
  if (grew) {
    // round the older codes again, 32 rows in flight; a lane takes its own
    // four channels of every row, so it also has their range
    const float ratio = __fdiv_rn(s_old, s);
    constexpr int kRows = 32;
    for (int r0 = 0; r0 < lo; r0 += kRows) {
      uint32_t w[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        w[i] = 0;
        if (r0 + i >= lo) continue;
        const uint8_t* row = codes + (r0 + i) * kHeadDim;
        if (kHalf) {
          w[i] = *reinterpret_cast<const uint16_t*>(row + c0) |
                 (uint32_t(*reinterpret_cast<const uint16_t*>(row + c1)) << 16);
        } else {
          w[i] = *reinterpret_cast<const uint32_t*>(row + c0);
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (r0 + i >= lo) break;
        uint8_t* row = codes + (r0 + i) * kHeadDim;
        const uint32_t u = recode4<kInt8>(w[i], ratio);
        if (kHalf) {
          *reinterpret_cast<uint16_t*>(row + c0) = uint16_t(u);
          *reinterpret_cast<uint16_t*>(row + c1) = uint16_t(u >> 16);
        } else {
          *reinterpret_cast<uint32_t*>(row + c0) = u;
        }
        const float2 f = dec2<kInt8>(u & 0xffffu), g = dec2<kInt8>(u >> 16);
        cl[0] = fminf(cl[0], f.x); ch[0] = fmaxf(ch[0], f.x);
        cl[1] = fminf(cl[1], f.y); ch[1] = fmaxf(ch[1], f.y);
        cl[2] = fminf(cl[2], g.x); ch[2] = fmaxf(ch[2], g.x);
        cl[3] = fminf(cl[3], g.y); ch[3] = fmaxf(ch[3], g.y);
      }
    }
  }
  if (!key) return;
  int8_t* bd = a.k_bounds + at * 2 * kHeadDim;
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    char2* pl = reinterpret_cast<char2*>(bd + (k ? c1 : c0));
    char2* ph = reinterpret_cast<char2*>(bd + kHeadDim + (k ? c1 : c0));
    int l0 = bound_lo<kInt8>(cl[k]), l1 = bound_lo<kInt8>(cl[k + 1]);
    int h0 = bound_hi<kInt8>(ch[k]), h1 = bound_hi<kInt8>(ch[k + 1]);
    if (lo > 0 && !grew) {     // the older tokens' bounds still hold
      const char2 ol = *pl, oh = *ph;
      l0 = min(l0, int(ol.x)); l1 = min(l1, int(ol.y));
      h0 = max(h0, int(oh.x)); h1 = max(h1, int(oh.y));
    }
    *pl = make_char2(char(l0), char(l1));
    *ph = make_char2(char(h0), char(h1));
  }
}

// ----------------------------------------------------------- many tokens
//
// A CTA takes a block of 128 slots of K or V for a group of heads, one head
// after the other: the heads' [128 tokens][128] bf16 boxes come in by TMA
// through a ring of stages, while the rotation's angles of the block's
// tokens stay in registers. 16 lanes share a token, eight channels each,
// four tokens per thread; the rotated block stays in registers between the
// maximum and the encoding, so each input is read once and each code
// written once. K keeps the channels' smallest and largest value, which
// give the block's maximum as well as its bounds. One barrier per head.
constexpr int kWrThreads = 512;
constexpr int kWrWarps = kWrThreads / 32;
constexpr int kWrLanes = 16;
constexpr int kWrStep = kWrThreads / kWrLanes;     // tokens per pass
constexpr int kWrPasses = kKv8Block / kWrStep;
constexpr int kWrStages = 4;
constexpr int kWrTile = kKv8Block * kHeadDim * 2;
constexpr uint64_t kWrWaitNs = 4000000000ull;
// shared memory (bytes): stages, channel ranges [2][lo, hi][warp][128],
// maxima [2][warp], barriers
constexpr int kWrChan = kWrStages * kWrTile;
constexpr int kWrMax = kWrChan + 2 * 2 * kWrWarps * kHeadDim * 4;
constexpr int kWrBars = kWrMax + 2 * kWrWarps * 4;
constexpr int kWrSmem = kWrBars + kWrStages * 8 + 128;
static_assert(kWrSmem <= 232448, "shared memory per CTA");

struct WriteItem {
  int b, h0, h1;
  bool key;
  int64_t base;       // first slot of the block
  int lo, hi;         // its new slots
  int64_t tok;        // token of the block's first slot (may be negative)
  bool any;
};

struct WriteGrid {
  int per_row;        // blocks a row's tokens can touch
  int groups, heads;  // head groups and heads in each
  int64_t items;      // 2 * B * per_row * groups
};

__device__ __forceinline__ WriteItem write_item(const Kv8WriteArgs& a,
                                                const WriteGrid& g,
                                                int64_t i) {
  WriteItem w;
  // all of K, then all of V; within each, heads of a block side by side
  const int64_t half = g.items / 2;
  w.key = i < half;
  if (!w.key) i -= half;
  const int64_t row_blk = i / g.groups;
  w.h0 = int(i - row_blk * g.groups) * g.heads;
  w.h1 = min(w.h0 + g.heads, a.H);
  w.b = int(row_blk / g.per_row);
  const NewSlots n = new_slots(a, w.b);
  w.base = (n.lo / kKv8Block + (row_blk - int64_t(w.b) * g.per_row)) *
           kKv8Block;
  w.any = n.lo < n.hi && w.base < n.hi;
  w.lo = int(max(n.lo - w.base, int64_t(0)));
  w.hi = int(min(n.hi - w.base, int64_t(kKv8Block)));
  w.tok = w.base - n.start;
  return w;
}

template <bool kInt8, bool kHalf>
__global__ void __launch_bounds__(kWrThreads, 1)
kv8_write_kernel(const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ Kv8WriteArgs a,
                 const WriteGrid grid, int* status) {
  extern __shared__ uint8_t dsmem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(dsmem_raw) + 127) & ~uintptr_t(127));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int s) { return sbase + kWrBars + 8u * s; };
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int c = t % kWrLanes, row0 = t / kWrLanes;
  if (t == 0) {
    for (int s = 0; s < kWrStages; ++s) mbar_init(bar(s), 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int nblk = (a.L + kKv8Block - 1) / kKv8Block;

  // loader (a lane of the last warp): runs kWrStages - 1 heads ahead over the same items
  int64_t ld_i = blockIdx.x;
  WriteItem ld{};
  int ld_h = 0, ld_n = 0;
  auto ld_seek = [&]() {
    while (ld_i < grid.items) {
      ld = write_item(a, grid, ld_i);
      ld_h = ld.h0;
      if (ld.any) return;
      ld_i += gridDim.x;
    }
  };
  auto ld_issue = [&]() {
    if (ld_i >= grid.items) return;
    const int s = ld_n % kWrStages;
    mbar_arrive_expect_tx(bar(s), kWrTile);
    // tokens before the first and behind the last one read as zeros
    tma_load_4d(sbase + s * kWrTile, ld.key ? &tm_k : &tm_v, bar(s), 0, ld_h,
                int(ld.tok), ld.b);
    ++ld_n;
    if (++ld_h >= ld.h1) {
      ld_i += gridDim.x;
      ld_seek();
    }
  };
  const bool loader = t == kWrThreads - 32;
  if (loader) {
    ld_seek();
    for (int s = 0; s < kWrStages - 1; ++s) ld_issue();
  }

  int n = 0;          // heads done
  for (int64_t i = blockIdx.x; i < grid.items; i += gridDim.x) {
    const WriteItem it = write_item(a, grid, i);
    if (!it.any) continue;
    const bool full = it.lo == 0 && it.hi == kKv8Block;
    // angles of the thread's tokens, pairs (4c, 4c + 1), (4c + 2, 4c + 3)
    float2 cc[kWrPasses][2], ss[kWrPasses][2];
    if (it.key) {
#pragma unroll
      for (int k = 0; k < kWrPasses; ++k) {
        const int r = row0 + k * kWrStep;
        int p = 0;
        if (r >= it.lo && r < it.hi)
          p = max(0, min(__ldg(a.positions + int64_t(it.b) * a.T + it.tok + r),
                         a.max_pos - 1));
        const float4* tab = reinterpret_cast<const float4*>(
            a.table + int64_t(p) * kHeadDim) + 2 * c;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 f = __ldg(tab + j);
          cc[k][j] = make_float2(f.x, f.z);
          ss[k][j] = make_float2(f.y, f.w);
        }
      }
    }
    for (int h = it.h0; h < it.h1; ++h, ++n) {
      const int64_t bh = int64_t(it.b) * a.H + h;
      const int64_t at = bh * nblk + it.base / kKv8Block;
      float* scale = (it.key ? a.scale[0] : a.scale[1]) + at;
      const float s_old = it.lo > 0 ? __ldcg(scale) : 0.f;
      const bool ok = mbar_wait(bar(n % kWrStages), (n / kWrStages) & 1,
                                nullptr, status, kWrWaitNs);
      const uint8_t* tile = smem + (n % kWrStages) * kWrTile;
      // x, y: first and second members of pairs 4c .. 4c + 3
      float2 x[kWrPasses][2], y[kWrPasses][2];
#pragma unroll
      for (int k = 0; k < kWrPasses; ++k) {
        const uint8_t* row = tile + (row0 + k * kWrStep) * (kHeadDim * 2);
        if (kHalf) {
          const uint2 u = *reinterpret_cast<const uint2*>(row + c * 8);
          const uint2 v = *reinterpret_cast<const uint2*>(row + 128 + c * 8);
          x[k][0] = make_float2(bf16lo_to_f32(u.x), bf16hi_to_f32(u.x));
          x[k][1] = make_float2(bf16lo_to_f32(u.y), bf16hi_to_f32(u.y));
          y[k][0] = make_float2(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x));
          y[k][1] = make_float2(bf16lo_to_f32(v.y), bf16hi_to_f32(v.y));
        } else {
          const uint4 u = *reinterpret_cast<const uint4*>(row + c * 16);
          x[k][0] = make_float2(bf16lo_to_f32(u.x), bf16lo_to_f32(u.y));
          y[k][0] = make_float2(bf16hi_to_f32(u.x), bf16hi_to_f32(u.y));
          x[k][1] = make_float2(bf16lo_to_f32(u.z), bf16lo_to_f32(u.w));
          y[k][1] = make_float2(bf16hi_to_f32(u.z), bf16hi_to_f32(u.w));
        }
        if (it.key) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            rotate(x[k][j].x, y[k][j].x, cc[k][j].x, ss[k][j].x);
            rotate(x[k][j].y, y[k][j].y, cc[k][j].y, ss[k][j].y);
          }
        }
      }
      float amax = 0.f;
      // value j of pass k: x of pairs 4c + j for j < 4, then their y
      auto val = [&](int k, int j) {
        const float2 v = j < 4 ? x[k][j / 2] : y[k][(j - 4) / 2];
        return (j & 1) ? v.y : v.x;
      };
      static_assert(kWrPasses == 4, "the maxima below take four values");
      if (it.key) {
        float mn[8], mx[8];
        bool some = false;
        if (full) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            mn[j] = min_nan(min3_nan(val(0, j), val(1, j), val(2, j)),
                            val(3, j));
            mx[j] = max_nan(max3_nan(val(0, j), val(1, j), val(2, j)),
                            val(3, j));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            mn[j] = INFINITY;
            mx[j] = -INFINITY;
#pragma unroll
            for (int k = 0; k < kWrPasses; ++k) {
              const int r = row0 + k * kWrStep;
              if (r >= it.lo && r < it.hi) {
                some = true;
                mn[j] = min_nan(mn[j], val(k, j));
                mx[j] = max_nan(mx[j], val(k, j));
              }
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          mn[j] = min_nan(mn[j], __shfl_xor_sync(0xffffffffu, mn[j], 16));
          mx[j] = max_nan(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 16));
        }
        float* chan = reinterpret_cast<float*>(smem + kWrChan) +
                      ((n & 1) * 2 * kWrWarps + warp) * kHeadDim;
        // lanes 0-15 keep the smallest values, the others the largest
        const bool low = lane < kWrLanes;
        float m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = low ? mn[j] : mx[j];
        if (!low) chan += kWrWarps * kHeadDim;
        if (kHalf) {    // channels 4c .. and 64 + 4c ..
          *reinterpret_cast<float4*>(chan + 4 * c) =
              make_float4(m[0], m[1], m[2], m[3]);
          *reinterpret_cast<float4*>(chan + 64 + 4 * c) =
              make_float4(m[4], m[5], m[6], m[7]);
        } else {        // channels 8c .., pairs side by side
          *reinterpret_cast<float4*>(chan + 8 * c) =
              make_float4(m[0], m[4], m[1], m[5]);
          *reinterpret_cast<float4*>(chan + 8 * c + 4) =
              make_float4(m[2], m[6], m[3], m[7]);
        }
        // a warp none of whose tokens is new has nothing to add
        if (full || __any_sync(0xffffffffu, some)) {
          amax = max3_abs_nan(max3_abs_nan(m[0], m[1], m[2]),
                              max3_abs_nan(m[3], m[4], m[5]),
                              max_nan(fabsf(m[6]), fabsf(m[7])));
        }
      } else {
#pragma unroll
        for (int k = 0; k < kWrPasses; ++k) {
          const int r = row0 + k * kWrStep;
          if (full || (r >= it.lo && r < it.hi)) {
            amax = max3_abs_nan(amax, x[k][0].x, x[k][0].y);
            amax = max3_abs_nan(amax, x[k][1].x, x[k][1].y);
            amax = max3_abs_nan(amax, y[k][0].x, y[k][0].y);
            amax = max3_abs_nan(amax, y[k][1].x, y[k][1].y);
          }
        }
      }
      amax = warp_max_abs(amax);
      float* red = reinterpret_cast<float*>(smem + kWrMax) +
                   (n & 1) * kWrWarps;
      if (lane == 0) red[warp] = amax;
      // all have read the tile: its stage is free
      if (!__syncthreads_and(ok)) {
        // a load did not land in time: wait for the others before leaving
        if (loader)
          for (int f = n + 1; f < ld_n; ++f)
            mbar_wait(bar(f % kWrStages), (f / kWrStages) & 1, nullptr,
                      status, kWrWaitNs);
        return;
      }
      if (loader) ld_issue();
#pragma unroll
      for (int w = 0; w < kWrWarps; w += 4) {
        const float4 m4 = *reinterpret_cast<const float4*>(red + w);
        amax = max_nan(amax, max_nan(max_nan(m4.x, m4.y), max_nan(m4.z, m4.w)));
      }
      const float s = block_scale<kInt8>(s_old, amax);
      const float inv = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
      const bool grew = it.lo > 0 && s > s_old;
      uint8_t* codes = static_cast<uint8_t*>(it.key ? a.codes[0] : a.codes[1]) +
                       (bh * a.L + it.base) * kHeadDim;
#pragma unroll
      for (int k = 0; k < kWrPasses; ++k) {
        const int r = row0 + k * kWrStep;
        if (!full && (r < it.lo || r >= it.hi)) continue;
        const float2 x0 = scaled(x[k][0], inv), x1 = scaled(x[k][1], inv);
        const float2 y0 = scaled(y[k][0], inv), y1 = scaled(y[k][1], inv);
        uint32_t w0, w1;
        if (kHalf) {
          w0 = enc4<kInt8>(x0.x, x0.y, x1.x, x1.y);
          w1 = enc4<kInt8>(y0.x, y0.y, y1.x, y1.y);
        } else {
          w0 = enc4<kInt8>(x0.x, y0.x, x0.y, y0.y);
          w1 = enc4<kInt8>(x1.x, y1.x, x1.y, y1.y);
        }
        if (!(inv > 0.f)) w0 = w1 = 0u;     // whatever the values are
        uint8_t* row = codes + r * kHeadDim;
        if (kHalf) {
          *reinterpret_cast<uint32_t*>(row + c * 4) = w0;
          *reinterpret_cast<uint32_t*>(row + 64 + c * 4) = w1;
        } else {
          *reinterpret_cast<uint2*>(row + c * 8) = make_uint2(w0, w1);
        }
      }
      if (t == 0) *scale = s;
      if (grew) {
        // the block's older codes, rounded again: four channels per thread
        const float ratio = __fdiv_rn(s_old, s);
        const int c4 = (t & 31) * 4;
        float lo4[4], hi4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          lo4[j] = INFINITY;
          hi4[j] = -INFINITY;
        }
        for (int r = warp; r < it.lo; r += kWrWarps) {
          uint32_t* p = reinterpret_cast<uint32_t*>(codes + r * kHeadDim + c4);
          const uint32_t w = recode4<kInt8>(*p, ratio);
          *p = w;
          const float2 f = dec2<kInt8>(w & 0xffffu), g = dec2<kInt8>(w >> 16);
          const float v[4] = {f.x, f.y, g.x, g.y};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            lo4[j] = fminf(lo4[j], v[j]);
            hi4[j] = fmaxf(hi4[j], v[j]);
          }
        }
        if (it.key) {
          // through the other half of the channel ranges
          float* chan = reinterpret_cast<float*>(smem + kWrChan) +
                        (((n & 1) ^ 1) * 2 * kWrWarps + warp) * kHeadDim + c4;
          *reinterpret_cast<float4*>(chan) =
              make_float4(lo4[0], lo4[1], lo4[2], lo4[3]);
          *reinterpret_cast<float4*>(chan + kWrWarps * kHeadDim) =
              make_float4(hi4[0], hi4[1], hi4[2], hi4[3]);
          __syncthreads();
        }
      }
      if (it.key && t < 2 * kHeadDim) {
        // thread t < 128: lower bound of channel t; then the upper bounds
        const bool upper = t >= kHeadDim;
        const int ch = t & (kHeadDim - 1);
        auto range = [&](int half) {
          const float* chan =
              reinterpret_cast<const float*>(smem + kWrChan) +
              (half * 2 + upper) * kWrWarps * kHeadDim + ch;
          float v[kWrWarps];
#pragma unroll
          for (int w = 0; w < kWrWarps; ++w) v[w] = chan[w * kHeadDim];
          float m = v[0];
#pragma unroll
          for (int w = 1; w < kWrWarps; ++w)
            m = upper ? fmaxf(m, v[w]) : fminf(m, v[w]);
          return m;
        };
        // encoding keeps the order
        const float m = range(n & 1);
        float code = dec2<kInt8>(code2<kInt8>(m, m, inv)).x;
        if (grew) {
          const float old = range((n & 1) ^ 1);
          code = upper ? fmaxf(code, old) : fminf(code, old);
        }
        int bound = upper ? bound_hi<kInt8>(code) : bound_lo<kInt8>(code);
        int8_t* bd = a.k_bounds + at * 2 * kHeadDim + t;
        if (it.lo > 0 && !grew)     // the older tokens' bounds still hold
          bound = upper ? max(bound, int(*bd)) : min(bound, int(*bd));
        *bd = int8_t(bound);
      }
      if (grew && it.key) __syncthreads();   // the ranges have been read
    }
  }
}

// ------------------------------------------------------------------ read
//
// out[b][t][h] = code * scale of slot start[b] + t, zeros outside
// [0, min(kv_len[b], L)). A CTA takes 32 tokens of one (row, head) of K or
// V, eight lanes per row of 128 codes, 16 codes each. Heads are neighbours
// in the grid, so that a token's heads, adjacent in the output, are written
// close in time. Bound by HBM: 128K tokens x 32 heads in 498 us, the rate of
// a plain copy; two, four and eight rows per thread took 513, 545 and 557.
constexpr int kRdThreads = 256;
constexpr int kRdTokens = kRdThreads / 8;

template <bool kInt8>
__global__ void __launch_bounds__(kRdThreads)
kv8_read_kernel(const __grid_constant__ Kv8ReadArgs a, int tiles) {
  pdl_wait();
  pdl_trigger();
  uint32_t e = blockIdx.x;
  const bool key = (e & 1) == 0;
  e >>= 1;
  const int h = int(e % uint32_t(a.H));
  e /= uint32_t(a.H);
  const int b = int(e / uint32_t(tiles));
  const int tok = int(e - uint32_t(b) * uint32_t(tiles)) * kRdTokens +
                  (threadIdx.x >> 3);
  const int c = threadIdx.x & 7;
  if (tok >= a.T) return;
  const int nblk = (a.L + kKv8Block - 1) / kKv8Block;
  const int64_t bh = int64_t(b) * a.H + h;
  const int64_t slot = int64_t(__ldg(a.start + b)) + tok;
  const int len = a.kv_len ? min(__ldg(a.kv_len + b), a.L) : a.L;
  uint4 w = make_uint4(0, 0, 0, 0);
  float s = 0.f;
  if (slot >= 0 && slot < len) {
    w = __ldg(static_cast<const uint4*>(key ? a.codes[0] : a.codes[1]) +
              (bh * a.L + slot) * 8 + c);
    s = __ldg((key ? a.scale[0] : a.scale[1]) + bh * nblk + slot / kKv8Block);
  }
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f0 = dec2<kInt8>(ws[k] & 0xffffu);
    const float2 f1 = dec2<kInt8>(ws[k] >> 16);
    o[2 * k] = pack_bf16x2(f0.x * s, f0.y * s);
    o[2 * k + 1] = pack_bf16x2(f1.x * s, f1.y * s);
  }
  uint4* dst = static_cast<uint4*>(key ? a.out[0] : a.out[1]) +
               ((int64_t(b) * a.T + tok) * a.H + h) * 16 + c * 2;
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

template <bool kInt8, bool kHalf>
cudaError_t launch_few(const Kv8WriteArgs& a, cudaStream_t st) {
  const int64_t items = int64_t(a.B) * a.H * 2 * (a.T > 1 ? 2 : 1);
  const int64_t grid = (items + kFewThreads / 32 - 1) / (kFewThreads / 32);
  return launch_dependent(kv8_write_few_kernel<kInt8, kHalf>,
                          dim3(unsigned(grid)), dim3(kFewThreads), 0, st, a,
                          items);
}

template <bool kInt8, bool kHalf>
cudaError_t launch_many(const Kv8WriteArgs& a, int* status, cudaStream_t st) {
  CUtensorMap mk, mv;
  if (!make_tokens_map(&mk, a.x[0], a.B, a.T, a.H) ||
      !make_tokens_map(&mv, a.x[1], a.B, a.T, a.H))
    return cudaErrorInvalidValue;
  const int sms = sm_count();
  WriteGrid g{};
  g.per_row = (a.T + kKv8Block - 1) / kKv8Block + 1;
  // as many heads per item as leave each SM four items or more: a longer
  // run reuses the angles, a shorter one spreads the work
  const int64_t tiles = 2 * int64_t(a.B) * g.per_row * a.H;
  g.heads = int(std::max<int64_t>(
      1, std::min<int64_t>({16, tiles / (4 * sms), a.H})));
  g.groups = (a.H + g.heads - 1) / g.heads;
  g.items = 2 * int64_t(a.B) * g.per_row * g.groups;
  const cudaError_t e = allow_smem<kv8_write_kernel<kInt8, kHalf>>(kWrSmem);
  if (e != cudaSuccess) return e;
  const int64_t ctas = std::min<int64_t>(g.items, sms);
  return launch_dependent(kv8_write_kernel<kInt8, kHalf>,
                          dim3(unsigned(ctas)), dim3(kWrThreads), kWrSmem, st,
                          mk, mv, a, g, status);
}

template <bool kInt8, bool kHalf>
cudaError_t launch_write(const Kv8WriteArgs& a, int* status, cudaStream_t st) {
  return a.T <= kFewTokens ? launch_few<kInt8, kHalf>(a, st)
                           : launch_many<kInt8, kHalf>(a, status, st);
}

}  // namespace

cudaError_t launch_kv8_write(const Kv8WriteArgs& a, int* status,
                             cudaStream_t st) {
  const cudaError_t e =
      a.int8 ? (a.half ? launch_write<true, true>(a, status, st)
                       : launch_write<true, false>(a, status, st))
             : (a.half ? launch_write<false, true>(a, status, st)
                       : launch_write<false, false>(a, status, st));
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_kv8_read(const Kv8ReadArgs& a, cudaStream_t st) {
  const int tiles = (a.T + kRdTokens - 1) / kRdTokens;
  const int64_t grid = int64_t(a.B) * a.H * tiles * 2;
  const cudaError_t e = launch_dependent(
      a.int8 ? kv8_read_kernel<true> : kv8_read_kernel<false>,
      dim3(unsigned(grid)), dim3(kRdThreads), 0, st, a, tiles);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

}  // namespace lwm
