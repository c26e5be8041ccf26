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
  n.start = ld_now(a.start + b);
  const int count = a.n_new ? max(0, min(ld_now(a.n_new + b), a.T)) : a.T;
  n.lo = n.start > 0 ? n.start : 0;
  n.hi = min(n.start + count, int64_t(a.L));
  return n;
}

// Blocks that a row's new slots lie in.
__device__ __forceinline__ int new_blocks(const NewSlots& n) {
  return n.lo < n.hi ? int((n.hi - 1) / kKv8Block - n.lo / kKv8Block) + 1 : 0;
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
// and 256 bounds and writes 128 codes. Bound by latency, half a microsecond
// per token: 4 tokens of 8 to 512 (row, head) pairs take 3.1 to 4.3 us, where
// the kernel for many tokens, which moves a whole block whatever is new in
// it, takes 5.8 to 14. The two meet at 12 tokens where there are few pairs
// (8 to 128 pairs: 5.8 to 6.4 against 5.8 to 6.6; 16 tokens 7.0 to 7.7
// against 5.8 to 6.7) and at 32 where each SM has several (512 pairs: 18.8
// against 18.2; 2048: 33 against 52; 4096: 77 against 105).
constexpr int kFewThreads = 128;
constexpr int kFewTokens = 12, kFewTokensOfMany = 32, kManyPairs = 512;

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
    const uint32_t w0 = ld_now(reinterpret_cast<const uint32_t*>(row + 2 * c0));
    const uint32_t w1 = ld_now(reinterpret_cast<const uint32_t*>(row + 2 * c1));
    x[0] = bf16lo_to_f32(w0);
    x[1] = bf16hi_to_f32(w0);
    x[2] = bf16lo_to_f32(w1);
    x[3] = bf16hi_to_f32(w1);
    if (key) {
      const int p = max(0, min(ld_now(a.positions + tok), a.max_pos - 1));
      // pairs 2 lane and 2 lane + 1
      const float4 cs = ld_now(reinterpret_cast<const float4*>(
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
// All (row, block of 128 slots, head) that the call touches, in this order,
// are cut into equal shares, one per CTA, whatever the rows' lengths are.
// The heads' [128 tokens][128] bf16 boxes, K and V, come in by TMA through a
// ring of stages, the angles of a block's tokens (512 bytes each) by bulk
// copies while the last V boxes of the block before are worked on. Two
// groups of eight warps take the boxes in turn, each with a loader and
// stages of its own, so that neither waits for the other; K and V alternate
// within each group, so that the instructions of the one and the traffic of
// the other even out. 16 lanes share a token, eight channels each (4c .. 4c + 3
// and the same 64 further up), eight tokens per thread; the rotated block
// stays in registers between the maximum and the encoding, so each input is
// read once and each code written once. K keeps the channels' smallest and
// largest value, which give the block's maximum as well as its bounds. One
// barrier of the group per box.
// 32K tokens x 32 heads (805 MB) take 145 us. The traffic alone would take
// 115 to 124 (an elementwise stream, a copy), the warps' work on boxes that
// come from L2 and go nowhere 114; the two overlap in part. One loader for
// both groups took 148 (147 without the rotation, 120 with V boxes in K's
// place: it is the chain from the box to its maximum and on to the codes
// that counts, not the arithmetic), all K before V 153, shares of whole runs
// of heads 164 for the same tokens in 32 rows, one group of 16 warps 187,
// and a CTA per block and head without TMA 536.
constexpr int kWrGroups = 2;
constexpr int kWrGroup = 256;                       // threads of a group
constexpr int kWrWarps = kWrGroup / 32;
constexpr int kWrThreads = kWrGroups * (kWrGroup + 32);  // and the loaders'
constexpr int kWrLanes = 16;
constexpr int kWrStep = kWrGroup / kWrLanes;        // tokens per pass
constexpr int kWrPasses = kKv8Block / kWrStep;
constexpr int kWrStages = 4;
constexpr int kWrTile = kKv8Block * kHeadDim * 2;
constexpr int kWrAngles = kKv8Block * kHeadDim * 4;  // 64 pairs per token
constexpr uint64_t kWrWaitNs = 4000000000ull;

// A box and where its codes go.
struct __align__(16) WriteBox {
  int64_t codes;      // first code of the block
  int64_t at;         // its scale
  int lo, hi;         // its new slots
  int flags;
  int item;           // counts the CTA's blocks (angles)
};
enum : int {
  kBoxKey = 1,
  kBoxEnd = 2,
  // Of every run of heads, each group waits for the angles, so that it never
  // is a run ahead of them, and says once that it needs them no more: at its
  // K boxes and the last of them, or at its V box where it has no K.
  kBoxAngles = 4,
  kBoxFree = 8,
};

// shared memory (bytes): stages, angles, channel ranges
// [group][box parity][lo, hi][warp][128], maxima [group][parity][warp],
// boxes, barriers
constexpr int kWrAng = kWrStages * kWrTile;
constexpr int kWrChan = kWrAng + kWrAngles;
constexpr int kWrChanHalf = 2 * kWrWarps * kHeadDim * 4;   // one parity
constexpr int kWrMax = kWrChan + kWrGroups * 2 * kWrChanHalf;
constexpr int kWrBox = kWrMax + kWrGroups * 2 * kWrWarps * 4;
constexpr int kWrBars = kWrBox + kWrStages * int(sizeof(WriteBox));
constexpr int wFull = 0, wEmpty = kWrStages, wAngles = 2 * kWrStages,
              wFree = wAngles + 1, kWrNumBars = wFree + 1;
constexpr int kWrSmem = kWrBars + kWrNumBars * 8 + 16 + 128;
static_assert(kWrSmem <= 232448, "shared memory per CTA");

// Barrier of a group; true if all its threads said so.
__device__ __forceinline__ bool group_all(int id, bool mine) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
      "bar.red.and.pred p, %1, 256, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(uint32_t(mine))
      : "memory");
  return all != 0;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src,
                                          uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Where a group finds its box and leaves what its threads exchange: the
// stage, the group and the parity of its boxes.
struct WriteWhere {
  uint8_t* smem;
  int stage, group, parity;
  __device__ __forceinline__ float* chan(int parity) const {
    return reinterpret_cast<float*>(smem + kWrChan +
                                    (group * 2 + parity) * kWrChanHalf);
  }
};

// One box by one group. kFull: every slot of the block is new. False if a
// warp of the group has given up.
template <bool kInt8, bool kHalf, bool kKey, bool kFull>
__device__ __forceinline__ bool write_box(const Kv8WriteArgs& a,
                                          const WriteBox& box,
                                          const WriteWhere& w) {
  const int t = threadIdx.x & (kWrGroup - 1);
  const int lane = t & 31, wg = t >> 5;
  const int c = t % kWrLanes, row0 = t / kWrLanes;
  float* scale = (kKey ? a.scale[0] : a.scale[1]) + box.at;
  float s_old = 0.f;
  if (!kFull && box.lo > 0) s_old = __ldcg(scale);
  // v[k][j]: channel 4c + j of token row0 + 16 k, then 64 + 4c + j - 4
  float v[kWrPasses][8];
#pragma unroll
  for (int k = 0; k < kWrPasses; ++k) {
    const uint8_t* row =
        w.smem + w.stage * kWrTile + (row0 + k * kWrStep) * (kHeadDim * 2);
    const uint2 u = *reinterpret_cast<const uint2*>(row + c * 8);
    const uint2 x = *reinterpret_cast<const uint2*>(row + 128 + c * 8);
    v[k][0] = bf16lo_to_f32(u.x); v[k][1] = bf16hi_to_f32(u.x);
    v[k][2] = bf16lo_to_f32(u.y); v[k][3] = bf16hi_to_f32(u.y);
    v[k][4] = bf16lo_to_f32(x.x); v[k][5] = bf16hi_to_f32(x.x);
    v[k][6] = bf16lo_to_f32(x.y); v[k][7] = bf16hi_to_f32(x.y);
    if (kKey) {
      const float4* ang = reinterpret_cast<const float4*>(
          w.smem + kWrAng + (row0 + k * kWrStep) * (kHeadDim * 4));
      if (kHalf) {          // pairs 4c .. 4c + 3
        const float4 p = ang[2 * c], q = ang[2 * c + 1];
        rotate(v[k][0], v[k][4], p.x, p.y);
        rotate(v[k][1], v[k][5], p.z, p.w);
        rotate(v[k][2], v[k][6], q.x, q.y);
        rotate(v[k][3], v[k][7], q.z, q.w);
      } else {              // pairs 2c, 2c + 1 and 32 + 2c, 33 + 2c
        const float4 p = ang[c], q = ang[16 + c];
        rotate(v[k][0], v[k][1], p.x, p.y);
        rotate(v[k][2], v[k][3], p.z, p.w);
        rotate(v[k][4], v[k][5], q.x, q.y);
        rotate(v[k][6], v[k][7], q.z, q.w);
      }
    }
  }
  auto on = [&](int k) {
    const int r = row0 + k * kWrStep;
    return r >= box.lo && r < box.hi;
  };
  float amax = 0.f;
  // the warp has read the box and its angles
  __syncwarp();
  if (lane == 0) {
    const uint32_t bars = smem_u32(w.smem) + kWrBars;
    mbar_arrive(bars + 8u * (wEmpty + w.stage));
    if (box.flags & kBoxFree) mbar_arrive(bars + 8u * wFree);
  }
  if (kKey) {
    // lanes 0-15 keep the smallest values of the warp's two tokens of each
    // pass, the others the largest
    const bool low = lane < kWrLanes;
    bool some = kFull;
    float m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float mn, mx;
      if (kFull) {
        mn = min_nan(v[0][j], v[1][j]);
        mx = max_nan(v[0][j], v[1][j]);
#pragma unroll
        for (int k = 2; k < kWrPasses; k += 2) {
          mn = min3_nan(mn, v[k][j], v[k + 1][j]);
          mx = max3_nan(mx, v[k][j], v[k + 1][j]);
        }
      } else {
        mn = INFINITY;
        mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < kWrPasses; ++k) {
          if (!on(k)) continue;
          some = true;
          mn = min_nan(mn, v[k][j]);
          mx = max_nan(mx, v[k][j]);
        }
      }
      const float got = __shfl_xor_sync(0xffffffffu, low ? mx : mn, 16);
      m[j] = low ? min_nan(mn, got) : max_nan(mx, got);
    }
    float* to =
        w.chan(w.parity) + (low ? wg : kWrWarps + wg) * kHeadDim + 4 * c;
    *reinterpret_cast<float4*>(to) = make_float4(m[0], m[1], m[2], m[3]);
    *reinterpret_cast<float4*>(to + 64) =
        make_float4(m[4], m[5], m[6], m[7]);
    // a warp none of whose tokens is new has nothing to add
    if (__any_sync(0xffffffffu, some))
      amax = max3_abs_nan(max3_abs_nan(m[0], m[1], m[2]),
                          max3_abs_nan(m[3], m[4], m[5]),
                          max_nan(fabsf(m[6]), fabsf(m[7])));
  } else {
#pragma unroll
    for (int k = 0; k < kWrPasses; ++k) {
      if (!kFull && !on(k)) continue;
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        amax = max3_abs_nan(amax, v[k][j], v[k][j + 1]);
    }
  }
  amax = warp_max_abs(amax);
  float* red = reinterpret_cast<float*>(w.smem + kWrMax) +
               (w.group * 2 + w.parity) * kWrWarps;
  if (lane == 0) red[wg] = amax;
  if (!group_all(1 + w.group, true)) return false;
  {
    const float4 p = *reinterpret_cast<const float4*>(red);
    const float4 q = *reinterpret_cast<const float4*>(red + 4);
    amax = max3_nan(max3_nan(p.x, p.y, p.z), max3_nan(p.w, q.x, q.y),
                    max_nan(q.z, q.w));
  }
  const float sc = block_scale<kInt8>(s_old, amax);
  const float inv = sc > 0.f ? __fdiv_rn(1.f, sc) : 0.f;
  const bool grew = !kFull && box.lo > 0 && sc > s_old;
  uint8_t* codes =
      static_cast<uint8_t*>(kKey ? a.codes[0] : a.codes[1]) + box.codes;
  uint8_t* mine = codes + row0 * kHeadDim + 4 * c;
#pragma unroll
  for (int k = 0; k < kWrPasses; ++k) {
    if (!kFull && !on(k)) continue;
    uint32_t w0 = enc4<kInt8>(
        __fmul_rn(v[k][0], inv), __fmul_rn(v[k][1], inv),
        __fmul_rn(v[k][2], inv), __fmul_rn(v[k][3], inv));
    uint32_t w1 = enc4<kInt8>(
        __fmul_rn(v[k][4], inv), __fmul_rn(v[k][5], inv),
        __fmul_rn(v[k][6], inv), __fmul_rn(v[k][7], inv));
    if (!(inv > 0.f)) w0 = w1 = 0u;       // whatever the values are
    *reinterpret_cast<uint32_t*>(mine + k * kWrStep * kHeadDim) = w0;
    *reinterpret_cast<uint32_t*>(mine + k * kWrStep * kHeadDim + 64) = w1;
  }
  if (t == 0) *scale = sc;
  float* old_chan = w.chan(w.parity ^ 1);
  if (grew) {
    // the block's older codes, rounded again: four channels per thread,
    // their range through the other half of the channel ranges
    const float ratio = __fdiv_rn(s_old, sc);
    const int c4 = lane * 4;
    float lo4[4], hi4[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo4[j] = INFINITY;
      hi4[j] = -INFINITY;
    }
    for (int r = wg; r < box.lo; r += kWrWarps) {
      uint32_t* p = reinterpret_cast<uint32_t*>(codes + r * kHeadDim + c4);
      const uint32_t u = recode4<kInt8>(*p, ratio);
      *p = u;
      const float2 f = dec2<kInt8>(u & 0xffffu), g = dec2<kInt8>(u >> 16);
      const float x[4] = {f.x, f.y, g.x, g.y};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo4[j] = fminf(lo4[j], x[j]);
        hi4[j] = fmaxf(hi4[j], x[j]);
      }
    }
    *reinterpret_cast<float4*>(old_chan + wg * kHeadDim + c4) =
        make_float4(lo4[0], lo4[1], lo4[2], lo4[3]);
    *reinterpret_cast<float4*>(old_chan + (kWrWarps + wg) * kHeadDim + c4) =
        make_float4(hi4[0], hi4[1], hi4[2], hi4[3]);
    named_barrier_sync(1 + w.group, kWrGroup);
  }
  if (kKey) {
    // thread t < 128: lower bound of channel t; then the upper bounds
    const bool upper = t >= kHeadDim;
    auto range = [&](const float* from) {
      const float* p = from + (upper ? kWrWarps * kHeadDim : 0) +
                       (t & (kHeadDim - 1));
      float m = p[0];
#pragma unroll
      for (int i = 1; i < kWrWarps; ++i) {
        const float x = p[i * kHeadDim];
        m = upper ? fmaxf(m, x) : fminf(m, x);
      }
      return m;
    };
    // encoding keeps the order
    const float m = range(w.chan(w.parity));
    float code = dec2<kInt8>(code2<kInt8>(m, m, inv)).x;
    if (grew) {
      const float old = range(old_chan);
      code = upper ? fmaxf(code, old) : fminf(code, old);
    }
    int bound = upper ? bound_hi<kInt8>(code) : bound_lo<kInt8>(code);
    int8_t* bd = a.k_bounds + box.at * 2 * kHeadDim + t;
    if (!kFull && box.lo > 0 && !grew)   // the older tokens' bounds still hold
      bound = upper ? max(bound, int(*bd)) : min(bound, int(*bd));
    *bd = int8_t(bound);
  }
  if (grew) named_barrier_sync(1 + w.group, kWrGroup);   // ranges are read
  return true;
}

template <bool kInt8, bool kHalf>
__global__ void __launch_bounds__(kWrThreads, 1)
kv8_write_kernel(const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ Kv8WriteArgs a, int* status) {
  extern __shared__ uint8_t dsmem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(dsmem_raw) + 127) & ~uintptr_t(127));
  const uint32_t sbase = smem_u32(smem);
  WriteBox* boxes = reinterpret_cast<WriteBox*>(smem + kWrBox);
  volatile int* abort_word =
      reinterpret_cast<volatile int*>(smem + kWrBars + kWrNumBars * 8);
  auto bar = [&](int i) { return sbase + kWrBars + 8u * i; };
  auto wait = [&](int i, int phase) {
    return mbar_wait(bar(i), phase & 1, abort_word, status, kWrWaitNs);
  };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWrNumBars; ++i)
      mbar_init(bar(i), i >= wEmpty && i < wEmpty + kWrStages ? kWrWarps
                        : i == wFree ? kWrGroups * kWrWarps
                                     : 1);
    fence_mbar_init();
    *abort_word = 0;
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int nblk = (a.L + kKv8Block - 1) / kKv8Block;

  if (warp >= kWrGroups * kWrWarps) {
    // -------------------------------------------- loaders, one per group
    // n counts the boxes of both groups, which take turns; each group has
    // every other stage. The first loader also fetches the angles.
    const int own = warp - kWrGroups * kWrWarps;
    static_assert(kWrGroups == 2 && kWrStages % 2 == 0, "a group's own stages");
    int n = 0, item = 0, angles = 0;
    bool ok = true;
    // rows 32 at a time, one per lane: its new slots, its blocks and those
    // of the rows up to it, `before` those of the rows below row0
    NewSlots mine;
    int count, upto, before = 0, row0 = 0;
    auto rows_at = [&](int row) {
      mine = NewSlots{0, 0, 0};
      if (row + lane < a.B) mine = new_slots(a, row + lane);
      count = new_blocks(mine);
      upto = count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
    };
    rows_at(0);
    int all = __shfl_sync(0xffffffffu, upto, 31);
    if (a.B > 32) {
      int more_rows = 0;
      for (int b = lane + 32; b < a.B; b += 32)
        more_rows += new_blocks(new_slots(a, b));
      all += __reduce_add_sync(0xffffffffu, more_rows);
    }
    // the CTA's share of all (row, block, head), heads innermost
    all *= a.H;
    const int C = gridDim.x, c = blockIdx.x;
    const int each = all / C, more = all - each * C;
    int u = each * c + min(c, more);
    const int u_end = u + each + (c < more);
    while (ok && u < u_end) {
      const int blk = u / a.H, h0 = u - blk * a.H;
      const int heads = min(a.H - h0, u_end - u);
      uint32_t hit;
      while ((hit = __ballot_sync(0xffffffffu, blk < before + upto)) == 0 &&
             row0 + 32 < a.B) {
        before += __shfl_sync(0xffffffffu, upto, 31);
        row0 += 32;
        rows_at(row0);
      }
      if (hit == 0) break;
      const int f = __ffs(hit) - 1, b = row0 + f;
      NewSlots ns;
      ns.start = __shfl_sync(0xffffffffu, mine.start, f);
      ns.lo = __shfl_sync(0xffffffffu, mine.lo, f);
      ns.hi = __shfl_sync(0xffffffffu, mine.hi, f);
      const int first_blk = before + __shfl_sync(0xffffffffu, upto - count, f);
      const int64_t base =
          (ns.lo / kKv8Block + (blk - first_blk)) * kKv8Block;
      u += heads;
      const int lo = int(max(ns.lo - base, int64_t(0)));
      const int hi = int(min(ns.hi - base, int64_t(kKv8Block)));
      const int64_t tok = base - ns.start;   // of the block's first slot
      if (own == 0) {
        if (item > 0) ok = wait(wFree, item - 1);
        if (!ok) break;
        // consecutive positions are consecutive rows of the table: one copy;
        // one per token (a quarter of the loader's time) only where they jump
        int p[kKv8Block / 32];
        const int32_t* pos = a.positions + int64_t(b) * a.T + tok;
#pragma unroll
        for (int k = 0; k < kKv8Block / 32; ++k) {
          const int r = lane + 32 * k;
          p[k] = r >= lo && r < hi
                     ? max(0, min(ld_now(pos + r), a.max_pos - 1))
                     : -1;
        }
        const int first =
            max(0, min(ld_now(pos + lo), a.max_pos - 1)) - lo;   // of slot 0
        bool run = true;
#pragma unroll
        for (int k = 0; k < kKv8Block / 32; ++k)
          run = run && (p[k] < 0 || p[k] == first + lane + 32 * k);
        run = __all_sync(0xffffffffu, run);
        if (lane == 0)
          mbar_arrive_expect_tx(bar(wAngles), (hi - lo) * (kHeadDim * 4));
        __syncwarp();
        if (run) {
          if (lane == 0)
            bulk_load(sbase + kWrAng + lo * (kHeadDim * 4),
                      a.table + int64_t(first + lo) * kHeadDim,
                      (hi - lo) * (kHeadDim * 4), bar(wAngles));
        } else {
#pragma unroll
          for (int k = 0; k < kKv8Block / 32; ++k)
            if (p[k] >= 0)
              bulk_load(sbase + kWrAng + (lane + 32 * k) * (kHeadDim * 4),
                        a.table + int64_t(p[k]) * kHeadDim, kHeadDim * 4,
                        bar(wAngles));
        }
        ++angles;
      }
      // K 0, K 1; V 0, K 2; K 3, V 1; V 2, K 4; ... V m - 2, V m - 1
      auto head_of = [&](int i, bool& key) {
        key = i < min(2, heads);
        if (key) return i;
        const int pair = (i >> 1) - 1;
        key = pair < heads - 2 && ((i ^ pair) & 1) != 0;
        return pair >= heads - 2 ? i - heads : key ? pair + 2 : pair;
      };
      // the group's last K, or its one V
      int last = 2 * heads - 2 + own;
      for (bool key = false; last > own; last -= 2) {
        head_of(last, key);
        if (key) break;
      }
      int i = own;
      for (; i < 2 * heads; i += 2) {
        bool key;
        const int h = h0 + head_of(i, key);
        const int at = n + i;
        const int s = at % kWrStages;
        if (at >= kWrStages) ok = wait(wEmpty + s, at / kWrStages - 1);
        if (!ok) break;
        if (lane == 0) {
          const int64_t bh = int64_t(b) * a.H + h;
          WriteBox x;
          x.codes = (bh * a.L + base) * kHeadDim;
          x.at = bh * nblk + base / kKv8Block;
          x.lo = lo;
          x.hi = hi;
          x.flags = (key ? kBoxKey : 0) |
                    (key || i == last ? kBoxAngles : 0) |
                    (i == last ? kBoxFree : 0);
          x.item = item;
          boxes[s] = x;
          mbar_arrive_expect_tx(bar(wFull + s), kWrTile);
          // tokens before the first and behind the last one read as zeros
          tma_load_4d(sbase + s * kWrTile, key ? &tm_k : &tm_v,
                      bar(wFull + s), 0, h, int(tok), b);
        }
        __syncwarp();
      }
      n += ok ? 2 * heads : i - own;
      ++item;
    }
    // the end, behind the group's boxes
    const int end = n + own;
    const bool ended = ok;
    if (ok) {
      const int s = end % kWrStages;
      if (end >= kWrStages) ok = wait(wEmpty + s, end / kWrStages - 1);
      if (ok && lane == 0) {
        boxes[s].flags = kBoxEnd;
        mbar_arrive(bar(wFull + s));
      }
      __syncwarp();
    }
    // no load is in flight when the CTA leaves, abandoned or not (the stage
    // that an end has taken was empty before)
    for (int m = max(own, ended && ok ? end - 2 : end - kWrStages); m < end;
         m += 2)
      mbar_wait(bar(wFull + m % kWrStages), (m / kWrStages) & 1, nullptr,
                status, kWrWaitNs);
    if (angles > 0)
      mbar_wait(bar(wAngles), (angles - 1) & 1, nullptr, status, kWrWaitNs);
    return;
  }

  // ---------------------------------------------------------------- groups
  const int group = warp / kWrWarps;
  for (int n = group, parity = 0;; n += kWrGroups, parity ^= 1) {
    const int s = n % kWrStages;
    // the end and a wait that gave up are agreed on, warp by warp here and by
    // the whole group at the box's barrier, so that no thread is left alone
    bool ok = __all_sync(0xffffffffu, wait(wFull + s, n / kWrStages));
    const WriteBox box = boxes[s];
    if (ok) ok = !(box.flags & kBoxEnd);
    if (ok && (box.flags & kBoxAngles))
      ok = __all_sync(0xffffffffu, wait(wAngles, box.item));
    if (!ok) {
      group_all(1 + group, false);
      break;
    }
    const bool key = box.flags & kBoxKey;
    const bool full = box.lo == 0 && box.hi == kKv8Block;
    const WriteWhere w{smem, s, group, parity};
    if (key)
      ok = full ? write_box<kInt8, kHalf, true, true>(a, box, w)
                : write_box<kInt8, kHalf, true, false>(a, box, w);
    else
      ok = full ? write_box<kInt8, kHalf, false, true>(a, box, w)
                : write_box<kInt8, kHalf, false, false>(a, box, w);
    if (!ok) break;
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
  const int64_t slot = int64_t(ld_now(a.start + b)) + tok;
  const int len = a.kv_len ? min(ld_now(a.kv_len + b), a.L) : a.L;
  uint4 w = make_uint4(0, 0, 0, 0);
  float s = 0.f;
  if (slot >= 0 && slot < len) {
    w = ld_now(static_cast<const uint4*>(key ? a.codes[0] : a.codes[1]) +
              (bh * a.L + slot) * 8 + c);
    s = ld_now((key ? a.scale[0] : a.scale[1]) + bh * nblk + slot / kKv8Block);
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
  const cudaError_t e =
      allow_smem<kv8_write_kernel<kInt8, kHalf>, kWrSmem>();
  if (e != cudaSuccess) return e;
  // never more CTAs than there can be (block, head) pairs
  const int64_t pairs =
      int64_t(a.B) * a.H * ((a.T + kKv8Block - 1) / kKv8Block + 1);
  const int64_t ctas = std::min<int64_t>(pairs, sm_count());
  return launch_dependent(kv8_write_kernel<kInt8, kHalf>,
                          dim3(unsigned(ctas)), dim3(kWrThreads), kWrSmem, st,
                          mk, mv, a, status);
}

template <bool kInt8, bool kHalf>
cudaError_t launch_write(const Kv8WriteArgs& a, int* status, cudaStream_t st) {
  const int few = int64_t(a.B) * a.H >= kManyPairs ? kFewTokensOfMany
                                                   : kFewTokens;
  return a.T <= few ? launch_few<kInt8, kHalf>(a, st)
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
