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
#include "kv8.cuh"

namespace lwm {
namespace {

constexpr int kWrThreads = 256;
constexpr int kWrLanes = 16;                       // lanes per token row
constexpr int kWrRows = kWrThreads / kWrLanes;     // rows per pass
constexpr int kWrPasses = kKv8Block / kWrRows;

// One CTA per (row, block touched, head, K or V): 16 lanes share a token,
// eight channels each, eight tokens per thread; the block stays in
// registers between the maximum and the encoding, so the input is read
// once and the codes are written once.
template <bool kInt8>
__global__ void __launch_bounds__(kWrThreads)
kv8_write_kernel(const Kv8WriteArgs a, int blocks_per_row) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[kWrThreads / 32];
  __shared__ float bmin[kWrThreads / 32][kHeadDim];
  __shared__ float bmax[kWrThreads / 32][kHeadDim];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int c = t % kWrLanes, row0 = t / kWrLanes;
  int64_t e = blockIdx.x;
  const int which = int(e & 1);
  e >>= 1;
  const int h = int(e % a.H);
  e /= a.H;
  const int blk_i = int(e % blocks_per_row);
  const int b = int(e / blocks_per_row);
  const bool key = which == 0;

  const int64_t start = a.start[b];
  const int n_new = a.n_new ? max(0, min(a.n_new[b], a.T)) : a.T;
  // slots [first, end) get the new tokens; older tokens lie below first
  const int64_t first = start > 0 ? start : 0;
  const int64_t end = min(start + n_new, int64_t(a.L));
  const int64_t base = (first / kKv8Block + blk_i) * kKv8Block;
  if (first >= end || base >= end) return;
  const int lo_new = int(max(first - base, int64_t(0)));
  const int hi_new = int(min(end - base, int64_t(kKv8Block)));
  const bool has_old = lo_new > 0;

  const int nblk = (a.L + kKv8Block - 1) / kKv8Block;
  const int64_t bh = int64_t(b) * a.H + h;
  const int64_t sc_i = bh * nblk + base / kKv8Block;
  uint8_t* codes = static_cast<uint8_t*>(a.codes[which]) +
                   (bh * a.L + base) * kHeadDim;
  const float s_old = has_old ? a.scale[which][sc_i] : 0.f;

  float x[kWrPasses][8];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kWrPasses; ++i) {
    const int r = row0 + i * kWrRows;
    const bool on = r >= lo_new && r < hi_new;
    uint4 w = make_uint4(0, 0, 0, 0);
    int p = 0;
    if (on) {
      const int64_t tok = int64_t(b) * a.T + (base + r - start);
      w = __ldg(reinterpret_cast<const uint4*>(a.x[which]) +
                (tok * a.H + h) * kWrLanes + c);
      if (key) p = max(0, min(__ldg(a.positions + tok), a.max_pos - 1));
    }
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[i][2 * k] = bf16lo_to_f32(ws[k]);
      x[i][2 * k + 1] = bf16hi_to_f32(ws[k]);
    }
    if (key) {
      const float4* tab = reinterpret_cast<const float4*>(
          a.table + int64_t(p) * kHeadDim);
      if (a.half) {
        // channels 8c' .. 8c'+7 pair with those 64 further up, held by the
        // lane eight away
        const float4* tc = tab + (c & 7) * 4;
        const bool low = c < 8;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 cs =
              on ? __ldg(tc + k) : make_float4(0.f, 0.f, 0.f, 0.f);
          const float cc[2] = {cs.x, cs.z}, ss[2] = {cs.y, cs.w};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float me = x[i][2 * k + u];
            const float other = __shfl_xor_sync(0xffffffffu, me, 8);
            x[i][2 * k + u] =
                low ? __fsub_rn(__fmul_rn(me, cc[u]), __fmul_rn(other, ss[u]))
                    : __fadd_rn(__fmul_rn(other, ss[u]), __fmul_rn(me, cc[u]));
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 cs =
              on ? __ldg(tab + c * 2 + k) : make_float4(0.f, 0.f, 0.f, 0.f);
          const float cc[2] = {cs.x, cs.z}, ss[2] = {cs.y, cs.w};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float p0 = x[i][4 * k + 2 * u], p1 = x[i][4 * k + 2 * u + 1];
            x[i][4 * k + 2 * u] =
                __fsub_rn(__fmul_rn(p0, cc[u]), __fmul_rn(p1, ss[u]));
            x[i][4 * k + 2 * u + 1] =
                __fadd_rn(__fmul_rn(p0, ss[u]), __fmul_rn(p1, cc[u]));
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = max_nan(amax, fabsf(x[i][k]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (lane == 0) red[warp] = amax;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kWrThreads / 32; ++k) amax = max_nan(amax, red[k]);

  constexpr float kRq = kInt8 ? 1.f / kInt8Max : 1.f / kE4m3Max;
  float s = max_nan(s_old, __fmul_rn(amax, kRq));
  if (s < kTinyScale) s = 0.f;
  if (!(s <= 3.402823466e38f)) s = __int_as_float(0x7fffffff);  // NaN
  const bool ok = s > 0.f;                        // false for NaN
  const float inv = ok ? __fdiv_rn(1.f, s) : 0.f;
  // older codes change only when the scale grew; a NaN leaves them
  const bool grew = has_old && ok && s > s_old;
  const float ratio = grew ? __fdiv_rn(s_old, s) : 1.f;

  float mn[8], mx[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    mn[k] = INFINITY;
    mx[k] = -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < kWrPasses; ++i) {
    const int r = row0 + i * kWrRows;
    uint2* at = reinterpret_cast<uint2*>(codes + r * kHeadDim + c * 8);
    const bool is_new = r >= lo_new && r < hi_new;
    if (!is_new && !(grew && r < lo_new)) continue;
    uint32_t w[4];
    if (is_new) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = ok ? enc2<kInt8>(__fmul_rn(x[i][2 * k], inv),
                                __fmul_rn(x[i][2 * k + 1], inv))
                  : 0u;
    } else {
      const uint2 old = *at;
      const uint32_t ow[4] = {old.x & 0xffffu, old.x >> 16, old.y & 0xffffu,
                              old.y >> 16};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = dec2<kInt8>(ow[k]);
        w[k] = enc2<kInt8>(__fmul_rn(f.x, ratio), __fmul_rn(f.y, ratio));
      }
    }
    *at = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    if (key) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = dec2<kInt8>(w[k]);
        mn[2 * k] = fminf(mn[2 * k], f.x);
        mx[2 * k] = fmaxf(mx[2 * k], f.x);
        mn[2 * k + 1] = fminf(mn[2 * k + 1], f.y);
        mx[2 * k + 1] = fmaxf(mx[2 * k + 1], f.y);
      }
    }
  }
  if (t == 0) a.scale[which][sc_i] = s;
  if (!key) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    mn[k] = fminf(mn[k], __shfl_xor_sync(0xffffffffu, mn[k], 16));
    mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 16));
  }
  if (lane < kWrLanes) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      bmin[warp][c * 8 + k] = mn[k];
      bmax[warp][c * 8 + k] = mx[k];
    }
  }
  __syncthreads();
  if (t < kHeadDim) {
    float m0 = INFINITY, m1 = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWrThreads / 32; ++w) {
      m0 = fminf(m0, bmin[w][t]);
      m1 = fmaxf(m1, bmax[w][t]);
    }
    constexpr float kUnit = kInt8 ? 1.f : kInt8Max / kE4m3Max;
    int lo = __float2int_rd(__fmul_rn(m0, kUnit));
    int hi = __float2int_ru(__fmul_rn(m1, kUnit));
    lo = max(-127, min(127, lo));
    hi = max(-127, min(127, hi));
    int8_t* bd = a.k_bounds + sc_i * 2 * kHeadDim;
    if (has_old && !grew) {  // the older tokens' bounds still hold
      lo = min(lo, int(bd[t]));
      hi = max(hi, int(bd[kHeadDim + t]));
    }
    bd[t] = int8_t(lo);
    bd[kHeadDim + t] = int8_t(hi);
  }
}

// out[b][t][h] = code * scale of slot start[b] + t, zeros outside
// [0, min(kv_len[b], L)). Eight lanes per row of 128 codes, 16 codes each.
template <bool kInt8>
__global__ void kv8_read_kernel(const Kv8ReadArgs a) {
  pdl_wait();
  pdl_trigger();
  const int which = blockIdx.y;
  const int nblk = (a.L + kKv8Block - 1) / kKv8Block;
  const int64_t n = int64_t(a.B) * a.T * a.H * 8;
  for (int64_t e = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; e < n;
       e += int64_t(gridDim.x) * blockDim.x) {
    const int c = int(e & 7);
    const int64_t row = e >> 3;              // (b, t, h)
    const int h = int(row % a.H);
    const int64_t bt = row / a.H;
    const int b = int(bt / a.T);
    const int64_t slot = int64_t(__ldg(a.start + b)) + (bt - int64_t(b) * a.T);
    const int len = a.kv_len ? min(__ldg(a.kv_len + b), a.L) : a.L;
    uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (slot >= 0 && slot < len) {
      const int64_t bh = int64_t(b) * a.H + h;
      const float s = __ldg(a.scale[which] + bh * nblk + slot / kKv8Block);
      const uint4 w = __ldg(
          reinterpret_cast<const uint4*>(a.codes[which]) +
          (bh * a.L + slot) * 8 + c);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f0 = dec2<kInt8>(ws[k] & 0xffffu);
        const float2 f1 = dec2<kInt8>(ws[k] >> 16);
        o[2 * k] = pack_bf16x2(f0.x * s, f0.y * s);
        o[2 * k + 1] = pack_bf16x2(f1.x * s, f1.y * s);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(a.out[which]) + e * 2;
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace

cudaError_t launch_kv8_write(const Kv8WriteArgs& a, cudaStream_t st) {
  const int per_row = (a.T + kKv8Block - 1) / kKv8Block + 1;
  const int64_t grid = int64_t(a.B) * per_row * a.H * 2;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const cudaError_t e = launch_dependent(
      a.int8 ? kv8_write_kernel<true> : kv8_write_kernel<false>,
      dim3(unsigned(grid)), dim3(kWrThreads), 0, st, a, per_row);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_kv8_read(const Kv8ReadArgs& a, cudaStream_t st) {
  const int64_t n = int64_t(a.B) * a.T * a.H * 8;
  const int threads = 256;
  const int64_t want = (n + threads - 1) / threads;
  const unsigned grid = unsigned(want < (1 << 20) ? want : (1 << 20));
  const cudaError_t e = launch_dependent(
      a.int8 ? kv8_read_kernel<true> : kv8_read_kernel<false>, dim3(grid, 2),
      dim3(threads), 0, st, a);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

}  // namespace lwm
