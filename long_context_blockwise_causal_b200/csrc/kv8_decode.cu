// Decode attention over the 8-bit cache: one query token per (row, head)
// against the visible slots [kv_start, kv_len) of its row, of all blocks or
// of a list of blocks. With q~ = R(pos) q and block scales ks, vs:
//   s_t = (q~ . k_t) ks_j / sqrt(D),  out = sum_t softmax(s)_t v_t vs_j.
//
// Work: a tile is one block of 128 slots of one (row, cache head); the G
// query heads that share a cache head go through a tile together. All tiles
// of the call, in the order (row, head, block), are cut into equal
// consecutive shares, one per CTA, whatever the rows' lengths are. A CTA
// that holds every tile of a (row, head) writes its result; the others
// leave (m, l, acc) in the workspace, at most two per CTA (the first and
// the last (row, head) of its share), and a second kernel joins them.
#include <algorithm>

#include "kv8.cuh"
#include "tc_kernels.cuh"

namespace lwm {
namespace {

struct Rows {
  const int32_t* kv_start;
  const int32_t* kv_len;
  int B, L, H, K;
  bool listed;
};

struct RowTiles {
  int start, len, t0, n;    // visible slots, first block, tiles per head
};

__device__ __forceinline__ RowTiles row_tiles(const Rows& r, int b) {
  RowTiles x;
  x.len = max(0, min(__ldg(r.kv_len + b), r.L));
  x.start = max(0, min(__ldg(r.kv_start + b), x.len));
  x.t0 = x.start / kKv8Block;
  x.n = x.len > x.start
            ? (r.listed ? r.K : (x.len + kKv8Block - 1) / kKv8Block - x.t0)
            : 0;
  return x;
}

// A warp's lanes together: tiles per head of rows [0, upto).
__device__ __forceinline__ int64_t tiles_before(const Rows& r, int upto) {
  int64_t s = 0;
  for (int b = threadIdx.x & 31; b < upto; b += 32) s += row_tiles(r, b).n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// A warp's lanes together: the row that holds tile u (counted over all rows
// and heads), and the tiles before that row.
__device__ __forceinline__ int find_row(const Rows& r, int64_t u,
                                        int64_t* before) {
  const int lane = threadIdx.x & 31;
  int64_t base = 0;
  for (int b0 = 0; b0 < r.B; b0 += 32) {
    int64_t n = b0 + lane < r.B ? int64_t(row_tiles(r, b0 + lane).n) * r.H : 0;
    int64_t inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, u < base + inc);
    if (hit) {
      const int f = __ffs(hit) - 1;
      *before = base + __shfl_sync(0xffffffffu, inc - n, f);
      return b0 + f;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  *before = base;
  return r.B;
}

// CTA c of C takes tiles [share(c), share(c + 1)).
__device__ __forceinline__ int64_t share(int64_t total, int C, int c) {
  return total * c / C;
}

// Partial result records: m[G], l[G], acc[G][128].
__host__ __device__ constexpr int part_stride(int G) {
  return G * (kHeadDim + 2);
}

constexpr int kSimpleThreads = 128;

template <bool kInt8>
__global__ void __launch_bounds__(kSimpleThreads)
kv8_decode_kernel(const Kv8DecodeArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float qs[kKv8MaxGroup][kHeadDim];
  __shared__ float ps[kKv8MaxGroup][kKv8Block];
  __shared__ float red[4];
  __shared__ int64_t where[4];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const Rows rows{a.kv_start, a.kv_len, a.B, a.L, a.H, a.K,
                  a.listed};
  if (warp == 0) {
    const int64_t total = tiles_before(rows, a.B) * a.H;
    const int64_t u0 = share(total, gridDim.x, blockIdx.x);
    const int64_t u1 = share(total, gridDim.x, blockIdx.x + 1);
    int64_t before = 0;
    const int b = u0 < u1 ? find_row(rows, u0, &before) : 0;
    if (lane == 0) {
      where[0] = u0;
      where[1] = u1;
      where[2] = b;
      where[3] = before;
    }
  }
  __syncthreads();
  int64_t u = where[0];
  const int64_t u0 = u, u1 = where[1];
  int b = int(where[2]);
  int64_t row_at = where[3];
  const int nblk = (a.L + kKv8Block - 1) / kKv8Block;
  const float scale = kLog2e / sqrtf(float(kHeadDim));
  auto reduce = [&](float x, bool is_max) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, x, o);
      x = is_max ? fmaxf(x, y) : x + y;
    }
    __syncthreads();
    if (lane == 0) red[warp] = x;
    __syncthreads();
    return is_max ? fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]))
                  : (red[0] + red[1]) + (red[2] + red[3]);
  };

  while (u < u1) {
    RowTiles rt = row_tiles(rows, b);
    if (u >= row_at + int64_t(rt.n) * a.H) {
      row_at += int64_t(rt.n) * a.H;
      ++b;
      continue;
    }
    const int h = int((u - row_at) / rt.n);
    const int64_t p0 = row_at + int64_t(h) * rt.n, p1 = p0 + rt.n;
    const int64_t ue = min(u1, p1);
    const int64_t bh = int64_t(b) * a.H + h;
    // rotated query
    __syncthreads();
    const int pos = max(0, min(__ldg(a.q_pos + b), a.max_pos - 1));
    for (int g = 0; g < a.G; ++g) {
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) +
                               (bh * a.G + g) * kHeadDim;
      const int k = a.half ? (t & 63) : (t >> 1);
      const bool low = a.half ? t < 64 : (t & 1) == 0;
      const int ia = a.half ? k : 2 * k, ib = a.half ? k + 64 : 2 * k + 1;
      const float2 cs = __ldg(reinterpret_cast<const float2*>(a.table) +
                              int64_t(pos) * (kHeadDim / 2) + k);
      const float qa = __bfloat162float(q[ia]), qb = __bfloat162float(q[ib]);
      qs[g][t] = (low ? qa * cs.x - qb * cs.y : qa * cs.y + qb * cs.x) * scale;
    }
    __syncthreads();
    float m[kKv8MaxGroup], l[kKv8MaxGroup], acc[kKv8MaxGroup];
    for (int g = 0; g < kKv8MaxGroup; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
      acc[g] = 0.f;
    }
    for (; u < ue; ++u) {
      const int j = int(u - p0);
      int blk = rt.t0 + j;
      if (a.listed) {
        const int32_t* list = a.blocks + bh * a.K;
        blk = __ldg(list + j);
        if (blk < rt.t0 || int64_t(blk) * kKv8Block >= rt.len ||
            (j > 0 && blk <= __ldg(list + j - 1)))
          continue;
      }
      const int slot = blk * kKv8Block + t;
      const bool seen = slot >= rt.start && slot < rt.len;
      const float ks = __ldg(a.k_scale + bh * nblk + blk);
      const float vs = __ldg(a.v_scale + bh * nblk + blk);
      float s[kKv8MaxGroup];
      for (int g = 0; g < kKv8MaxGroup; ++g) s[g] = 0.f;
      if (seen) {
        const uint4* kr = reinterpret_cast<const uint4*>(
            static_cast<const uint8_t*>(a.k) +
            (bh * a.L + slot) * kHeadDim);
        for (int i = 0; i < 8; ++i) {
          const uint4 w = __ldg(kr + i);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
          for (int e = 0; e < 8; ++e) {
            const float2 f = dec2<kInt8>((ws[e >> 1] >> (16 * (e & 1))) &
                                         0xffffu);
            for (int g = 0; g < a.G; ++g) {
              s[g] = fmaf(f.x, qs[g][16 * i + 2 * e], s[g]);
              s[g] = fmaf(f.y, qs[g][16 * i + 2 * e + 1], s[g]);
            }
          }
        }
      }
      for (int g = 0; g < a.G; ++g) {
        const float x = seen ? s[g] * ks : -INFINITY;
        const float mn = fmaxf(m[g], reduce(x, true));
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float alpha = exp2f(m[g] - mu);
        const float p = seen ? exp2f(x - mu) : 0.f;
        m[g] = mn;
        l[g] = l[g] * alpha + p;
        acc[g] *= alpha;
        ps[g][t] = p;
      }
      __syncthreads();
      // thread t: channel t
      const int lo = max(0, rt.start - blk * kKv8Block);
      const int hi = min(kKv8Block, rt.len - blk * kKv8Block);
      float o[kKv8MaxGroup];
      for (int g = 0; g < kKv8MaxGroup; ++g) o[g] = 0.f;
      const uint8_t* vr = static_cast<const uint8_t*>(a.v) +
                          (bh * a.L + int64_t(blk) * kKv8Block) * kHeadDim;
      for (int i = lo; i < hi; ++i) {
        const float f = dec2<kInt8>(vr[i * kHeadDim + t]).x;
        for (int g = 0; g < a.G; ++g) o[g] = fmaf(f, ps[g][i], o[g]);
      }
      for (int g = 0; g < a.G; ++g) acc[g] = fmaf(o[g], vs, acc[g]);
      __syncthreads();
    }
    const bool whole = p0 >= u0 && p1 <= u1;
    float* rec = a.part + (int64_t(blockIdx.x) * 2 + (p0 < u0 ? 0 : 1)) *
                              part_stride(a.G);
    for (int g = 0; g < a.G; ++g) {
      const float lt = reduce(l[g], false);
      if (whole) {
        const int64_t o = bh * a.G + g;
        static_cast<__nv_bfloat16*>(a.out)[o * kHeadDim + t] =
            __float2bfloat16_rn(lt == 0.f ? 0.f : acc[g] / lt);
        if (t == 0)
          a.lse[o] = lt == 0.f ? -INFINITY : (m[g] + log2f(lt)) * kLn2;
      } else {
        rec[2 * a.G + g * kHeadDim + t] = acc[g];
        if (t == 0) {
          rec[g] = m[g];
          rec[a.G + g] = lt;
        }
      }
    }
  }
}

// One CTA per (row, cache head): joins the parts of a (row, head) that more
// than one CTA of the decode kernel worked on, and writes (0, -inf) for a
// row that sees nothing.
__global__ void __launch_bounds__(kHeadDim)
kv8_combine_kernel(const Kv8DecodeArgs a, int C) {
  pdl_wait();
  pdl_trigger();
  __shared__ int64_t where[2];
  const int t = threadIdx.x;
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const Rows rows{a.kv_start, a.kv_len, a.B, a.L, a.H, a.K,
                  a.listed};
  if (t < 32) {
    const int64_t total = tiles_before(rows, a.B) * a.H;
    const int64_t before = tiles_before(rows, b) * a.H;
    if (t == 0) {
      where[0] = total;
      where[1] = before;
    }
  }
  __syncthreads();
  const int64_t total = where[0];
  const int n = row_tiles(rows, b).n;
  const int64_t o0 = int64_t(blockIdx.x) * a.G;
  if (n == 0) {
    for (int g = 0; g < a.G; ++g) {
      static_cast<__nv_bfloat16*>(a.out)[(o0 + g) * kHeadDim + t] =
          __float2bfloat16_rn(0.f);
      if (t == 0) a.lse[o0 + g] = -INFINITY;
    }
    return;
  }
  const int64_t p0 = where[1] + int64_t(h) * n, p1 = p0 + n;
  const int c0 = int(((p0 + 1) * C - 1) / total);
  const int c1 = int((p1 * C - 1) / total);
  if (c0 == c1) return;       // one CTA held it all
  for (int g = 0; g < a.G; ++g) {
    float M = -INFINITY;
    for (int c = c0; c <= c1; ++c) {
      if (share(total, C, c) == share(total, C, c + 1)) continue;
      const float* rec =
          a.part + (int64_t(c) * 2 + (c == c0)) * part_stride(a.G);
      M = fmaxf(M, rec[g]);
    }
    const float mu = M == -INFINITY ? 0.f : M;
    float l = 0.f, acc = 0.f;
    for (int c = c0; c <= c1; ++c) {
      if (share(total, C, c) == share(total, C, c + 1)) continue;
      const float* rec =
          a.part + (int64_t(c) * 2 + (c == c0)) * part_stride(a.G);
      const float w = exp2f(rec[g] - mu);
      l += rec[a.G + g] * w;
      acc += rec[2 * a.G + g * kHeadDim + t] * w;
    }
    static_cast<__nv_bfloat16*>(a.out)[(o0 + g) * kHeadDim + t] =
        __float2bfloat16_rn(l == 0.f ? 0.f : acc / l);
    if (t == 0) a.lse[o0 + g] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
  }
}

}  // namespace

int kv8_decode_grid(int B, int L, int H, int K) {
  const int64_t per = K >= 0 ? K : (L + kKv8Block - 1) / kKv8Block;
  const int64_t most = int64_t(B) * H * per;
  return int(std::max<int64_t>(1, std::min<int64_t>(most, 148 * 8)));
}

size_t kv8_part_floats(int B, int L, int H, int G, int K) {
  return size_t(kv8_decode_grid(B, L, H, K)) * 2 * part_stride(G);
}

cudaError_t launch_kv8_decode(const Kv8DecodeArgs& a, cudaStream_t st) {
  const int C = kv8_decode_grid(a.B, a.L, a.H, a.listed ? a.K : -1);
  cudaError_t e = launch_dependent(
      a.int8 ? kv8_decode_kernel<true> : kv8_decode_kernel<false>, dim3(C),
      dim3(kSimpleThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  note_launch();
  e = launch_dependent(kv8_combine_kernel, dim3(a.B * a.H), dim3(kHeadDim), 0,
                       st, a, C);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

}  // namespace lwm
