// Block selection on the 8-bit cache's key bounds.
//
// For one query token per (row, head): q~ = R(pos) q in fp64 (the table's
// angles), codes qi = rint(q~ * (127 / max |q~|)) in [-127, 127], and for a
// block with bounds lo, hi (int8) and scale s
//   score = fp32( sum_d max(qi_d lo_d, qi_d hi_d) * s * (max |q~| / 127) ),
// an upper bound, up to the constant 127 / Q and qi's rounding, of the
// block's q . k. The sum is a dot product of whole numbers, exact in any
// order: max(a lo, a hi) is max(a, 0) hi + min(a, 0) lo. The score of the
// heads that share a cache head is their largest. The K best visible blocks
// are listed in ascending order, the first n_sink and the last n_recent
// among them always; then blocks whose score is NaN; ties go to the lowest
// index.
#include "kv8.cuh"

namespace lwm {
namespace {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 256;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same shared-memory word in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_load(const uint32_t* p,
                                              uint32_t rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at)
               : "memory");
  return v;
}

// Ranking order as an unsigned word: forced blocks, NaN, then by score.
__device__ __forceinline__ uint32_t rank_key(float s, bool forced) {
  if (forced) return 0xffffffffu;
  if (s != s) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(s + 0.f);   // -0 ranks as +0
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// Sum over the block's threads of (x, y), for every thread.
__device__ __forceinline__ uint2 block_prefix(uint32_t x, uint2* buf,
                                              uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) buf[warp].x = inc;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    const uint32_t y = buf[w].x;
    if (w < warp) before += y;
    all += y;
  }
  __syncthreads();
  *total = all;
  return make_uint2(before + inc - x, before + inc);
}

// A cluster of C CTAs per (row, cache head); CTA r scores the r-th share of
// the visible blocks into its shared memory, and the cluster finds the K-th
// best key by four rounds of 8-bit counting over all its shares.
__global__ void __launch_bounds__(kSelThreads)
kv8_select_kernel(const Kv8SelectArgs a, int C) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float score[];                    // [share]
  __shared__ __align__(16) int8_t qc[kKv8MaxGroup][2 * kHeadDim];
  __shared__ double qs[kKv8MaxGroup];
  __shared__ double qmax[kSelWarps];
  __shared__ uint32_t hist[4][kSelBins];
  __shared__ uint32_t counts[2];                      // above, equal
  __shared__ uint2 scan[kSelWarps];
  __shared__ uint32_t pick[2];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int r = int(cluster_rank());
  const int64_t bh = blockIdx.x / C;
  const int b = int(bh / a.H), h = int(bh % a.H);

  const int len = max(0, min(__ldg(a.kv_len + b), a.L));
  const int start = max(0, min(__ldg(a.kv_start + b), len));
  const int j0 = start / kKv8Block;
  const int j1 = len > start ? (len + kKv8Block - 1) / kKv8Block : j0;
  const int nv = j1 - j0;
  const int share = (nv + C - 1) / C;
  const int i0 = min(r * share, nv), n = min(share, nv - i0);
  const int nblk = (a.L + kKv8Block - 1) / kKv8Block;

  for (int i = t; i < 4 * kSelBins; i += kSelThreads)
    hist[i / kSelBins][i % kSelBins] = 0;

  // query codes: qc[g] = (min(qi, 0), max(qi, 0)), as the bounds lie
  const int p = max(0, min(__ldg(a.q_pos + b), a.max_pos - 1));
  for (int g = 0; g < a.G; ++g) {
    double x = 0.0;
    const int d = t & (kHeadDim - 1);
    {
      const __nv_bfloat16* q =
          static_cast<const __nv_bfloat16*>(a.q) +
          (int64_t(b) * a.H * a.G + h * a.G + g) * kHeadDim;
      const int k = a.half ? (d & 63) : (d >> 1);
      const bool low = a.half ? d < 64 : (d & 1) == 0;
      const int i_a = a.half ? k : 2 * k, i_b = a.half ? k + 64 : 2 * k + 1;
      const float2 cs = __ldg(reinterpret_cast<const float2*>(a.table) +
                              int64_t(p) * (kHeadDim / 2) + k);
      const double qa = double(__bfloat162float(q[i_a]));
      const double qb = double(__bfloat162float(q[i_b]));
      x = low ? __dsub_rn(__dmul_rn(qa, double(cs.x)),
                          __dmul_rn(qb, double(cs.y)))
              : __dadd_rn(__dmul_rn(qa, double(cs.y)),
                          __dmul_rn(qb, double(cs.x)));
    }
    double m = fabs(x);
    bool bad = !(m <= 1e300);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) qmax[warp] = m;
    bad = __syncthreads_or(bad);
    m = 0.0;
#pragma unroll
    for (int w = 0; w < kHeadDim / 32; ++w) m = fmax(m, qmax[w]);
    int qi = 0;
    if (m > 0.0 && !bad) qi = __double2int_rn(__dmul_rn(x, 127.0 / m));
    qi = max(-127, min(127, qi));
    if (t < kHeadDim) {
      qc[g][d] = int8_t(min(qi, 0));
      qc[g][kHeadDim + d] = int8_t(max(qi, 0));
    }
    // a query with a NaN or an infinity scores every block alike
    if (t == 0) qs[g] = bad ? 0.0 : __dmul_rn(m, 1.0 / 127.0);
    __syncthreads();
  }

  // scores: 16 lanes per block, 16 of its 256 bounds each
  {
    const int l16 = lane & 15;
    const int step = kSelWarps * 2;
    const int8_t* bounds =
        a.k_bounds + (bh * nblk + j0 + i0) * (2 * kHeadDim);
    const float* ks = a.k_scale + bh * nblk + j0 + i0;
    for (int i = warp * 2; i < n; i += step) {
      const int blk = i + (lane >> 4);
      const bool on = blk < n;
      int4 w = make_int4(0, 0, 0, 0);
      float s = 0.f;
      if (on) {
        w = __ldg(reinterpret_cast<const int4*>(
                bounds + int64_t(blk) * (2 * kHeadDim)) + l16);
        s = __ldg(ks + blk);
      }
      float best = -INFINITY;
      for (int g = 0; g < a.G; ++g) {
        const int4 q = *reinterpret_cast<const int4*>(&qc[g][l16 * 16]);
        int dot = __dp4a(w.x, q.x, 0);
        dot = __dp4a(w.y, q.y, dot);
        dot = __dp4a(w.z, q.z, dot);
        dot = __dp4a(w.w, q.w, dot);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
          dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const float v =
            float(__dmul_rn(__dmul_rn(double(dot), double(s)), qs[g]));
        best = max_nan(best, v);
      }
      if (on && l16 == 0) score[blk] = best;
    }
  }
  __syncthreads();

  auto forced = [&](int i) {      // i: index among this CTA's blocks
    const int k = i0 + i;
    return k < a.n_sink || k >= nv - a.n_recent;
  };
  uint32_t bar = 0, quota = 0;    // take keys above bar, quota equal to it
  const bool all = nv <= a.K;
  if (!all) {
    uint32_t prefix = 0, mask = 0;
    uint32_t left = uint32_t(a.K);
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      for (int i = t; i < n; i += kSelThreads) {
        const uint32_t key = rank_key(score[i], forced(i));
        if ((key & mask) == prefix)
          atomicAdd(&hist[pass][(key >> shift) & 255u], 1u);
      }
      if (C > 1) cluster_sync(); else __syncthreads();
      // thread t counts bin 255 - t over the cluster: best bins first
      uint32_t cnt = 0;
      const int bin = kSelBins - 1 - t;
      if (C > 1) {
        for (int c = 0; c < C; ++c) cnt += peer_load(&hist[pass][bin], c);
      } else {
        cnt = hist[pass][bin];
      }
      uint32_t total;
      const uint2 pr = block_prefix(cnt, scan, &total);
      if (pr.x < left && left <= pr.y) {
        pick[0] = uint32_t(bin);
        pick[1] = left - pr.x;
      }
      __syncthreads();
      prefix |= pick[0] << shift;
      mask |= 255u << shift;
      left = pick[1];
      __syncthreads();
    }
    bar = prefix;
    quota = left;
  }

  // how many each CTA lists, then the lists in ascending order
  uint32_t above = 0, equal = 0;
  if (t < 2) counts[t] = 0;
  __syncthreads();
  for (int i = t; i < n; i += kSelThreads) {
    if (all) {
      ++above;
    } else {
      const uint32_t key = rank_key(score[i], forced(i));
      above += key > bar;
      equal += key == bar;
    }
  }
  if (above) atomicAdd(&counts[0], above);
  if (equal) atomicAdd(&counts[1], equal);
  if (C > 1) cluster_sync(); else __syncthreads();
  uint32_t at = 0, eq_before = 0;
  for (int c = 0; c < r; ++c) {
    at += peer_load(&counts[0], c);
    eq_before += peer_load(&counts[1], c);
  }
  at += min(eq_before, quota);
  uint32_t eq_left = quota - min(eq_before, quota);
  int32_t* blocks = a.blocks + bh * a.K;
  float* out_s = a.scores + bh * a.K;
  for (int i = 0; i < n; i += kSelThreads) {
    const int k = i + t;
    bool gt = false, eq = false;
    if (k < n) {
      if (all) {
        gt = true;
      } else {
        const uint32_t key = rank_key(score[k], forced(k));
        gt = key > bar;
        eq = key == bar;
      }
    }
    uint32_t n_eq, n_take;
    const uint2 pe = block_prefix(eq ? 1u : 0u, scan, &n_eq);
    const bool take = gt || (eq && pe.x < eq_left);
    const uint2 pt = block_prefix(take ? 1u : 0u, scan, &n_take);
    if (take) {
      blocks[at + pt.x] = j0 + i0 + k;
      out_s[at + pt.x] = score[k];
    }
    at += n_take;
    eq_left -= min(eq_left, n_eq);
  }
  // the rest of a short list
  if (r == 0)
    for (int i = nv + t; i < a.K; i += kSelThreads) {
      blocks[i] = -1;
      out_s[i] = -INFINITY;
    }
  // no CTA leaves while another may still read its counts
  if (C > 1) cluster_sync();
}

}  // namespace

cudaError_t launch_kv8_select(const Kv8SelectArgs& a, cudaStream_t st) {
  const int nblk = (a.L + kKv8Block - 1) / kKv8Block;
  int C = 1;
  while (C < 8 && nblk > 128 * C) C *= 2;
  const int64_t grid = int64_t(a.B) * a.H * C;
  const size_t smem = size_t((nblk + C - 1) / C) * sizeof(float);
  cudaError_t e = allow_smem<kv8_select_kernel>(int(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(C);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kv8_select_kernel, a, C);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

}  // namespace lwm
