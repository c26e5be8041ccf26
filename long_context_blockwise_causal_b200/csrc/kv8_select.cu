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
#include "tc_kernels.cuh"

namespace lwm {
namespace {

constexpr int kSelPasses = 3;                // digits of up to 11 bits
constexpr int kSelBins = 2048;
constexpr int kSelMost = 8;                  // CTAs per cluster
// bytes of the scores of the longest row
constexpr int kSelMostSmem = kKv8SelectMaxLen / kKv8Block * 4;
static_assert(kSelMostSmem <= 160 * 1024,
              "a row's scores fit one CTA's shared memory");

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores to the cluster's first CTA, where this CTA would have *p.
__device__ __forceinline__ void first_store(const float* p, float v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
               : "=r"(at)
               : "r"(smem_u32(p)));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v)
               : "memory");
}

// Ranking order as an unsigned word: by score, NaN above all.
__device__ __forceinline__ uint32_t rank_key(float s) {
  if (s != s) return 0xff800001u;
  const uint32_t u = __float_as_uint(s + 0.f);   // -0 ranks as +0
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_score(uint32_t k) {
  if (k == 0xff800001u) return __int_as_float(0x7fffffff);
  return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k);
}

// Sum of x over the threads before this one.
template <int Warps>
__device__ __forceinline__ uint32_t block_prefix(uint32_t x, uint32_t* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) buf[warp] = inc;
  __syncthreads();
  uint32_t before = 0;
#pragma unroll
  for (int w = 0; w < Warps; ++w) before += w < warp ? buf[w] : 0u;
  return before + inc - x;
}

// Adds up N values (a power of two, at most 16) over the 16 lanes that share
// a block, halving the number of values a lane holds while it can: lane l
// ends with the total of value l mod N.
template <int N>
__device__ __forceinline__ int sum16(int (&v)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    // of 2 o values, those whose index has bit o go to the lanes that have it
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const int keep = up ? v[i + o] : v[i];
      const int give = up ? v[i] : v[i + o];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (int o = N; o < 16; o <<= 1)
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

// A cluster of C CTAs per (row, cache head). CTA r scores the r-th share of
// the visible blocks into the shared memory of the first CTA, which finds
// the K-th best key by three rounds of digit counting and writes the list;
// counting over the shares of all CTAs cost more in exchanges (23 us for
// three rounds over 8 CTAs) than one CTA takes for everything. Scoring reads
// 256 bytes per block: 16 lanes share a block, a warp keeps several pairs of
// blocks in flight, the first of them while the query is made ready. 1M slots
// x 32 heads (67 MB) take 23.6 us in turns over eight caches, 18.2 where the
// bounds are still in L2; 2 of them go to the digits of 512 of 8192 blocks
// (a list that takes every block needs none). 4 rows x 8 heads x 32K with 4
// query heads each are latency: 6.7 us, of which 3.3 for a call of a single
// block, 2.2 for the digits. GP: G rounded up to a power of two.
template <int GP, int Threads>
struct Sel {
  // 512 threads, one CTA per SM, for few long rows; 256 threads, four CTAs
  // per SM, for many rows
  static constexpr int kFlight = Threads == 512 ? 8 : 4;
  static constexpr int kPerSm = Threads == 512 ? 1 : 4;
  // pairs whose sums are finished together: one step of fp64 serves all of
  // them (scores are rounded from fp64, whose conversions are slow)
  static constexpr int kJoint = 16 / GP < kFlight ? 16 / GP : kFlight;
};

template <int GP, int Threads>
__global__ void __launch_bounds__(Threads, Sel<GP, Threads>::kPerSm)
kv8_select_kernel(const __grid_constant__ Kv8SelectArgs a, int C) {
  constexpr int kSelThreads = Threads;
  constexpr int kSelWarps = Threads / 32;
  constexpr int kSelFlight = Sel<GP, Threads>::kFlight;
  extern __shared__ __align__(16) float score[];      // [visible blocks]
  __shared__ __align__(16) int8_t qc[GP][2 * kHeadDim];
  __shared__ double qs[GP];
  __shared__ __align__(16) uint32_t hist[kSelPasses][kSelBins];
  __shared__ uint32_t scan[kSelWarps];
  __shared__ uint2 runs[kSelWarps], span[kSelWarps];
  __shared__ uint32_t pick[2];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int r = int(cluster_rank());
  const int64_t bh = blockIdx.x / C;
  const int b = int(bh / a.H);
  for (int i = t; i < kSelPasses * kSelBins; i += kSelThreads)
    hist[0][i] = 0;
  // a CTA that has arrived is running: its memory may be written
  if (C > 1) cluster_arrive();
  pdl_wait();
  pdl_trigger();

  const int len = max(0, min(ld_now(a.kv_len + b), a.L));
  const int start = max(0, min(ld_now(a.kv_start + b), len));
  const int j0 = start / kKv8Block;
  const int j1 = len > start ? (len + kKv8Block - 1) / kKv8Block : j0;
  const int nv = j1 - j0;
  const int share = (nv + C - 1) / C;
  const int i0 = min(r * share, nv), n = min(share, nv - i0);
  const int nblk = (a.L + kKv8Block - 1) / kKv8Block;

  const int l16 = lane & 15;
  const int8_t* bounds =
      a.k_bounds + (bh * nblk + j0 + i0) * (2 * kHeadDim) + l16 * 16;
  const float* ks = a.k_scale + bh * nblk + j0 + i0;
  int4 w[kSelFlight];
  // blocks i, i + 1 (one per half warp) and those of the next flights
  auto fetch = [&](int i) {
#pragma unroll
    for (int f = 0; f < kSelFlight; ++f) {
      const int blk = i + f * kSelWarps * 2 + (lane >> 4);
      w[f] = make_int4(0, 0, 0, 0);
      if (blk < n)
        w[f] = ld_now(reinterpret_cast<const int4*>(
            bounds + int64_t(blk) * (2 * kHeadDim)));
    }
  };
  fetch(warp * 2);

  // query codes: qc[g] = (min(qi, 0), max(qi, 0)), as the bounds lie; a warp
  // per head, two pairs of the rotation per lane
  const int p = max(0, min(ld_now(a.q_pos + b), a.max_pos - 1));
  for (int g = warp; g < GP; g += kSelWarps) {
    const int c0 = a.half ? 2 * lane : 4 * lane;       // channels c0, c0 + 1,
    const int c1 = a.half ? 64 + 2 * lane : c0 + 2;    // c1, c1 + 1
    double x[4] = {0.0, 0.0, 0.0, 0.0};
    if (g < a.G) {
      const char* q = static_cast<const char*>(a.q) +
                      (bh * a.G + g) * (kHeadDim * 2);
      const uint32_t w0 = ld_now(reinterpret_cast<const uint32_t*>(q + 2 * c0));
      const uint32_t w1 = ld_now(reinterpret_cast<const uint32_t*>(q + 2 * c1));
      const float4 cs = ld_now(reinterpret_cast<const float4*>(
                                  a.table + int64_t(p) * kHeadDim) + lane);
      const double f[4] = {bf16lo_to_f32(w0), bf16hi_to_f32(w0),
                           bf16lo_to_f32(w1), bf16hi_to_f32(w1)};
      auto turn = [](double u, double v, double c, double s, double& ru,
                     double& rv) {
        ru = __dsub_rn(__dmul_rn(u, c), __dmul_rn(v, s));
        rv = __dadd_rn(__dmul_rn(u, s), __dmul_rn(v, c));
      };
      if (a.half) {
        turn(f[0], f[2], cs.x, cs.y, x[0], x[2]);
        turn(f[1], f[3], cs.z, cs.w, x[1], x[3]);
      } else {
        turn(f[0], f[1], cs.x, cs.y, x[0], x[1]);
        turn(f[2], f[3], cs.z, cs.w, x[2], x[3]);
      }
    }
    double m = 0.0;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      bad = bad || !(fabs(x[k]) <= 1e300);
      m = fmax(m, fabs(x[k]));
    }
    bad = __any_sync(0xffffffffu, bad);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
    const double f = m > 0.0 && !bad ? 127.0 / m : 0.0;
    int qi[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      qi[k] = f > 0.0 ? __double2int_rn(__dmul_rn(x[k], f)) : 0;
      qi[k] = max(-127, min(127, qi[k]));
    }
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const int c = k ? c1 : c0;
      *reinterpret_cast<char2*>(&qc[g][c]) =
          make_char2(char(min(qi[k], 0)), char(min(qi[k + 1], 0)));
      *reinterpret_cast<char2*>(&qc[g][kHeadDim + c]) =
          make_char2(char(max(qi[k], 0)), char(max(qi[k + 1], 0)));
    }
    // a query with a NaN or an infinity scores every block alike
    if (lane == 0) qs[g] = bad ? 0.0 : __dmul_rn(m, 1.0 / 127.0);
  }
  __syncthreads();
  if (C > 1) cluster_wait();

  // scores: 16 lanes per block, 16 of its 256 bounds each
  {
    constexpr int kJoint = Sel<GP, Threads>::kJoint, kSums = kJoint * GP;
    const int mine = l16 % GP;                 // the head and, of the pairs
    const int my_pair = l16 % kSums / GP;      // finished together, the one
    const double my_qs = qs[mine];             // whose total comes here
    // one head: its codes stay in registers
    int4 q1 = make_int4(0, 0, 0, 0);
    if (GP == 1) q1 = *reinterpret_cast<const int4*>(&qc[0][l16 * 16]);
    for (int i = warp * 2; i < n; i += kSelWarps * 2 * kSelFlight) {
      if (i > warp * 2) fetch(i);
#pragma unroll
      for (int f0 = 0; f0 < kSelFlight; f0 += kJoint) {
        const int first = i + f0 * kSelWarps * 2;
        if (first >= n) break;
        const int blk = first + my_pair * kSelWarps * 2 + (lane >> 4);
        const float s = blk < n ? ld_now(ks + blk) : 0.f;
        int dot[kSums];
#pragma unroll
        for (int g = 0; g < GP; ++g) {
          const int4 q = GP == 1 ? q1
                                 : *reinterpret_cast<const int4*>(
                                       &qc[g][l16 * 16]);
#pragma unroll
          for (int f = 0; f < kJoint; ++f) {
            const int4 x = w[f0 + f];
            int d = __dp4a(x.x, q.x, 0);
            d = __dp4a(x.y, q.y, d);
            d = __dp4a(x.z, q.z, d);
            dot[f * GP + g] = __dp4a(x.w, q.w, d);
          }
        }
        const int total = sum16<kSums>(dot);
        float v = float(
            __dmul_rn(__dmul_rn(double(total), double(s)), my_qs));
        if (GP > 1 && mine >= a.G) v = -INFINITY;
#pragma unroll
        for (int o = GP / 2; o > 0; o >>= 1)
          v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (l16 < kSums && mine == 0 && blk < n) {
          if (r == 0)
            score[blk] = v;
          else
            first_store(score + i0 + blk, v);
        }
      }
    }
  }
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
    if (r > 0) return;
  } else {
    __syncthreads();
  }

  // scores become ranking keys, four per thread and step; past the last
  // block lie keys of 0, below every score's
  uint4* key4 = reinterpret_cast<uint4*>(score);
  const int n4 = (nv + 3) / 4;
  // forced blocks are listed whatever they score
  const int first_free = min(a.n_sink, nv);
  const int last_free = max(first_free, nv - min(a.n_recent, nv));
  uint32_t lo = 0xffffffffu, hi = 0u;   // the free keys' range
  for (int i = t; i < n4; i += kSelThreads) {
    const float4 f = reinterpret_cast<const float4*>(score)[i];
    const float v[4] = {f.x, f.y, f.z, f.w};
    uint32_t k[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      k[j] = 4 * i + j < nv ? rank_key(v[j]) : 0u;
      if (4 * i + j >= first_free && 4 * i + j < last_free) {
        lo = min(lo, k[j]);
        hi = max(hi, k[j]);
      }
    }
    key4[i] = make_uint4(k[0], k[1], k[2], k[3]);
  }
  uint32_t bar = 0, quota = 0;    // take keys above bar, quota equal to it
  const bool all = nv <= a.K;
  uint32_t left = uint32_t(max(0, a.K - first_free - (nv - last_free)));
  if (!all && left == 0) bar = 0xffffffffu;
  if (!all && left > 0) {
    // the range's 2048 parts tell the keys apart
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) span[warp] = make_uint2(lo, hi);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      lo = min(lo, span[w].x);
      hi = max(hi, span[w].y);
    }
    // keys in [lo, lo + 2^bits) hold the one that is left-th from the top
    int bits = 32 - __clz(hi - lo);
#pragma unroll 1
    for (int pass = 0; bits > 0; ++pass) {
      const int shift = max(bits - 11, 0);
      const uint32_t parts = 1u << (bits - shift);
      // keys outside the range do not count: those below it wrap around to
      // 2^24 - 2 or more, as no two keys are further apart than 0xff000002,
      // and a range below some of them has 21 bits at most
      for (int i = t; i < n4; i += kSelThreads) {
        const uint4 k = key4[i];
        const uint32_t d[4] = {(k.x - lo) >> shift, (k.y - lo) >> shift,
                               (k.z - lo) >> shift, (k.w - lo) >> shift};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (d[j] < parts && 4 * i + j >= first_free && 4 * i + j < last_free)
            atomicAdd(&hist[pass][d[j]], 1u);
      }
      __syncthreads();
      // a thread counts a run of digits, the largest first
      constexpr int kRun = kSelBins / kSelThreads;
      const uint4* bins = reinterpret_cast<const uint4*>(
          &hist[pass][kSelBins - kRun * (t + 1)]);
      uint32_t c[kRun], mine = 0;
#pragma unroll
      for (int j = 0; j < kRun / 4; ++j) {
        const uint4 x = bins[j];
        c[kRun - 1 - 4 * j] = x.x;
        c[kRun - 2 - 4 * j] = x.y;
        c[kRun - 3 - 4 * j] = x.z;
        c[kRun - 4 - 4 * j] = x.w;
      }
#pragma unroll
      for (int j = 0; j < kRun; ++j) mine += c[j];
      uint32_t before = block_prefix<kSelWarps>(mine, scan);
      if (before < left && left <= before + mine) {
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
          if (before < left && left <= before + c[j]) {
            pick[0] = uint32_t(kSelBins - kRun * t - 1 - j);
            pick[1] = left - before;
          }
          before += c[j];
        }
      }
      __syncthreads();
      lo += pick[0] << shift;
      left = pick[1];
      bits = shift;
      __syncthreads();
    }
    bar = lo;
    quota = left;
  } else {
    __syncthreads();              // the keys are in place
  }

  // The list in ascending order: warp w takes the w-th run of blocks, four
  // per lane, counts its keys above the bar and at it, and places them
  // behind the runs before.
  auto takes = [&](int i, bool (&gt)[4], bool (&eq)[4]) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (i < n4) x = key4[i];
    const uint32_t k[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = 4 * i + j;
      gt[j] = at < nv && (all || at < first_free || at >= last_free ||
                          k[j] > bar);
      eq[j] = at < nv && !gt[j] && k[j] == bar;
    }
  };
  const int run = (n4 + kSelThreads - 1) / kSelThreads * 32;
  const int i_lo = warp * run, i_hi = min(i_lo + run, n4);
  uint32_t above = 0, equal = 0;
  for (int i = i_lo; i < i_hi; i += 32) {
    bool gt[4], eq[4];
    takes(i + lane, gt, eq);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      above += gt[j];
      equal += eq[j];
    }
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) runs[warp] = make_uint2(above, equal);
  __syncthreads();
  uint32_t at = 0, eq_at = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    at += w < warp ? runs[w].x : 0u;
    eq_at += w < warp ? runs[w].y : 0u;
  }
  int32_t* blocks = a.blocks + bh * a.K;
  float* out_s = a.scores + bh * a.K;
  const uint32_t below = (1u << lane) - 1u;
  for (int i = i_lo; i < i_hi; i += 32) {
    bool gt[4], eq[4];
    takes(i + lane, gt, eq);
    uint32_t g0 = at, e0 = eq_at;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t mg = __ballot_sync(0xffffffffu, gt[j]);
      const uint32_t me = __ballot_sync(0xffffffffu, eq[j]);
      g0 += __popc(mg & below);
      e0 += __popc(me & below);
      at += __popc(mg);
      eq_at += __popc(me);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (gt[j] || (eq[j] && e0 < quota)) {
        const uint32_t to = g0 + min(e0, quota);
        blocks[to] = j0 + 4 * (i + lane) + j;
        out_s[to] = key_score(reinterpret_cast<const uint32_t*>(
            score)[4 * (i + lane) + j]);
      }
      g0 += gt[j];
      e0 += eq[j];
    }
  }
  // the rest of a short list
  for (int i = nv + t; i < a.K; i += kSelThreads) {
    blocks[i] = -1;
    out_s[i] = -INFINITY;
  }
}

template <int GP, int Threads>
cudaError_t launch_rows(const Kv8SelectArgs& a, int C, cudaStream_t st) {
  const int nblk = (a.L + kKv8Block - 1) / kKv8Block;
  const int64_t grid = int64_t(a.B) * a.H * C;
  const size_t smem = size_t(nblk + 3) / 4 * 16;
  const cudaError_t e =
      allow_smem<kv8_select_kernel<GP, Threads>, kSelMostSmem>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(Threads);
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
  return cudaLaunchKernelEx(&cfg, kv8_select_kernel<GP, Threads>, a, C);
}

// Few (row, head) pairs: a cluster of large CTAs each, as long as there are
// SMs for all of them at once and more than 64 blocks for each. In turns over
// caches that do not fit L2: 32 pairs of 1M slots 23.6 us over clusters of 4,
// 30 over 2, 33.6 over 8 (two rounds); 8 pairs with 4 query heads each 21.5
// over 8, 29 over 4; 32 pairs of 256 blocks 6.6 over 2, 7.1 in one small CTA
// each; at 129 blocks that is even (6.1 and 5.6 for 8 pairs). More than 512
// blocks of as many pairs as SMs: one large CTA each (128 pairs of 1024 blocks
// 12.6, small ones 19.2). Many pairs, or short rows: one small CTA each, four
// to an SM (512 pairs of 256 blocks 12.8 us, large ones 27).
template <int GP>
cudaError_t launch_group(const Kv8SelectArgs& a, cudaStream_t st) {
  const int nblk = (a.L + kKv8Block - 1) / kKv8Block;
  const int64_t pairs = int64_t(a.B) * a.H;
  const int sms = sm_count();
  int C = 1;
  while (C < kSelMost && pairs * C * 2 <= sms && nblk > 128 * C) C *= 2;
  return C > 1 || (nblk > 512 && pairs <= sms)
             ? launch_rows<GP, 512>(a, C, st)
             : launch_rows<GP, 256>(a, C, st);
}

}  // namespace

cudaError_t launch_kv8_select(const Kv8SelectArgs& a, cudaStream_t st) {
  const cudaError_t e = a.G == 1   ? launch_group<1>(a, st)
                        : a.G == 2 ? launch_group<2>(a, st)
                        : a.G <= 4 ? launch_group<4>(a, st)
                        : a.G <= 8 ? launch_group<8>(a, st)
                                   : launch_group<16>(a, st);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

}  // namespace lwm
