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

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

struct Rows {
  const int32_t* kv_start;
  const int32_t* kv_len;
  const int32_t* q_pos;
  int max_pos, B, L, H, K;
  bool listed;
};

// Tiles are counted in 32 bits (the host refuses a call of more).
struct RowTiles {
  int start, len, t0, n;    // visible slots, first block, tiles per head
  int pos;                  // of the query
};

__device__ __forceinline__ RowTiles row_tiles(const Rows& r, int b) {
  RowTiles x;
  const int len = __ldcg(r.kv_len + b), start = __ldcg(r.kv_start + b);
  const int pos = __ldcg(r.q_pos + b);
  x.len = max(0, min(len, r.L));
  x.start = max(0, min(start, x.len));
  x.pos = max(0, min(pos, r.max_pos - 1));
  x.t0 = x.start / kKv8Block;
  x.n = x.len > x.start
            ? (r.listed ? r.K : (x.len + kKv8Block - 1) / kKv8Block - x.t0)
            : 0;
  return x;
}

// A warp's lanes together: tiles per head of rows [0, upto).
__device__ __forceinline__ int tiles_before(const Rows& r, int upto) {
  int s = 0;
  for (int b = threadIdx.x & 31; b < upto; b += 32) s += row_tiles(r, b).n;
  return __reduce_add_sync(0xffffffffu, s);
}

// CTA c of C takes tiles [first(c), first(c + 1)): the first `more` CTAs
// take one tile more than the others.
struct Shares {
  int each, more;
  __device__ __forceinline__ Shares(int total, int C)
      : each(total / C), more(total - each * C) {}
  __device__ __forceinline__ int first(int c) const {
    return each * c + min(c, more);
  }
  // The CTA that holds tile u.
  __device__ __forceinline__ int holder(int u) const {
    const int cut = (each + 1) * more;
    return u < cut ? u / (each + 1) : more + (u - cut) / each;
  }
};

// Where a CTA starts: its tiles [u0, u1), the row that holds u0 and the
// tiles before that row.
struct Start {
  int u0, u1, b, row_at;
  RowTiles rt;
};

// A warp's lanes together, one row per lane.
__device__ __forceinline__ Start find_start(const Rows& r, int C, int c) {
  const int lane = threadIdx.x & 31;
  RowTiles mine{};
  if (lane < r.B) mine = row_tiles(r, lane);
  int sum = mine.n;
  for (int b = lane + 32; b < r.B; b += 32) sum += row_tiles(r, b).n;
  const Shares sh(__reduce_add_sync(0xffffffffu, sum) * r.H, C);
  Start s;
  s.u0 = sh.first(c);
  s.u1 = sh.first(c + 1);
  s.b = s.row_at = 0;
  if (s.u0 >= s.u1) return s;
  int base = 0;
  for (int b0 = 0; b0 < r.B; b0 += 32) {
    if (b0 > 0) {
      mine.n = 0;
      if (b0 + lane < r.B) mine = row_tiles(r, b0 + lane);
    }
    const int n = mine.n * r.H;
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, s.u0 < base + inc);
    if (hit) {
      const int f = __ffs(hit) - 1;
      s.b = b0 + f;
      s.row_at = base + __shfl_sync(0xffffffffu, inc - n, f);
      s.rt.start = __shfl_sync(0xffffffffu, mine.start, f);
      s.rt.len = __shfl_sync(0xffffffffu, mine.len, f);
      s.rt.t0 = __shfl_sync(0xffffffffu, mine.t0, f);
      s.rt.n = __shfl_sync(0xffffffffu, mine.n, f);
      s.rt.pos = __shfl_sync(0xffffffffu, mine.pos, f);
      return s;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  s.u1 = s.u0;   // lengths that change during the call: no work, no fault
  return s;
}

// Partial result records: m[G], l[G], padding to 16 bytes, acc[G][128].
__host__ __device__ constexpr int part_acc(int G) { return (2 * G + 3) & ~3; }
__host__ __device__ constexpr int part_stride(int G) {
  return part_acc(G) + G * kHeadDim;
}

// ---------------------------------------------------------------- kernel
//
// Both products run on the tensor cores straight on the codes, so no code
// is ever converted on the CUDA cores:
//   S[128 slots][n] = K tile (A, K-major)      . Q  (B: n rows of 128 codes)
//   O[128 dims][n]  = V tile (A, read MN-major) . P  (B: n rows of 128 codes)
// Q and P become codes of the cache's type: a number is the sum of a few
// codes (terms), each carrying what the ones before it left, and each term
// of each head is one column n; products of codes are exact and the columns
// are added up in fp32. e4m3: terms 1/16 apart, 5 for q (2^-20 of a channel,
// or 2^-34 of the largest), 4 for p (2^-16 of a weight at most, 2^-21 on
// average, or 2^-30 of the largest). int8: terms 1/254 apart, 3 for q (2^-22
// of the largest channel) and 3 for p (2^-24 of the largest weight). Weights
// are taken against the tile's own maximum, so what the terms cannot hold is
// small against the tile's own sum, however far the running maximum lies
// above it. With these terms out is off by less than fp32 sums in another
// order are (2-norm of 2048 slots, before rounding: 3e-7); three terms for
// an e4m3 weight left 1.4e-5, which turned roundings of out to bf16.
//
// Softmax warps: four per group of at most 8 heads; thread t of a group is
// slot t of S (scores, maximum, weights) and channel t of O (accumulator).
// The warp after them issues the products, the last one walks the tiles and
// loads them by TMA. The products of one tile run while the softmax works
// on the next: S, P and, up to 8 heads, O are double buffered.
//
// Bound by HBM (256 bytes per slot and cache head) up to 8 query heads per
// cache head: a 1M-slot cache of 32 heads in 1.17 ms call after call (7.3
// TB/s; 1.24 in turns over three caches), 16 rows x 32K x 8 heads in 158 to
// 161 us with 1 to 4 query heads each (6.7 TB/s) and 172 to 174 with 8 (6.2);
// with 16 the softmax warps' instructions bound it (665 a warp and tile; 246
// to 260 us, int8 250 to 257; an e4m3 weight of three terms, one fewer than
// now, 626 and 240). A kernel that decoded the codes on the CUDA cores took
// 18.8 ms for the 1M-slot cache. What a call costs beside
// the traffic is about 7 us: the walk to the first tile and its query (5 us
// to the first scores), the last tile's product, and joining the parts (2).
constexpr int kDecRing = 8;              // tile descriptions
constexpr int kDecPerSm = 2;             // CTAs
constexpr uint64_t kDecWaitNs = 4000000000ull;
constexpr int kTile = kKv8Block * kHeadDim;   // bytes of K or V of one tile

enum : int {
  kFirst = 1,     // first tile of its (row, head) in this CTA
  kLast = 2,
  kWhole = 4,     // the CTA holds every tile of the (row, head)
  kSlot1 = 8,     // partial result goes to the CTA's second record
  kEnd = 16,      // no tile: the CTA's work is done
};
struct __align__(8) Tile {
  int b, h, blk, flags;
  int lo, hi;     // visible slots of the block (lo >= hi: nothing to read)
  int pos, pad;   // of the query
};

template <bool kInt8, int GP>
struct Dec {
  static constexpr int kGroups = GP > 8 ? 2 : 1;        // of softmax warps
  static constexpr int kHeads = GP / kGroups;           // per group
  static constexpr int kThreads = 128 * kGroups + 64;
  static constexpr int kPerSm = kDecPerSm;
  static constexpr int kQTerms = kInt8 ? 3 : 5;
  static constexpr int kPTerms = kInt8 ? 3 : 4;
  static constexpr int kNq = (kQTerms * GP + 15) / 16 * 16;
  static constexpr int kNp = (kPTerms * GP + 15) / 16 * 16;
  // O is double buffered where the columns allow: 16 heads of e4m3 have one,
  // which is read before the next tile's weights are handed over
  static constexpr int kOBufs = 2 * kNq + 2 * kNp <= 256 ? 2 : 1;
  static constexpr int kCols = 2 * kNq + kOBufs * kNp;
  static constexpr int kTmem = kCols <= 64 ? 64 : kCols <= 128 ? 128 : 256;
  static_assert(kCols <= 256, "CTAs share the SM's 512 columns");
  // factor of the first term
  static constexpr float kPScale = kInt8 ? 127.f : 256.f;
  static constexpr int kQExp = kInt8 ? 6 : 8;  // |q~| 2^(kQExp - e) < 2^kQExp
  // shared memory, from a 1024-byte boundary
  static constexpr int kQBytes = kNq * kHeadDim;
  static constexpr int kPBytes = kNp * kKv8Block;
  static constexpr int kStats = 4 * kHeads;  // floats: see stats below
  static constexpr int kSmall = kQBytes + 2 * kPBytes + 448 +
                                (2 * 4 + 2 + 4) * GP * 4 +
                                kGroups * 8 * kStats * 4;
  // as many tiles as the CTA's part of 227 KB holds, V with the odd one.
  // With three stages, a K tile is refilled together with its V tile: the
  // two then load side by side, 7.4 TB/s from a 1M-token cache, where
  // refilling it as soon as its scores are done gave 7.1. With fewer, the
  // earlier refill wins (16 heads, 16 x 32K, weights of three terms: 233
  // against 264 us).
  static constexpr int kRoom = 233472 / kPerSm - 2048 - kSmall;
  static constexpr int kTiles = kRoom / kTile < 6 ? kRoom / kTile : 6;
  static constexpr int kKStages = kTiles / 2, kVStages = kTiles - kKStages;
  static constexpr bool kEarlyK = kKStages < 3;
  static_assert(kKStages >= 2, "the next tile loads while one is worked on");
  static constexpr int kV = kKStages * kTile;
  static constexpr int kQ = kTiles * kTile;
  static constexpr int kP = kQ + kQBytes;
  static constexpr int kRingAt = kP + 2 * kPBytes;
  static constexpr int kMaxAt = kRingAt + kDecRing * int(sizeof(Tile));
  static constexpr int kQsAt = kMaxAt + 2 * 4 * GP * 4;
  static constexpr int kSumAt = kQsAt + 2 * GP * 4;
  static constexpr int kStatsAt = (kSumAt + 4 * GP * 4 + 15) / 16 * 16;
  static constexpr int kBars = kStatsAt + kGroups * 4 * 2 * kStats * 4;
  static constexpr int bKFull = 0, bKEmpty = kKStages, bVFull = 2 * kKStages,
                       bVEmpty = bVFull + kVStages,
                       bTok = bVEmpty + kVStages,
                       bS = bTok + kDecRing, bP = bS + 2, bO = bP + 2,
                       bQ = bO + 2, bDone = bQ + 2, kNumBars = bDone + 1;
  static constexpr int kTail = kBars + kNumBars * 8;  // tmem base, abort word
  static constexpr int kSmem = kTail + 16 + 1024;
  static_assert(kPerSm * (kSmem + 1024) <= 233472, "shared memory per SM");
  static_assert(kVStages + 2 < kDecRing, "descriptions outlive their tiles");
};

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t* r) {
  static_assert(N == 1 || N == 2 || N == 4 || N == 8, "columns");
  if constexpr (N == 1) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];"
                 : "=r"(r[0]) : "r"(at));
  } else if constexpr (N == 2) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1]) : "r"(at));
  } else if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, "
        "[%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
          "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(at));
  }
}

// N floats that every thread of a warp reads.
template <int N>
__device__ __forceinline__ void lds(const float* p, float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + i);
      v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = p[i];
  }
}

// One 32-code step of a product: D[tmem] (+)= A . B^T.
template <bool kInt8>
__device__ __forceinline__ void mma8(uint32_t d, uint64_t a, uint64_t b,
                                     uint32_t idesc, uint32_t accumulate) {
  if constexpr (kInt8) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// Instruction descriptor, M = 128: e4m3 x e4m3 -> f32, or s8 x s8 -> s32;
// a_mn: A is MN-major. Fields as in idesc_bf16.
template <bool kInt8>
__device__ constexpr uint32_t idesc8(int N, int a_mn) {
  return (kInt8 ? (2u << 4) | (1u << 7) | (1u << 10) : (1u << 4)) |
         (uint32_t(a_mn) << 15) | (uint32_t(N >> 3) << 17) | (8u << 24);
}

// Factor from one term to the next.
template <bool kInt8>
constexpr float kStepOf = kInt8 ? 254.f : 16.f;

template <bool kInt8>
__device__ __forceinline__ float term_value(uint32_t w) {
  return kInt8 ? float(int(w)) : __uint_as_float(w);
}

// x += y, x *= y and x += y z of N numbers, two at a time where there are
// two.
template <int N>
__device__ __forceinline__ void add_all(float (&x)[N], const float (&y)[N]) {
  if constexpr (N == 1) x[0] += y[0];
#pragma unroll
  for (int g = 0; g + 1 < N; g += 2) {
    const float2 v = add2(make_float2(x[g], x[g + 1]),
                          make_float2(y[g], y[g + 1]));
    x[g] = v.x;
    x[g + 1] = v.y;
  }
}
template <int N>
__device__ __forceinline__ void mul_all(float (&x)[N], const float (&y)[N]) {
  if constexpr (N == 1) x[0] *= y[0];
#pragma unroll
  for (int g = 0; g + 1 < N; g += 2) {
    const float2 v = mul2(make_float2(x[g], x[g + 1]),
                          make_float2(y[g], y[g + 1]));
    x[g] = v.x;
    x[g + 1] = v.y;
  }
}
template <int N>
__device__ __forceinline__ void mul_all(float (&x)[N], float y) {
  float all[N];
#pragma unroll
  for (int g = 0; g < N; ++g) all[g] = y;
  mul_all(x, all);
}
template <int N>
__device__ __forceinline__ void fma_all(float (&x)[N], const float (&y)[N],
                                        const float (&z)[N]) {
  if constexpr (N == 1) x[0] = fmaf(y[0], z[0], x[0]);
#pragma unroll
  for (int g = 0; g + 1 < N; g += 2) {
    const float2 v = fma2(make_float2(y[g], y[g + 1]),
                          make_float2(z[g], z[g + 1]),
                          make_float2(x[g], x[g + 1]));
    x[g] = v.x;
    x[g + 1] = v.y;
  }
}

// The numbers whose terms are r[0..N)[g], two at a time where there are two.
template <bool kInt8, int N, int GH>
__device__ __forceinline__ void join_terms(const uint32_t (&r)[N][GH],
                                           float (&x)[GH]) {
  constexpr float kDown = 1.f / kStepOf<kInt8>;
#pragma unroll
  for (int g = 0; g < GH; g += 2) {
    if constexpr (GH > 1) {
      float2 v = make_float2(term_value<kInt8>(r[N - 1][g]),
                             term_value<kInt8>(r[N - 1][g + 1]));
#pragma unroll
      for (int n = N - 2; n >= 0; --n)
        v = fma2(v, make_float2(kDown, kDown),
                 make_float2(term_value<kInt8>(r[n][g]),
                             term_value<kInt8>(r[n][g + 1])));
      x[g] = v.x;
      x[g + 1] = v.y;
    } else {
      x[0] = term_value<kInt8>(r[N - 1][0]);
#pragma unroll
      for (int n = N - 2; n >= 0; --n)
        x[0] = fmaf(x[0], kDown, term_value<kInt8>(r[n][0]));
    }
  }
}

// Barrier of a group of softmax warps; true if all its threads said so.
__device__ __forceinline__ bool softmax_all(int id, bool mine) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
      "bar.red.and.pred p, %1, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(uint32_t(mine))
      : "memory");
  return all != 0;
}

// The next term of (a, b): its two codes, and what they leave, scaled up.
template <bool kInt8>
__device__ __forceinline__ uint32_t next_term(float& a, float& b) {
  constexpr float kStep = kStepOf<kInt8>;
  if constexpr (kInt8) {
    const float ra = rintf(a), rb = rintf(b);
    const uint32_t w = uint32_t(int(ra) & 255) | (uint32_t(int(rb) & 255) << 8);
    a = (a - ra) * kStep;
    b = (b - rb) * kStep;
    return w;
  } else {
    const uint32_t w = enc2_e4m3(a, b);
    const float2 f = dec2_e4m3(w);
    // (x - f) 16, exact: f 16 and the difference are
    const float2 r = fma2(make_float2(a, b), make_float2(kStep, kStep),
                          make_float2(f.x * -kStep, f.y * -kStep));
    a = r.x;
    b = r.y;
    return w;
  }
}

// Stores a code to (Row + h0, t) of a K-major operand of 128-byte rows,
// 128-byte swizzle (16-byte column c of row r lies at c ^ (r & 7)); h0 is 0
// or a multiple of 8, at the address of (h0, t), so that the others are an
// exclusive or and a constant away. (Worked out for each code, 24 addresses
// took 150 of a thread's 850 instructions per tile.)
template <int Row>
__device__ __forceinline__ void st_code(uint32_t at, uint32_t code) {
  asm volatile("st.shared.u8 [%0+%2], %1;" ::"r"(at ^ ((Row & 7) << 4)),
               "r"(code), "n"((Row >> 3) * 1024 + (Row & 7) * 128)
               : "memory");
}

// The terms of y[0..GH), heads h0 .. of GP, to rows n GP + h0 .. of an
// operand.
template <bool kInt8, int GP, int Terms, int GH, int N = 0, int G = 0>
__device__ __forceinline__ void st_terms(uint32_t at, float (&y)[GH]) {
  if constexpr (N < Terms) {
    float none = 0.f;
    constexpr bool kTwo = G + 1 < GH;
    const uint32_t w = next_term<kInt8>(y[G], kTwo ? y[(G + 1) % GH] : none);
    st_code<N * GP + G>(at, w);
    if constexpr (kTwo) st_code<N * GP + G + 1>(at, w >> 8);
    constexpr bool kDone = G + 2 >= GH;
    st_terms<kInt8, GP, Terms, GH, kDone ? N + 1 : N, kDone ? 0 : G + 2>(at, y);
  }
}

// Walks the CTA's tiles: every readable one, and one empty tile for a
// (row, head) whose list holds none.
struct Walker {
  Rows rows;
  const int32_t* blocks;
  int u, u0, u1, row_at, b;
  RowTiles rt;
  // current (row, head): tiles [j, je) are left
  int h, j, je, seg_flags;
  bool emitted;
  // of a listed call: entry j of the list, fetched ahead, and the one before
  const int32_t* list;
  int entry, left;

  __device__ __forceinline__ void open() {   // at tile u < u1
    while (u >= row_at + rt.n * rows.H) {
      row_at += rt.n * rows.H;
      if (++b >= rows.B) {     // as in find_start
        u = u1;
        return;
      }
      rt = row_tiles(rows, b);
    }
    h = (u - row_at) / rt.n;
    const int p0 = row_at + h * rt.n, p1 = p0 + rt.n;
    j = u - p0;
    je = min(u1, p1) - p0;
    seg_flags = (p0 >= u0 && p1 <= u1 ? kWhole : 0) | (p0 < u0 ? 0 : kSlot1);
    emitted = false;
    u += je - j;
    if (rows.listed) {
      list = blocks + (int64_t(b) * rows.H + h) * rows.K;
      entry = ld_now(list + j);
      left = j > 0 ? ld_now(list + j - 1) : -1;
    }
  }
  // False at the end of the CTA's share.
  __device__ __forceinline__ bool next(Tile& t) {
    for (;;) {
      if (j >= je) {
        if (!emitted && je >= 0) {            // nothing readable: one empty
          emitted = true;
          t.b = b; t.h = h; t.blk = 0; t.lo = t.hi = 0;
          t.flags = seg_flags | kFirst;
          t.pos = rt.pos;
          return true;
        }
        if (u >= u1) return false;
        open();
        continue;
      }
      int blk = rt.t0 + j;
      bool ok = true;
      if (rows.listed) {
        blk = entry;
        if (j + 1 < je) entry = ld_now(list + j + 1);
        ok = blk >= rt.t0 && int64_t(blk) * kKv8Block < rt.len && blk > left;
        left = blk;
      }
      ++j;
      if (!ok) continue;
      t.b = b; t.h = h; t.blk = blk;
      t.lo = max(0, rt.start - blk * kKv8Block);
      t.hi = min(kKv8Block, rt.len - blk * kKv8Block);
      t.flags = seg_flags | (emitted ? 0 : kFirst);
      t.pos = rt.pos;
      emitted = true;
      return true;
    }
  }
};

template <bool kInt8, int GP>
__global__ void __launch_bounds__(Dec<kInt8, GP>::kThreads,
                                  Dec<kInt8, GP>::kPerSm)
kv8_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ Kv8DecodeArgs a) {
  using C = Dec<kInt8, GP>;
  extern __shared__ uint8_t dsmem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(dsmem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  Tile* ring = reinterpret_cast<Tile*>(smem + C::kRingAt);
  float* wmax = reinterpret_cast<float*>(smem + C::kMaxAt);   // [2][4][GP]
  float* qscale = reinterpret_cast<float*>(smem + C::kQsAt);  // [2][GP]
  float* wsum = reinterpret_cast<float*>(smem + C::kSumAt);   // [4][GP]
  float* stats = reinterpret_cast<float*>(smem + C::kStatsAt);
  volatile int* abort_word =
      reinterpret_cast<volatile int*>(smem + C::kTail + 4);
  auto bar = [&](int i) { return sbase + C::kBars + 8u * i; };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kMmaWarp = 4 * C::kGroups, kLoadWarp = kMmaWarp + 1;

  // set up while the kernel before this one may still run
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i) {
      const bool by_warps = i >= C::bP && i < C::bP + 2;
      const bool by_warps_q = i >= C::bQ && i < C::bQ + 2;
      mbar_init(bar(i), by_warps || by_warps_q ? 4 * C::kGroups : 1);
    }
    fence_mbar_init();
    *abort_word = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(sbase + C::kTail, C::kTmem);
    tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<uint32_t*>(smem + C::kTail);
  pdl_wait();
  pdl_trigger();
  auto wait = [&](int i, int phase) {
    return mbar_wait(bar(i), phase & 1, abort_word, a.status, kDecWaitNs);
  };
  const int nblk = (a.L + kKv8Block - 1) / kKv8Block;

  if (warp == kLoadWarp) {
    // ------------------------------------------------------ tiles and TMA
    Walker w;
    w.rows = Rows{a.kv_start, a.kv_len, a.q_pos, a.max_pos,
                  a.B, a.L, a.H, a.K, a.listed};
    w.blocks = a.blocks;
    const Start st = find_start(w.rows, gridDim.x, blockIdx.x);
    w.u0 = w.u = st.u0;
    w.u1 = st.u1;
    w.b = st.b;
    w.row_at = st.row_at;
    w.rt = st.rt;
    w.j = 0;
    w.je = -1;
    w.emitted = true;
    if (lane == 0) {
      auto load = [&](const CUtensorMap* map, int full, uint32_t at,
                      const Tile& x) {
        if (x.lo < x.hi) {
          mbar_arrive_expect_tx(bar(full), kTile);
          tma_load_3d(at, map, bar(full), 0, x.blk * kKv8Block,
                      x.b * a.H + x.h);
        } else {
          mbar_arrive(bar(full));
        }
      };
      auto load_v = [&](int i, const Tile& x) {
        const int s = i % C::kVStages;
        if (i >= C::kVStages && !wait(C::bVEmpty + s, i / C::kVStages - 1))
          return false;
        load(&tm_v, C::bVFull + s, sbase + C::kV + s * kTile, x);
        return true;
      };
      Tile cur, nxt;
      bool more = w.next(cur), ok = true;
      int i = 0, nv = 0;
      for (; more && ok; ++i) {
        more = w.next(nxt);
        if (!more || (nxt.flags & kFirst)) cur.flags |= kLast;
        const int s = i % C::kKStages;
        // the first query's loads go before the flood of all CTAs' first
        // tiles, in which they took 7 us instead of 1
        if (i == 1) ok = wait(C::bQ, 0);
        if (i >= C::kKStages)
          ok = ok && wait(C::bKEmpty + s, i / C::kKStages - 1);
        if (!ok) break;
        load(&tm_k, C::bKFull + s, sbase + s * kTile, cur);
        ring[i % kDecRing] = cur;
        mbar_arrive(bar(C::bTok + i % kDecRing));
        ok = load_v(i, cur);
        nv += ok;
        cur = nxt;
      }
      if (ok) {
        ring[i % kDecRing].flags = kEnd;
        mbar_arrive(bar(C::bTok + i % kDecRing));
      }
      // no load is in flight when the CTA leaves, abandoned or not
      for (int f = max(0, i - C::kKStages); f < i; ++f)
        mbar_wait(bar(C::bKFull + f % C::kKStages), (f / C::kKStages) & 1,
                  nullptr, a.status, kDecWaitNs);
      for (int f = max(0, nv - C::kVStages); f < nv; ++f)
        mbar_wait(bar(C::bVFull + f % C::kVStages), (f / C::kVStages) & 1,
                  nullptr, a.status, kDecWaitNs);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      constexpr uint32_t idq = idesc8<kInt8>(C::kNq, 0);
      constexpr uint32_t idp = idesc8<kInt8>(C::kNp, 1);
      int seg = -1;
      // scores of tile i
      auto qk = [&](int i) {
        if (!wait(C::bTok + i % kDecRing, i / kDecRing)) return 2;
        const int flags = ring[i % kDecRing].flags;
        if (flags & kEnd) return 1;
        const bool live = ring[i % kDecRing].lo < ring[i % kDecRing].hi;
        const int s = i % C::kKStages;
        if (flags & kFirst) {
          ++seg;
          if (!wait(C::bQ + (seg & 1), seg >> 1)) return 2;
        }
        if (!wait(C::bKFull + s, i / C::kKStages)) return 2;
        tc_fence_after();
        if (live) {
          const uint64_t kd = sdesc_sw128(sbase + s * kTile, 16, 1024);
          const uint64_t qd =
              sdesc_sw128(sbase + C::kQ, 16, 1024);
#pragma unroll
          for (int k = 0; k < kHeadDim / 32; ++k)
            mma8<kInt8>(tmem + (i & 1) * C::kNq, kd + 2 * k, qd + 2 * k, idq,
                        k > 0);
        }
        if (C::kEarlyK) mma_commit(bar(C::bKEmpty + s));
        mma_commit(bar(C::bS + (i & 1)));
        return 0;
      };
      // weights times values of tile i
      auto pv = [&](int i) {
        const int s = i % C::kVStages;
        if (!wait(C::bP + (i & 1), i >> 1) ||
            !wait(C::bVFull + s, i / C::kVStages))
          return false;
        tc_fence_after();
        if (ring[i % kDecRing].lo < ring[i % kDecRing].hi) {
          const uint64_t vd =
              sdesc_sw128(sbase + C::kV + s * kTile, kTile, 1024);
          const uint64_t pd =
              sdesc_sw128(sbase + C::kP + (i & 1) * C::kPBytes, 16, 1024);
#pragma unroll
          for (int k = 0; k < kKv8Block / 32; ++k)
            mma8<kInt8>(tmem + 2 * C::kNq + i % C::kOBufs * C::kNp,
                        vd + uint64_t(k * (32 * kHeadDim >> 4)), pd + 2 * k,
                        idp, k > 0);
        }
        if (!C::kEarlyK) mma_commit(bar(C::bKEmpty + i % C::kKStages));
        mma_commit(bar(C::bVEmpty + s));
        mma_commit(bar(C::bO + (i & 1)));
        return true;
      };
      int state = qk(0);
      for (int i = 0; state == 0; ++i) {
        // the next tile's scores go first, unless they wait for a query
        // that the softmax makes after this tile's weights
        const bool last = ring[i % kDecRing].flags & kLast;
        if (!last && (state = qk(i + 1)) == 2) break;
        if (!pv(i)) break;
        if (last) state = qk(i + 1);
      }
      // no product is running when the CTA leaves
      mma_commit(bar(C::bDone));
      mbar_wait(bar(C::bDone), 0, nullptr, a.status, kDecWaitNs);
    }
  } else {
    // ------------------------------------------------------------- softmax
    constexpr int GH = C::kHeads;         // this group's heads: h0 + g
    const int t = threadIdx.x & 127, quad = warp & 3;
    const int group = C::kGroups == 1 ? 0 : warp >> 2;
    const int h0 = group * GH, sync_id = 1 + group;
    const uint32_t my_tmem = tmem + (uint32_t(quad * 32) << 16) + h0;
    int seg = -1;
    // Query of a (row, head), thread t channel t: its two members of the
    // rotation and their angle are fetched ahead of the tile that needs
    // them, ...
    uint32_t q_raw[GH];
    float2 q_cs;
    const bool low = a.half ? t < 64 : (t & 1) == 0;
    auto fetch_q = [&](const Tile& x) {
      const int k = a.half ? (t & 63) : (t >> 1);
      q_cs = ld_now(reinterpret_cast<const float2*>(a.table) +
                   int64_t(x.pos) * (kHeadDim / 2) + k);
      const uint16_t* q = static_cast<const uint16_t*>(a.q) +
                          ((int64_t(x.b) * a.H + x.h) * a.G + h0) * kHeadDim;
#pragma unroll
      for (int g = 0; g < GH; ++g) {
        q_raw[g] = 0;
        if (h0 + g >= a.G) continue;
        const uint16_t* row = q + g * kHeadDim;
        q_raw[g] =
            a.half ? ld_now(row + k) | (uint32_t(ld_now(row + k + 64)) << 16)
                   : ld_now(reinterpret_cast<const uint32_t*>(row) + k);
      }
    };
    // ... then rotated and split into terms. Called when the scores of the
    // (row, head) before are all done, so that the terms may overwrite its
    // own; buf: which of two sets of scales.
    auto make_q = [&](int buf) {
      float x[GH];
#pragma unroll
      for (int g = 0; g < GH; ++g) {
        const float qa = bf16lo_to_f32(q_raw[g]), qb = bf16hi_to_f32(q_raw[g]);
        x[g] = low ? qa * q_cs.x - qb * q_cs.y : qa * q_cs.y + qb * q_cs.x;
      }
      float big[GH];
#pragma unroll
      for (int g = 0; g < GH; ++g) {
        // a NaN or an infinity counts as the largest magnitude
        const float m = fabsf(x[g]);
        big[g] = warp_max(m <= 3.402823466e38f ? m : INFINITY);
      }
      if (lane == 0)
#pragma unroll
        for (int g = 0; g < GH; ++g) wsum[quad * GP + h0 + g] = big[g];
      named_barrier_sync(sync_id, 128);
      float y[GH];
#pragma unroll
      for (int g = 0; g < GH; ++g) {
        const float* w = wsum + h0 + g;
        const float m = fmaxf(fmaxf(w[0], w[GP]),
                              fmaxf(w[2 * GP], w[3 * GP]));
        const bool fine = m <= 3.402823466e38f;
        // m < 2^e; the factor 2^k is exact, and so are its products
        const int e = int(__float_as_uint(m) >> 23) - 126;
        const int k = min(C::kQExp - e, 126);
        y[g] = fine ? x[g] * __uint_as_float(uint32_t(127 + k) << 23) : 0.f;
        if (t == 0)
          qscale[buf * GP + h0 + g] =
              fine ? kLog2e / sqrtf(float(kHeadDim)) *
                         __uint_as_float(uint32_t(127 - k) << 23)
                   : __int_as_float(0x7fffffff);
      }
      st_terms<kInt8, GP, C::kQTerms>(sbase + C::kQ + h0 * kHeadDim + t, y);
      fence_proxy_async_smem();
      // all of wsum has been read and qscale written before anyone goes on
      named_barrier_sync(sync_id, 128);
      if (lane == 0) mbar_arrive(bar(C::bQ + buf));
    };

    float l[GH], acc[GH];
    // Lane g (mod GH) of every warp follows head h0 + g: its running maximum m
    // and, per tile, what all threads need of it, passed on through the
    // warp's own stats [tile parity][4][GH]: the tile's maximum, the factors
    // of the sums so far and of the tile's, and the tile's for the values.
    const int my_head = lane & (GH - 1);
    float m = -INFINITY;
    auto stats_of = [&](int i) {
      return stats + (warp * 2 + (i & 1)) * C::kStats;
    };
    bool pending = false;
    // a wait that gave up is agreed on at the next barrier of these warps,
    // so that none is left at a barrier alone
    bool ok = wait(C::bTok, 0);
    bool go = softmax_all(sync_id, ok);
    Tile cur = ring[0];
    // scales of a tile, fetched while the tile before it is worked on
    float ks = 0.f, vs = 0.f, ks_next = 0.f, vs_next = 0.f;
    auto fetch = [&](const Tile& x) {
      if (x.lo >= x.hi) return;
      const int64_t i = (int64_t(x.b) * a.H + x.h) * nblk + x.blk;
      ks_next = ld_now(a.k_scale + i);
      vs_next = ld_now(a.v_scale + i);
    };
    if (go && !(cur.flags & kEnd)) {
      fetch_q(cur);
      fetch(cur);
      make_q(0);
      seg = 0;
    }
    // adds the product of tile i, whose weights were scaled by alpha, beta
    auto add_o = [&](int i, bool live) {
      ok = wait(C::bO + (i & 1), i >> 1) && ok;
      if (!live) return;
      tc_fence_after();
      uint32_t r[C::kPTerms][GH];
      const uint32_t at = my_tmem + 2 * C::kNq + i % C::kOBufs * C::kNp;
#pragma unroll
      for (int n = 0; n < C::kPTerms; ++n) tmem_ld<GH>(at + n * GP, r[n]);
      float al[GH], be[GH];
      lds<GH>(stats_of(i) + GH, al);
      lds<GH>(stats_of(i) + 3 * GH, be);
      tmem_wait_ld();
      float o[GH];
      join_terms<kInt8>(r, o);
      mul_all(acc, al);
      fma_all(acc, o, be);
      tc_fence_before();
    };

    for (int i = 0; go && !(cur.flags & kEnd); ++i) {
      const bool live = cur.lo < cur.hi;
      ok = wait(C::bTok + (i + 1) % kDecRing, (i + 1) / kDecRing) && ok;
      const Tile nxt = ring[(i + 1) % kDecRing];
      ks = ks_next;
      vs = vs_next;
      const bool new_q = !(nxt.flags & kEnd) && (nxt.flags & kFirst);
      // (two groups of warps leave too few registers to hold it so long)
      if (C::kGroups == 1 && ok && new_q) fetch_q(nxt);
      if (ok && !(nxt.flags & kEnd)) fetch(nxt);
      if (cur.flags & kFirst) {
        m = -INFINITY;
#pragma unroll
        for (int g = 0; g < GH; ++g) {
          l[g] = 0.f;
          acc[g] = 0.f;
        }
      }
      ok = wait(C::bS + (i & 1), i >> 1) && ok;
      tc_fence_after();
      if (!live) {
        go = softmax_all(sync_id, ok);
        if (!go) break;
      }
      if (live) {
        float s[GH];
        {
          const uint32_t at = my_tmem + (i & 1) * C::kNq;
          uint32_t r[C::kQTerms][GH];
#pragma unroll
          for (int n = 0; n < C::kQTerms; ++n) tmem_ld<GH>(at + n * GP, r[n]);
          float qs[GH];
          lds<GH>(qscale + (seg & 1) * GP + h0, qs);
          tmem_wait_ld();
          tc_fence_before();
          const bool seen = t >= cur.lo && t < cur.hi;
          join_terms<kInt8>(r, s);
          mul_all(qs, ks);
          mul_all(s, qs);
#pragma unroll
          for (int g = 0; g < GH; ++g) s[g] = seen ? s[g] : -INFINITY;
        }
        float* wm = wmax + (i & 1) * 4 * GP + h0;
        float mx = 0.f;
#pragma unroll
        for (int g = 0; g < GH; ++g) {
          const float x = warp_max(s[g]);
          mx = my_head == g ? x : mx;
        }
        if (lane < GH) wm[quad * GP + lane] = mx;
        go = softmax_all(sync_id, ok);
        if (!go) break;
        {
          const float mt = fmaxf(fmaxf(wm[my_head], wm[GP + my_head]),
                                 fmaxf(wm[2 * GP + my_head],
                                       wm[3 * GP + my_head]));
          const float mn = fmaxf(m, mt);
          const float mu = mn == -INFINITY ? 0.f : mn;
          const float al = ex2(m - mu), be = ex2(mt - mu);
          m = mn;
          if (lane < GH) {
            float* st = stats_of(i) + lane;
            st[0] = mt == -INFINITY ? 0.f : -mt;
            st[GH] = al;
            st[2 * GH] = be;
            st[3 * GH] = be * (vs * (1.f / C::kPScale));
          }
          __syncwarp();
        }
        float p[GH];
        {
          float mt[GH], al[GH], be[GH];
          lds<GH>(stats_of(i), mt);
          lds<GH>(stats_of(i) + GH, al);
          lds<GH>(stats_of(i) + 2 * GH, be);
          add_all(s, mt);
#pragma unroll
          for (int g = 0; g < GH; ++g) p[g] = ex2(s[g]);
          mul_all(l, al);
          fma_all(l, p, be);
          mul_all(p, C::kPScale);
        }
        st_terms<kInt8, GP, C::kPTerms>(
            sbase + C::kP + (i & 1) * C::kPBytes + h0 * kKv8Block + t, p);
        if (!kInt8 && group == 0 && (t < cur.lo || t >= cur.hi)) {
          // an unseen slot's weight is 0, but its codes may be NaN
          ok = wait(C::bVFull + i % C::kVStages, i / C::kVStages) && ok;
          uint4* row = reinterpret_cast<uint4*>(
              smem + C::kV + (i % C::kVStages) * kTile + t * kHeadDim);
#pragma unroll
          for (int k = 0; k < kHeadDim / 16; ++k)
            row[k] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      // the product of the tile before ran meanwhile; where there is one O,
      // it is read before these weights let the next product write it
      if (C::kOBufs == 1 && pending) add_o(i - 1, true);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::bP + (i & 1)));
      // the next (row, head)'s query
      if (new_q) {
        if (C::kGroups > 1) fetch_q(nxt);
        make_q((seg + 1) & 1);
      }
      if (C::kOBufs == 2 && pending) add_o(i - 1, true);
      pending = live;
      if (cur.flags & kLast) {
        add_o(i, live);
        pending = false;
#pragma unroll
        for (int g = 0; g < GH; ++g) {
          float x = l[g];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
            x += __shfl_xor_sync(0xffffffffu, x, o);
          if (lane == 0) wsum[quad * GP + h0 + g] = x;
        }
        named_barrier_sync(sync_id, 128);
        const int64_t o0 = (int64_t(cur.b) * a.H + cur.h) * a.G;
        float* rec = a.part + (int64_t(blockIdx.x) * 2 +
                               ((cur.flags & kSlot1) ? 1 : 0)) *
                                  part_stride(a.G);
#pragma unroll
        for (int g = 0; g < GH; ++g) {
          const int hq = h0 + g;
          if (hq >= a.G) break;
          const float* w = wsum + hq;
          const float lt = (w[0] + w[GP]) + (w[2 * GP] + w[3 * GP]);
          if (cur.flags & kWhole) {
            static_cast<__nv_bfloat16*>(a.out)[(o0 + hq) * kHeadDim + t] =
                __float2bfloat16_rn(lt == 0.f ? 0.f : acc[g] / lt);
            if (t == g)
              a.lse[o0 + hq] = lt == 0.f ? -INFINITY : (m + log2f(lt)) * kLn2;
          } else {
            rec[part_acc(a.G) + hq * kHeadDim + t] = acc[g];
            if (t == g) {
              rec[hq] = m;
              rec[a.G + hq] = lt;
            }
          }
        }
        named_barrier_sync(sync_id, 128);   // wsum is free again
        ++seg;
      }
      cur = nxt;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// One CTA per (row, query head): joins the parts of a (row, cache head) that
// more than one CTA of the decode kernel worked on, and writes (0, -inf) for
// a row that sees nothing. A pass takes up to 64 parts: their maxima and
// sums by one thread each, their accumulators by eight groups of 32 lanes
// (four channels per lane), every group an eighth of the parts.
// Which parts they are follows from the rows' lengths, which are read before
// pdl_wait(), while the last tiles are worked on: every CTA of the decode
// kernel has waited for the work before it when it lets this kernel begin,
// so they are final then, in L2, where row_tiles() reads them.
constexpr int kJoinThreads = 256;
constexpr int kJoinGroups = kJoinThreads / 32;
constexpr int kJoinParts = 64;

__global__ void __launch_bounds__(kJoinThreads)
kv8_combine_kernel(const Kv8DecodeArgs a, int C) {
  __shared__ int where[2];
  __shared__ float wt[kJoinParts];
  __shared__ float4 part[kJoinGroups][32];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int bh = blockIdx.x / a.G, g = blockIdx.x - bh * a.G;
  const int b = bh / a.H, h = bh - b * a.H;
  const Rows rows{a.kv_start, a.kv_len, a.q_pos, a.max_pos,
                  a.B, a.L, a.H, a.K, a.listed};
  if (warp < 2) {
    const int n = tiles_before(rows, warp == 0 ? a.B : b) * a.H;
    if (lane == 0) where[warp] = n;
  }
  const int n = row_tiles(rows, b).n;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                       int64_t(blockIdx.x) * kHeadDim;
  if (n == 0) {
    if (t < kHeadDim) out[t] = __float2bfloat16_rn(0.f);
    if (t == 0) a.lse[blockIdx.x] = -INFINITY;
    return;
  }
  const Shares sh(where[0], C);
  const int p0 = where[1] + h * n;
  const int c0 = sh.holder(p0), c1 = sh.holder(p0 + n - 1);
  if (c0 == c1) return;       // one CTA held it all
  // CTA c0's part is its second record, those after it have theirs first
  auto record = [&](int c) {
    return a.part + (int64_t(c) * 2 + (c == c0)) * part_stride(a.G);
  };
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c0; c <= c1; c += kJoinParts) {
    const int k = min(kJoinParts, c1 + 1 - c);
    // the accumulators come in while their weights are worked out
    constexpr int kMine = kJoinParts / kJoinGroups;
    float4 x[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int j = warp + i * kJoinGroups;
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < k)
        x[i] = __ldcg(reinterpret_cast<const float4*>(
                          record(c + j) + part_acc(a.G) + g * kHeadDim) +
                      lane);
    }
    // every warp forms the pass's maximum and sum (lane: parts lane, + 32)
    float mp[2], lp[2];
    float mx = m;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = lane + 32 * i;
      mp[i] = j < k ? __ldcg(record(c + j) + g) : -INFINITY;
      lp[i] = j < k ? __ldcg(record(c + j) + a.G + g) : 0.f;
      mx = fmaxf(mx, mp[i]);
    }
    mx = warp_max(mx);
    const float mu = mx == -INFINITY ? 0.f : mx;
    const float old = exp2f(m - mu);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float w = exp2f(mp[i] - mu);
      sum += lp[i] * w;
      if (warp == 0) wt[lane + 32 * i] = w;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * old + sum;
    m = mx;
    acc.x *= old; acc.y *= old; acc.z *= old; acc.w *= old;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int j = warp + i * kJoinGroups;
      if (j >= k) break;
      const float w = wt[j];
      acc.x = fmaf(x[i].x, w, acc.x);
      acc.y = fmaf(x[i].y, w, acc.y);
      acc.z = fmaf(x[i].z, w, acc.z);
      acc.w = fmaf(x[i].w, w, acc.w);
    }
    __syncthreads();
  }
  part[warp][lane] = acc;
  __syncthreads();
  if (warp > 0) return;
#pragma unroll
  for (int i = 1; i < kJoinGroups; ++i) {
    const float4 x = part[i][lane];
    acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  reinterpret_cast<uint2*>(out)[lane] =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                 pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0)
    a.lse[blockIdx.x] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// The same where there are more (row, cache head) pairs than CTAs in the
// decode kernel, so that most are whole and the others have few parts: one
// CTA per cut between two shares, a warp per query head. Cut c lies before
// tile first(c); the pair it runs through is joined at its first cut.
__global__ void __launch_bounds__(kJoinThreads)
kv8_combine_cuts_kernel(const Kv8DecodeArgs a, int C) {
  __shared__ Start at;
  __shared__ int tiles;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const Rows rows{a.kv_start, a.kv_len, a.q_pos, a.max_pos,
                  a.B, a.L, a.H, a.K, a.listed};
  if (warp == 0) {
    const Start s = find_start(rows, C, blockIdx.x + 1);
    if (lane == 0) at = s;
  } else if (warp == 1) {
    const int n = tiles_before(rows, a.B) * a.H;
    if (lane == 0) tiles = n;
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  // rows that see nothing
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (row_tiles(rows, b).n > 0) continue;
    // (a row's query heads fit 32 bits, its channels need not)
    const int64_t heads = int64_t(a.H) * a.G, q0 = b * heads;
    for (int64_t i = t; i < heads * (kHeadDim / 2); i += kJoinThreads)
      reinterpret_cast<uint32_t*>(a.out)[q0 * (kHeadDim / 2) + i] = 0u;
    for (int64_t i = t; i < heads; i += kJoinThreads)
      a.lse[q0 + i] = -INFINITY;
  }
  // a call of one CTA has no cut; and there may be no tiles behind one
  if (int(blockIdx.x) + 1 >= C || at.u0 >= at.u1) return;
  const Shares sh(tiles, C);
  const int h = (at.u0 - at.row_at) / at.rt.n;
  const int p0 = at.row_at + h * at.rt.n;
  const int c0 = sh.holder(p0), c1 = sh.holder(p0 + at.rt.n - 1);
  if (c0 != int(blockIdx.x)) return;     // starts at the cut, or cut before
  const int64_t q0 = (int64_t(at.b) * a.H + h) * a.G;
  for (int g = warp; g < a.G; g += kJoinThreads / 32) {
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0; c <= c1; ++c) {
      const float* rec =
          a.part + (int64_t(c) * 2 + (c == c0)) * part_stride(a.G);
      const float mp = __ldcg(rec + g), lp = __ldcg(rec + a.G + g);
      const float4 x = __ldcg(reinterpret_cast<const float4*>(
                                  rec + part_acc(a.G) + g * kHeadDim) + lane);
      const float mx = fmaxf(m, mp);
      const float mu = mx == -INFINITY ? 0.f : mx;
      const float old = exp2f(m - mu), w = exp2f(mp - mu);
      m = mx;
      l = l * old + lp * w;
      acc.x = acc.x * old + x.x * w;
      acc.y = acc.y * old + x.y * w;
      acc.z = acc.z * old + x.z * w;
      acc.w = acc.w * old + x.w * w;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) +
                             (q0 + g) * kHeadDim)[lane] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                   pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0)
      a.lse[q0 + g] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

}  // namespace

int kv8_decode_grid(int B, int L, int H, int K) {
  // every SM's CTAs at once, never more than there can be tiles
  const int64_t per = K >= 0 ? K : (L + kKv8Block - 1) / kKv8Block;
  const int64_t most = int64_t(B) * H * per;
  return int(
      std::max<int64_t>(1, std::min<int64_t>(most, kDecPerSm * sm_count())));
}

size_t kv8_part_floats(int B, int L, int H, int G, int K) {
  return size_t(kv8_decode_grid(B, L, H, K)) * 2 * part_stride(G);
}

namespace {

template <bool kInt8, int GP>
cudaError_t launch_tiles(const Kv8DecodeArgs& a, int C, cudaStream_t st) {
  using D = Dec<kInt8, GP>;
  CUtensorMap mk, mv;
  // an empty cache issues no load; the maps then only need valid shapes
  const void* k = a.L > 0 ? a.k : a.part;
  const void* v = a.L > 0 ? a.v : a.part;
  const int L = std::max(a.L, 1);
  if (!make_codes_map(&mk, k, int64_t(a.B) * a.H, L) ||
      !make_codes_map(&mv, v, int64_t(a.B) * a.H, L))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<kv8_decode_kernel<kInt8, GP>, D::kSmem>();
  if (e != cudaSuccess) return e;
  return launch_dependent(kv8_decode_kernel<kInt8, GP>, dim3(C),
                          dim3(D::kThreads), D::kSmem, st, mk, mv, a);
}

template <bool kInt8>
cudaError_t launch_group(const Kv8DecodeArgs& a, int C, cudaStream_t st) {
  if (a.G == 1) return launch_tiles<kInt8, 1>(a, C, st);
  if (a.G == 2) return launch_tiles<kInt8, 2>(a, C, st);
  if (a.G <= 4) return launch_tiles<kInt8, 4>(a, C, st);
  if (a.G <= 8) return launch_tiles<kInt8, 8>(a, C, st);
  return launch_tiles<kInt8, 16>(a, C, st);
}

}  // namespace

cudaError_t launch_kv8_decode(const Kv8DecodeArgs& a, cudaStream_t st) {
  const int C = kv8_decode_grid(a.B, a.L, a.H, a.listed ? a.K : -1);
  cudaError_t e =
      a.int8 ? launch_group<true>(a, C, st) : launch_group<false>(a, C, st);
  if (e != cudaSuccess) return e;
  note_launch();
  e = int64_t(a.B) * a.H > C
          ? launch_dependent(kv8_combine_cuts_kernel,
                             dim3(std::max(C - 1, 1)), dim3(kJoinThreads), 0,
                             st, a, C)
          : launch_dependent(kv8_combine_kernel, dim3(a.B * a.H * a.G),
                             dim3(kJoinThreads), 0, st, a, C);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

}  // namespace lwm
