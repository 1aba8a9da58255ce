// Sampling from logits and sampled verification of drafted tokens.
//
//   p_i = exp(x_i / T) / sum exp(x_j / T);  with e_i given exponential variates the largest
//   p_i / e_i is token i with probability p_i (a race of exponential clocks).
//   A node's children are tried in their order with r = p at first: child c of token x and
//   draft distribution q is accepted when u_c q(x) < r(x); else r becomes max(r - q, 0)
//   divided by its sum.  With none accepted, the next token is drawn from r.
//
// Three kernels, all over rows of n_vocab logits in tiles of 8 elements a thread:
//   row_stats   one pass over every row, cut into pieces: sums of 2^(x s - m), s = log2(e) / T,
//               m a whole number: the largest score's, of the unrounded product;
//   verify      a cluster walks an entry's tree: the tests need single logits and the sums,
//               so only a draw, and a rejection with more children to come, read a row; its
//               tiles go round the cluster's blocks;
//   sample      a cluster draws a row's token: x s - log2(e), largest.
//
// Precision.  Which token wins and whether a test passes is decided by comparing numbers, so
// what is compared is exact to far below the gaps: sums are 64-bit whole numbers of fp32
// weights (m being whole, moving it shifts them); a test's probabilities are 2^frac in fp32
// times an exact power of two and the sum (3e-7); in a race a thread counts its keys from its
// winner's, and of the threads' candidates those that single fp32 operations cannot tell apart
// (within 2^-9) are compared again as 64-bit whole numbers of 2^-32.  Whole numbers, because an SM
// has two lanes for fp64 here: 480 draws in blocks of two tiles took 69 us with fp64 sums and
// winners, 45 without.  What rejections leave is a difference of probabilities and keeps their
// absolute error; where it is small the entry is walked again with two floats a weight (kLittle).
//
// Bound: the logits' bytes at the copy rate.  480 draws over 32768 tokens: 20.5 us, 0.91 of it.
// 32 chains of 16 rows, f32, drafts drawn: 34.5 us, 24 of them the sums (0.83 of it), then the
// walk and the draw, some fifteen dependent steps.  A small call is latency: 16 bf16 rows of
// 8192 8.4 us.
#include "verify.h"

#include "cache.cuh"

#include <math_constants.h>

#include <algorithm>

namespace dflash {

namespace {

constexpr int kThreads = 256;              // of row_stats and sample
constexpr int kWalkThreads = 512;          // of verify: few entries, whole rows
constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596303e-8f;   // log2(e) in two parts
constexpr float kUnit = 0x1p40f;           // of sums
constexpr float kCold = 0x1p-20f;          // temperatures below it (and not below 0) count as 0
constexpr float kLeastVariate = 0x1p-126f; // variates below it count as 0 (lg2 takes them so)
constexpr float kScoreMost = 0x1p30f;      // scores x log2(e) / T of this magnitude count as infinite
constexpr int kLeast = -(1 << 30);         // the reference of a sum of nothing

// ------------------------------------------------------------------ clusters

DF_DEVICE uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
DF_DEVICE void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Block `rank`'s copy of a shared variable.
template <typename V>
DF_DEVICE V peer(const V* at, uint32_t rank) {
  static_assert(sizeof(V) == 4 || sizeof(V) == 8, "a word or two");
  uint32_t a = (uint32_t)__cvta_generic_to_shared(at);
  asm("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(rank));
  V v;
  if constexpr (sizeof(V) == 4) {
    uint32_t w;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(w) : "r"(a) : "memory");
    memcpy(&v, &w, 4);
  } else {
    unsigned long long w;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(w) : "r"(a) : "memory");
    memcpy(&v, &w, 8);
  }
  return v;
}

DF_DEVICE float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
DF_DEVICE float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------------ rows

// Element k of a thread's eight of the tile that begins at `tile0`.  VEC: eight neighbours
// (vector loads: every row 16-byte aligned); else every NT-th (threads of the block), so that a
// warp's loads of any alignment are whole lines.
template <bool VEC, int NT>
DF_DEVICE int element(int tile0, int k) {
  return VEC ? tile0 + 8 * (int)threadIdx.x + k : tile0 + k * NT + (int)threadIdx.x;
}

// A thread's eight elements of a tile; `none` behind the row's end.
template <int EL, bool VEC, int NT>
DF_DEVICE void load8(const char* row, int tile0, int V, float none, float (&x)[8]) {
  if (VEC && tile0 + 8 * (int)threadIdx.x + 8 <= V) {
    const char* at = row + (size_t)element<true, NT>(tile0, 0) * EL;
    if constexpr (EL == 4) {
      const float4 a = *reinterpret_cast<const float4*>(at), b = *reinterpret_cast<const float4*>(at + 16);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(at);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = element<VEC, NT>(tile0, k);
    if constexpr (EL == 4)
      x[k] = i < V ? reinterpret_cast<const float*>(row)[i] : none;
    else
      x[k] = i < V ? bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(row)[i]) : none;
  }
}
DF_DEVICE float logit(const char* row, int el, int i) {
  return el == 4 ? reinterpret_cast<const float*>(row)[i] : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(row)[i]);
}

enum Heat { kBadHeat, kGreedy, kWarm };
DF_DEVICE Heat heat_of(float t) {
  if (!(t >= 0.f) || t > 1.f / kCold) return kBadHeat;
  return t < kCold ? kGreedy : kWarm;
}
DF_DEVICE float heat_at(const float* temperature, int row) { return temperature ? temperature[row] : 1.f; }

// log2(e) / t in two parts.
struct Slope {
  float hi, lo;
};
DF_DEVICE Slope slope_of(float t) {
  Slope s;
  s.hi = __fdiv_rn(kLog2e, t);
  s.lo = __fdividef(fmaf(-s.hi, t, kLog2e) + kLog2eRest, t);
  return s;
}
// 2^(y - m) = 2^(y + at) by for the whole number m of a sum: fp32 does not hold all of them
// beyond 2^24, and what it leaves (up to 64) is a power of two of its own.
struct Reference {
  float at, by;
};
DF_DEVICE Reference reference_of(int m) {
  const float at = (float)-m;
  return {at, __int_as_float((127 - m - (int)at) << 23)};
}
// 2^(x s - m) to 2e-7: the exponent with its rounding errors kept.
DF_DEVICE float weight_of(float x, float s, int m) {
  // (beyond 2^24 all of this is whole: `left` adds up exactly)
  // (__fmul_rn: a product whose rounding is taken off again is not to be fused into a sum)
  const float p = __fmul_rn(x, s), mf = (float)-m, left = (float)(-m - (int)mf), y = p + mf, bb = y - p, a = y + left;
  if (!(a > -200.f)) return a != a ? a : 0.f;
  const float rest = fmaf(x, s, -p) + ((p - (y - bb)) + (mf - bb)), k = rintf(a);
  return ldexpf(exp2f((a - k) + rest), (int)fminf(k, 200.f));
}
// Powers of two as whole numbers of 2^-32: x log2(e) / t, and log2 of a variate or a share
// (to 4e-8), within 2^62 and 2^61, so that their difference fits.
DF_DEVICE long long score_of(float x, Slope s) {
  const float p = x * s.hi;
  if (!(fabsf(p) < kScoreMost)) return p > 0.f ? 1ll << 62 : -(1ll << 62);
  return __float2ll_rn(p * 0x1p32f) + __float2ll_rn((fmaf(x, s.hi, -p) + x * s.lo) * 0x1p32f);
}
// What wins over them all, equal to itself: a variate of 0.
constexpr long long kWins = 0x7fffffffffffffffll;
DF_DEVICE long long log2_of(float e) {
  if (!(e > 0.f)) return -(1ll << 61);
  if (e == CUDART_INF_F) return 1ll << 61;
  int k;
  float f = frexpf(e, &k);   // [1/2, 1)
  if (f < 0.7071f) {
    f *= 2.f;
    --k;
  }
  return (long long)k * (1ll << 32) + __float2ll_rn(log2f(f) * 0x1p32f);
}

// ------------------------------------------------------------------ reductions

// The larger key, the lower index of equal ones (-1: none).
DF_DEVICE void best_of(long long& v, int& i, long long v2, int i2) {
  if (i2 >= 0 && (i < 0 || v2 > v || (v2 == v && i2 < i))) {
    v = v2;
    i = i2;
  }
}
// ... of the warp's lanes that have one: usually a single one.
DF_DEVICE void warp_best(long long& v, int& i) {
  unsigned has = __ballot_sync(0xffffffffu, i >= 0);
  if (!has) return;
  const int at = __ffs(has) - 1;
  long long bv = __shfl_sync(0xffffffffu, v, at);
  int bi = __shfl_sync(0xffffffffu, i, at);
  for (has &= has - 1; has; has &= has - 1) {
    const int k = __ffs(has) - 1;
    const long long v2 = __shfl_sync(0xffffffffu, v, k);
    best_of(bv, bi, v2, __shfl_sync(0xffffffffu, i, k));
  }
  v = bv;
  i = bi;
}
// A float's bits in its order (a whole number), and back.
DF_DEVICE int order_of(float x) {
  const int b = __float_as_int(x == 0.f ? 0.f : x);
  return b < 0 ? b ^ 0x7fffffff : b;
}
DF_DEVICE float largest(float x) {   // of the warp
  const int b = __reduce_max_sync(0xffffffffu, order_of(x));
  return __int_as_float(b < 0 ? b ^ 0x7fffffff : b);
}

DF_DEVICE int largest(int x) { return __reduce_max_sync(0xffffffffu, x); }

// What a block tells its cluster, twice: a block may write one while others read the other.
struct Told {
  long long v[2];
  float key[2];
  int i[2], n[2];   // n: candidates; -1: something is bad
  unsigned part[2];
};
template <int NT>
struct Shared {
  Told told;
  long long w_v[NT / 32];
  int w_i[NT / 32];
  float w_f[NT / 32];
  unsigned w_part[NT / 32];
  int turn;      // which of the two is next (the same in all blocks)
};

template <int N>
DF_DEVICE long long lane_sum(long long v) {   // of lanes 0 .. N - 1 (a power of two), in all of them
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return __shfl_sync(0xffffffffu, v, 0);
}

// Sum of v over the cluster (all threads, the same everywhere).
template <int NT>
DF_DEVICE long long cluster_total(long long v, Shared<NT>& s, int S) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = s.turn;
  v = lane_sum<32>(v);
  if (lane == 0) s.w_v[warp] = v;
  __syncthreads();
  const long long sum = lane_sum<NT / 32>(lane < NT / 32 ? s.w_v[lane] : 0ll);
  if (threadIdx.x == 0) {
    s.told.v[k] = sum;
    s.turn = k ^ 1;
  }
  if (S == 1) {
    __syncthreads();
    return sum;
  }
  cluster_sync();
  return lane_sum<8>(lane < S ? peer(&s.told.v[k], lane) : 0ll);
}

// The largest of the cluster.
template <int NT>
DF_DEVICE int cluster_largest(int v, Shared<NT>& s, int S) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = s.turn;
  v = largest(v);
  if (lane == 0) s.w_i[warp] = v;
  __syncthreads();
  v = largest(lane < NT / 32 ? s.w_i[lane] : v);
  if (threadIdx.x == 0) {
    s.told.i[k] = v;
    s.turn = k ^ 1;
  }
  if (S == 1) {
    __syncthreads();
    return v;
  }
  cluster_sync();
  return largest(lane < S ? peer(&s.told.i[k], lane) : v);
}

// The cluster's winner among the threads' candidates (float key in powers of two, index; -1:
// none).  Where others come within 2^-9 and a rounding of the largest, they are compared by
// exact(), of the thread's own (a race in some hundreds).  bad: any thread's flag.  PART: and the
// sum of the threads' parts.
template <bool PART, int NT, typename F>
DF_DEVICE int cluster_winner(float key, int i, bool& bad, F exact, Shared<NT>& s, int S, unsigned* part = nullptr) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int k = s.turn;
  const float mine = i >= 0 ? key : -CUDART_INF_F;
  const float w = largest(mine);
  if (lane == 0) s.w_f[warp] = w;
  if constexpr (PART) {
    const unsigned u = __reduce_add_sync(0xffffffffu, *part);
    if (lane == 0) s.w_part[warp] = u;
  }
  const int any = __syncthreads_or(bad);
  float top = largest(lane < NT / 32 ? s.w_f[lane] : -CUDART_INF_F);
  auto near = [](float key, float top) { return key == top || key >= top - 0x1p-9f - fabsf(top) * 0x1p-20f; };
  bool in = i >= 0 && near(mine, top);
  if (in) s.told.i[k] = i;   // (one of them: all that is needed of a single one)
  const int n = __syncthreads_count(in);
  if constexpr (PART) {
    const unsigned u = __reduce_add_sync(0xffffffffu, lane < NT / 32 ? s.w_part[lane] : 0u);
    if (threadIdx.x == 0) s.told.part[k] = u;
  }
  if (threadIdx.x == 0) {
    s.told.key[k] = top;
    s.told.n[k] = any ? -1 : n;
    s.turn = k ^ 1;
  }
  auto meet = [&] {
    if (S == 1)
      __syncthreads();
    else
      cluster_sync();
  };
  meet();
  float their = lane < S ? peer(&s.told.key[k], lane) : -CUDART_INF_F;
  int their_n = lane < S ? peer(&s.told.n[k], lane) : 0, their_i = lane < S ? peer(&s.told.i[k], lane) : -1;
  if constexpr (PART) *part = __reduce_add_sync(0xffffffffu, lane < S ? peer(&s.told.part[k], lane) : 0u);
  bad = __any_sync(0xffffffffu, their_n < 0);
  if (bad) return -1;
  top = largest(their_n > 0 ? their : -CUDART_INF_F);
  const bool close = their_n > 0 && near(their, top);
  const unsigned who = __ballot_sync(0xffffffffu, close);
  if (!who) return -1;
  const int first = __ffs(who) - 1;
  if ((who & (who - 1)) == 0 && __shfl_sync(0xffffffffu, their_n, first) == 1) return __shfl_sync(0xffffffffu, their_i, first);
  // ---- too close
  k ^= 1;
  in = in && near(mine, top);
  long long v = in ? exact() : 0;
  i = in ? i : -1;
  warp_best(v, i);
  if (lane == 0) {
    s.w_v[warp] = v;
    s.w_i[warp] = i;
  }
  __syncthreads();
  if (warp == 0) {
    v = lane < NT / 32 ? s.w_v[lane] : 0;
    i = lane < NT / 32 ? s.w_i[lane] : -1;
    warp_best(v, i);
    if (lane == 0) {
      s.told.v[k] = v;
      s.told.i[k] = i;
      s.turn = k ^ 1;
    }
  }
  meet();
  v = lane < S ? peer(&s.told.v[k], lane) : 0;
  i = lane < S ? peer(&s.told.i[k], lane) : -1;
  warp_best(v, i);
  return i;
}

// ------------------------------------------------------------------ sums of rows

// A sum whose reference moves up from m to `to`.
DF_DEVICE long long shifted(long long z, int m, int to) { return z >> min((unsigned)to - (unsigned)m, 63u); }

// Tiles of a batch: 64 bytes of a thread in flight.
template <int EL>
constexpr int kBatch = EL == 2 ? 4 : 2;
// A batch adds 64 at most (kBatchMost), and every thread of every piece (of two tiles or more) may have
// one that is not full: a row's sum stays within 63 bits.
constexpr float kBatchMost = 64.f;
constexpr int pieces_most(int V) { return ((V + 8 * kThreads - 1) / (8 * kThreads) + 1) / 2; }
static_assert((kVocabMost / (8 * kBatch<4>) + kThreads * pieces_most(kVocabMost)) * (double)kBatchMost * kUnit < 0x1p62,
              "a row's sum overflows");

// Piece `g` of P of a row: the tiles g, g + P, ..  A thread adds up 2^(x s - m), m its first
// batch's largest score, rounded up; a later batch of more than 64 makes it move m and shift
// its sum.
template <int EL, bool VEC>
DF_DEVICE void row_piece(const char* row, int V, float temperature, bool draft, int g, int P, Piece* out) {
  constexpr int kTile = 8 * kThreads;
  constexpr int kTiles = kBatch<EL>;
  __shared__ long long w_v[kThreads / 32];
  __shared__ int w_m[kThreads / 32], w_i[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Heat heat = heat_of(temperature);
  if (heat == kBadHeat || (draft && heat == kGreedy)) {   // (a greedy drafter's row is not needed)
    if (threadIdx.x == 0) *out = {heat == kBadHeat ? kNoPiece : kGreedyPiece, 0, -1};
    return;
  }
  if (heat == kGreedy) {
    float top = -CUDART_INF_F;
    int at = -1;
    bool bad = false;
    for (int t0 = g * kTile; t0 < V; t0 += P * kTile) {
      float x[8];
      load8<EL, VEC, kThreads>(row, t0, V, -CUDART_INF_F, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        bad |= !(x[k] < CUDART_INF_F);
        if (x[k] > top) {
          top = x[k];
          at = element<VEC, kThreads>(t0, k);
        }
      }
    }
    long long v = order_of(top);
    warp_best(v, at);
    if (lane == 0) {
      w_v[warp] = v;
      w_i[warp] = at;
    }
    const int any = __syncthreads_or(bad);
    if (warp == 0) {
      v = lane < kThreads / 32 ? w_v[lane] : 0;
      at = lane < kThreads / 32 ? w_i[lane] : -1;
      warp_best(v, at);
      if (lane == 0) *out = {any ? kNoPiece : kGreedyPiece, (int)v, at};
    }
    return;
  }
  const float sc = slope_of(temperature).hi;
  long long sum = 0;
  bool bad = false;
  int m = kLeast;                            // nothing seen
  Reference ref = reference_of(m);
  for (int t0 = g * kTile; t0 < V; t0 += kTiles * P * kTile) {
    float x[kTiles][8];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) load8<EL, VEC, kThreads>(row, t0 + j * P * kTile, V, -CUDART_INF_F, x[j]);
    for (bool again = false;; again = true) {
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) part[k & 3] += ex2(fmaf(x[j][k], sc, ref.at));
      const float b = ((part[0] + part[1]) + (part[2] + part[3])) * ref.by;
      if (b <= kBatchMost || again) {
        bad |= !(b <= kBatchMost);           // NaN or infinite
        sum += __float2ll_rn(b * kUnit);
        break;
      }
      float top = -CUDART_INF_F;
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, x[j][k]);
      // its score, rounded (a step of it is up to 64), and what the rounding left
      const float score = ceilf(top * sc);
      if (b == b && score <= -kScoreMost) break;   // (counts as -inf: nothing to add)
      if (!(score > -kScoreMost && score < kScoreMost)) continue;
      const int to = (int)score + (int)ceilf(fmaf(top, sc, -score));
      if (to > m) {
        sum = m > kLeast ? shifted(sum, m, to) : 0;
        m = to;
        ref = reference_of(m);
      }
    }
  }
  // one reference for all: the largest
  const int w = largest(m);
  if (lane == 0) w_m[warp] = w;
  __syncthreads();
  const int top = largest(lane < kThreads / 32 ? w_m[lane] : kLeast);
  sum = lane_sum<32>(m > kLeast ? shifted(sum, m, top) : 0ll);
  if (lane == 0) w_v[warp] = sum;
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    sum = w_v[0];
#pragma unroll
    for (int j = 1; j < kThreads / 32; ++j) sum += w_v[j];
    *out = {any ? kNoPiece : sum, top, 0};
  }
}

// Grid: P pieces of every row of the target's logits, then the drafter's.
template <int ELT, int ELD, bool VEC>
__global__ void __launch_bounds__(kThreads) row_stats_kernel(const __grid_constant__ VerifyParams p) {
  pdl_wait();
  pdl_trigger();   // (behind the wait: the walk may then read what earlier launches wrote ahead of its own)
  const int P = p.pieces, r = blockIdx.x / P, g = blockIdx.x - r * P, d = r - p.rows.T;
  if (d < 0)
    row_piece<ELT, VEC>(p.target.at + (size_t)r * p.target.ld, p.V, heat_at(p.target.temperature, r), false, g, P,
                        p.stats + blockIdx.x);
  else if (d < p.draft.rows)   // (a call without rows has blocks for one)
    row_piece<ELD, VEC>(p.draft.at + (size_t)d * p.draft.ld, p.V, heat_at(p.draft.temperature, d), true, g, P,
                        p.stats + blockIdx.x);
}

// A row's probabilities: p_i = 2^(x_i s - m) inv.  inv -1: all on token m (a target of
// temperature 0) or not needed (a drafter's); NaN: not a distribution.
struct RowStats {
  float inv, s;
  int m;
};

// Row `r` from its pieces, by `G` neighbouring lanes (a power of two, all of the warp's lanes
// call; the result is theirs alike).
DF_DEVICE RowStats row_of(const Piece* pieces, int P, int r, float s, int G) {
  const int lane = threadIdx.x & (G - 1);
  long long z = 0, v = 0;
  int top = kLeast, arg = -1, greedy = 0, bad = 0;
  for (int g0 = 0; g0 < P; g0 += G) {
    const Piece x = g0 + lane < P ? pieces[(size_t)r * P + g0 + lane] : Piece{0, kLeast, -1};
    bad |= x.z == kNoPiece;
    if (x.z == kGreedyPiece) {
      greedy = 1;
      best_of(v, arg, (long long)x.m, x.arg);
    } else if (x.z >= 0) {
      const int to = max(top, x.m);
      z = shifted(z, top, to) + shifted(x.z, x.m, to);
      top = to;
    }
  }
  for (int o = G >> 1; o > 0; o >>= 1) {
    const int to = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    z = shifted(z, top, to);
    z += __shfl_xor_sync(0xffffffffu, z, o);
    top = to;
    const long long v2 = __shfl_xor_sync(0xffffffffu, v, o);
    best_of(v, arg, v2, __shfl_xor_sync(0xffffffffu, arg, o));
    greedy |= __shfl_xor_sync(0xffffffffu, greedy, o);
    bad |= __shfl_xor_sync(0xffffffffu, bad, o);
  }
  if (bad || (!greedy && z <= 0)) return {CUDART_NAN_F, s, 0};
  if (greedy) return {-1.f, s, arg};
  return {__fdiv_rn(kUnit, __ll2float_rn(z)), s, top};
}

// ------------------------------------------------------------------ draws

// The winner of the race over a row's probabilities (bad: a NaN or +inf among the logits).
// barred(i): tokens that have no share any more.
template <int EL, bool VEC, int NT, typename F>
DF_DEVICE int race(const char* row, const char* noise, int V, float temperature, bool& bad, F barred, Shared<NT>& s,
                   int S) {
  constexpr int kTiles = 2, kTile = 8 * NT;
  const Slope slope = slope_of(temperature);
  const float sc = slope.hi, most = kScoreMost / sc;
  // keys are counted from the winner's: close ones are small then, whatever the scores (with a
  // variate of 0 it is infinite, and no key comes after it)
  float top = -kScoreMost, from = 0.f;
  int at = -1;
  for (int t0 = cluster_rank() * kTile; t0 < V; t0 += kTiles * S * kTile) {
    float x[kTiles][8], e[kTiles][8];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      load8<EL, VEC, NT>(row, t0 + j * S * kTile, V, -CUDART_INF_F, x[j]);
      load8<4, VEC, NT>(noise, t0 + j * S * kTile, V, 1.f, e[j]);
    }
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        bad |= !(x[j][k] < most);
        const float l = lg2(e[j][k]);
        if (fmaf(x[j][k], sc, -from) - l > top && !barred(element<VEC, NT>(t0 + j * S * kTile, k))) {
          from = fmaf(x[j][k], sc, -l);
          top = fmaf(x[j][k], sc, -from) - l;
          at = element<VEC, NT>(t0 + j * S * kTile, k);
        }
      }
  }
  return cluster_winner<false>(from == CUDART_INF_F ? from : top + from, at, bad, [&] {
    const float e = reinterpret_cast<const float*>(noise)[at];
    return e >= kLeastVariate ? score_of(logit(row, EL, at), slope) - log2_of(e) : kWins;
  }, s, S);
}

template <int EL, bool VEC>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleParams p, int S) {
  constexpr int kTile = 8 * kThreads;
  __shared__ Shared<kThreads> s;
  pdl_trigger();
  pdl_wait();
  if (threadIdx.x == 0) s.turn = 0;
  __syncthreads();
  const int t = blockIdx.x / S, r = p.rows ? p.rows[t] : t;
  const float temperature = heat_at(p.logits.temperature, t);
  const Heat heat = heat_of(temperature);
  const bool lead = cluster_rank() == 0 && threadIdx.x == 0;
  if (r < 0 || r >= p.n_rows || heat == kBadHeat) {   // (the whole cluster)
    if (lead) {
      set_status(p.status, heat == kBadHeat ? DEV_BAD_PROBS : DEV_BAD_ROWS);
      p.tokens[t] = -1;
    }
    return;
  }
  const char* row = p.logits.at + (size_t)r * p.logits.ld;
  bool bad = false;
  int i;
  if (heat == kGreedy) {
    float top = -CUDART_INF_F;
    i = -1;
    for (int t0 = cluster_rank() * kTile; t0 < p.V; t0 += S * kTile) {
      float x[8];
      load8<EL, VEC, kThreads>(row, t0, p.V, -CUDART_INF_F, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        bad |= !(x[k] < CUDART_INF_F);
        if (x[k] > top) {
          top = x[k];
          i = element<VEC, kThreads>(t0, k);
        }
      }
    }
    i = cluster_winner<false>(top, i, bad, [&] { return (long long)order_of(top); }, s, S);
  } else {
    i = race<EL, VEC>(row, p.noise + (size_t)t * p.noise_ld, p.V, temperature, bad, [](int) { return false; }, s, S);
  }
  if (lead) {
    if (bad || i < 0) {
      set_status(p.status, DEV_BAD_PROBS);
      i = -1;
    }
    p.tokens[t] = i;
  }
  if (S > 1) cluster_sync();
}

// ------------------------------------------------------------------ the walk

struct Node {
  float p, q;          // the target's and the drafter's probability of its token (before: its logits)
  RowStats own, from;  // its row of the target; the row of the drafter that its token was drawn from
  int token, row;      // row: of the drafter
  float u;
  short parent, first; // first child (0: none)
  short is;            // bits of Is
};
enum Is { kNoRow = 1, kGreedyRow = 2, kNoToken = 4, kNoDraft = 8, kSure = 16, kTaken = 32 };   // (kTaken: as a first child)

enum Act { kUpdate, kDraw, kDrawRest, kEnd, kBad, kCareful };

// Less than this part of the target's mass left at a node: the entry is walked again, carefully.  p
// and q are known to some 5e-7 of themselves here, so that a part m left as their difference is
// known to 5e-7 / m: to 1e-5 at least.  A rejection that leaves m has the probability m, so the
// second walk is as rare as it is slow: of one rejected draft over 32768 tokens 29 us instead of 9 (over
// 151936 68, 14), of two argmax siblings 18 instead of 8.
constexpr float kLittle = 0x1p-4f;

// Which of a thread's elements of a tile are among `n` barred tokens.
template <bool VEC, int NT>
DF_DEVICE unsigned barred_of(const int* barred, int n, int tile0) {
  unsigned mask = 0;
  for (int j = 0; j < n; ++j) {
    const unsigned off = (unsigned)(barred[j] - tile0);
    if (off < 8u * NT && (VEC ? off >> 3 : off % NT) == threadIdx.x) mask |= 1u << (VEC ? off & 7 : off / NT);
  }
  return mask;
}

// ---- careful passes: weights as two floats, to 2^-38

struct Two {
  float hi, lo;
};
// 2^(j / 64) for j = -32 .. 32
constexpr int kPowers = 65;
DF_DEVICE void make_powers(Two* power) {
  if (threadIdx.x < kPowers) {
    const double w = exp2(((int)threadIdx.x - 32) / 64.0);
    power[threadIdx.x] = {(float)w, (float)(w - (float)w)};
  }
}
// 2^(x s - m), at most about 1: the exponent as two floats (product and sums with what their
// roundings left), k + j / 64 + g, |g| < 1 / 100, and a polynomial in g.  (__fmul_rn: products
// whose rounding is taken off again are not to be fused into a sum.)
DF_DEVICE Two two_of(float x, Slope s, int m, const Two* power) {
  const float p = __fmul_rn(x, s.hi), mf = (float)-m, left = (float)(-m - (int)mf), y = p + mf, bb = y - p, a = y + left;
  if (!(a > -160.f)) return {0.f, 0.f};
  const float l = ((p - (y - bb)) + (mf - bb)) + (fmaf(x, s.hi, -p) + x * s.lo);
  const float t = a + l, cc = t - a, rest = (a - (t - cc)) + (l - cc);
  const float k = rintf(t), j = rintf((t - k) * 64.f), g = fmaf(j, -0x1p-6f, t - k);
  constexpr float kLn2 = 0.693147182f, kLn2Rest = -1.90465430e-9f;   // ln 2 in two parts; ln^n 2 / n!
  const float h = __fmul_rn(g, kLn2), q = g * g * fmaf(g, fmaf(g, 0.00961812911f, 0.0555041087f), 0.240226507f);
  const float v = fmaf(g, kLn2, -h) + (g * kLn2Rest + q), e = h + v, e2 = (h - e) + v + rest * kLn2 * (1.f + e);
  const Two c = power[(int)j + 32];
  const float w = __fmul_rn(c.hi, e), hi = c.hi + w, lo = ((c.hi - hi) + w) + (fmaf(c.hi, e, -w) + (c.lo + fmaf(c.hi, e2, c.lo * e)));
  const float by = __int_as_float((127 + (int)fminf(fmaxf(k, -126.f), 100.f)) << 23);
  return {hi * by, lo * by};
}
// Units of a careful sum, 2^-60: references are such that sums are at most 1.
constexpr float kFine = 0x1p60f;
DF_DEVICE long long fine_of(Two w) { return __float2ll_rn(w.hi * kFine) + __float2ll_rn(w.lo * kFine); }
// A reference as high as a row's sum.
DF_DEVICE int above_sum(RowStats st) {
  int k;
  frexpf(__fdiv_rn(1.f, st.inv), &k);
  return st.m + k;
}

// r at node `cur` of a careful walk: the target's p (by 2^(x s - m)), or (`written`) s_r, without
// the tokens of s_barred; `total` is its sum, `exact` what it was when it was last added up.
struct Rest {
  int m, written, n_barred;
  double total, exact;
  float ratio, ratio_rest, inv;
};
// A row, its slope, and its sum as the first pass left it.
struct Row {
  const char* at;
  Slope s;
  RowStats sum;
};

// All blocks of a cluster: r is added up, and with a drafter's row (at: not null) becomes
// max(r - q, 0), written.  What would leave nothing (by rounding, or u beyond its range) leaves r
// as it was.
template <int ELT, int ELD, bool VEC, int NT>
__device__ void take_off(const Row& row, const Row& draft, int V, int S, Rest& w, Shared<NT>& sh, const int* s_barred,
                         float* s_r, const Two* power) {
  constexpr int kTile = 8 * NT;
  const int tid = threadIdx.x, rank = cluster_rank(), hop = S * kTile;
  const bool written = w.written;
  const Slope s = row.s, s_d = draft.s;
  auto barred = [&](int t0) { return barred_of<VEC, NT>(s_barred, w.n_barred, t0); };
  int m = above_sum(row.sum), m_d = 0;
  float scale = 1.f;   // of s_r: so that its sum is at most 1
  if (written) {
    int k;
    frexpf((float)w.exact, &k);
    scale = ldexpf(1.f, -k);
  }
  if (ELD && draft.at) m_d = above_sum(draft.sum);
  long long z = 0, z_d = 0;
  while (true) {
    z = 0;
    const bool both = ELD && draft.at && z_d == 0;
    int at = 0;
    for (int t0 = rank * kTile; t0 < V; t0 += hop, at += kTile) {
      float x[8], y[8];
      if (!written) load8<ELT, VEC, NT>(row.at, t0, V, -CUDART_INF_F, x);
      if (ELD && both) load8<ELD ? ELD : 4, VEC, NT>(draft.at, t0, V, -CUDART_INF_F, y);
      const unsigned out = barred(t0);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const Two v = written ? Two{s_r[at + element<VEC, NT>(t0, k) - t0] * scale, 0.f} : two_of(x[k], s, m, power);
        if (!(out >> k & 1)) z += fine_of(v);
        if (ELD && both) z_d += fine_of(two_of(y[k], s_d, m_d, power));
      }
    }
    z = cluster_total(z, sh, S);
    if (both) z_d = cluster_total(z_d, sh, S);
    if (z >= 1ll << 46) break;
    // without the barred tokens it is small: a lower reference (a token may have lost half a unit)
    if (z > 0) {
      const int k = __clzll(z + V) - 4;
      if (written)
        scale = ldexpf(scale, k);
      else
        m -= k;
      continue;
    }
    int top = kLeast;   // the largest score
    for (int t0 = rank * kTile; t0 < V && !written; t0 += hop) {
      float x[8];
      load8<ELT, VEC, NT>(row.at, t0, V, -CUDART_INF_F, x);
      const unsigned out = barred(t0);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = __fmul_rn(x[k], s.hi);
        if (!(out >> k & 1) && v > -kScoreMost) top = max(top, (int)ceilf(v) + (int)ceilf(fmaf(x[k], s.hi, -v)));
      }
    }
    top = cluster_largest(top, sh, S);
    if (top > kLeast) {
      m = top + 19;
      continue;
    }
    if (w.n_barred == 0) break;   // (nothing is left: r as it was before the last one)
    __syncthreads();
    if (tid == 0) --w.n_barred;
    m = above_sum(row.sum);
    __syncthreads();
  }
  __syncthreads();   // (all have read the sums)
  if (tid == 0) {
    w.m = m;
    w.total = w.exact = (double)z * 0x1p-60 / scale;
  }
  if constexpr (ELD > 0) {
    if (draft.at) {
      if (tid == 0) {
        const double c = w.total / ((double)z_d * 0x1p-60);
        w.ratio = (float)c;
        w.ratio_rest = (float)(c - (float)c);
        w.inv = (float)(1.0 / w.total);
      }
      __syncthreads();
      const float c = w.ratio, c2 = w.ratio_rest, inv = w.inv;
      for (int pass = written ? 0 : 1; pass < 2; ++pass) {   // (nothing left leaves s_r as it is: added up first)
        long long units = 0;
        int at = 0;
        for (int t0 = rank * kTile; t0 < V; t0 += hop, at += kTile) {
          float x[8], y[8];
          load8<ELD, VEC, NT>(draft.at, t0, V, -CUDART_INF_F, y);
          if (!written) load8<ELT, VEC, NT>(row.at, t0, V, -CUDART_INF_F, x);
          const unsigned out = barred(t0);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float* const to = s_r + (at + element<VEC, NT>(t0, k) - t0);
            const Two a = written ? Two{*to, 0.f} : two_of(x[k], s, m, power), b = two_of(y[k], s_d, m_d, power);
            const float v = __fmul_rn(b.hi, c), v2 = fmaf(b.hi, c, -v) + fmaf(b.hi, c2, b.lo * c);
            const float r = out >> k & 1 ? 0.f : fmaxf(((a.hi - v) + (a.lo - v2)) * inv, 0.f);
            units += __float2ll_rn(r * kFine);
            if (pass == 1) *to = r;
          }
        }
        const double left = (double)cluster_total(units, sh, S) * 0x1p-60;
        if (!(left > 0x1p-34)) return;   // (known to some 2^-37)
        if (tid == 0 && pass == 1) w.total = w.exact = left;
      }
      if (tid == 0) {
        w.written = 1;
        w.n_barred = 0;
      }
    }
  }
  if (S > 1) cluster_sync();   // (s_r is there for all blocks)
  __syncthreads();
}

// The walk from node `cur` on, the path's last: every difference from numbers with bits to spare.  All
// threads walk.  Returns the token behind the path (-1: none).
template <int ELT, int ELD, bool VEC, int NT>
__device__ __noinline__ int walk_carefully(const VerifyParams& p, int lo, int n, int S, const char* noise, const Node* s_node,
                                           int* s_barred, float* s_r, short* s_path, int* s_len, int cur, Shared<NT>& sh) {
  constexpr int kTile = 8 * NT;
  __shared__ Rest w;
  __shared__ Two s_power[kPowers];
  const int tid = threadIdx.x, rank = cluster_rank(), V = p.V;
  make_powers(s_power);
  bool bad = false;
  int len = *s_len;
  while (true) {
    const int is_row = s_node[cur].is;
    if (is_row & kNoRow) return -1;
    const float temperature = heat_at(p.target.temperature, lo + cur);
    const Row row = {p.target.at + (size_t)(lo + cur) * p.target.ld, slope_of(temperature), s_node[cur].own};
    __syncthreads();
    if (tid == 0) {
      w.written = w.n_barred = 0;
      w.total = w.exact = 0.0;   // (not added up: the first child's test is settled)
    }
    __syncthreads();
    auto take = [&](int child) {
      Row draft = {nullptr, {0.f, 0.f}, {1.f, 0.f, 0}};
      if (ELD && child >= 0) {
        const int d = s_node[child].row;
        draft = {p.draft.at + (size_t)d * p.draft.ld, slope_of(heat_at(p.draft.temperature, d)), s_node[child].from};
      }
      take_off<ELT, ELD, VEC, NT>(row, draft, V, S, w, sh, s_barred, s_r, s_power);
    };
    int next = -1;
    bool first = true;
    for (int j = cur + 1; j < n && next < 0 && len < p.max_path; ++j) {
      if (s_node[j].parent != cur) continue;
      const int is = s_node[j].is, token = s_node[j].token;
      if (is & kNoToken) {
        if (rank == 0 && tid == 0) set_status(p.status, DEV_BAD_TOKEN);
        continue;
      }
      if (is & kNoDraft) return -1;
      double r = s_node[j].p;
      bool taken = is & kTaken;
      if (!first && !(is_row & kGreedyRow)) {
        if (w.total < kLittle * w.exact || w.exact == 0.0) take(-1);
        bool out = false;
        for (int k = 0; k < w.n_barred; ++k) out |= s_barred[k] == token;
        r = 0.0;
        if (!out && w.written) {
          const int tile = token / kTile;
          r = (double)peer(s_r + tile / S * kTile + (token - tile * kTile), tile % S) / w.total;
        } else if (!out) {
          const Two t = two_of(logit(row.at, ELT, token), row.s, w.m, s_power);
          r = ((double)t.hi + t.lo) / w.total;
        }
        taken = (double)s_node[j].u * (double)s_node[j].q < r;
      }
      if (taken) {
        next = j;
      } else if (!(is_row & kGreedyRow)) {
        if (!(is & kSure)) {
          take(j);
        } else if (r > 0.0) {
          __syncthreads();   // (all have read s_barred and the sums)
          if (tid == 0) {
            s_barred[w.n_barred++] = token;
            w.total -= r * w.total;
          }
          __syncthreads();
        }
      }
      first = false;
    }
    if (next >= 0) {
      cur = next;
      if (tid == 0) s_path[len] = (short)cur;
      ++len;
      continue;
    }
    if (tid == 0) *s_len = len;
    if (is_row & kGreedyRow) return s_node[cur].own.m;
    // ---- the token behind the path: from what is left, or (only barred tokens: u beyond its range)
    // from what was before the last ones were
    for (bool again = false;; again = true) {
      if (again) {
        __syncthreads();
        take(-1);
      }
      const int n_barred = w.n_barred;
      int token;
      if (!w.written) {
        token = race<ELT, VEC>(row.at, noise, V, temperature, bad, [&](int i) {
          for (int j = 0; j < n_barred; ++j)
            if (s_barred[j] == i) return true;
          return false;
        }, sh, S);
      } else {
        float best = 0.f, at_e = 1.f;   // best / at_e is the largest so far
        int win = -1, at = 0;
        const float inv = (float)(1.0 / w.total);
        for (int t0 = rank * kTile; t0 < V; t0 += S * kTile, at += kTile) {
          float z[8];
          load8<4, VEC, NT>(noise, t0, V, CUDART_NAN_F, z);
          const unsigned out = barred_of<VEC, NT>(s_barred, n_barred, t0);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int i = element<VEC, NT>(t0, k);
            const float r = s_r[at + i - t0] * inv;
            if (r > 0.f && z[k] >= 0.f && r * at_e > best * z[k] && !(out >> k & 1)) {
              best = r;
              win = i;
              at_e = z[k];
            }
          }
        }
        token = cluster_winner<false>(lg2(best) - lg2(at_e), win, bad,
                                      [&] { return at_e >= kLeastVariate ? log2_of(best) - log2_of(at_e) : kWins; }, sh, S);
      }
      if (token >= 0 || n_barred == 0 || again) return token;
    }
  }
}

// A cluster per entry; its blocks walk alike, from the same numbers.  r is the target's p
// without the tokens of s_barred, until a rejection with other children behind it makes the
// blocks write it down (s_r, each its tiles); `total` is its sum.
template <int ELT, int ELD, bool VEC>
__global__ void __launch_bounds__(kWalkThreads, 1) verify_kernel(const __grid_constant__ VerifyParams p, int S, int most) {
  constexpr int NT = kWalkThreads, kTile = 8 * NT;
  extern __shared__ __align__(16) char smem[];
  __shared__ Shared<NT> s;
  __shared__ int s_act, s_child, s_cur, s_len, s_from, s_n_barred, s_written, s_seen;
  __shared__ float s_mass;   // of the target's at the node, what rejections have left
  __shared__ double s_total;
  // (`most`: nodes of an entry that there is room for)
  Node* s_node = reinterpret_cast<Node*>(smem);
  int* s_barred = reinterpret_cast<int*>(s_node + most);
  float* s_r = reinterpret_cast<float*>(s_barred + (most + 3) / 4 * 4);
  short* s_path = reinterpret_cast<short*>(s_r + (ELD ? p.rest : 0));
  pdl_trigger();
  const int e = blockIdx.x / S, rank = cluster_rank(), tid = threadIdx.x, lane = tid & 31, V = p.V;
  const bool lead = rank == 0 && tid == 0;
  int32_t* path = p.path + (size_t)e * p.max_path;
  const char* noise = reinterpret_cast<const char*>(p.noise + (size_t)e * p.noise_ld);
  int lo, n;
  const bool fits = entry_rows(p.rows, e, lo, n) && n <= most;
  if (!fits || n == 0) {   // (the whole cluster)
    pdl_wait();
    if (!fits && lead) set_status(p.status, DEV_BAD_ROWS);
    if (rank == 0)
      for (int j = tid; j < p.max_path; j += NT) path[j] = -1;
    if (lead) p.n_path[e] = 0;
    return;
  }
  auto target_row = [&](int node) { return p.target.at + (size_t)(lo + node) * p.target.ld; };
  auto draft_of = [&](int node) { return p.draft_row ? p.draft_row[lo + node] : lo + node; };
  auto draft_row = [&](int d) { return p.draft.at + (size_t)d * p.draft.ld; };
  // every node's test, should the walk come to it: first what the sums are not needed for
  for (int i = tid; i < n; i += NT) {
    const int up = p.parents[lo + i];
    Node nd;
    nd.parent = i > 0 && up >= 0 && up < i ? up : -1;
    nd.token = p.tokens[lo + i];
    nd.u = p.uniform[lo + i];
    nd.p = nd.q = 0.f;
    nd.row = 0;
    nd.first = 0;
    nd.own.s = slope_of(heat_at(p.target.temperature, lo + i)).hi;
    nd.from.s = 0.f;
    nd.is = nd.token >= 0 && nd.token < V ? 0 : kNoToken;
    if (nd.parent >= 0 && !nd.is) {
      nd.p = logit(target_row(up), ELT, nd.token);
      if constexpr (ELD > 0) {
        const int d = draft_of(i);
        if (d >= 0 && d < p.draft.rows) {
          nd.q = logit(draft_row(d), ELD, nd.token);
          nd.from.s = slope_of(heat_at(p.draft.temperature, d)).hi;
          nd.row = d;
        } else {
          nd.is |= kNoDraft;
        }
      }
    }
    s_node[i] = nd;
  }
  for (int t0 = (rank * NT + tid) * 32; t0 < V; t0 += S * NT * 32)   // the draw's variates towards L2
    asm volatile("prefetch.global.L2 [%0];" ::"l"(noise + (size_t)t0 * 4));
  if (tid == 0) {
    s.turn = 0;
    s_cur = 0;
    s_len = 1;
    s_path[0] = 0;
    s_from = 1;
    s_n_barred = 0;
    s_written = 0;
    s_seen = 0;
    s_total = 1.0;
    s_mass = 1.f;
  }
  pdl_wait();
  __syncthreads();
  // G lanes a node: as many as a row has pieces
  int G = 1;
  while (G < p.pieces && G < 32) G *= 2;
  for (int i0 = tid / 32 * (32 / G); i0 < n; i0 += NT / G) {
    const int i = min(i0 + (tid & 31) / G, n - 1);
    const bool mine = (tid & (G - 1)) == 0 && i0 + (tid & 31) / G < n;
    const RowStats st = row_of(p.stats, p.pieces, lo + i, s_node[i].own.s, G);
    if (mine) s_node[i].own = st;
    if constexpr (ELD > 0) {
      const RowStats sd = row_of(p.stats, p.pieces, p.rows.T + s_node[i].row, s_node[i].from.s, G);
      if (mine) s_node[i].from = sd;
    }
  }
  __syncthreads();
  for (int i = tid; i < n; i += NT) {
    Node& nd = s_node[i];
    short is = nd.is;
    is |= nd.own.inv != nd.own.inv ? kNoRow : nd.own.inv < 0.f ? kGreedyRow : 0;
    float q = 1.f;
    if constexpr (ELD > 0) {
      if (nd.from.inv != nd.from.inv)
        is |= kNoDraft;
      else if (nd.from.inv < 0.f)
        is |= kSure;
      else
        q = weight_of(nd.q, nd.from.s, nd.from.m) * nd.from.inv;
    } else {
      is |= kSure;
    }
    nd.q = q;
    if (nd.parent >= 0) {
      const RowStats st = s_node[nd.parent].own;
      nd.p = st.inv < 0.f ? (nd.token == st.m ? 1.f : 0.f) : weight_of(nd.p, st.s, st.m) * st.inv;
      if ((double)nd.u * (double)q < (double)nd.p) is |= kTaken;
      // (the parent's first child: no node between is its child)
      bool least = true;
      for (int j = nd.parent + 1; j < i && least; ++j) least = s_node[j].parent != nd.parent;
      if (least) s_node[nd.parent].first = i;
    }
    nd.is = is;
  }
  __syncthreads();

  while (true) {
    // ---- the first warp walks until a row has to be read
    if (tid < 32) {
      int cur = s_cur, len = s_len, from = s_from, barred = s_n_barred, written = s_written, child = -1, act = -1;
      double total = s_total;
      float mass = s_mass;
      bool fresh = from == 1 && len == 1;   // no child of cur has been tried
      while (act < 0) {
        const int row = s_node[cur].is;
        if (row & kNoRow) {
          act = kBad;
          break;
        }
        int next = -1;   // the first child of cur from `from` on
        if (len < p.max_path) {
          if (fresh) {
            next = s_node[cur].first - 1;
            if (next >= 0) ++next;
          } else {
            for (int b = from; b < n && next < 0; b += 32) {
              const unsigned is = __ballot_sync(0xffffffffu, b + lane < n && s_node[min(b + lane, n - 1)].parent == cur);
              if (is) next = b + __ffs(is) - 1;
            }
          }
        }
        if (next < 0) {
          act = row & kGreedyRow ? kEnd : child >= 0 ? kDrawRest : kDraw;
          break;
        }
        if (child >= 0) {   // the rejected child's distribution has to be taken off first
          act = kUpdate;
          break;
        }
        if (mass < kLittle) {   // (its test needs what is left)
          act = kCareful;
          break;
        }
        const Node& nd = s_node[next];
        const int is = nd.is;
        from = next + 1;
        if (is & kNoToken) {
          if (lead) set_status(p.status, DEV_BAD_TOKEN);
          fresh = false;
          continue;
        }
        if (is & kNoDraft) {
          act = kBad;
          break;
        }
        bool taken = is & kTaken;
        double r = nd.p;
        if (!(row & kGreedyRow) && (barred || written)) {
          int out = 0;
          for (int j = lane; j < barred; j += 32) out |= s_barred[j] == nd.token;
          const bool gone = __any_sync(0xffffffffu, out);
          if (written && !gone) {
            const int tile = nd.token / kTile;
            r = (double)peer(s_r + tile / S * kTile + (nd.token - tile * kTile), tile % S);
          }
          r = gone ? 0.0 : r / total;
          taken = (double)nd.u * (double)nd.q < r;
        }
        if (taken) {
          if (lane == 0) s_path[len] = next;
          ++len;
          cur = next;
          barred = written = 0;
          total = 1.0;
          mass = 1.f;
          fresh = true;
          continue;
        }
        fresh = false;
        if (row & kGreedyRow) continue;
        if (!(is & kSure)) {
          child = next;
        } else if (r > 0.0) {
          if (lane == 0) s_barred[barred] = nd.token;
          ++barred;
          total -= r * total;
          mass *= (float)(1.0 - r);
          __syncwarp();
        }
      }
      if (lane == 0) {
        s_act = act;
        s_child = child;
        s_cur = cur;
        s_len = len;
        s_from = from;
        s_n_barred = barred;
        s_written = written;
        s_total = total;
        s_mass = mass;
      }
    }
    __syncthreads();
    if (s_act != kUpdate || s_mass < kLittle) break;

    // ---- r becomes max(r - q, 0), written down
    if constexpr (ELD > 0) {
      if (S > 1 && s_seen) cluster_sync();   // no block changes s_r while the walk of another looks into it
      const int cur = s_cur, barred = s_n_barred, written = s_written;
      const RowStats st = s_node[cur].own, sd = s_node[s_child].from;
      const Reference ref = reference_of(st.m), ref_d = reference_of(sd.m);
      const float inv = (written ? 1.f : st.inv * ref.by) / (float)s_total, inv_d = sd.inv * ref_d.by;
      const char *row = target_row(cur), *row_d = draft_row(s_node[s_child].row);
      long long units = 0;   // of 2^-50 (r adds up to at most 1)
      float x[2][8], y[2][8];
      auto fetch = [&](int t0, float(&x)[8], float(&y)[8]) {
        load8<ELD, VEC, NT>(row_d, t0, V, -CUDART_INF_F, y);
        if (!written) load8<ELT, VEC, NT>(row, t0, V, -CUDART_INF_F, x);
      };
      auto take = [&](int t0, int at, const float(&x)[8], const float(&y)[8]) {
        float part = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int i = element<VEC, NT>(t0, k);
          float r = written ? s_r[at + i - t0] : ex2(fmaf(x[k], st.s, ref.at));
          for (int j = 0; j < barred; ++j)
            if (s_barred[j] == i) r = 0.f;
          r = fmaxf(fmaf(r, inv, -ex2(fmaf(y[k], sd.s, ref_d.at)) * inv_d), 0.f);
          s_r[at + i - t0] = r;
          part += r;
        }
        units += __float2ll_rn(part * 0x1p50f);
      };
      const int hop = S * kTile;
      int t0 = rank * kTile, at = 0;
      fetch(t0, x[0], y[0]);
      for (; t0 < V; t0 += 2 * hop, at += 2 * kTile) {   // (the next tile on its way under a tile's arithmetic)
        fetch(t0 + hop, x[1], y[1]);
        take(t0, at, x[0], y[0]);
        if (t0 + hop >= V) break;
        fetch(t0 + 2 * hop, x[0], y[0]);
        take(t0 + hop, at + kTile, x[1], y[1]);
      }
      const double sum = (double)cluster_total(units, s, S) * 0x1p-50;
      if (tid == 0) {
        s_written = 1;
        s_total = sum;
        s_mass *= (float)sum;
        s_n_barred = 0;
        s_seen = 1;
      }
      __syncthreads();
    }
  }

  // ---- the token behind the path
  int act = s_act;
  const int cur = s_cur, barred = s_n_barred, written = s_written;
  // (tokens barred beside a drafter's distribution: what is left is not added up here)
  if (act == kUpdate || (act == kDrawRest && (barred || s_mass < kLittle)) || (act == kDraw && written && s_mass < kLittle))
    act = kCareful;
  const RowStats st = s_node[cur].own;
  const float temperature = heat_at(p.target.temperature, lo + cur);
  auto is_barred = [&](int i) {
    for (int j = 0; j < barred; ++j)
      if (s_barred[j] == i) return true;
    return false;
  };
  int token = act == kEnd ? st.m : -1;
  bool bad = false;
  if (act == kDrawRest || (act == kDraw && written)) {
    const bool less = ELD > 0 && act == kDrawRest;   // a last child's q comes off on the way
    RowStats sd = {1.f, 0.f, 0};
    const char* row_d = nullptr;
    if (less) {
      sd = s_node[s_child].from;
      row_d = draft_row(s_node[s_child].row);
    }
    const Reference ref = reference_of(st.m), ref_d = reference_of(sd.m);
    const float inv0 = (written ? 1.f : st.inv) / (float)s_total, inv = written ? inv0 : inv0 * ref.by, inv_d = sd.inv * ref_d.by;
    const char* row = target_row(cur);
    float best = 0.f, at_x = 0.f, at_y = 0.f, at_e = 1.f;   // best / at_e is the largest so far
    int win = -1;
    float part = 0.f;   // of what is left
    float x[2][8], y[2][8], z[2][8];
    auto fetch = [&](int t0, float(&x)[8], float(&y)[8], float(&z)[8]) {
      load8<4, VEC, NT>(noise, t0, V, CUDART_NAN_F, z);
      if constexpr (ELD > 0) {
        if (less) load8<ELD, VEC, NT>(row_d, t0, V, -CUDART_INF_F, y);
      }
      if (!written) load8<ELT, VEC, NT>(row, t0, V, -CUDART_INF_F, x);
    };
    auto take = [&](int t0, int at, float(&x)[8], const float(&y)[8], const float(&z)[8]) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = element<VEC, NT>(t0, k);
        if (written) x[k] = s_r[at + i - t0];
        float r = (written ? x[k] : ex2(fmaf(x[k], st.s, ref.at))) * inv;
        if (less) {
          r = r - ex2(fmaf(y[k], sd.s, ref_d.at)) * inv_d;
          part += fmaxf(r, 0.f);
        }
        // (r / z above the best, without a quotient)
        if (r > 0.f && z[k] >= 0.f && r * at_e > best * z[k] && !is_barred(i)) {
          best = r;
          win = i;
          at_x = x[k];
          at_e = z[k];
          if (less) at_y = y[k];
        }
      }
    };
    const int hop = S * kTile;
    int t0 = rank * kTile, at = 0;
    fetch(t0, x[0], y[0], z[0]);
    for (; t0 < V; t0 += 2 * hop, at += 2 * kTile) {
      fetch(t0 + hop, x[1], y[1], z[1]);
      take(t0, at, x[0], y[0], z[0]);
      if (t0 + hop >= V) break;
      fetch(t0 + 2 * hop, x[0], y[0], z[0]);
      take(t0 + hop, at + kTile, x[1], y[1], z[1]);
    }
    const float top = lg2(best) - lg2(at_e);
    unsigned parts = (unsigned)__float2int_rn(part * 0x1p30f);
    token = cluster_winner<ELD != 0>(top, win, bad, [&] {
      float r = (written ? at_x : weight_of(at_x, st.s, st.m)) * inv0;
      if (less) r = fmaf(-weight_of(at_y, sd.s, sd.m), sd.inv, r);
      return at_e >= kLeastVariate ? log2_of(r) - log2_of(at_e) : kWins;
    }, s, S, &parts);
    if (less && s_mass * ((float)parts * 0x1p-30f) < kLittle) act = kCareful;
  }
  if (act == kDraw && !written)
    token = race<ELT, VEC>(target_row(cur), noise, V, temperature, bad, is_barred, s, S);
  // (and where tokens are barred and nothing else is to be drawn)
  if (act == kCareful || (act == kDraw && token < 0 && barred > 0 && !bad)) {
    token = walk_carefully<ELT, ELD, VEC, NT>(p, lo, n, S, noise, s_node, s_barred, s_r, s_path, &s_len, cur, s);
    __syncthreads();
  }
  const bool none = token < 0 || bad;
  if (rank == 0) {
    const int len = none ? 0 : s_len;
    for (int j = tid; j < p.max_path; j += NT) path[j] = j < len ? s_path[j] : -1;
    if (tid == 0) {
      p.n_path[e] = len;
      if (none)
        set_status(p.status, DEV_BAD_PROBS);
      else
        p.id_last[e] = token;
    }
  }
  if (S > 1) cluster_sync();   // no block ends while another reads what it told
}

// ------------------------------------------------------------------ launches

bool vector_rows(const void* at, int64_t ld_bytes) {
  return ((reinterpret_cast<uintptr_t>(at) | (uint64_t)ld_bytes) & 15) == 0;
}
bool vector_rows(const Logits& x) { return vector_rows(x.at, x.ld); }

// Blocks of a cluster: as many as keep the launch within `most` blocks, at least `least`, no
// more than a row has tiles.
int cluster_of(int64_t rows, int tiles, int most, int least) {
  int S = 1;
  while (S < 8 && (S < least || (rows * 2 * S <= most && 2 * S <= tiles))) S *= 2;
  return S;
}

template <typename K, typename... A>
cudaError_t launch_clusters(K* kernel, int64_t rows, int S, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * S));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {(unsigned)S, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int kSms = 152;
constexpr size_t kRestMost = sizeof(float) * (kVocabMost / 8);   // a block's share of the largest vocabulary
constexpr size_t kNodeBytes = sizeof(Node) + sizeof(int) + sizeof(short);
constexpr size_t kSmemMost = kRestMost + kTreeMax * kNodeBytes + 16;
static_assert(kVocabMost % (8 * 8 * kWalkThreads) == 0, "whole tiles");
static_assert(kSmemMost <= 225 * 1024, "shared memory");

template <int ELT, int ELD, bool VEC>
cudaError_t verify_as(VerifyParams& p, cudaStream_t st) {
  const int rows = p.rows.T + (ELD ? p.draft.rows : 0);
  // pieces of a row: enough blocks for six rounds of the GPU's, each of two tiles at least
  p.pieces = std::min(std::max(rows > 0 ? kSms * 30 / rows : 1, 1), pieces_most(p.V));
  // (without rows too: the walk may start ahead of this launch's end, not of what came before)
  const cudaError_t e = launch_dependent(row_stats_kernel<ELT, ELD ? ELD : 4, VEC>, dim3(std::max(rows, 1) * p.pieces),
                                         kThreads, 0, st, p);
  if (e != cudaSuccess) return e;
  const int walk_tiles = (p.V + 8 * kWalkThreads - 1) / (8 * kWalkThreads), most = kVocabMost / (8 * 8 * kWalkThreads);
  const int W = cluster_of(p.rows.n_seq, walk_tiles, kSms, (walk_tiles + most - 1) / most);
  const int nodes = std::max(std::min(p.rows.T, kTreeMax), 1);
  p.rest = ELD ? 8 * kWalkThreads * ((walk_tiles + W - 1) / W) : 0;
  return launch_clusters(verify_kernel<ELT, ELD, VEC>, p.rows.n_seq, W, kWalkThreads,
                         nodes * kNodeBytes + 16 + sizeof(float) * p.rest, st, p, W, nodes);
}

template <int ELT, int ELD>
cudaError_t verify_by_rows(VerifyParams& p, cudaStream_t st) {
  const bool vec = vector_rows(p.target) && (!ELD || vector_rows(p.draft)) && vector_rows(p.noise, p.noise_ld * 4);
  return vec ? verify_as<ELT, ELD, true>(p, st) : verify_as<ELT, ELD, false>(p, st);
}

template <int ELT>
cudaError_t verify_by_draft(VerifyParams& p, cudaStream_t st) {
  return !p.draft.at ? verify_by_rows<ELT, 0>(p, st) : p.draft.el == 4 ? verify_by_rows<ELT, 4>(p, st)
                                                                       : verify_by_rows<ELT, 2>(p, st);
}

template <int ELT, int ELD>
cudaError_t raise_smem() {
  const cudaError_t e = cudaFuncSetAttribute(verify_kernel<ELT, ELD, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kSmemMost);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(verify_kernel<ELT, ELD, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMost);
}

template <int EL>
cudaError_t sample_as(const SampleParams& p, cudaStream_t st) {
  const int S = cluster_of(p.T, (p.V + 8 * kThreads - 1) / (8 * kThreads), kSms * 4, 1);
  return vector_rows(p.logits) && vector_rows(p.noise, p.noise_ld)
             ? launch_clusters(sample_kernel<EL, true>, p.T, S, kThreads, 0, st, p, S)
             : launch_clusters(sample_kernel<EL, false>, p.T, S, kThreads, 0, st, p, S);
}

}  // namespace

cudaError_t configure_verify() {
  cudaError_t e = raise_smem<2, 0>();
  if (e == cudaSuccess) e = raise_smem<4, 0>();
  if (e == cudaSuccess) e = raise_smem<2, 2>();
  if (e == cudaSuccess) e = raise_smem<2, 4>();
  if (e == cudaSuccess) e = raise_smem<4, 2>();
  if (e == cudaSuccess) e = raise_smem<4, 4>();
  return e;
}

cudaError_t launch_verify(VerifyParams p, cudaStream_t st) {
  return p.target.el == 4 ? verify_by_draft<4>(p, st) : verify_by_draft<2>(p, st);
}

cudaError_t launch_sample(const SampleParams& p, cudaStream_t st) {
  return p.logits.el == 4 ? sample_as<4>(p, st) : sample_as<2>(p, st);
}

}  // namespace dflash
