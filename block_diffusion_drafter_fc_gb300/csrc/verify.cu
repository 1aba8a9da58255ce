// Sampling from logits and sampled verification of drafted tokens.
//
//   p_i = exp(x_i / T) / sum exp(x_j / T);  with e_i given exponential variates the largest
//   p_i / e_i is token i with probability p_i (a race of exponential clocks).
//   A node's children are tried in their order with r = p at first: child c of token x and
//   draft distribution q is accepted when u_c q(x) < r(x); else r becomes max(r - q, 0)
//   divided by its sum.  With none accepted, the next token is drawn from r.
//
// Three kernels, all over rows of n_vocab logits cut into tiles of 2048, a row's tiles going
// round the blocks of a cluster (1 to 8; sums and maxima through distributed shared memory):
//   row_stats   one pass over every row: sum of 2^(x s - m), s = log2(e) / T, m a whole number;
//   verify      a cluster walks an entry's tree: the tests need single logits and the sums,
//               so only a draw, and a rejection with more children to come, read a row;
//   sample      a cluster draws a row's token: x s - log2(e), largest.
//
// Precision.  Which token wins and whether a test passes is decided by comparing numbers, so
// what is compared is exact to far below the gaps: sums are fp64 of fp32 weights (m being a
// whole number, moving it rescales exactly), tests are fp64, and in a race the candidates that
// fp32 cannot tell apart (a block's within 2^-9) are compared again in fp64.
//
// Bound: the logits' bytes at the copy rate; a small call by latency.
#include "verify.h"

#include "cache.cuh"

#include <math_constants.h>

namespace dflash {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 8 * kThreads;        // elements of a row that a block takes at once, 8 a thread
constexpr double kLog2e = 1.4426950408889634;
constexpr float kCold = 0x1p-20f;          // temperatures below it (and not below 0) count as 0
constexpr float kScoreMost = 0x1p30f;      // scores x log2(e) / T of this magnitude count as infinite

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
// (vector loads: every row 16-byte aligned); else every 256th, so that a warp's loads of any
// alignment are whole lines.
template <bool VEC>
DF_DEVICE int element(int tile0, int k) {
  return VEC ? tile0 + 8 * (int)threadIdx.x + k : tile0 + k * kThreads + (int)threadIdx.x;
}

// A thread's eight elements of a tile; `none` behind the row's end.
template <int EL, bool VEC>
DF_DEVICE void load8(const char* row, int tile0, int V, float none, float (&x)[8]) {
  if (VEC && tile0 + 8 * (int)threadIdx.x + 8 <= V) {
    const char* at = row + (size_t)element<true>(tile0, 0) * EL;
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
    const int i = element<VEC>(tile0, k);
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

// ------------------------------------------------------------------ reductions

DF_DEVICE double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// The larger key, the lower index of equal ones; NaN never wins.
DF_DEVICE void best_of(double& v, int& i, double v2, int i2) {
  if (i2 >= 0 && (i < 0 || v2 > v || (v2 == v && i2 < i))) {
    v = v2;
    i = i2;
  }
}
DF_DEVICE void warp_best(double& v, int& i) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double v2 = __shfl_xor_sync(0xffffffffu, v, o);
    const int i2 = __shfl_xor_sync(0xffffffffu, i, o);
    best_of(v, i, v2, i2);
  }
}

// What a block tells its cluster, twice: a block may write one while others read the other.
struct Told {
  double v[2];
  int i[2], bad[2];
};
struct Shared {
  Told told;
  double w_v[kThreads / 32];
  int w_i[kThreads / 32];
  float w_f[kThreads / 32];
  int turn;      // which of the two is next (the same in all blocks)
};

// Sum of v over the cluster (all threads, the same everywhere).
DF_DEVICE double cluster_total(double v, Shared& s, int S) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = s.turn;
  v = warp_sum(v);
  if (lane == 0) s.w_v[warp] = v;
  __syncthreads();
  double sum = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) sum += s.w_v[w];
  if (threadIdx.x == 0) {
    s.told.v[k] = sum;
    s.turn = k ^ 1;
  }
  if (S == 1) {
    __syncthreads();
    return sum;
  }
  cluster_sync();
  double all = 0.0;
  for (int r = 0; r < S; ++r) all += peer(&s.told.v[k], r);
  return all;
}

// The cluster's winner among the threads' candidates (float key in powers of two, index; -1:
// none): those within 2^-9 and a rounding of the block's largest are compared by exact(i).
// bad: any thread's flag.
template <typename F>
DF_DEVICE int cluster_winner(float key, int i, bool& bad, F exact, Shared& s, int S) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = s.turn;
  const float mine = i >= 0 ? key : -CUDART_INF_F;
  const float w = warp_max(mine);
  if (lane == 0) s.w_f[warp] = w;
  const int any = __syncthreads_or(bad);
  float top = s.w_f[0];
#pragma unroll
  for (int j = 1; j < kThreads / 32; ++j) top = fmaxf(top, s.w_f[j]);
  const float near = top - 0x1p-9f - fabsf(top) * 0x1p-20f;
  double v = 0.0;
  if (i >= 0) {
    if (mine >= near || mine == top)
      v = exact(i);
    else
      i = -1;
  }
  warp_best(v, i);
  if (lane == 0) {
    s.w_v[warp] = v;
    s.w_i[warp] = i;
  }
  __syncthreads();
  if (warp == 0) {
    v = lane < kThreads / 32 ? s.w_v[lane] : 0.0;
    i = lane < kThreads / 32 ? s.w_i[lane] : -1;
    warp_best(v, i);
    if (lane == 0) {
      s.told.v[k] = v;
      s.told.i[k] = i;
      s.told.bad[k] = any;
      s.turn = k ^ 1;
    }
  }
  if (S == 1)
    __syncthreads();
  else
    cluster_sync();
  v = 0.0;
  i = -1;
  int b = 0;
  for (int r = 0; r < S; ++r) {
    best_of(v, i, peer(&s.told.v[k], r), peer(&s.told.i[k], r));
    b |= peer(&s.told.bad[k], r);
  }
  bad = b != 0;
  return i;
}

// ------------------------------------------------------------------ sums of rows

// Rows 0 .. target_rows - 1 of the target's logits, then the drafter's.  A cluster per row.
//
// A thread adds up 2^(x s - m) for the first m that keeps a batch's sum below 2^40 (its first
// batch's largest, rounded up); larger scores later make it move m and rescale, exactly.
template <int EL, bool VEC>
DF_DEVICE void row_stats(const char* row, int V, float temperature, bool draft, RowStats* out, Shared& s, int S) {
  constexpr int kTiles = EL == 2 ? 4 : 2;    // tiles of a batch: 64 bytes of a thread in flight
  const Heat heat = heat_of(temperature);
  const int rank = cluster_rank();
  if (heat == kBadHeat || (draft && heat == kGreedy)) {   // (a greedy drafter's row is not needed)
    if (rank == 0 && threadIdx.x == 0) *out = {heat == kBadHeat ? (double)CUDART_NAN_F : -1.0, 0, -1};
    return;
  }
  if (heat == kGreedy) {
    float top = -CUDART_INF_F;
    int at = -1;
    bool bad = false;
    for (int t0 = rank * kTile; t0 < V; t0 += S * kTile) {
      float x[8];
      load8<EL, VEC>(row, t0, V, -CUDART_INF_F, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        bad |= !(x[k] < CUDART_INF_F);
        if (x[k] > top) {
          top = x[k];
          at = element<VEC>(t0, k);
        }
      }
    }
    const int arg = cluster_winner(top, at, bad, [&](int i) { return (double)logit(row, EL, i); }, s, S);
    if (rank == 0 && threadIdx.x == 0) *out = {bad || arg < 0 ? (double)CUDART_NAN_F : -1.0, 0, arg};
    return;
  }
  const float sc = (float)(kLog2e / temperature);
  double sum = 0.0;
  float m = -kScoreMost;                     // nothing seen
  for (int t0 = rank * kTile; t0 < V; t0 += kTiles * S * kTile) {
    float x[kTiles][8];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) load8<EL, VEC>(row, t0 + j * S * kTile, V, -CUDART_INF_F, x[j]);
    for (bool again = false;; again = true) {
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) part[k & 3] += ex2(fmaf(x[j][k], sc, -m));
      const float b = (part[0] + part[1]) + (part[2] + part[3]);
      if (b < 0x1p40f || again) {
        sum += (double)b;
        break;
      }
      float top = -CUDART_INF_F;             // (of a batch with NaN: of its numbers; its sum stays NaN)
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, x[j][k] * sc);
      const float to = top < kScoreMost ? ceilf(top) : m;
      if (to > m) {
        sum = ldexp(sum, (int)fmaxf(m - to, -2000.f));
        m = to;
      }
    }
  }
  // one reference for all: the largest
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = s.turn;
  const float w = warp_max(m);
  if (lane == 0) s.w_f[warp] = w;
  __syncthreads();
  float top = s.w_f[0];
#pragma unroll
  for (int j = 1; j < kThreads / 32; ++j) top = fmaxf(top, s.w_f[j]);
  if (S > 1) {
    if (threadIdx.x == 0) {
      s.told.v[k] = (double)top;
      s.turn = k ^ 1;
    }
    cluster_sync();
    for (int r = 0; r < S; ++r) top = fmaxf(top, (float)peer(&s.told.v[k], r));
  }
  // (a NaN or an infinite sum stays what it is)
  const double z = cluster_total(sum == 0.0 ? 0.0 : ldexp(sum, (int)fmaxf(m - top, -2000.f)), s, S);
  if (rank == 0 && threadIdx.x == 0)
    *out = {z > 0.0 && z < CUDART_INF ? z : (double)CUDART_NAN_F, (int)top, -1};
}

template <int ELT, int ELD, bool VEC>
__global__ void __launch_bounds__(kThreads) row_stats_kernel(const __grid_constant__ VerifyParams p, int target_rows,
                                                             int S) {
  __shared__ Shared s;
  pdl_trigger();
  pdl_wait();
  if (threadIdx.x == 0) s.turn = 0;
  __syncthreads();
  const int r = blockIdx.x / S, d = r - target_rows;
  if (d < 0)
    row_stats<ELT, VEC>(p.target.at + (size_t)r * p.target.ld, p.V, heat_at(p.target.temperature, r), false, p.stats + r, s, S);
  else
    row_stats<ELD, VEC>(p.draft.at + (size_t)d * p.draft.ld, p.V, heat_at(p.draft.temperature, d), true, p.stats + r, s, S);
  if (S > 1) cluster_sync();   // no block ends while another reads what it told
}

// ------------------------------------------------------------------ draws

// The winner of the race over a row's probabilities (bad: a NaN or +inf among the logits).
// barred(i): tokens that have no share any more.
template <int EL, bool VEC, typename F>
DF_DEVICE int race(const char* row, const char* noise, int V, float temperature, bool& bad, F barred, Shared& s, int S) {
  constexpr int kTiles = 2;
  const double sd = kLog2e / temperature;
  const float sc = (float)sd;
  const float most = kScoreMost / sc;
  float top = -kScoreMost;
  int at = -1;
  for (int t0 = cluster_rank() * kTile; t0 < V; t0 += kTiles * S * kTile) {
    float x[kTiles][8], e[kTiles][8];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      load8<EL, VEC>(row, t0 + j * S * kTile, V, -CUDART_INF_F, x[j]);
      load8<4, VEC>(noise, t0 + j * S * kTile, V, 1.f, e[j]);
    }
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        bad |= !(x[j][k] < most);
        const float key = fmaf(x[j][k], sc, -lg2(e[j][k]));
        if (key > top && !barred(element<VEC>(t0 + j * S * kTile, k))) {
          top = key;
          at = element<VEC>(t0 + j * S * kTile, k);
        }
      }
  }
  return cluster_winner(top, at, bad, [&](int i) {
    return (double)logit(row, EL, i) * sd - log2((double)reinterpret_cast<const float*>(noise)[i]);
  }, s, S);
}

template <int EL, bool VEC>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleParams p, int S) {
  __shared__ Shared s;
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
      load8<EL, VEC>(row, t0, p.V, -CUDART_INF_F, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        bad |= !(x[k] < CUDART_INF_F);
        if (x[k] > top) {
          top = x[k];
          i = element<VEC>(t0, k);
        }
      }
    }
    i = cluster_winner(top, i, bad, [&](int j) { return (double)logit(row, EL, j); }, s, S);
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
  double p, q;    // the target's and the drafter's probability of its token (q -1: drafted with certainty)
  int parent, token;
  float u;
  int heat;       // of the target's row: 0, 1 (greedy) or 2 (no distribution)
};

enum Act { kUpdate, kDraw, kDrawRest, kEnd, kBad };

// A cluster per entry; its blocks walk alike, from the same numbers.  r is the target's p
// without the tokens of s_barred, until a rejection with other children behind it makes the
// blocks write it down (s_r, each its tiles); `total` is its sum.
template <int ELT, int ELD, bool VEC>
__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyParams p, int S) {
  extern __shared__ float s_r[];
  __shared__ Shared s;
  __shared__ Node s_node[kTreeMax];
  __shared__ int s_path[kTreeMax], s_barred[kTreeMax];
  __shared__ int s_act, s_child, s_cur, s_len, s_from, s_n_barred, s_written;
  __shared__ double s_total;
  pdl_trigger();
  pdl_wait();
  const int e = blockIdx.x / S, rank = cluster_rank(), tid = threadIdx.x, lane = tid & 31, V = p.V;
  const bool lead = rank == 0 && tid == 0;
  int32_t* path = p.path + (size_t)e * p.max_path;
  int lo, n;
  const bool fits = entry_rows(p.rows, e, lo, n) && n <= kTreeMax;
  if (!fits || n == 0) {   // (the whole cluster)
    if (!fits && lead) set_status(p.status, DEV_BAD_ROWS);
    if (rank == 0)
      for (int j = tid; j < p.max_path; j += kThreads) path[j] = -1;
    if (lead) p.n_path[e] = 0;
    return;
  }
  auto target_row = [&](int node) { return p.target.at + (size_t)(lo + node) * p.target.ld; };
  auto target_heat = [&](int node) { return heat_at(p.target.temperature, lo + node); };
  auto draft_of = [&](int node) { return p.draft_row ? p.draft_row[lo + node] : lo + node; };
  // x's share of its row, in fp64
  auto share = [](float x, float temperature, const RowStats& st) {
    return exp2((double)x * (double)(float)(kLog2e / temperature) - st.m) / st.z;
  };
  // every node's test, should the walk come to it
  for (int i = tid; i < n; i += kThreads) {
    const RowStats own = p.stats[lo + i];
    const int up = p.parents[lo + i], x = p.tokens[lo + i];
    Node nd = {0.0, -1.0, i > 0 && up >= 0 && up < i ? up : -1, x, p.uniform[lo + i],
               own.z != own.z ? 2 : own.z < 0.0 ? 1 : 0};
    if (nd.parent >= 0 && x >= 0 && x < V) {
      const RowStats st = p.stats[lo + up];
      nd.p = st.z < 0.0 ? (x == st.arg ? 1.0 : 0.0) : share(logit(target_row(up), ELT, x), target_heat(up), st);
      if constexpr (ELD > 0) {
        const int d = draft_of(i);
        if (d < 0 || d >= p.draft.rows) {
          nd.q = CUDART_NAN;
        } else {
          const RowStats sd = p.stats[p.rows.T + d];
          if (!(sd.z < 0.0))
            nd.q = share(logit(p.draft.at + (size_t)d * p.draft.ld, ELD, x), heat_at(p.draft.temperature, d), sd);
        }
      }
    }
    s_node[i] = nd;
  }
  if (tid == 0) {
    s.turn = 0;
    s_cur = 0;
    s_len = 1;
    s_path[0] = 0;
    s_from = 1;
    s_n_barred = 0;
    s_written = 0;
    s_total = 1.0;
  }
  __syncthreads();

  while (true) {
    // ---- the first warp walks until a row has to be read
    if (tid < 32) {
      int cur = s_cur, len = s_len, from = s_from, barred = s_n_barred, written = s_written, child = -1, act = -1;
      double total = s_total;
      while (act < 0) {
        const int heat = s_node[cur].heat;
        if (heat == 2) {
          act = kBad;
          break;
        }
        int next = -1;   // the first child of cur from `from` on
        if (len < p.max_path)
          for (int b = from; b < n && next < 0; b += 32) {
            const unsigned is = __ballot_sync(0xffffffffu, b + lane < n && s_node[min(b + lane, n - 1)].parent == cur);
            if (is) next = b + __ffs(is) - 1;
          }
        if (next < 0) {
          act = heat == 1 ? kEnd : child >= 0 ? kDrawRest : kDraw;
          break;
        }
        if (child >= 0) {   // the rejected child's distribution has to be taken off first
          act = kUpdate;
          break;
        }
        const Node nd = s_node[next];
        from = next + 1;
        if (nd.token < 0 || nd.token >= V) {
          if (lead) set_status(p.status, DEV_BAD_TOKEN);
          continue;
        }
        if (nd.q != nd.q) {
          act = kBad;
          break;
        }
        double r = nd.p;
        if (heat == 0) {
          int out = 0;
          for (int j = lane; j < barred; j += 32) out |= s_barred[j] == nd.token;
          const bool gone = __any_sync(0xffffffffu, out) || !(total > 0.0);
          if (written && !gone) {
            const int tile = nd.token / kTile;
            r = (double)peer(s_r + tile / S * kTile + (nd.token - tile * kTile), tile % S);
          }
          r = gone ? 0.0 : r / total;
        }
        const bool sure = nd.q < 0.0;
        if ((double)nd.u * (sure ? 1.0 : nd.q) < r) {
          if (lane == 0) s_path[len] = next;
          ++len;
          cur = next;
          barred = written = 0;
          total = 1.0;
        } else if (heat == 0 && !sure) {
          child = next;
        } else if (heat == 0 && r > 0.0) {
          if (lane == 0) s_barred[barred] = nd.token;
          ++barred;
          total -= r * total;
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
      }
    }
    // (no block changes s_r while the walk of another may still look into it)
    if (S > 1)
      cluster_sync();
    else
      __syncthreads();
    if (s_act != kUpdate) break;

    // ---- r becomes max(r - q, 0), written down
    if constexpr (ELD > 0) {
      const int cur = s_cur, d = draft_of(s_child), barred = s_n_barred, written = s_written;
      const RowStats st = p.stats[lo + cur], sd = p.stats[p.rows.T + d];
      const float sc = (float)(kLog2e / target_heat(cur)), scd = (float)(kLog2e / heat_at(p.draft.temperature, d));
      const float inv = (float)(1.0 / ((written ? 1.0 : st.z) * s_total)), inv_d = (float)(1.0 / sd.z);
      const char *row = target_row(cur), *row_d = p.draft.at + (size_t)d * p.draft.ld;
      double sum = 0.0;
      for (int t0 = rank * kTile, at = 0; t0 < V; t0 += S * kTile, at += kTile) {
        float x[8], y[8];
        load8<ELD, VEC>(row_d, t0, V, -CUDART_INF_F, y);
        if (!written) load8<ELT, VEC>(row, t0, V, -CUDART_INF_F, x);
        float part = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int i = element<VEC>(t0, k);
          float r = written ? s_r[at + i - t0] : ex2(fmaf(x[k], sc, (float)-st.m));
          for (int j = 0; j < barred; ++j)
            if (s_barred[j] == i) r = 0.f;
          r = fmaxf(fmaf(r, inv, -ex2(fmaf(y[k], scd, (float)-sd.m)) * inv_d), 0.f);
          s_r[at + i - t0] = r;
          part += r;
        }
        sum += (double)part;
      }
      sum = cluster_total(sum, s, S);
      if (tid == 0) {   // (nothing left, by rounding alone: the target's own)
        s_written = sum > 0.0;
        s_total = sum > 0.0 ? sum : 1.0;
        s_n_barred = 0;
      }
      __syncthreads();
    }
  }

  // ---- the token behind the path
  const int act = s_act, cur = s_cur, barred = s_n_barred, written = s_written;
  const RowStats st = p.stats[lo + cur];
  const char* noise = reinterpret_cast<const char*>(p.noise + (size_t)e * p.noise_ld);
  const float* noise_f = reinterpret_cast<const float*>(noise);
  auto is_barred = [&](int i) {
    for (int j = 0; j < barred; ++j)
      if (s_barred[j] == i) return true;
    return false;
  };
  int token = act == kEnd ? st.arg : -1;
  bool bad = false;
  if (act == kDrawRest || (act == kDraw && written)) {
    const bool less = ELD > 0 && act == kDrawRest;   // a last child's q comes off on the way
    const int d = less ? draft_of(s_child) : 0;
    RowStats sd = {1.0, 0, 0};
    double sdd = 0.0;
    const char* row_d = nullptr;
    if (less) {
      sd = p.stats[p.rows.T + d];
      sdd = (double)(float)(kLog2e / heat_at(p.draft.temperature, d));
      row_d = p.draft.at + (size_t)d * p.draft.ld;
    }
    const double st_s = (double)(float)(kLog2e / target_heat(cur)), all = (written ? 1.0 : st.z) * s_total;
    const float sc = (float)st_s, scd = (float)sdd, inv = (float)(1.0 / all), inv_d = (float)(1.0 / sd.z);
    const char* row = target_row(cur);
    float top = -CUDART_INF_F;
    int win = -1;
    for (int t0 = rank * kTile, at = 0; t0 < V; t0 += S * kTile, at += kTile) {
      float x[8], y[8], z[8];
      load8<4, VEC>(noise, t0, V, 1.f, z);
      if constexpr (ELD > 0) {
        if (less) load8<ELD, VEC>(row_d, t0, V, -CUDART_INF_F, y);
      }
      if (!written) load8<ELT, VEC>(row, t0, V, -CUDART_INF_F, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = element<VEC>(t0, k);
        float r = (written ? s_r[at + i - t0] : ex2(fmaf(x[k], sc, (float)-st.m))) * inv;
        if (less) r = r - ex2(fmaf(y[k], scd, (float)-sd.m)) * inv_d;
        const float key = lg2(r) - lg2(z[k]);   // (NaN for what is not positive)
        if (i < V && r > 0.f && key > top && !is_barred(i)) {
          top = key;
          win = i;
        }
      }
    }
    token = cluster_winner(top, win, bad, [&](int i) {
      const int tile = i / kTile;
      double r = written ? (double)s_r[tile / S * kTile + (i - tile * kTile)] : exp2((double)logit(row, ELT, i) * st_s - st.m);
      r /= all;
      if constexpr (ELD > 0)
        if (less) r -= exp2((double)logit(row_d, ELD, i) * sdd - sd.m) / sd.z;
      return log2(fmax(r, 0.0)) - log2((double)noise_f[i]);
    }, s, S);
  }
  // (a rest that rounding left nothing of: the target's own)
  if (token < 0 && (act == kDraw || act == kDrawRest)) {
    const bool rest = act == kDraw && !written;
    token = race<ELT, VEC>(target_row(cur), noise, V, target_heat(cur), bad, [&](int i) { return rest && is_barred(i); }, s, S);
    if (token < 0 && rest && barred > 0)
      token = race<ELT, VEC>(target_row(cur), noise, V, target_heat(cur), bad, [](int) { return false; }, s, S);
  }
  const bool none = token < 0 || bad;
  if (rank == 0) {
    const int len = none ? 0 : s_len;
    for (int j = tid; j < p.max_path; j += kThreads) path[j] = j < len ? s_path[j] : -1;
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

// Blocks of a cluster: as many as keep the GPU's blocks within `most`, at least `least`, no
// more than a row has tiles.
int cluster_of(int64_t rows, int V, int most, int least) {
  int S = 1;
  const int tiles = (V + kTile - 1) / kTile;
  while (S < 8 && (S < least || (rows * 2 * S <= most && 2 * S <= tiles))) S *= 2;
  return S;
}

template <typename K, typename... A>
cudaError_t launch_clusters(K* kernel, int64_t rows, int S, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * S));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {(unsigned)S, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int kBlocks = 152 * 8;   // blocks that the GPU holds at once
constexpr size_t kRestMost = sizeof(float) * kTile * (kVocabMost / 8 / kTile);

template <int ELT, int ELD, bool VEC>
cudaError_t verify_as(const VerifyParams& p, cudaStream_t st) {
  const int rows = p.rows.T + (ELD ? p.draft.rows : 0);
  const int S = cluster_of(rows, p.V, kBlocks, 1);
  cudaError_t e = cudaSuccess;
  if (rows > 0)
    e = launch_clusters(row_stats_kernel<ELT, ELD ? ELD : 4, VEC>, rows, S, 0, st, p, p.rows.T, S);
  if (e != cudaSuccess) return e;
  const int tiles = (p.V + kTile - 1) / kTile, most = (int)(kRestMost / sizeof(float) / kTile);
  const int W = cluster_of(p.rows.n_seq, p.V, kBlocks / 4, (tiles + most - 1) / most);
  const size_t smem = ELD ? sizeof(float) * kTile * ((tiles + W - 1) / W) : 0;
  return launch_clusters(verify_kernel<ELT, ELD, VEC>, p.rows.n_seq, W, smem, st, p, W);
}

template <int ELT, int ELD>
cudaError_t verify_by_rows(const VerifyParams& p, cudaStream_t st) {
  const bool vec = vector_rows(p.target) && (!ELD || vector_rows(p.draft)) && vector_rows(p.noise, p.noise_ld * 4);
  return vec ? verify_as<ELT, ELD, true>(p, st) : verify_as<ELT, ELD, false>(p, st);
}

template <int ELT>
cudaError_t verify_by_draft(const VerifyParams& p, cudaStream_t st) {
  return !p.draft.at ? verify_by_rows<ELT, 0>(p, st) : p.draft.el == 4 ? verify_by_rows<ELT, 4>(p, st)
                                                                       : verify_by_rows<ELT, 2>(p, st);
}

template <int ELT, int ELD>
cudaError_t raise_smem() {
  const cudaError_t e = cudaFuncSetAttribute(verify_kernel<ELT, ELD, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kRestMost);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(verify_kernel<ELT, ELD, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRestMost);
}

template <int EL>
cudaError_t sample_as(const SampleParams& p, cudaStream_t st) {
  const int S = cluster_of(p.T, p.V, kBlocks, 1);
  return vector_rows(p.logits) && vector_rows(p.noise, p.noise_ld)
             ? launch_clusters(sample_kernel<EL, true>, p.T, S, 0, st, p, S)
             : launch_clusters(sample_kernel<EL, false>, p.T, S, 0, st, p, S);
}

}  // namespace

cudaError_t configure_verify() {
  cudaError_t e = raise_smem<2, 2>();
  if (e == cudaSuccess) e = raise_smem<2, 4>();
  if (e == cudaSuccess) e = raise_smem<4, 2>();
  if (e == cudaSuccess) e = raise_smem<4, 4>();
  return e;
}

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t st) {
  return p.target.el == 4 ? verify_by_draft<4>(p, st) : verify_by_draft<2>(p, st);
}

cudaError_t launch_sample(const SampleParams& p, cudaStream_t st) {
  return p.logits.el == 4 ? sample_as<4>(p, st) : sample_as<2>(p, st);
}

}  // namespace dflash
