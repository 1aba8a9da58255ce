// Tree attention with f32 storage, on the fp32 units.
//
// Streaming kernel as in tree_attention.cu (the same ring, ranges of work and
// join; chunks of 32 slots, four warps, a quarter of a chunk's slots each, a fifth
// warp for the copies), with both products as fp32 multiply-adds from shared
// memory: exact products, fp32 sums, pairs of them by fma.rn.f32x2.  Why not
// mma.sync with operands split into tf32 hi + lo and three products: m16n8k8
// keeps a scheduler busy for 32 clocks, so that leaves 43 products a clock and SM
// of the fp32 units' 128 (238 us against 145 for four trees of 9..33 nodes over
// 1000..4100 slots, 32 / 8 heads of 128).
//
// Tiles have 16 rows whatever a tree's size: a tile of 48 rows (12 warps, one
// block per SM) reads a page's rows a third as often, but was no faster at 48
// rows per kv head (79.5 us against 78.7), slower at 20 (75 against 57) and 64
// (134 against 100) and gained only at 132 (197 against 207).  Two blocks per SM:
// with three, 128 registers a thread spill (16 rows 45 us against 37).
//
// Bound: up to a tile of rows by the latency of its chunks (16 rows over the
// slots above 37 us, their pages' bytes 12), beyond it by shared memory: a lane's
// 4 x 4 products with K take 8 reads of 16 bytes for 64 multiply-adds, 4 x 2 over
// all of head_dim would take 12 (198 us).
//
// A lane's share.  Scores: 4 rows x 4 slots over a quarter of head_dim, then one
// of those rows with the four quarters added up.  Values: 8 neighbouring rows (4
// where head_dim is 32) and every sixteenth (eighth) 16-byte piece of a slot's
// row, the warp's weights through shared memory.  Eight neighbouring lanes read
// eight different pieces of the swizzled tiles: no bank conflicts.
#include "tree_stream.cuh"

namespace dflash {

using namespace tree;

namespace {

DF_DEVICE uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
DF_DEVICE float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
DF_DEVICE void fma2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
DF_DEVICE uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

DF_DEVICE void lds(uint64_t& a, uint64_t& b, uint32_t at) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(at));
}

// the warps that compute
template <int N>
DF_DEVICE void sync_tile() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

constexpr int kPad = 16;   // floats between slots of a warp's weights

constexpr int TR = 16;                       // rows of a tile
constexpr int kAll = kThreads + 32;          // one warp more copies
constexpr int kPerSm = 2;                    // blocks per SM

template <int HD>
__global__ void __launch_bounds__(kAll, kPerSm) attend_f32_kernel(const __grid_constant__ StreamParams p) {
  using G = Geo<4, HD>;
  constexpr int NS = G::WS / 2;                 // slots of a lane in the products with K (x 4 rows)
  constexpr int DG = HD == 32 ? 8 : 16;         // lanes along head_dim in the product with V
  constexpr int NX = HD / (4 * DG);             // 16-byte pieces of a lane
  constexpr int PR = DG / 2;                    // rows of a lane
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int S = p.stages;
  uint8_t* s_q = sm + S * G::kHalf;
  float* s_w = reinterpret_cast<float*>(s_q + TR * G::kRowB);           // [4 warps][8 slots][kPad]
  float* s_fade = s_w + kConsumers * G::WS * kPad;                 // [4][16]
  float2* s_ml = reinterpret_cast<float2*>(s_fade + kConsumers * 16);   // [4][TR]
  uint64_t* full = reinterpret_cast<uint64_t*>(s_ml + kConsumers * TR);
  uint64_t* empty = full + S;
  long long* s_warp = reinterpret_cast<long long*>(empty + S);          // [16]
  long long* s_end = s_warp + 16;
  Entry* s_e = reinterpret_cast<Entry*>(s_end + p.a.rows.n_seq);
  float* s_o = reinterpret_cast<float*>(s_q);   // [TR][HD], once the tile's scores are done
  __shared__ volatile int s_abort;

  const CacheView& c = p.a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      bar_init(&full[i], 1);
      bar_init(&empty[i], kConsumers);
    }
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_trigger();
  pdl_wait();
  plan_entries(p.a, cutting<4>(TR), s_e, s_end, s_warp, kAll, blockIdx.x == 0);
  __syncthreads();
  const long long U = s_end[p.a.rows.n_seq - 1];
  const int Gr = blocks_used(U, gridDim.x, kMinUnits), b = blockIdx.x;
  Cut d = {0, 0, 0, 0, -1, 0};
  if (b >= Gr || U == 0) {
    if (tid == 0) p.cuts[b] = d;
    return;
  }
  const long long ub0 = range_begin(U, Gr, b), ub1 = range_begin(U, Gr, b + 1);
  const int s_first = find_entry(s_end, p.a.rows.n_seq, ub0);
  const int grp = p.a.grp;
  if (warp == kConsumers) {
    Copies<4, HD> cp;
    cp.u = ub0;
    cp.s = s_first;
    cp.open(p, s_e, s_end, ub1, TR);
    while (cp.more) cp.issue(p, sm, full, empty, s_e, s_end, ub1, TR, &s_abort);
    cp.drain(S, full);
    return;
  }

  // scores: quarter kg of each 16 floats of head_dim, rows r0 + (j & 1) + 8 (j >> 1), slots sg + 2 i;
  // softmax: row rs
  const int kg = lane & 3, r0 = 4 * ((lane >> 2) & 1) + 2 * ((lane >> 3) & 1), sg = lane >> 4;
  const int rs = r0 + (kg >> 1) + 8 * (kg & 1);
  const int pr = PR * (lane / DG), dg = lane % DG;    // values: rows pr ..
  float* w = s_w + warp * G::WS * kPad;               // [slot][row]
  // Offsets of a lane's first pieces in the swizzled tiles (rows of 8 pieces); its
  // next piece is 4 on, the other half of the same 128 bytes.
  uint32_t at_q[2], at_k[4];   // (slots sg + 2 i and sg + 2 i + 8 alike)
#pragma unroll
  for (int j = 0; j < 2; ++j) at_q[j] = su32(s_q) + (r0 + j) * 128 + ((kg ^ ((r0 + j) & 7)) << 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) at_k[i] = su32(sm) + (warp * G::WS + sg + 2 * i) * 128 + ((kg ^ (sg + 2 * i)) << 4);
  const uint32_t at_v = su32(sm) + warp * G::WS * 128 + (dg >> 3) * G::CS * 128;
  float* fades = s_fade + warp * 16;                  // [row]
  const float scale = p.a.scale * kLog2e;
  long long u = ub0;
  int s = s_first, st = 0, ph = 0;   // the ring's next stage, its phase
  auto step = [&] {
    if (++st == S) st = 0, ph ^= 1;
  };
  Segment g;
  while (next_segment(p.a, cutting<4>(TR), s_e, s_end, u, ub1, s, g)) {
    const Entry x = s_e[g.s];
    const int rows = min(TR, x.n * grp - g.row0), end = x.len + x.n;
    const int all = x.len + (p.a.mask ? 0 : g.row0 / grp + 1);   // slots that all rows see
    sync_tile<kThreads>();   // the previous tile's sums have been read
    for (int i = tid; i < TR * (G::kRowB / 16); i += kThreads) {
      const int r = i / (G::kRowB / 16), pc = i - r * (G::kRowB / 16);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int node = (g.row0 + r) / grp, h = g.kvh * grp + (g.row0 + r) - node * grp;
        v = *reinterpret_cast<const uint4*>(p.a.q + (size_t)(x.lo + node) * p.a.q_ld + (size_t)h * G::kRowB + pc * 16);
      }
      *reinterpret_cast<uint4*>(s_q + swz<G::kRowB>(TR, r, pc)) = v;
    }
    sync_tile<kThreads>();
    uint64_t o[PR][NX][2];
    float m = -CUDART_INF_F, l = 0.f;
    const int node = (g.row0 + rs) / grp;
#pragma unroll
    for (int r = 0; r < PR; ++r)
#pragma unroll
      for (int k = 0; k < NX; ++k) o[r][k][0] = o[r][k][1] = 0;

    for (int ch = g.c0; ch < g.c1; ++ch) {
      const int slot0 = ch * G::CS + warp * G::WS;
      // ---- scores
      bar_wait(&full[st], (uint32_t)ph, &s_abort, c.status);
      uint64_t acc[4][NS];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < NS; ++i) acc[j][i] = 0;
      const uint32_t kb = st * G::kHalf;
#pragma unroll
      for (int x = 0; x < HD / 16; ++x) {
        uint64_t kv[NS][2];
#pragma unroll
        for (int i = 0; i < NS; ++i)
          lds(kv[i][0], kv[i][1], ((kb + at_k[i & 3]) ^ ((x & 1) * 64)) + (i >> 2) * 1024 + (x >> 1) * G::CS * 128);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint64_t q0, q1;
          lds(q0, q1, (at_q[j & 1] ^ ((x & 1) * 64)) + (j >> 1) * 1024 + (x >> 1) * TR * 128);
#pragma unroll
          for (int i = 0; i < NS; ++i) fma2(acc[j][i], q0, kv[i][0]);
#pragma unroll
          for (int i = 0; i < NS; ++i) fma2(acc[j][i], q1, kv[i][1]);
        }
      }
      __syncwarp();
      if (lane == 0 && !s_abort) bar_arrive(&empty[st]);
      step();
      // ---- what a row does not attend to; running maximum, weights
      const bool masked = slot0 + G::WS > all;
      float sc[NS], top = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        // the quarters' sums: half of the rows to the neighbour, then half of the rest
        float y[4], z[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = unpack2(acc[j][i]);
          y[j] = f.x + f.y;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
          z[j] = (kg & 1 ? y[j + 2] : y[j]) + __shfl_xor_sync(0xffffffffu, kg & 1 ? y[j] : y[j + 2], 1);
        sc[i] = (kg & 2 ? z[1] : z[0]) + __shfl_xor_sync(0xffffffffu, kg & 2 ? z[0] : z[1], 2);
        if (masked) {
          const int slot = slot0 + sg + 2 * i, at = slot - x.len;
          bool sees = slot < end;
          if (sees && at >= 0 && rs < rows)
            sees = p.a.mask ? (p.a.mask[(size_t)(x.lo + node) * p.a.words + (at >> 5)] >> (at & 31)) & 1 : at <= node;
          if (!sees) sc[i] = -CUDART_INF_F;
        }
        top = fmaxf(top, sc[i]);
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
      const float mn = fmaxf(m, top * scale);
      const float use = mn == -CUDART_INF_F ? 0.f : mn;   // nothing attended yet
      const float fade = ex2(m - use);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const float y = ex2(fmaf(sc[i], scale, -use));
        sum += y;
        w[(sg + 2 * i) * kPad + rs] = y;
      }
      l = l * fade + sum;
      if (sg == 0) fades[rs] = fade;
      const bool faded = __any_sync(0xffffffffu, mn != m);
      m = mn;
      __syncwarp();
      // ---- values: rows pr .. pr + PR - 1, pieces dg + DG k
      if (faded)
#pragma unroll
        for (int r = 0; r < PR; ++r) {
          const uint64_t f = pack2(fades[pr + r], fades[pr + r]);
#pragma unroll
          for (int k = 0; k < NX; ++k) {
            o[r][k][0] = mul2(o[r][k][0], f);
            o[r][k][1] = mul2(o[r][k][1], f);
          }
        }
      bar_wait(&full[st], (uint32_t)ph, &s_abort, c.status);
      const uint32_t vb = at_v + st * G::kHalf;
      // (slots past the last node may hold anything: 0 x NaN is NaN)
      const int ns = min(G::WS, end - slot0);
#pragma unroll
      for (int i = 0; i < G::WS; ++i) {
        if (i >= ns) break;
        uint64_t v[NX][2];
#pragma unroll
        for (int k = 0; k < NX; ++k) lds(v[k][0], v[k][1], vb + i * 128 + (((dg & 7) ^ i) << 4) + k * (DG / 8) * G::CS * 128);
        float ys[PR];
#pragma unroll
        for (int r = 0; r < PR; r += 4) *reinterpret_cast<float4*>(ys + r) = *reinterpret_cast<const float4*>(w + i * kPad + pr + r);
#pragma unroll
        for (int r = 0; r < PR; ++r) {
          const uint64_t f = pack2(ys[r], ys[r]);
#pragma unroll
          for (int k = 0; k < NX; ++k) {
            fma2(o[r][k][0], f, v[k][0]);
            fma2(o[r][k][1], f, v[k][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0 && !s_abort) bar_arrive(&empty[st]);
      step();
    }

    // ---- the four warps' parts of the tile, added up in warp order
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    if (sg == 0) s_ml[warp * TR + rs] = make_float2(m, l);
    const bool whole = g.c0 == 0 && g.c1 == g.nch;
    sync_tile<kThreads>();   // (and every warp is done with Q)
    float wt[PR];      // this warp's weight in its lanes' rows
#pragma unroll
    for (int r = 0; r < PR; ++r) {
      float top = -CUDART_INF_F, sum = 0.f;
#pragma unroll
      for (int k = 0; k < kConsumers; ++k) top = fmaxf(top, s_ml[k * TR + pr + r].x);
      const float use = top == -CUDART_INF_F ? 0.f : top;
#pragma unroll
      for (int k = 0; k < kConsumers; ++k) {
        const float2 y = s_ml[k * TR + pr + r];
        sum += ex2(y.x - use) * y.y;
      }
      wt[r] = ex2(s_ml[warp * TR + pr + r].x - use) * (!whole ? 1.f : sum > 0.f ? 1.f / sum : 0.f);
    }
#pragma unroll 1
    for (int k0 = 0; k0 < kConsumers; ++k0) {
      if (warp == k0)
#pragma unroll
        for (int r = 0; r < PR; ++r)
#pragma unroll
          for (int k = 0; k < NX; ++k) {
            float4* at = reinterpret_cast<float4*>(s_o + (pr + r) * HD + (dg + DG * k) * 4);
            const float2 f0 = unpack2(o[r][k][0]), f1 = unpack2(o[r][k][1]);
            float4 y = k0 ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
            y.x += f0.x * wt[r];
            y.y += f0.y * wt[r];
            y.z += f1.x * wt[r];
            y.w += f1.y * wt[r];
            *at = y;
          }
      sync_tile<kThreads>();
    }
    // this block's partial rows: slot 0 if its range starts in the tile, else 1
    const int slot = 2 * b + (ub0 >= g.u0 ? 0 : 1);
    for (int i = tid; i < rows * (HD / 4); i += kThreads) {
      const int r = i / (HD / 4), pc = i - r * (HD / 4);
      const float4 y = *reinterpret_cast<const float4*>(s_o + r * HD + pc * 4);
      const int node = (g.row0 + r) / grp, h = g.kvh * grp + (g.row0 + r) - node * grp;
      if (whole)
        *reinterpret_cast<float4*>(p.a.out + (size_t)(x.lo + node) * p.a.out_ld + (size_t)h * G::kRowB + pc * 16) = y;
      else
        *reinterpret_cast<float4*>(p.part_o + ((size_t)slot * TR + r) * HD + pc * 4) = y;
      if (pc) continue;
      float top = -CUDART_INF_F, sum = 0.f;
      for (int k = 0; k < kConsumers; ++k) top = fmaxf(top, s_ml[k * TR + r].x);
      const float use = top == -CUDART_INF_F ? 0.f : top;
      for (int k = 0; k < kConsumers; ++k) sum += ex2(s_ml[k * TR + r].x - use) * s_ml[k * TR + r].y;
      if (!whole)
        p.part_ml[(size_t)slot * TR + r] = make_float2(top, sum);
      else if (p.a.lse)
        p.a.lse[(size_t)(x.lo + node) * c.n_head + h] = sum > 0.f ? (top + log2f(sum)) * kLn2 : -CUDART_INF_F;
    }
    // the block with a cut tile's first chunk describes it to the join
    if (tid == 0 && g.c0 == 0 && !whole)
      d = {x.lo, g.row0, g.kvh, rows, block_of(U, Gr, g.u0 + (long long)(g.nch - 1) * g.w), slot};
  }
  if (tid == 0) p.cuts[b] = d;
}

template <int HD>
size_t fixed_smem(int n_seq) {
  return 1024 + TR * HD * 4 + kConsumers * (Geo<4, HD>::WS * kPad + 16) * 4 + kConsumers * TR * 8 + 16 * 8 +
         (size_t)n_seq * (sizeof(long long) + sizeof(Entry));
}

template <int HD>
cudaError_t f32_as(const AttendParams& a, const AttendWork& w, cudaStream_t st) {
  size_t smem;
  const StreamParams p = stream_params<4, HD>(a, w, TR, fixed_smem<HD>(a.rows.n_seq), smem);
  const cudaError_t e = launch_dependent(attend_f32_kernel<HD>, dim3(kPerSm * w.sms), kAll, smem, st, p);
  if (e != cudaSuccess) return e;
  return launch_join<4, HD>(a, w, TR, kPerSm * w.sms, st);
}

template <int HD>
cudaError_t raise_smem() {
  return cudaFuncSetAttribute(attend_f32_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemTwo);
}

}  // namespace

cudaError_t configure_attend_f32() {
  cudaError_t e = raise_smem<32>();
  if (e == cudaSuccess) e = raise_smem<64>();
  if (e == cudaSuccess) e = raise_smem<128>();
  return e;
}

cudaError_t launch_attend_f32(const AttendParams& a, const AttendWork& w, cudaStream_t st) {
  return a.c.hd == 32 ? f32_as<32>(a, w, st) : a.c.hd == 64 ? f32_as<64>(a, w, st) : f32_as<128>(a, w, st);
}

}  // namespace dflash
