// Attention of the rows of a call (tree nodes, a causal chain, single tokens)
// over their sequences' cache pages.
//
//   out[t][h] = sum_p w_p V[p],  w = softmax over the attended slots p of
//   scale q[t][h] . K[p];  lse[t][h] = ln sum_p exp(scale q[t][h] . K[p]).
//
// One pass over the slots with a running maximum m and sum l: a new score s
// changes them to m' = max(m, s), l' = l e^(m-m') + e^(s-m'), and the weighted
// sum of values likewise.  Parts of a row's slots join the same way.
//
// Streaming kernel, for calls with few rows per kv head (decoding, small trees)
// and for f32 storage: the bound is the read of the pages.  The call's work is
// one list of units (a tile of 16 or 32 rows of one kv head's query group x a
// chunk of slots), cut into equal ranges, one per resident block, so that one
// long sequence is spread over the whole GPU and many short ones are balanced;
// a tile cut by ranges leaves partial rows in scratch, which a second, dependent
// launch joins in block order (a warp per row: joining in the tile's last block
// took 40 of 78 us for a 16-node chain over 2048 slots).  K and V chunks come through a ring of shared-memory
// stages (TMA, one box per page and 128 bytes of a row), across tiles; four
// warps each take a quarter of a chunk's slots for all rows of the tile, with
// their own m, l and sums (no exchange until the tile ends), on mma.sync.  Warp
// 0 also refills the stage of the chunk before the current one: a fifth, copying
// warp would leave the others 168 registers instead of 255 (two blocks per SM),
// and the 32-row tiles spill at that.
//
// bf16: products of bf16 operands are exact in fp32; the weights are split
// into bf16 hi + lo (2^-17), which costs one more mma per tile and is free
// here.  f32: every operand is split into tf32 hi + lo and three products are
// kept (2^-21 of a product's size).
#include "tree_common.cuh"

namespace dflash {

using namespace tree;

namespace {

constexpr int kConsumers = 4;
constexpr int kThreads = 32 * kConsumers;
constexpr int kMinUnits = 3;   // a block's least share of a call's units

template <int EL, int HD>
struct Geo {
  static constexpr int CS = EL == 2 ? 64 : 32;            // slots of a chunk
  static constexpr int WS = CS / kConsumers;              // slots of a warp
  static constexpr int kRowB = HD * EL;                   // bytes of a row
  static constexpr int kBoxB = kRowB < 128 ? kRowB : 128; // bytes of a row within a box
  static constexpr int kBoxes = kRowB / kBoxB;
  static constexpr int kHalf = CS * kRowB;                // bytes of a K or V chunk
};

// Offset of 16-byte piece `c` of row r in a block of `rows` rows as the copies
// lay it out: boxes of 128-byte (64-byte) rows, swizzled.
template <int RowB>
DF_DEVICE int swz(int rows, int r, int c) {
  if constexpr (RowB >= 128)
    return (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  else
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

DF_DEVICE void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
DF_DEVICE void ldsm2(uint32_t (&r)[2], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}
DF_DEVICE void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
DF_DEVICE void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo with both in tf32 (11 significant bits each)
DF_DEVICE void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
}

// every chunk one unit, a tile two besides
template <int EL>
DF_DEVICE Cutting cutting(int tile) {
  return {tile, Geo<EL, 64>::CS, 0, 1, 1, 2};
}

struct StreamParams {
  CUtensorMap tm;     // pages as [rows of (page, layer, k|v, head)][page_size][hd]
  AttendParams a;
  float* part_o;      // [2 blocks][rows of a tile][hd]
  float2* part_ml;    // [2 blocks][rows of a tile] (maximum in powers of two, sum)
  Cut* cuts;          // [blocks]
  int stages, box_rows;
};

// The copies of a block's chunks, run ahead of their use by one warp: K, then V
// of every chunk of every segment.
template <int EL, int HD>
struct Copies {
  using G = Geo<EL, HD>;
  long long u;
  int s, it = 0, ch = 0, kv = 0;
  int base = 0, row = 0;    // lane i holds the tensor row of page base + i
  bool more = false;
  Segment g;

  DF_DEVICE void open(const StreamParams& p, const Entry* e, const long long* end, long long u1, int tile) {
    more = next_segment(p.a, cutting<EL>(tile), e, end, u, u1, s, g);
    ch = g.c0;
    base = -64;
  }
  DF_DEVICE void issue(const StreamParams& p, uint8_t* sm, uint64_t* full, uint64_t* empty, const Entry* e,
                       const long long* end, long long u1, int tile, volatile int* abort) {
    if (!more) return;
    const CacheView& c = p.a.c;
    const int lane = threadIdx.x & 31, S = p.stages, st = it % S;
    const int none = c.n_pages * c.n_layer * 2 * c.n_head_kv;   // past the tensor: reads as zero
    if (kv == 0 && ((ch * G::CS + G::CS - 1) >> c.ps_log2) > base + 31) {
      const Entry x = e[g.s];
      base = (ch * G::CS) >> c.ps_log2;
      row = none;
      if (base + lane <= (x.len + x.n - 1) >> c.ps_log2) {
        const int t = c.table[(size_t)x.q * c.max_pages + base + lane];
        if (t >= 0 && t < c.n_pages)
          row = (t * c.n_layer + p.a.layer) * 2 * c.n_head_kv + g.kvh;
        else
          set_status(c.status, DEV_BAD_PAGE);
      }
    }
    int stop = 0;
    if (lane == 0) {
      bar_wait(&empty[st], (uint32_t)((it / S) & 1) ^ 1, abort, c.status);
      stop = *abort;
      if (!stop) bar_expect(&full[st], G::kHalf);
    }
    if (__shfl_sync(0xffffffffu, stop, 0)) {
      more = false;
      return;
    }
    uint8_t* dst = sm + st * G::kHalf;
    for (int i = 0; i < G::CS; i += p.box_rows) {
      const int slot = ch * G::CS + i;
      const int r = __shfl_sync(0xffffffffu, row, ((slot >> c.ps_log2) - base) & 31);
      if (lane == 0)
#pragma unroll
        for (int x4 = 0; x4 < G::kBoxes; ++x4)
          tma3d(dst + x4 * G::CS * G::kBoxB + i * G::kBoxB, &p.tm, x4 * (G::kBoxB / EL), slot & (c.ps - 1),
                r == none ? none : r + kv * c.n_head_kv, &full[st]);
    }
    ++it;
    if (kv ^= 1) return;
    if (++ch == g.c1) open(p, e, end, u1, tile);
  }
  // no copy may still be landing when the block ends
  DF_DEVICE void drain(int S, uint64_t* full) {
    if ((threadIdx.x & 31) == 0)
      for (int j = max(0, it - S); j < it; ++j) {
        const long long t0 = clock64();
        while (!bar_try(&full[j % S], (uint32_t)((j / S) & 1)) && clock64() - t0 < kWait) {
        }
      }
  }
};

template <int EL, int HD, int MT>
__global__ void __launch_bounds__(kThreads, 2) attend_stream_kernel(const __grid_constant__ StreamParams p) {
  using G = Geo<EL, HD>;
  constexpr int TR = 16 * MT;                 // rows of a tile
  constexpr int NV = HD / 8;                  // 8-wide column blocks of the output
  constexpr int kQ = TR * G::kRowB;           // bytes of Q (f32: hi, then lo)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int S = p.stages;
  uint8_t* s_q = sm + S * G::kHalf;
  float* s_o = reinterpret_cast<float*>(s_q + (EL == 4 ? 2 : 1) * kQ);    // two 16 x HD tiles
  float2* s_ml = reinterpret_cast<float2*>(s_o + 2 * 16 * HD);            // [2][16]
  uint64_t* full = reinterpret_cast<uint64_t*>(s_ml + 32);
  uint64_t* empty = full + S;
  long long* s_warp = reinterpret_cast<long long*>(empty + S);            // [8]
  long long* s_end = s_warp + 8;
  Entry* s_e = reinterpret_cast<Entry*>(s_end + p.a.rows.n_seq);
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
  plan_entries(p.a, cutting<EL>(TR), s_e, s_end, s_warp, kThreads, blockIdx.x == 0);
  __syncthreads();
  const long long U = s_end[p.a.rows.n_seq - 1];
  // fewer blocks than launched where their shares would get too small
  const int Gr = blocks_used(U, gridDim.x, kMinUnits), b = blockIdx.x;
  Cut d = {0, 0, 0, 0, -1, 0};
  if (b >= Gr || U == 0) {
    if (tid == 0) p.cuts[b] = d;
    return;
  }
  const long long ub0 = range_begin(U, Gr, b), ub1 = range_begin(U, Gr, b + 1);
  const int s_first = find_entry(s_end, p.a.rows.n_seq, ub0);
  const int grp = c.n_head / c.n_head_kv;

  Copies<EL, HD> cp;
  cp.u = ub0;
  cp.s = s_first;
  if (warp == 0) {
    cp.open(p, s_e, s_end, ub1, TR);
    for (int i = 0; i < S; ++i) cp.issue(p, sm, full, empty, s_e, s_end, ub1, TR, &s_abort);
  }

  // -------------------------------------------------------------------- rows
  const int gr = lane >> 2, qd = lane & 3;    // fragment row and column pair
  const float scale = p.a.scale * kLog2e;
  long long u = ub0;
  int s = s_first, it = 0;
  Segment g;
  while (next_segment(p.a, cutting<EL>(TR), s_e, s_end, u, ub1, s, g)) {
    const Entry x = s_e[g.s];
    const int rows = min(TR, x.n * grp - g.row0), end = x.len + x.n;
    // Q: row r is head kvh grp + (row0 + r) % grp of node (row0 + r) / grp
    __syncthreads();   // the previous tile's Q and sums have been read
    for (int i = tid; i < TR * (G::kRowB / 16); i += 32 * kConsumers) {
      const int r = i / (G::kRowB / 16), pc = i - r * (G::kRowB / 16);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int node = (g.row0 + r) / grp, h = g.kvh * grp + (g.row0 + r) - node * grp;
        v = *reinterpret_cast<const uint4*>(p.a.q + (size_t)(x.lo + node) * p.a.q_ld + (size_t)h * G::kRowB + pc * 16);
      }
      uint8_t* d = s_q + swz<G::kRowB>(TR, r, pc);
      if constexpr (EL == 2) {
        *reinterpret_cast<uint4*>(d) = v;
      } else {
        uint4 hi, lo;
        split_tf32(__uint_as_float(v.x), hi.x, lo.x);
        split_tf32(__uint_as_float(v.y), hi.y, lo.y);
        split_tf32(__uint_as_float(v.z), hi.z, lo.z);
        split_tf32(__uint_as_float(v.w), hi.w, lo.w);
        *reinterpret_cast<uint4*>(d) = hi;
        *reinterpret_cast<uint4*>(d + kQ) = lo;
      }
    }
    __syncthreads();
    float o[MT][NV][4], m[MT][2], l[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      m[t][0] = m[t][1] = -CUDART_INF_F;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[t][j][k] = 0.f;
    }
    constexpr int NS = G::WS / 8;             // 8-slot blocks of the warp's slots
    for (int ch = g.c0; ch < g.c1; ++ch) {
      const int slot0 = ch * G::CS + warp * G::WS;
      // ---- scores
      float sc[MT][NS][4];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[t][j][k] = 0.f;
      const uint8_t* kb = sm + (it % S) * G::kHalf;
      if (warp == 0 && it > 0) cp.issue(p, sm, full, empty, s_e, s_end, ub1, TR, &s_abort);
      bar_wait(&full[it % S], (uint32_t)((it / S) & 1), &s_abort, c.status);
      const uint32_t kbase = su32(kb), qbase = su32(s_q);
      if constexpr (EL == 2) {
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          uint32_t kf[4];   // (slots 0-7, k 0-7), (slots 0-7, k 8-15), (slots 8-15, ..)
          ldsm4(kf, kbase + swz<G::kRowB>(G::CS, warp * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            uint32_t qf[4];
            ldsm4(qf, qbase + swz<G::kRowB>(TR, t * 16 + (lane & 15), 2 * k + (lane >> 4)));
            mma_bf16_16816(sc[t][0], qf, kf[0], kf[1]);
            mma_bf16_16816(sc[t][1], qf, kf[2], kf[3]);
          }
        }
      } else {
#pragma unroll 4
        for (int k = 0; k < HD / 8; ++k) {
          uint32_t kf[2], kh[2], kl[2];
          ldsm2(kf, kbase + swz<G::kRowB>(G::CS, warp * 8 + (lane & 7), 2 * k + ((lane >> 3) & 1)));
          split_tf32(__uint_as_float(kf[0]), kh[0], kl[0]);
          split_tf32(__uint_as_float(kf[1]), kh[1], kl[1]);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            uint32_t qh[4], ql[4];
            const uint32_t qa = qbase + swz<G::kRowB>(TR, t * 16 + (lane & 15), 2 * k + (lane >> 4));
            ldsm4(qh, qa);
            ldsm4(ql, qa + kQ);
            mma_tf32(sc[t][0], ql, kh[0], kh[1]);
            mma_tf32(sc[t][0], qh, kl[0], kl[1]);
            mma_tf32(sc[t][0], qh, kh[0], kh[1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0 && !s_abort) bar_arrive(&empty[it % S]);
      ++it;
      // ---- what a row does not attend to
      if (slot0 + G::WS > x.len) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int r = t * 16 + hf * 8 + gr, node = (g.row0 + r) / grp;
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int slot = slot0 + j * 8 + qd * 2 + k, at = slot - x.len;
                bool sees = slot < end;
                if (sees && at >= 0 && r < rows)
                  sees = p.a.mask ? (p.a.mask[(size_t)(x.lo + node) * p.a.words + (at >> 5)] >> (at & 31)) & 1 : at <= node;
                if (!sees) sc[t][j][hf * 2 + k] = -CUDART_INF_F;
              }
          }
      }
      // ---- running maximum, weights
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float top = -CUDART_INF_F;
#pragma unroll
          for (int j = 0; j < NS; ++j) top = fmaxf(top, fmaxf(sc[t][j][hf * 2], sc[t][j][hf * 2 + 1]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)) * scale;
          const float mo = m[t][hf], mn = fmaxf(mo, top);
          const float use = mn == -CUDART_INF_F ? 0.f : mn;   // nothing attended yet
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float w = ex2(fmaf(sc[t][j][hf * 2 + k], scale, -use));
              sc[t][j][hf * 2 + k] = w;
              sum += w;
            }
          const float fade = ex2(mo - use);
          l[t][hf] = l[t][hf] * fade + sum;
          m[t][hf] = mn;
          if (__any_sync(0xffffffffu, mn != mo)) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
              o[t][j][hf * 2] *= fade;
              o[t][j][hf * 2 + 1] *= fade;
            }
          }
        }
      // ---- values
      const int st = it % S;
      if (warp == 0) cp.issue(p, sm, full, empty, s_e, s_end, ub1, TR, &s_abort);
      bar_wait(&full[st], (uint32_t)((it / S) & 1), &s_abort, c.status);
      uint8_t* vb = sm + st * G::kHalf;
      const uint32_t vbase = su32(vb);
      const bool ragged = slot0 + G::WS > end;
      if (ragged) {
        // slots past the last node may hold anything: 0 x NaN is NaN
        for (int i = lane; i < G::WS * (G::kRowB / 16); i += 32) {
          const int r = i / (G::kRowB / 16), pc = i - r * (G::kRowB / 16);
          if (slot0 + r >= end)
            *reinterpret_cast<uint4*>(vb + swz<G::kRowB>(G::CS, warp * G::WS + r, pc)) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      if constexpr (EL == 2) {
        uint32_t ph[MT][4], pl[MT][4];   // weights as the A operand: the score fragment's layout
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          split_bf16x2(sc[t][0][0], sc[t][0][1], ph[t][0], pl[t][0]);
          split_bf16x2(sc[t][0][2], sc[t][0][3], ph[t][1], pl[t][1]);
          split_bf16x2(sc[t][1][0], sc[t][1][1], ph[t][2], pl[t][2]);
          split_bf16x2(sc[t][1][2], sc[t][1][3], ph[t][3], pl[t][3]);
        }
#pragma unroll
        for (int j = 0; j < NV; j += 2) {
          uint32_t vf[4];   // (slots 0-7, dims j), (slots 8-15, dims j), (.., dims j + 1)
          ldsm4t(vf, vbase + swz<G::kRowB>(G::CS, warp * 16 + (lane & 15), j + (lane >> 4)));
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            mma_bf16_16816(o[t][j], pl[t], vf[0], vf[1]);
            mma_bf16_16816(o[t][j], ph[t], vf[0], vf[1]);
            mma_bf16_16816(o[t][j + 1], pl[t], vf[2], vf[3]);
            mma_bf16_16816(o[t][j + 1], ph[t], vf[2], vf[3]);
          }
        }
      } else {
        // k index t of the product is slot 2t, t + 4 is slot 2t + 1: the score
        // fragment is the A operand as it stands
        uint32_t ph[MT][4], pl[MT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          split_tf32(sc[t][0][0], ph[t][0], pl[t][0]);
          split_tf32(sc[t][0][2], ph[t][1], pl[t][1]);
          split_tf32(sc[t][0][1], ph[t][2], pl[t][2]);
          split_tf32(sc[t][0][3], ph[t][3], pl[t][3]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          uint32_t vh[2], vl[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int d = j * 8 + gr;
            const float v = *reinterpret_cast<const float*>(
                vb + swz<G::kRowB>(G::CS, warp * 8 + 2 * qd + k, d >> 2) + (d & 3) * 4);
            split_tf32(v, vh[k], vl[k]);
          }
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            mma_tf32(o[t][j], pl[t], vh[0], vh[1]);
            mma_tf32(o[t][j], ph[t], vl[0], vl[1]);
            mma_tf32(o[t][j], ph[t], vh[0], vh[1]);
          }
        }
      }
      if (ragged) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0 && !s_abort) bar_arrive(&empty[st]);
      ++it;
    }

    // ---- the four warps' parts: 2 and 3 into 0 and 1, then 1 into 0
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {   // the row's sum over its four lanes
        l[t][hf] += __shfl_xor_sync(0xffffffffu, l[t][hf], 1);
        l[t][hf] += __shfl_xor_sync(0xffffffffu, l[t][hf], 2);
      }
#pragma unroll
      for (int step = 2; step >= 1; step >>= 1) {
        __syncthreads();
        if (warp >= step && warp < 2 * step) {
          const int w = warp - step;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int r = hf * 8 + gr;
            if (qd == 0) s_ml[w * 16 + r] = make_float2(m[t][hf], l[t][hf]);
#pragma unroll
            for (int j = 0; j < NV; ++j)
              *reinterpret_cast<float2*>(s_o + (w * 16 + r) * HD + ((j ^ (r & (NV < 8 ? NV - 1 : 7))) * 8 + qd * 2)) =
                  make_float2(o[t][j][hf * 2], o[t][j][hf * 2 + 1]);
          }
        }
        __syncthreads();
        if (warp < step) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int r = hf * 8 + gr;
            const float2 x2 = s_ml[warp * 16 + r];
            const float mn = fmaxf(m[t][hf], x2.x), use = mn == -CUDART_INF_F ? 0.f : mn;
            const float fa = ex2(m[t][hf] - use), fb = ex2(x2.x - use);
            m[t][hf] = mn;
            l[t][hf] = l[t][hf] * fa + x2.y * fb;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
              const float2 v = *reinterpret_cast<const float2*>(s_o + (warp * 16 + r) * HD + ((j ^ (r & (NV < 8 ? NV - 1 : 7))) * 8 + qd * 2));
              o[t][j][hf * 2] = o[t][j][hf * 2] * fa + v.x * fb;
              o[t][j][hf * 2 + 1] = o[t][j][hf * 2 + 1] * fa + v.y * fb;
            }
          }
        }
      }
    }

    auto out_row = [&](int r, char*& dst, float*& lse) {
      const int node = (g.row0 + r) / grp, h = g.kvh * grp + (g.row0 + r) - node * grp;
      dst = p.a.out + (size_t)(x.lo + node) * p.a.out_ld + (size_t)h * G::kRowB;
      lse = p.a.lse ? p.a.lse + (size_t)(x.lo + node) * c.n_head + h : nullptr;
    };
    const bool whole = g.c0 == 0 && g.c1 == g.nch;
    // this block's partial rows: slot 0 if its range starts in the tile, else 1
    const int slot = 2 * b + (ub0 >= g.u0 ? 0 : 1);
    if (warp == 0) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int r = t * 16 + hf * 8 + gr;
          if (r >= rows) continue;
          if (whole) {
            const float inv = l[t][hf] > 0.f ? 1.f / l[t][hf] : 0.f;
            char* dst;
            float* lse;
            out_row(r, dst, lse);
            if (lse && qd == 0) *lse = l[t][hf] > 0.f ? (m[t][hf] + log2f(l[t][hf])) * kLn2 : -CUDART_INF_F;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
              const float a = o[t][j][hf * 2] * inv, bb = o[t][j][hf * 2 + 1] * inv;
              if constexpr (EL == 2)
                *reinterpret_cast<uint32_t*>(dst + (j * 8 + qd * 2) * 2) = pack_bf16x2(a, bb);
              else
                *reinterpret_cast<float2*>(dst + (j * 8 + qd * 2) * 4) = make_float2(a, bb);
            }
          } else {
            float* po = p.part_o + ((size_t)slot * TR + r) * HD;
            if (qd == 0) p.part_ml[(size_t)slot * TR + r] = make_float2(m[t][hf], l[t][hf]);
#pragma unroll
            for (int j = 0; j < NV; ++j)
              *reinterpret_cast<float2*>(po + j * 8 + qd * 2) = make_float2(o[t][j][hf * 2], o[t][j][hf * 2 + 1]);
          }
        }
    }
    // the block with a cut tile's first chunk describes it to the join
    if (tid == 0 && g.c0 == 0 && !whole) {
      d.lo = x.lo;
      d.row0 = g.row0;
      d.kvh = g.kvh;
      d.rows = rows;
      d.last = block_of(U, Gr, g.u0 + (long long)(g.nch - 1) * g.w);
      d.slot = slot;
    }
  }
  if (warp == 0) cp.drain(S, full);
  if (tid == 0) p.cuts[b] = d;
}

template <int EL, int HD, int MT>
size_t fixed_smem(int n_seq) {
  return 1024 + (EL == 4 ? 2 : 1) * 16 * MT * HD * EL + 2 * 16 * HD * 4 + 32 * 8 + 8 * 8 +
         (size_t)n_seq * (sizeof(long long) + sizeof(Entry));
}
constexpr size_t kSmemTwo = 114 * 1024 - 512;   // dynamic shared memory of a block, two blocks per SM
constexpr int kStagesMost = 12;

template <int EL, int HD, int MT>
cudaError_t stream_as(const AttendParams& a, const AttendWork& w, cudaStream_t st) {
  using G = Geo<EL, HD>;
  StreamParams p;
  p.tm = *w.tm;
  p.a = a;
  p.part_o = w.part_o;
  p.part_ml = w.part_ml;
  p.cuts = w.cuts;
  p.box_rows = a.c.ps < G::CS ? a.c.ps : G::CS;
  const size_t fixed = fixed_smem<EL, HD, MT>(a.rows.n_seq);
  p.stages = (int)((kSmemTwo - fixed) / (G::kHalf + 16));
  if (p.stages > kStagesMost) p.stages = kStagesMost;
  const size_t smem = fixed + (size_t)p.stages * (G::kHalf + 16);
  const cudaError_t e = launch_dependent(attend_stream_kernel<EL, HD, MT>, dim3(2 * w.sms), kThreads, smem, st, p);
  if (e != cudaSuccess) return e;
  return launch_join<EL, HD>(a, w, 16 * MT, 2 * w.sms, st);
}

template <int EL, int HD>
cudaError_t stream_hd(const AttendParams& a, const AttendWork& w, cudaStream_t st) {
  const long long rows = (long long)a.max_tree * (a.c.n_head / a.c.n_head_kv);
  return rows <= 16 ? stream_as<EL, HD, 1>(a, w, st) : stream_as<EL, HD, 2>(a, w, st);
}

template <int EL, int HD, int MT>
cudaError_t raise_smem() {
  return cudaFuncSetAttribute(attend_stream_kernel<EL, HD, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)kSmemTwo);
}

}  // namespace

bool attend_on_umma(int el, int hd) { return el == 2 && hd >= 64; }

int attend_chunk(int el, int hd) { return attend_on_umma(el, hd) ? 128 : el == 2 ? 64 : 32; }

// two parts per block: 256-row tiles, one block per SM, or 32-row tiles, two
size_t attend_part_rows(int el, int hd) { return 2 * (size_t)kAttendSms * (attend_on_umma(el, hd) ? 256 : 2 * 32); }

cudaError_t configure_attend() {
  cudaError_t e = configure_attend_umma();
  auto both = [&](cudaError_t x) { if (e == cudaSuccess) e = x; };
  both(raise_smem<2, 32, 1>());
  both(raise_smem<2, 32, 2>());
  both(raise_smem<4, 32, 1>());
  both(raise_smem<4, 32, 2>());
  both(raise_smem<4, 64, 1>());
  both(raise_smem<4, 64, 2>());
  both(raise_smem<4, 128, 1>());
  both(raise_smem<4, 128, 2>());
  return e;
}

cudaError_t launch_attend(const AttendParams& a, const AttendWork& w, cudaStream_t st) {
  if (attend_on_umma(a.c.el, a.c.hd)) return launch_attend_umma(a, w, st);
  if (a.c.el == 2) return stream_hd<2, 32>(a, w, st);
  return a.c.hd == 32 ? stream_hd<4, 32>(a, w, st) : a.c.hd == 64 ? stream_hd<4, 64>(a, w, st)
                                                                : stream_hd<4, 128>(a, w, st);
}

}  // namespace dflash
