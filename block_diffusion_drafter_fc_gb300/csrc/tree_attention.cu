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
// Streaming kernel, here for bf16 heads of 32 (tree_attention_umma.cu has the
// larger bf16 heads, tree_attention_f32.cu f32).  The call's work is one list of
// units (a tile of 16 or 32 rows of one kv head's query group x a chunk of slots),
// cut into equal ranges, one per resident block, so that one long sequence is
// spread over the whole GPU and many short ones are balanced; a tile cut by ranges
// leaves partial rows in scratch, which a second, dependent launch joins in block
// order (a warp per row: joining in the tile's last block took 40 of 78 us for a
// 16-node chain over 2048 slots).  K and V chunks come through a ring of
// shared-memory stages (TMA, one box per page and 128 bytes of a row), across
// tiles; four warps each take a quarter of a chunk's slots for all rows of the
// tile, with their own m, l and sums (no exchange until the tile ends), on
// mma.sync.  Warp 0 also refills the stage of the chunk before the current one.
// A chunk of 64 slots of 32 dims is too short a product to feed tcgen05 for, and
// the bound is the latency of its steps.
//
// Products of bf16 operands are exact in fp32; the weights are split into bf16
// hi + lo (2^-17), which costs one more mma per tile and is free here.
#include "tree_stream.cuh"

namespace dflash {

using namespace tree;

namespace {

DF_DEVICE void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
DF_DEVICE void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
template <int HD, int MT, typename E>
__global__ void __launch_bounds__(kThreads, 2) attend_stream_kernel(const __grid_constant__ StreamParams p) {
  constexpr int EL = 2;
  using G = Geo<EL, HD>;
  constexpr int TR = 16 * MT;                 // rows of a tile
  constexpr int NV = HD / 8;                  // 8-wide column blocks of the output
  constexpr int kQ = TR * G::kRowB;           // bytes of Q
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int S = p.stages;
  uint8_t* s_q = sm + S * G::kHalf;
  float* s_o = reinterpret_cast<float*>(s_q + kQ);    // two 16 x HD tiles
  float2* s_ml = reinterpret_cast<float2*>(s_o + 2 * 16 * HD);            // [2][16]
  uint64_t* full = reinterpret_cast<uint64_t*>(s_ml + 32);
  uint64_t* empty = full + S;
  long long* s_warp = reinterpret_cast<long long*>(empty + S);            // [8]
  long long* s_end = s_warp + 8;
  const int entries = E::count(p.a);
  E* s_e = reinterpret_cast<E*>(s_end + entries);
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
  const long long U = s_end[entries - 1];
  // fewer blocks than launched where their shares would get too small
  const int Gr = blocks_used(U, gridDim.x, kMinUnits), b = blockIdx.x;
  Cut d = {0, 0, 0, 0, -1, 0};
  if (b >= Gr || U == 0) {
    if (tid == 0) p.cuts[b] = d;
    return;
  }
  const long long ub0 = range_begin(U, Gr, b), ub1 = range_begin(U, Gr, b + 1);
  const int s_first = find_entry(s_end, entries, ub0);
  const int grp = p.a.grp;

  Copies<EL, HD, E> cp;
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
    const E x = s_e[g.s];
    const int rows = min(TR, x.n * grp - g.row0), end = x.len + x.nodes();
    const int all = x.len + (p.a.mask || !x.nodes() ? 0 : g.row0 / grp + 1);   // slots that all rows see
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
      *reinterpret_cast<uint4*>(d) = v;
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
      const int slot0 = x.base() + ch * G::CS + warp * G::WS;
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
      __syncwarp();
      if (lane == 0 && !s_abort) bar_arrive(&empty[it % S]);
      ++it;
      // ---- what a row does not attend to
      if (slot0 + G::WS > all) {
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
          const bool last_word = whole && x.alone();
          if (E::kParts && last_word && qd == 0) {
            const int node = (g.row0 + r) / grp;
            p.a.row_ml[part_row(p.a, x.pass(), x.lo + node, g.kvh * grp + g.row0 + r - node * grp)] = make_float2(0.f, kDone);
          }
          if (last_word) {
            const float inv = l[t][hf] > 0.f ? 1.f / l[t][hf] : 0.f;
            char* dst;
            float* lse;
            out_row(r, dst, lse);
            if (lse && qd == 0) *lse = l[t][hf] > 0.f ? (m[t][hf] + log2f(l[t][hf])) * kLn2 : -CUDART_INF_F;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
              const float a = o[t][j][hf * 2] * inv, bb = o[t][j][hf * 2 + 1] * inv;
              *reinterpret_cast<uint32_t*>(dst + (j * 8 + qd * 2) * 2) = pack_bf16x2(a, bb);
            }
          } else {
            const int node = (g.row0 + r) / grp;
            const size_t at = E::kParts && whole ? part_row(p.a, x.pass(), x.lo + node, g.kvh * grp + g.row0 + r - node * grp)
                                                 : (size_t)slot * TR + r;
            float* po = (E::kParts && whole ? p.a.row_o : p.part_o) + at * HD;
            if (qd == 0) (E::kParts && whole ? p.a.row_ml : p.part_ml)[at] = make_float2(m[t][hf], l[t][hf]);
            if (E::kParts && !whole && g.c0 == 0 && qd == 0)   // the cut tile's first block tells where its parts are
              p.a.row_ml[part_row(p.a, x.pass(), x.lo + node, g.kvh * grp + g.row0 + r - node * grp)] =
                  parts_at(b, block_of(U, Gr, g.u0 + (long long)(g.nch - 1) * g.w), slot, r);
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

template <int HD, int MT, typename E>
size_t fixed_smem(int entries) {
  return 1024 + 16 * MT * HD * 2 + 2 * 16 * HD * 4 + 32 * 8 + 8 * 8 +
         (size_t)entries * (sizeof(long long) + sizeof(E));
}

template <int HD, int MT, typename E>
cudaError_t stream_as(const AttendParams& a, const AttendWork& w, cudaStream_t st) {
  size_t smem;
  const StreamParams p = stream_params<2, HD>(a, w, 16 * MT, fixed_smem<HD, MT, E>(a.n_group + a.rows.n_seq), smem);
  const cudaError_t e = launch_dependent(attend_stream_kernel<HD, MT, E>, dim3(2 * w.sms), kThreads, smem, st, p);
  if (e != cudaSuccess) return e;
  return launch_join<2, HD, E>(a, w, 16 * MT, 2 * w.sms, st);
}

template <int HD, int MT, typename E>
cudaError_t raise_smem() {
  return cudaFuncSetAttribute(attend_stream_kernel<HD, MT, E>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemTwo);
}

}  // namespace

bool attend_on_umma(int el, int hd) { return el == 2 && hd >= 64; }

int attend_chunk(int el, int hd) { return attend_on_umma(el, hd) ? 128 : el == 2 ? 64 : 32; }

// two parts per block: 256-row tiles, one block per SM, or 32-row tiles, two
size_t attend_part_rows(int el, int hd) { return 2 * (size_t)kAttendSms * (attend_on_umma(el, hd) ? 256 : 2 * 32); }

cudaError_t configure_attend() {
  cudaError_t e = configure_attend_umma();
  if (e == cudaSuccess) e = configure_attend_f32();
  if (e == cudaSuccess) e = raise_smem<32, 1, Entry>();
  if (e == cudaSuccess) e = raise_smem<32, 2, Entry>();
  if (e == cudaSuccess) e = raise_smem<32, 1, PartEntry>();
  if (e == cudaSuccess) e = raise_smem<32, 2, PartEntry>();
  return e;
}

cudaError_t launch_attend(const AttendParams& a, const AttendWork& w, cudaStream_t st) {
  if (a.c.el == 4) return launch_attend_f32(a, w, st);
  if (attend_on_umma(a.c.el, a.c.hd)) return launch_attend_umma(a, w, st);
  // 32-row tiles once a call has entries (groups) of more than 16 rows per kv head
  if (a.n_group)
    return (long long)a.rows.T * a.grp <= 16 ? stream_as<32, 1, PartEntry>(a, w, st) : stream_as<32, 2, PartEntry>(a, w, st);
  const long long rows = (long long)a.max_tree * a.grp;
  return rows <= 16 ? stream_as<32, 1, Entry>(a, w, st) : stream_as<32, 2, Entry>(a, w, st);
}

}  // namespace dflash
