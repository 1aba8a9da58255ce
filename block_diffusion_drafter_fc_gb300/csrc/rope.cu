// Rotary positions, and the same fused with the write of keys and values into
// the cache pages.
//
// Pair (a, b) of a head at position p turns by t = p f_j: (a cos t - b sin t,
// b cos t + a sin t), times the layout's magnitude factor; the gradient turns
// by -t.  f_j arrives as turns per position scaled by 2^64 (an unsigned 64-bit
// integer): p f_j modulo 2^64 is then the exact fraction of a turn whatever the
// position, one integer multiply instead of an fp64 product and its range
// reduction, and sincospif sees an argument in [-1, 1).  The fraction is
// rounded to fp32 (2^-25 of a half turn: 1e-7 in cos and sin).
//
// Both kernels move every value once: bytes in + bytes out at the copy rate is
// the floor.  A block takes a run of items (an item: two vectors of 16 bytes,
// holding whole pairs) of one or more rows, issues all its loads, then fills
// the (cos, sin) table of its rows in shared memory - shared by the rows' heads
// - while they are in flight.  16381 rows x 20 heads of 128 f32: 52.5 us, 0.94 of the
// copy rate; append of 8192 rows of 32 + 8 + 8 bf16 heads: 38.8 us, 0.77.
#include "rope.cuh"

namespace dflash {

using namespace rope;

namespace {

template <int EL, int VB, int U>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeParams p, int rows_per_block, int span) {
  using V = typename Vec<VB>::T;
  constexpr int E = VB / EL;
  extern __shared__ float2 cs[];   // [rows][rd / 2]
  __shared__ int s_pos[kMaxRows];
  pdl_trigger();
  pdl_wait();
  const int ipr = p.hd / (2 * E), items = p.n_heads * ipr, half = p.r.rd / 2;
  const Span sp = block_span(p.T, rows_per_block, items, span, blockIdx.x, blockIdx.y);
  const int width = sp.it1 - sp.it0, total = sp.n_rows * width;
  if (threadIdx.x < sp.n_rows) {
    const int q = p.pos[sp.row0 + threadIdx.x];
    s_pos[threadIdx.x] = q;
    if (q < 0 && blockIdx.y == 0) set_status(p.status, DEV_BAD_POSITION);
  }
  V v0[U], v1[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int g = threadIdx.x + u * kThreads;
    if (g >= total) continue;
    const int r = g / width, it = sp.it0 + g - r * width, h = it / ipr;
    int o0, o1;
    item_offsets<E>(p.r, it - h * ipr, o0, o1);
    const char* src = p.x + (size_t)(sp.row0 + r) * p.x_ld + (size_t)h * p.hd * EL;
    v0[u] = *reinterpret_cast<const V*>(src + o0 * EL);
    v1[u] = *reinterpret_cast<const V*>(src + o1 * EL);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < sp.n_rows * half; e += kThreads) {
    const int r = e / half;
    cs[e] = angle(p.r, s_pos[r], e - r * half, p.backward);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int g = threadIdx.x + u * kThreads;
    if (g >= total) continue;
    const int r = g / width, it = sp.it0 + g - r * width, h = it / ipr, i = it - h * ipr;
    if (s_pos[r] < 0) continue;
    int o0, o1;
    if (item_offsets<E>(p.r, i, o0, o1)) turn<EL, VB>(v0[u], v1[u], cs + r * half + i * E, p.r.interleaved);
    char* dst = p.out + (size_t)(sp.row0 + r) * p.out_ld + (size_t)h * p.hd * EL;
    *reinterpret_cast<V*>(dst + o0 * EL) = v0[u];
    *reinterpret_cast<V*>(dst + o1 * EL) = v1[u];
  }
}

// Rows of q heads, then k heads, then v heads.  One warp per row finds the
// row's entry (the number of range starts at or below it: ranges ascend) and the
// page of its slot: five dependent loads, which a block makes for all of its rows
// at once while its first values are in flight.  Then the block streams its
// items, U a thread, the next U in flight while the last are turned and written.
// NORM: every q and k head is divided by its root mean square and multiplied by the
// weights before it is turned, in registers: its lanes hold it whole.  8192 rows of 32 + 8 +
// 8 heads: 56 us (without norms 39).
template <int EL, int VB, int U, bool NORM>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendParams p, int rows_per_block, int span,
                                                          uint32_t width_magic) {
  using V = typename Vec<VB>::T;
  constexpr int E = VB / EL;
  extern __shared__ float2 cs[];
  __shared__ int s_pos[kMaxRows];       // -1: the row does nothing
  __shared__ long long s_dst[kMaxRows]; // its slot's row of (layer, k, head 0), -1: not written
  pdl_trigger();
  pdl_wait();
  const CacheView& c = p.c;
  const int ipr = c.hd / (2 * E), li = __ffs(ipr) - 1, half = p.r.rd / 2;   // (ipr is a power of two)
  const int hq = p.q ? c.n_head : 0, heads = hq + 2 * c.n_head_kv, items = heads * ipr;
  // (a large call's block has all items of its rows: append_shape; the constants save 1 us of 40 there)
  const Span sp = U == 1 ? block_span(p.rows.T, rows_per_block, items, span, blockIdx.x, blockIdx.y)
                         : block_span(p.rows.T, rows_per_block, items, items, blockIdx.x, 0);
  const int width = sp.it1 - sp.it0, total = sp.n_rows * width;
  V v[2][U][2];
  auto load = [&](int g0, V (&x)[U][2]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + threadIdx.x + u * kThreads;
      if (g >= total) continue;
      const int r = small_quotient(g, width_magic), it = sp.it0 + g - r * width, h = it >> li;
      int o0, o1;
      item_offsets<E>(p.r, it - (h << li), o0, o1);
      const size_t t = sp.row0 + r;
      const char* src = h < hq ? p.q + t * p.q_ld + (size_t)h * c.hd * EL
                        : h < hq + c.n_head_kv ? p.k + t * p.k_ld + (size_t)(h - hq) * c.hd * EL
                                               : p.v + t * p.v_ld + (size_t)(h - hq - c.n_head_kv) * c.hd * EL;
      x[u][0] = *reinterpret_cast<const V*>(src + o0 * EL);
      x[u][1] = *reinterpret_cast<const V*>(src + o1 * EL);
    }
  };
  load(0, v[0]);
  // (a thread's items are all at the same place of their heads: kThreads and a row's items
  // are multiples of a head's)
  V wq[2], wk[2];
  if constexpr (NORM) {
    int o0, o1;
    item_offsets<E>(p.r, (sp.it0 + (int)threadIdx.x) & (ipr - 1), o0, o1);
    const char* nq = hq ? p.q_norm : p.k_norm;
    wq[0] = *reinterpret_cast<const V*>(nq + o0 * EL);
    wq[1] = *reinterpret_cast<const V*>(nq + o1 * EL);
    wk[0] = *reinterpret_cast<const V*>(p.k_norm + o0 * EL);
    wk[1] = *reinterpret_cast<const V*>(p.k_norm + o1 * EL);
  }
  const int lane = threadIdx.x & 31;
  const bool first = blockIdx.y == 0 && lane == 0;   // one report per row
  for (int r = threadIdx.x >> 5; r < sp.n_rows; r += kThreads / 32) {
    const int t = sp.row0 + r;
    int below = 0;
    for (int i = lane; i <= p.rows.n_seq; i += 32) below += p.rows.row_start[i] <= t;
    below = __reduce_add_sync(0xffffffffu, below);
    const int s = below - 1;
    int pos = -1;
    long long dst = -1;
    int lo = 0, n = 0;
    if (s >= 0 && s < p.rows.n_seq && entry_rows(p.rows, s, lo, n) && t >= lo && t < lo + n) {
      const int q = entry_sequence(p.rows, s, c.max_seq);
      int dup = 0;
      if (p.rows.seqs && q >= 0)
        for (int i = lane; i < s; i += 32) dup |= p.rows.seqs[i] == q;
      const bool twice = __any_sync(0xffffffffu, dup);
      const int len = q >= 0 ? c.length[q] : -1;
      if (q < 0 || twice) {
        if (first) set_status(c.status, DEV_BAD_SEQ);
      } else if (len < 0) {
        if (first) set_status(c.status, DEV_BAD_ROWS);
      } else {
        const long long at = (long long)len + (p.depth ? p.depth[t] : t - lo);
        if (at < 0 || at > 0x7fffffffLL) {
          if (first) set_status(c.status, DEV_BAD_POSITION);
        } else {
          pos = (int)at;
          const long long slot = (long long)len + (t - lo), idx = slot >> c.ps_log2;
          const int page = idx < c.max_pages ? c.table[(size_t)q * c.max_pages + idx] : -1;
          if (page >= 0 && page < c.n_pages && c.refs[page] <= 1)
            dst = (long long)page_row(c, page, p.layer, 0, 0, (int)(slot & (c.ps - 1)));
          else if (first)
            set_status(c.status, DEV_BAD_PAGE);
        }
      }
    }
    if (lane == 0) {
      s_pos[r] = pos;
      s_dst[r] = dst;
    }
  }
  // ranges that are no ranges are reported once
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int s = threadIdx.x; s < p.rows.n_seq; s += kThreads) {
      int lo, n;
      if (!entry_rows(p.rows, s, lo, n)) set_status(c.status, DEV_BAD_ROWS);
    }
  __syncthreads();
  for (int e = threadIdx.x; e < sp.n_rows * half; e += kThreads) {
    const int r = e / half;
    cs[e] = angle(p.r, s_pos[r], e - r * half, false);
  }
  __syncthreads();
  const size_t head_bytes = (size_t)c.ps * c.hd * EL;   // one (page, layer, k|v, head)
  auto store = [&](int g0, V (&x)[U][2]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + threadIdx.x + u * kThreads;
      float f[2 * E];
      if constexpr (NORM) {   // (with all lanes: a head's may be the last ones of a warp)
        unpack<EL, VB>(x[u][0], f);
        unpack<EL, VB>(x[u][1], f + E);
        norm_head<E>(f, ipr, p.per_dim, p.eps);
      }
      if (g >= total) continue;
      const int r = small_quotient(g, width_magic), it = sp.it0 + g - r * width, h = it >> li, i = it - (h << li);
      if (s_pos[r] < 0) continue;
      int o0, o1;
      const bool rot = item_offsets<E>(p.r, i, o0, o1);
      if constexpr (NORM) {
        if (h < hq + c.n_head_kv) {
          float w[2 * E];
          unpack<EL, VB>(h < hq ? wq[0] : wk[0], w);
          unpack<EL, VB>(h < hq ? wq[1] : wk[1], w + E);
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) f[e] *= w[e];
          if (rot) turn<E>(f, cs + r * half + i * E, p.r.interleaved);
          x[u][0] = pack<EL, VB>(f);
          x[u][1] = pack<EL, VB>(f + E);
        }
      } else if (rot && h < hq + c.n_head_kv) {
        turn<EL, VB>(x[u][0], x[u][1], cs + r * half + i * E, p.r.interleaved);
      }
      char* dst;
      if (h < hq) {
        dst = p.q_out + (size_t)(sp.row0 + r) * p.q_out_ld + (size_t)h * c.hd * EL;
      } else {
        if (s_dst[r] < 0) continue;
        dst = c.pages + s_dst[r] + (h - hq) * head_bytes;   // v follows the k heads
      }
      *reinterpret_cast<V*>(dst + o0 * EL) = x[u][0];
      *reinterpret_cast<V*>(dst + o1 * EL) = x[u][1];
    }
  };
  constexpr int kStep = U * kThreads;
  for (int g0 = 0; g0 < total; g0 += 2 * kStep) {
    if (g0 + kStep < total) load(g0 + kStep, v[1]);
    store(g0, v[0]);
    if (g0 + kStep >= total) break;
    if (g0 + 2 * kStep < total) load(g0 + 2 * kStep, v[0]);
    store(g0 + kStep, v[1]);
  }
}

template <int EL, int VB>
cudaError_t rope_as(const RopeParams& p, cudaStream_t st) {
  const Shape s = shape_of(p.T, p.n_heads * (p.hd / (2 * (VB / EL))), p.r.rd);
  const dim3 grid(s.gx, s.gy);
  return s.u == 4 ? launch_dependent(rope_kernel<EL, VB, 4>, grid, kThreads, s.smem, st, p, s.rows, s.span)
                  : launch_dependent(rope_kernel<EL, VB, 1>, grid, kThreads, s.smem, st, p, s.rows, s.span);
}

template <int EL, int VB, bool NORM>
cudaError_t append_as(const AppendParams& p, cudaStream_t st) {
  const int heads = (p.q ? p.c.n_head : 0) + 2 * p.c.n_head_kv, items = heads * (p.c.hd / (2 * (VB / EL)));
  const Shape s = append_shape(p.rows.T, items, p.r.rd);
  const dim3 grid(s.gx, s.gy);
  const uint32_t magic = append_magic(s, items);
  return s.u == 1 ? launch_dependent(append_kernel<EL, VB, 1, NORM>, grid, kThreads, s.smem, st, p, s.rows, s.span, magic)
                  : launch_dependent(append_kernel<EL, VB, 2, NORM>, grid, kThreads, s.smem, st, p, s.rows, s.span, magic);
}

}  // namespace

// 16-byte vectors hold whole pairs when rd is a multiple of two of them (16
// bf16 or 8 f32 dims); a bf16 rotary_dim that is an odd multiple of 8 takes
// 8-byte vectors.
cudaError_t launch_rope(const RopeParams& p, cudaStream_t st) {
  if (p.el == 4) return rope_as<4, 16>(p, st);
  return p.r.rd % 16 == 0 ? rope_as<2, 16>(p, st) : rope_as<2, 8>(p, st);
}

template <bool NORM>
static cudaError_t append_by_type(const AppendParams& p, cudaStream_t st) {
  if (p.c.el == 4) return append_as<4, 16, NORM>(p, st);
  return p.r.rd % 16 == 0 ? append_as<2, 16, NORM>(p, st) : append_as<2, 8, NORM>(p, st);
}

cudaError_t launch_append(const AppendParams& p, cudaStream_t st) {
  return p.k_norm ? append_by_type<true>(p, st) : append_by_type<false>(p, st);
}

}  // namespace dflash
