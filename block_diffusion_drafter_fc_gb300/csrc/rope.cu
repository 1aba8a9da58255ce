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
  extern __shared__ __align__(16) float2 cs[];   // [rows][rd / 2]
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
    cs[r * half + pair_at<E, true>(e - r * half, p.r.rd)] = angle(p.r, s_pos[r], e - r * half, p.backward);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int g = threadIdx.x + u * kThreads;
    if (g >= total) continue;
    const int r = g / width, it = sp.it0 + g - r * width, h = it / ipr, i = it - h * ipr;
    if (s_pos[r] < 0) continue;
    int o0, o1;
    if (item_offsets<E>(p.r, i, o0, o1)) turn<EL, VB, true>(v0[u], v1[u], cs + r * half, i, p.r);
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
template <int EL, int VB, int U>
__global__ void __launch_bounds__(kThreads, U == 2 ? 4 : 0) append_kernel(AppendParams p, int rows_per_block, int span,
                                                          uint32_t width_magic) {
  using V = typename Vec<VB>::T;
  constexpr int E = VB / EL;
  extern __shared__ __align__(16) float2 cs[];
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
  const int lane = threadIdx.x & 31;
  const bool first = blockIdx.y == 0 && lane == 0;   // one report per row
  for (int r = threadIdx.x >> 5; r < sp.n_rows; r += kThreads / 32) {
    const int t = sp.row0 + r;
    int pos;
    long long dst;
    append_row(p, t, lane, first, pos, dst);
    if (lane == 0) {
      s_pos[r] = pos;
      s_dst[r] = dst;
    }
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) report_ranges(p.rows, c.status);
  __syncthreads();
  for (int e = threadIdx.x; e < sp.n_rows * half; e += kThreads) {
    const int r = e / half;
    cs[r * half + pair_at<E, false>(e - r * half, p.r.rd)] = angle(p.r, s_pos[r], e - r * half, false);
  }
  __syncthreads();
  const size_t head_bytes = (size_t)c.ps * c.hd * EL;   // one (page, layer, k|v, head)
  auto store = [&](int g0, V (&x)[U][2]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + threadIdx.x + u * kThreads;
      if (g >= total) continue;
      const int r = small_quotient(g, width_magic), it = sp.it0 + g - r * width, h = it >> li, i = it - (h << li);
      if (s_pos[r] < 0) continue;
      int o0, o1;
      const bool rot = item_offsets<E>(p.r, i, o0, o1);
      if (rot && h < hq + c.n_head_kv) turn<EL, VB, false>(x[u][0], x[u][1], cs + r * half, i, p.r);
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

template <int EL, int VB>
cudaError_t append_as(const AppendParams& p, cudaStream_t st) {
  const int heads = (p.q ? p.c.n_head : 0) + 2 * p.c.n_head_kv, items = heads * (p.c.hd / (2 * (VB / EL)));
  const Shape s = append_shape(p.rows.T, items, p.r.rd);
  const dim3 grid(s.gx, s.gy);
  const uint32_t magic = append_magic(s, items);
  return s.u == 1 ? launch_dependent(append_kernel<EL, VB, 1>, grid, kThreads, s.smem, st, p, s.rows, s.span, magic)
                  : launch_dependent(append_kernel<EL, VB, 2>, grid, kThreads, s.smem, st, p, s.rows, s.span, magic);
}

}  // namespace

// 16-byte vectors hold whole pairs when rd is a multiple of two of them (16
// bf16 or 8 f32 dims); a bf16 rotary_dim that is an odd multiple of 8 takes
// 8-byte vectors.
cudaError_t launch_rope(const RopeParams& p, cudaStream_t st) {
  if (p.el == 4) return rope_as<4, 16>(p, st);
  return p.r.rd % 16 == 0 ? rope_as<2, 16>(p, st) : rope_as<2, 8>(p, st);
}

cudaError_t launch_append(const AppendParams& p, cudaStream_t st) {
  if (p.k_norm) return launch_norm_append(p, st);
  if (p.c.el == 4) return append_as<4, 16>(p, st);
  return p.r.rd % 16 == 0 ? append_as<2, 16>(p, st) : append_as<2, 8>(p, st);
}

}  // namespace dflash
