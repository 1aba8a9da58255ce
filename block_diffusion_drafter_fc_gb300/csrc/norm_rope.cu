// Norm of every query and key head and its rotation in one pass, and the gradient.
//
//   n = x / sqrt(mean(x^2) + eps) over a head's dims, y = R(p) (w * n), R the rotation of
//   rope.cu (dims from rotary_dim on keep w * n).
//   With g = R(p)^T dy:  dw = sum over rows and heads of g * n,  dn = g * w,
//   dx = (dn - n mean(dn * n)) / sqrt(mean(x^2) + eps).
//
// A head lies with 2 to 16 neighbouring lanes (an item of two vectors each, rope.cuh), so
// its sums are shuffles and every value is read and written once: bytes at the copy rate
// are the floor.  All arithmetic is fp32; y and dx are rounded once, to their type.
#include "rope.cuh"

namespace dflash {

using namespace rope;

namespace {

// Row `t`'s item `it`: its part, head's bytes and place in the head.
struct Where {
  int part, i;
  size_t head;   // bytes from the row's start
};
DF_DEVICE Where where(const NormRopeParams& p, int it, int li, int hd_bytes) {
  const int h = it >> li, k = h >= p.part[0].heads;
  return {k, it - (h << li), (size_t)(h - (k ? p.part[0].heads : 0)) * hd_bytes};
}

template <int EL, int VB, int U>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p,
                                                             int rows_per_block, int span, uint32_t width_magic) {
  using V = typename Vec<VB>::T;
  constexpr int E = VB / EL;
  extern __shared__ float2 cs[];   // [rows][rd / 2]
  __shared__ int s_pos[kMaxRows];
  pdl_trigger();
  pdl_wait();
  const int ipr = p.hd / (2 * E), li = __ffs(ipr) - 1, half = p.r.rd / 2, hb = p.hd * EL;
  const int items = (p.part[0].heads + p.part[1].heads) * ipr;
  const Span sp = U == 1 ? block_span(p.T, rows_per_block, items, span, blockIdx.x, blockIdx.y)
                         : block_span(p.T, rows_per_block, items, items, blockIdx.x, 0);
  const int width = sp.it1 - sp.it0, total = sp.n_rows * width;
  V v[2][U][2], w[2][2];
  auto load = [&](int g0, V (&x)[U][2]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + threadIdx.x + u * kThreads;
      if (g >= total) continue;
      const int r = small_quotient(g, width_magic);
      const Where at = where(p, sp.it0 + g - r * width, li, hb);
      int o0, o1;
      item_offsets<E>(p.r, at.i, o0, o1);
      const NormRopePart& q = p.part[at.part];
      const char* src = q.x + (size_t)(sp.row0 + r) * q.x_ld + at.head;
      x[u][0] = *reinterpret_cast<const V*>(src + o0 * EL);
      x[u][1] = *reinterpret_cast<const V*>(src + o1 * EL);
    }
  };
  load(0, v[0]);
  {   // (a thread's items are all at the same place of their heads)
    int o0, o1;
    item_offsets<E>(p.r, (sp.it0 + (int)threadIdx.x) & (ipr - 1), o0, o1);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (p.part[k].heads) {
        w[k][0] = *reinterpret_cast<const V*>(p.part[k].w + o0 * EL);
        w[k][1] = *reinterpret_cast<const V*>(p.part[k].w + o1 * EL);
      }
  }
  if (threadIdx.x < sp.n_rows) {
    const int q = p.pos[sp.row0 + threadIdx.x];
    s_pos[threadIdx.x] = q;
    if (q < 0 && blockIdx.y == 0) set_status(p.status, DEV_BAD_POSITION);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < sp.n_rows * half; e += kThreads) {
    const int r = e / half;
    cs[e] = angle(p.r, s_pos[r], e - r * half, false);
  }
  __syncthreads();
  auto store = [&](int g0, V (&x)[U][2]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + threadIdx.x + u * kThreads;
      float f[2 * E], y[2 * E];
      unpack<EL, VB>(x[u][0], f);
      unpack<EL, VB>(x[u][1], f + E);
      norm_head<E>(f, ipr, p.per_dim, p.eps);   // (all lanes)
      if (g >= total) continue;
      const int r = small_quotient(g, width_magic);
      if (s_pos[r] < 0) continue;
      const Where at = where(p, sp.it0 + g - r * width, li, hb);
      unpack<EL, VB>(at.part ? w[1][0] : w[0][0], y);
      unpack<EL, VB>(at.part ? w[1][1] : w[0][1], y + E);
#pragma unroll
      for (int e = 0; e < 2 * E; ++e) f[e] *= y[e];
      int o0, o1;
      if (item_offsets<E>(p.r, at.i, o0, o1)) turn<E>(f, cs + r * half + at.i * E, p.r.interleaved);
      const NormRopePart& q = p.part[at.part];
      char* dst = q.out + (size_t)(sp.row0 + r) * q.out_ld + at.head;
      *reinterpret_cast<V*>(dst + o0 * EL) = pack<EL, VB>(f);
      *reinterpret_cast<V*>(dst + o1 * EL) = pack<EL, VB>(f + E);
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

// Rows [T b / G, T (b + 1) / G) of block b of G, `rows` at a time (the table of their angles
// fills the dynamic shared memory).  The weights' gradients stay in registers: a thread's
// items are all at the same place of their heads; at the end the block adds up its threads'
// in order and leaves them for norm_rope_sums_kernel.
template <int EL, int VB>
__global__ void __launch_bounds__(kThreads) norm_rope_grad_kernel(const __grid_constant__ NormRopeParams p, int rows) {
  using V = typename Vec<VB>::T;
  constexpr int E = VB / EL;
  extern __shared__ float2 cs[];   // [rows][rd / 2]
  __shared__ int s_pos[kMaxRows];
  __shared__ float s_dw[kThreads / 32][128];
  pdl_trigger();
  pdl_wait();
  const int ipr = p.hd / (2 * E), li = __ffs(ipr) - 1, half = p.r.rd / 2, hb = p.hd * EL;
  const int items = (p.part[0].heads + p.part[1].heads) * ipr, G = gridDim.x;
  const int row1 = (int)((long long)p.T * (blockIdx.x + 1) / G);
  const int place = threadIdx.x & (ipr - 1);
  int o0, o1;
  const bool rot = item_offsets<E>(p.r, place, o0, o1);
  V w[2][2];
  float dw[2][2 * E];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (p.part[k].heads) {
      w[k][0] = *reinterpret_cast<const V*>(p.part[k].w + o0 * EL);
      w[k][1] = *reinterpret_cast<const V*>(p.part[k].w + o1 * EL);
    }
#pragma unroll
    for (int e = 0; e < 2 * E; ++e) dw[k][e] = 0.f;
  }
  V v[2][4];   // x and dy of the next item and of the one before it
  for (int row0 = (int)((long long)p.T * blockIdx.x / G); row0 < row1; row0 += rows) {
    const int n_rows = min(rows, row1 - row0), total = n_rows * items;
    auto load = [&](int g, V (&x)[4]) {
      if (g >= total) return;
      const int r = g / items;
      const Where at = where(p, g - r * items, li, hb);
      const NormRopePart& q = p.part[at.part];
      const char* src = q.x + (size_t)(row0 + r) * q.x_ld + at.head;
      const char* dy = q.dy + (size_t)(row0 + r) * q.dy_ld + at.head;
      x[0] = *reinterpret_cast<const V*>(src + o0 * EL);
      x[1] = *reinterpret_cast<const V*>(src + o1 * EL);
      x[2] = *reinterpret_cast<const V*>(dy + o0 * EL);
      x[3] = *reinterpret_cast<const V*>(dy + o1 * EL);
    };
    load(threadIdx.x, v[0]);
    __syncthreads();   // the last rows' angles have been read
    if (threadIdx.x < n_rows) {
      const int q = p.pos[row0 + threadIdx.x];
      s_pos[threadIdx.x] = q;
      if (q < 0) set_status(p.status, DEV_BAD_POSITION);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n_rows * half; e += kThreads) {
      const int r = e / half;
      cs[e] = angle(p.r, s_pos[r], e - r * half, true);
    }
    __syncthreads();
    auto step = [&](int g, V (&x)[4]) {
      const bool on = g < total;
      const int r = on ? g / items : 0;
      const Where at = where(p, on ? g - r * items : 0, li, hb);
      float n[2 * E], d[2 * E], y[2 * E];
      unpack<EL, VB>(x[0], n);
      unpack<EL, VB>(x[1], n + E);
      unpack<EL, VB>(x[2], d);
      unpack<EL, VB>(x[3], d + E);
      const float inv = norm_head<E>(n, ipr, p.per_dim, p.eps);
      if (rot) turn<E>(d, cs + r * half + place * E, p.r.interleaved);
      const bool used = on && s_pos[r] >= 0;
      if (used) {
        if (at.part) {
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) dw[1][e] = fmaf(d[e], n[e], dw[1][e]);
        } else {
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) dw[0][e] = fmaf(d[e], n[e], dw[0][e]);
        }
      }
      unpack<EL, VB>(at.part ? w[1][0] : w[0][0], y);
      unpack<EL, VB>(at.part ? w[1][1] : w[0][1], y + E);
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * E; ++e) {
        d[e] *= y[e];
        dot = fmaf(d[e], n[e], dot);
      }
      dot = head_sum(dot, ipr) * p.per_dim;   // (all lanes)
      if (!used) return;
#pragma unroll
      for (int e = 0; e < 2 * E; ++e) d[e] = inv * fmaf(-n[e], dot, d[e]);
      const NormRopePart& q = p.part[at.part];
      char* dst = q.out + (size_t)(row0 + r) * q.out_ld + at.head;
      *reinterpret_cast<V*>(dst + o0 * EL) = pack<EL, VB>(d);
      *reinterpret_cast<V*>(dst + o1 * EL) = pack<EL, VB>(d + E);
    };
    for (int g0 = 0; g0 < total; g0 += 2 * kThreads) {
      load(g0 + kThreads + threadIdx.x, v[1]);
      step(g0 + threadIdx.x, v[0]);
      if (g0 + kThreads >= total) break;
      load(g0 + 2 * kThreads + threadIdx.x, v[0]);
      step(g0 + kThreads + threadIdx.x, v[1]);
    }
  }
  // lanes at the same place of a head, then the warps in order
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!p.part[k].heads) continue;
#pragma unroll
    for (int e = 0; e < 2 * E; ++e)
      for (int o = ipr; o < 32; o <<= 1) dw[k][e] += __shfl_xor_sync(0xffffffffu, dw[k][e], o);
    __syncthreads();
    if ((threadIdx.x & 31) < ipr) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        s_dw[threadIdx.x >> 5][o0 + e] = dw[k][e];
        s_dw[threadIdx.x >> 5][o1 + e] = dw[k][E + e];
      }
    }
    __syncthreads();
    if (threadIdx.x < p.hd) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) sum += s_dw[i][threadIdx.x];
      p.sums[((size_t)blockIdx.x * 2 + k) * p.hd + threadIdx.x] = sum;
    }
  }
}

// The blocks' sums of the weights' gradients, each thread every eighth block's of a dim,
// the eight in order.  One block per part.
__global__ void __launch_bounds__(1024) norm_rope_sums_kernel(const __grid_constant__ NormRopeParams p, int blocks) {
  __shared__ float s[8][128];
  pdl_trigger();
  pdl_wait();
  const int k = blockIdx.x, d = threadIdx.x & 127, i0 = threadIdx.x >> 7;
  if (!p.part[k].heads) return;
  float sum = 0.f;
  if (d < p.hd)
#pragma unroll 8
    for (int i = i0; i < blocks; i += 8) sum += p.sums[((size_t)i * 2 + k) * p.hd + d];
  s[i0][d] = sum;
  __syncthreads();
  if (i0 == 0 && d < p.hd) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += s[i][d];
    p.part[k].dw[d] = sum;
  }
}

template <int EL, int VB>
cudaError_t norm_rope_as(const NormRopeParams& p, cudaStream_t st) {
  const int items = (p.part[0].heads + p.part[1].heads) * (p.hd / (2 * (VB / EL)));
  const Shape s = append_shape(p.T, items, p.r.rd);
  const dim3 grid(s.gx, s.gy);
  const uint32_t magic = append_magic(s, items);
  return s.u == 1 ? launch_dependent(norm_rope_kernel<EL, VB, 1>, grid, kThreads, s.smem, st, p, s.rows, s.span, magic)
                  : launch_dependent(norm_rope_kernel<EL, VB, 2>, grid, kThreads, s.smem, st, p, s.rows, s.span, magic);
}

template <int EL, int VB>
cudaError_t norm_rope_grad_as(const NormRopeParams& p, cudaStream_t st) {
  const int blocks = p.T < kNormBlocks ? p.T : kNormBlocks;
  const int rows = (p.T + blocks - 1) / blocks < kAppendRows ? (p.T + blocks - 1) / blocks : kAppendRows;
  const size_t smem = sizeof(float) * 2 * rows * (p.r.rd / 2);
  const cudaError_t e = launch_dependent(norm_rope_grad_kernel<EL, VB>, dim3(blocks), kThreads, smem, st, p, rows);
  if (e != cudaSuccess) return e;
  return launch_dependent(norm_rope_sums_kernel, dim3(2), 1024, 0, st, p, blocks);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t st) {
  if (p.el == 4) return norm_rope_as<4, 16>(p, st);
  return p.r.rd % 16 == 0 ? norm_rope_as<2, 16>(p, st) : norm_rope_as<2, 8>(p, st);
}

cudaError_t launch_norm_rope_grad(const NormRopeParams& p, cudaStream_t st) {
  if (p.el == 4) return norm_rope_grad_as<4, 16>(p, st);
  return p.r.rd % 16 == 0 ? norm_rope_grad_as<2, 16>(p, st) : norm_rope_grad_as<2, 8>(p, st);
}

}  // namespace dflash
