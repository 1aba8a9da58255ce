// Norm of every query and key head and its rotation in one pass: of rows, fused with the
// append of keys and values to the cache, and the gradient.
//
//   n = x / sqrt(mean(x^2) + eps) over a head's dims, y = R(p) (w * n), R the rotation of
//   rope.cu (dims from rotary_dim on keep w * n).
//   With g = R(p)^T dy:  dw = sum over rows and heads of g * n,  dn = g * w,
//   dx = (dn - n mean(dn * n)) / sqrt(mean(x^2) + eps).
//
// Every value is read and written once: bytes at the copy rate are the floor.  All arithmetic
// is fp32; y and dx are rounded once, to their type.
//
// A head lies with 2 to 16 neighbouring lanes (an item of two vectors each, rope.cuh), so its
// sums are shuffles.  A thread owns an item of the row and walks down rows: its head, weights
// and addresses' steps do not change, and the next rows' loads are under way.  (Walking along
// a row's items instead, as the append of rope.cu does, took 370 instructions an item, 60% of
// the issue slots, and 46 us for the append of 8192 rows, 56 for the gradient of 8191; now 39
// and 51.5, 0.76 and 0.72 of the copy rate.)
#include "rope.cuh"

#include <algorithm>

namespace dflash {

using namespace rope;

namespace {

constexpr int kMost = norm::kThreads, kRows = norm::kMaxRows;
constexpr int kGradRows = 2 * kRows;   // a gradient's: an even number of rounds, whatever rows lie side by side

// Queries, keys and (of the append) values.
struct NormRows {
  RopeView r;
  int T, hd, heads[3];
  const char* x[3];
  const char* w[2];
  char* out[2];
  int64_t x_ld[3], out_ld[2];   // bytes
  float per_dim, eps;
  const int32_t* pos;
  unsigned* status;
  AppendParams a;               // of the append: rows, pages
};

// A row's angles: two pairs' cosines and sines (16 bytes) of every item, then of their next
// two, so that neighbouring lanes read neighbouring words.
template <int E>
DF_DEVICE void put_angle(float* row, const RopeView& r, int pos, int j, bool backward) {
  const int i = j / E, e = j - i * E;
  float* at = row + ((e >> 1) * (r.rd / (2 * E)) + i) * 4 + (e & 1);
  const float2 cs = angle(r, pos, j, backward);
  at[0] = cs.x;
  at[2] = cs.y;
}
template <int E>
DF_DEVICE void turn_item(float (&f)[2 * E], const float* row, int i, const RopeView& r) {
  const float4* t4 = reinterpret_cast<const float4*>(row) + i;
  const int step = r.rd / (2 * E);
  auto pair = [](float& x, float& y, float c, float s) {
    const float a = x, b = y;
    x = a * c - b * s;
    y = b * c + a * s;
  };
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float4 t = t4[e / 2 * step];
    if (r.interleaved) {
      pair(f[2 * e], f[2 * e + 1], t.x, t.z);
      pair(f[2 * e + 2], f[2 * e + 3], t.y, t.w);
    } else {
      pair(f[e], f[E + e], t.x, t.z);
      pair(f[e + 1], f[E + e + 1], t.y, t.w);
    }
  }
}

// Two fp32 operations at a time.
DF_DEVICE void mul2(float& x, float& y, float a, float b) {
  asm("{\n .reg .b64 p, q;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n mul.rn.f32x2 p, p, q;\n"
      " mov.b64 {%0, %1}, p;\n}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
DF_DEVICE void fma2(float& x, float& y, float a0, float a1, float b0, float b1) {   // += a b
  asm("{\n .reg .b64 p, q, d;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %5};\n mov.b64 d, {%0, %1};\n"
      " fma.rn.f32x2 d, p, q, d;\n mov.b64 {%0, %1}, d;\n}"
      : "+f"(x), "+f"(y)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// Sum over the 2, 4, 8 or 16 neighbouring lanes that hold a head (all lanes of the warp).
DF_DEVICE float head_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int E>
DF_DEVICE float dot_item(const float (&a)[2 * E], const float (&b)[2 * E]) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int e = 0; e < 2 * E; e += 2) fma2(s0, s1, a[e], a[e + 1], b[e], b[e + 1]);
  return s0 + s1;
}
// 1 / root mean square of the head.
template <int E>
DF_DEVICE float norm_of(const float (&f)[2 * E], int lanes, float per_dim, float eps) {
  return rsqrtf(fmaf(head_sum(dot_item<E>(f, f), lanes), per_dim, eps));
}

// A thread's column: item `it` of the rows.
template <int E>
struct Column {
  int part, h, place, o0, o1;   // part: 0 queries, 1 keys, 2 values
  bool rot;
  DF_DEVICE Column(const int (&heads)[3], const RopeView& r, int hd, int it) {
    const int ipr = hd / (2 * E);
    h = it / ipr;
    place = it - h * ipr;
    part = h < heads[0] ? 0 : h < heads[0] + heads[1] ? 1 : 2;
    h -= part == 0 ? 0 : part == 1 ? heads[0] : heads[0] + heads[1];
    rot = item_offsets<E>(r, place, o0, o1);
  }
};

template <int EL, int VB, bool CACHE>
__global__ void __launch_bounds__(kMost, 3) norm_rows_kernel(const __grid_constant__ NormRows p, norm::Shape s) {
  using V = typename Vec<VB>::T;
  constexpr int E = VB / EL, kAhead = 2;   // rows on their way
  extern __shared__ __align__(16) float cs[];   // [rows][rd]
  __shared__ int s_pos[kRows];
  __shared__ long long s_dst[kRows];
  pdl_trigger();
  pdl_wait();
  const int ipr = p.hd / (2 * E), items = (p.heads[0] + p.heads[1] + p.heads[2]) * ipr, tid = threadIdx.x;
  const int row0 = blockIdx.x * s.rows, n_rows = min(s.rows, p.T - row0), side = tid / s.cols;
  const int it = blockIdx.y * s.cols + tid - side * s.cols;
  const bool real = side < s.side && it < items;
  const Column<E> c(p.heads, p.r, p.hd, real ? it : 0);
  const char* src = p.x[c.part] + (size_t)(row0 + side) * p.x_ld[c.part] + (size_t)c.h * p.hd * EL;
  const int64_t step = p.x_ld[c.part] * s.side;
  V v[kAhead][2];
  auto load = [&](int r, V (&x)[2]) {
    if (real && r < n_rows) {
      x[0] = *reinterpret_cast<const V*>(src + c.o0 * EL);
      x[1] = *reinterpret_cast<const V*>(src + c.o1 * EL);
    }
    src += step;
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) load(side + j * s.side, v[j]);
  float w[2 * E];
  if (c.part < 2) {
    unpack<EL, VB>(*reinterpret_cast<const V*>(p.w[c.part] + c.o0 * EL), w);
    unpack<EL, VB>(*reinterpret_cast<const V*>(p.w[c.part] + c.o1 * EL), w + E);
  }
  const bool first = blockIdx.y == 0;
  if constexpr (CACHE) {
    // (few entries: a lane a row, all rows at once; rows of a warp one after another are five
    // dependent loads each)
    const int lane = tid & 31;
    if (p.a.rows.n_seq <= 32) {
      if (tid < n_rows) append_row_alone(p.a, row0 + tid, first, s_pos[tid], s_dst[tid]);
    } else {
      for (int r = tid >> 5; r < n_rows; r += blockDim.x >> 5) {
        int pos;
        long long dst;
        append_row(p.a, row0 + r, lane, first && lane == 0, pos, dst);
        if (lane == 0) {
          s_pos[r] = pos;
          s_dst[r] = dst;
        }
      }
    }
    if (blockIdx.x == 0 && first) report_ranges(p.a.rows, p.status);
  } else if (tid < n_rows) {
    const int q = p.pos[row0 + tid];
    s_pos[tid] = q;
    if (q < 0 && first) set_status(p.status, DEV_BAD_POSITION);
  }
  __syncthreads();
  const int half = p.r.rd / 2;
  for (int e = tid; e < n_rows * half; e += blockDim.x) {
    const int r = e / half;
    put_angle<E>(cs + r * p.r.rd, p.r, s_pos[r], e - r * half, false);
  }
  __syncthreads();
  // where the column's results go: rows of out, or slots of the pages
  const bool paged = CACHE && c.part > 0;
  char* dst0;
  int64_t out_step = 0;
  if (paged) {
    dst0 = p.a.c.pages + (size_t)(c.h + (c.part == 2 ? p.heads[1] : 0)) * p.a.c.ps * p.hd * EL;
  } else {
    out_step = p.out_ld[c.part & 1] * s.side;
    dst0 = p.out[c.part & 1] + (size_t)(row0 + side) * p.out_ld[c.part & 1] + (size_t)c.h * p.hd * EL;
  }
  const bool warp_norms = __any_sync(0xffffffffu, c.part < 2);
  const int steps = (n_rows + s.side - 1) / s.side;
  for (int k0 = 0; k0 < steps; k0 += kAhead) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (k0 + j >= steps) break;
      const int r = side + (k0 + j) * s.side;
      V x[2] = {v[j][0], v[j][1]};
      load(r + kAhead * s.side, v[j]);
      const bool on = real && r < n_rows && s_pos[r] >= 0;
      if (warp_norms) {
        float f[2 * E];
        unpack<EL, VB>(x[0], f);
        unpack<EL, VB>(x[1], f + E);
        const float inv = norm_of<E>(f, ipr, p.per_dim, p.eps);   // (all lanes)
        if (on && c.part < 2) {
#pragma unroll
          for (int e = 0; e < 2 * E; e += 2) {
            mul2(f[e], f[e + 1], inv, inv);
            mul2(f[e], f[e + 1], w[e], w[e + 1]);
          }
          if (c.rot) turn_item<E>(f, cs + r * p.r.rd, c.place, p.r);
          x[0] = pack<EL, VB>(f);
          x[1] = pack<EL, VB>(f + E);
        }
      }
      char* dst = dst0;
      if (paged) {
        const long long at = r < n_rows ? s_dst[r] : -1;
        if (!on || at < 0) continue;
        dst += at;
      } else {
        dst0 += out_step;
        if (!on) continue;
      }
      *reinterpret_cast<V*>(dst + c.o0 * EL) = x[0];
      *reinterpret_cast<V*>(dst + c.o1 * EL) = x[1];
    }
  }
}

// The weights' gradients stay in registers (a thread's items are all at the same place of
// their heads); at the end the block adds up its threads' in order and leaves them for
// norm_sums_kernel.
template <int EL, int VB>
__global__ void __launch_bounds__(kMost, 2) norm_rope_grad_kernel(const __grid_constant__ NormRopeParams p, norm::Shape s) {
  using V = typename Vec<VB>::T;
  constexpr int E = VB / EL, kAhead = 2;
  extern __shared__ __align__(16) float cs[];   // [rows][rd], then the threads' sums
  __shared__ int s_pos[kGradRows];
  pdl_trigger();
  pdl_wait();
  const int heads[3] = {p.part[0].heads, p.part[1].heads, 0};
  const int ipr = p.hd / (2 * E), items = (heads[0] + heads[1]) * ipr, tid = threadIdx.x;
  const int row0 = blockIdx.x * s.rows, n_rows = min(s.rows, p.T - row0), side = tid / s.cols;
  const int it = blockIdx.y * s.cols + tid - side * s.cols;
  const bool real = side < s.side && it < items;
  const Column<E> c(heads, p.r, p.hd, real ? it : 0);
  const NormRopePart& q = p.part[c.part];
  const size_t head = (size_t)c.h * p.hd * EL;
  const char* src = q.x + (size_t)(row0 + side) * q.x_ld + head;
  const char* dys = q.dy + (size_t)(row0 + side) * q.dy_ld + head;
  char* dst = q.out + (size_t)(row0 + side) * q.out_ld + head;
  const int64_t step = q.x_ld * s.side, dy_step = q.dy_ld * s.side, out_step = q.out_ld * s.side;
  V v[kAhead][4];
  auto load = [&](int r, V (&x)[4]) {
    if (real && r < n_rows) {
      x[0] = *reinterpret_cast<const V*>(src + c.o0 * EL);
      x[1] = *reinterpret_cast<const V*>(src + c.o1 * EL);
      x[2] = *reinterpret_cast<const V*>(dys + c.o0 * EL);
      x[3] = *reinterpret_cast<const V*>(dys + c.o1 * EL);
    }
    src += step;
    dys += dy_step;
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) load(side + j * s.side, v[j]);
  float w[2 * E], dw[2 * E];
  unpack<EL, VB>(*reinterpret_cast<const V*>(q.w + c.o0 * EL), w);
  unpack<EL, VB>(*reinterpret_cast<const V*>(q.w + c.o1 * EL), w + E);
#pragma unroll
  for (int e = 0; e < 2 * E; ++e) dw[e] = 0.f;
  const int half = p.r.rd / 2, batch = kGradRows / (kAhead * s.side) * kAhead * s.side;   // rows whose angles are there
  for (int b0 = 0; b0 < n_rows; b0 += batch) {
    const int nb = min(batch, n_rows - b0), steps = (nb + s.side - 1) / s.side;
    __syncthreads();   // the last rows' angles have been read
    if (tid < nb) {
      const int t = p.pos[row0 + b0 + tid];
      s_pos[tid] = t;
      if (t < 0 && blockIdx.y == 0) set_status(p.status, DEV_BAD_POSITION);
    }
    __syncthreads();
    for (int e = tid; e < nb * half; e += blockDim.x) {
      const int r = e / half;
      put_angle<E>(cs + r * p.r.rd, p.r, s_pos[r], e - r * half, true);
    }
    __syncthreads();
    for (int k0 = 0; k0 < steps; k0 += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (k0 + j >= steps) break;
        const int r = side + (k0 + j) * s.side;   // within the batch
        float n[2 * E], d[2 * E];
        unpack<EL, VB>(v[j][0], n);
        unpack<EL, VB>(v[j][1], n + E);
        unpack<EL, VB>(v[j][2], d);
        unpack<EL, VB>(v[j][3], d + E);
        load(b0 + r + kAhead * s.side, v[j]);
        const bool on = real && r < nb && s_pos[r] >= 0;
        const float inv = norm_of<E>(n, ipr, p.per_dim, p.eps);
#pragma unroll
        for (int e = 0; e < 2 * E; e += 2) mul2(n[e], n[e + 1], inv, inv);
        if (c.rot) turn_item<E>(d, cs + min(r, nb - 1) * p.r.rd, c.place, p.r);
        if (on) {
#pragma unroll
          for (int e = 0; e < 2 * E; e += 2) fma2(dw[e], dw[e + 1], d[e], d[e + 1], n[e], n[e + 1]);
        }
#pragma unroll
        for (int e = 0; e < 2 * E; e += 2) mul2(d[e], d[e + 1], w[e], w[e + 1]);
        const float dot = -head_sum(dot_item<E>(d, n), ipr) * p.per_dim;   // (all lanes)
        if (on) {
#pragma unroll
          for (int e = 0; e < 2 * E; e += 2) {
            fma2(d[e], d[e + 1], n[e], n[e + 1], dot, dot);
            mul2(d[e], d[e + 1], inv, inv);
          }
          *reinterpret_cast<V*>(dst + c.o0 * EL) = pack<EL, VB>(d);
          *reinterpret_cast<V*>(dst + c.o1 * EL) = pack<EL, VB>(d + E);
        }
        dst += out_step;
      }
    }
  }
  // the block's sums by dim: all threads of the part at the dim's place, in order
  __syncthreads();
  float* sums = cs;   // [thread][2 E]
#pragma unroll
  for (int e = 0; e < 2 * E; ++e) sums[tid * 2 * E + e] = real ? dw[e] : 0.f;
  __syncthreads();
  const int it0 = blockIdx.y * s.cols, it1 = min(it0 + s.cols, items);
  for (int e = tid; e < 2 * p.hd; e += blockDim.x) {
    const int part = e >= p.hd, d = e - part * p.hd, h0 = part ? heads[0] : 0, h1 = h0 + heads[part];
    // dim d's place and number among its item's
    const int rd = p.r.rd;
    int place, at;
    if (d >= rd || p.r.interleaved) {
      place = d / (2 * E);
      at = d - place * 2 * E;
    } else {
      const int y = d >= rd / 2 ? d - rd / 2 : d;
      place = y / E;
      at = y - place * E + (d >= rd / 2 ? E : 0);
    }
    float sum = 0.f;
    for (int k = 0; k < s.side; ++k)
      for (int h = h0; h < h1; ++h) {
        const int i = h * ipr + place;
        if (i >= it0 && i < it1) sum += sums[(k * s.cols + i - it0) * 2 * E + at];
      }
    p.sums[((size_t)(blockIdx.y * gridDim.x + blockIdx.x) * 2) * p.hd + e] = sum;
  }
}

// The blocks' sums of the weights' gradients: grid (parts, 32 dims each), a warp every 32nd
// block's, the warps in order.
__global__ void __launch_bounds__(1024) norm_sums_kernel(const __grid_constant__ NormRopeParams p, int blocks) {
  __shared__ float s[32][32];
  pdl_trigger();
  pdl_wait();
  const int k = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = blockIdx.y * 32 + lane;
  if (!p.part[k].heads) return;
  const float* from = p.sums + k * p.hd + d;
  float sum = 0.f;
#pragma unroll 16
  for (int i = warp; i < blocks; i += 32) sum += from[(size_t)i * 2 * p.hd];
  s[warp][lane] = sum;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int i = 1; i < 32; ++i) sum += s[i][lane];
    p.part[k].dw[d] = sum;
  }
}

template <int EL, int VB, bool CACHE>
cudaError_t norm_rows_as(const NormRows& p, cudaStream_t st) {
  const norm::Shape s = norm::shape_of(p.T, (p.heads[0] + p.heads[1] + p.heads[2]) * (p.hd / (2 * (VB / EL))), 65536 / 80);
  return launch_dependent(norm_rows_kernel<EL, VB, CACHE>, dim3(s.gx, s.gy), s.threads, sizeof(float) * s.rows * p.r.rd,
                          st, p, s);
}

template <bool CACHE>
cudaError_t norm_rows(const NormRows& p, int el, cudaStream_t st) {
  if (el == 4) return norm_rows_as<4, 16, CACHE>(p, st);
  return p.r.rd % 16 == 0 ? norm_rows_as<2, 16, CACHE>(p, st) : norm_rows_as<2, 8, CACHE>(p, st);
}

template <int EL, int VB>
cudaError_t norm_rope_grad_as(const NormRopeParams& p, cudaStream_t st) {
  constexpr int E = VB / EL;
  const norm::Shape s = norm::sum_shape_of(p.T, (p.part[0].heads + p.part[1].heads) * (p.hd / (2 * E)), 65536 / 128, kNormBlocks);
  const size_t smem = sizeof(float) * std::max(kGradRows * p.r.rd, s.threads * 2 * E);
  const cudaError_t e = launch_dependent(norm_rope_grad_kernel<EL, VB>, dim3(s.gx, s.gy), s.threads, smem, st, p, s);
  if (e != cudaSuccess) return e;
  return launch_dependent(norm_sums_kernel, dim3(2, p.hd / 32), 1024, 0, st, p, s.gx * s.gy);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t st) {
  NormRows n = {};
  n.r = p.r;
  n.T = p.T;
  n.hd = p.hd;
  for (int k = 0; k < 2; ++k) {
    n.heads[k] = p.part[k].heads;
    n.x[k] = p.part[k].x;
    n.w[k] = p.part[k].w;
    n.out[k] = p.part[k].out;
    n.x_ld[k] = p.part[k].x_ld;
    n.out_ld[k] = p.part[k].out_ld;
  }
  n.per_dim = p.per_dim;
  n.eps = p.eps;
  n.pos = p.pos;
  n.status = p.status;
  return norm_rows<false>(n, p.el, st);
}

cudaError_t launch_norm_append(const AppendParams& a, cudaStream_t st) {
  NormRows n = {};
  n.r = a.r;
  n.T = a.rows.T;
  n.hd = a.c.hd;
  n.heads[0] = a.q ? a.c.n_head : 0;
  n.heads[1] = n.heads[2] = a.c.n_head_kv;
  n.x[0] = a.q;
  n.x[1] = a.k;
  n.x[2] = a.v;
  n.w[0] = a.q_norm;
  n.w[1] = a.k_norm;
  n.out[0] = a.q_out;
  n.x_ld[0] = a.q_ld;
  n.x_ld[1] = a.k_ld;
  n.x_ld[2] = a.v_ld;
  n.out_ld[0] = a.q_out_ld;
  n.per_dim = a.per_dim;
  n.eps = a.eps;
  n.status = a.c.status;
  n.a = a;
  return norm_rows<true>(n, a.c.el, st);
}

cudaError_t launch_norm_rope_grad(const NormRopeParams& p, cudaStream_t st) {
  if (p.el == 4) return norm_rope_grad_as<4, 16>(p, st);
  return p.r.rd % 16 == 0 ? norm_rope_grad_as<2, 16>(p, st) : norm_rope_grad_as<2, 8>(p, st);
}

}  // namespace dflash
