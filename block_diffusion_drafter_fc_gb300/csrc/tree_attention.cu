// Attention of the rows of a call (tree nodes, a causal chain, single tokens)
// over their sequences' cache pages.
//
//   out[t][h] = sum_p w_p V[p],  w = softmax over the attended slots p of
//   scale q[t][h] . K[p];  lse[t][h] = ln sum_p exp(scale q[t][h] . K[p]).
//
// One pass over the slots with a running maximum m and sum l: a new score s
// changes them to m' = max(m, s), l' = l e^(m-m') + e^(s-m'), and the weighted
// sum of values likewise.
//
// Simple form: one block per (row, head); each warp takes every fourth run of
// 32 slots, a lane scores one slot, and the warp adds the 32 weighted value
// rows with a lane per dims.
#include "cache.cuh"

#include <math_constants.h>

namespace dflash {

namespace {

constexpr int kWarps = 4;

template <int EL>
DF_DEVICE float load_el(const char* p) {
  return EL == 4 ? *reinterpret_cast<const float*>(p)
                 : bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(p));
}

template <int EL, int HD>
__global__ void __launch_bounds__(kWarps * 32) attend_kernel(AttendParams p) {
  __shared__ float s_q[HD];
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][HD];
  const CacheView& c = p.c;
  const int t = blockIdx.x, h = blockIdx.y, kvh = h / (c.n_head / c.n_head_kv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int below = 0;
  for (int i = lane; i <= p.rows.n_seq; i += 32) below += p.rows.row_start[i] <= t;
  const int s = __reduce_add_sync(0xffffffffu, below) - 1;
  int lo, n;
  if (s < 0 || s >= p.rows.n_seq) return;
  if (!entry_rows(p.rows, s, lo, n) || n > p.max_tree) {
    if (threadIdx.x == 0) set_status(c.status, DEV_BAD_ROWS);
    return;
  }
  const int q = entry_sequence(p.rows, s, c.max_seq);
  const int len = q >= 0 ? c.length[q] : 0;
  if (q < 0 || len < 0 || (long long)len + n > (long long)c.max_pages * c.ps) {
    if (threadIdx.x == 0) set_status(c.status, q < 0 ? DEV_BAD_SEQ : DEV_BAD_ROWS);
    return;
  }
  for (int d = threadIdx.x; d < HD; d += blockDim.x)
    s_q[d] = load_el<EL>(p.q + (size_t)t * p.q_ld + ((size_t)h * HD + d) * EL);
  __syncthreads();
  float m = -CUDART_INF_F, l = 0.f, o[HD / 32];
#pragma unroll
  for (int k = 0; k < HD / 32; ++k) o[k] = 0.f;
  const int end = len + n;
  for (int p0 = warp * 32; p0 < end; p0 += kWarps * 32) {
    const int slot = p0 + lane, node = slot - len;
    bool sees = slot < end;
    if (sees && node >= 0)
      sees = p.mask ? (p.mask[(size_t)t * p.words + (node >> 5)] >> (node & 31)) & 1 : node <= t - lo;
    int page = slot < end ? c.table[(size_t)q * c.max_pages + (slot >> c.ps_log2)] : -1;
    if (slot < end && (page < 0 || page >= c.n_pages)) {
      set_status(c.status, DEV_BAD_PAGE);
      page = -1;
    }
    sees = sees && page >= 0;
    float x = -CUDART_INF_F;
    const char* vrow = nullptr;
    if (sees) {
      const char* krow = c.pages + page_row(c, page, p.layer, 0, kvh, slot & (c.ps - 1));
      vrow = c.pages + page_row(c, page, p.layer, 1, kvh, slot & (c.ps - 1));
      x = 0.f;
      for (int d = 0; d < HD; ++d) x += s_q[d] * load_el<EL>(krow + d * EL);
      x *= p.scale;
    }
    const float top = fmaxf(m, warp_max(x));
    if (top == -CUDART_INF_F) continue;
    const float w = expf(x - top), fade = expf(m - top);
    l = l * fade + warp_sum(w);
    m = top;
#pragma unroll
    for (int k = 0; k < HD / 32; ++k) o[k] *= fade;
    for (int i = 0; i < 32; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const char* v = reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, (unsigned long long)vrow, i));
      if (!v) continue;
#pragma unroll
      for (int k = 0; k < HD / 32; ++k) o[k] += wi * load_el<EL>(v + (k * 32 + lane) * EL);
    }
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int k = 0; k < HD / 32; ++k) s_o[warp][k * 32 + lane] = o[k];
  __syncthreads();
  float top = -CUDART_INF_F, total = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  float f[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    f[w] = top == -CUDART_INF_F ? 0.f : expf(s_m[w] - top);
    total += f[w] * s_l[w];
  }
  for (int d = threadIdx.x; d < HD; d += blockDim.x) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += f[w] * s_o[w][d];
    v = total > 0.f ? v / total : 0.f;
    char* dst = p.out + (size_t)t * p.out_ld + ((size_t)h * HD + d) * EL;
    if (EL == 4)
      *reinterpret_cast<float*>(dst) = v;
    else
      *reinterpret_cast<uint16_t*>(dst) = f32_to_bf16_bits(v);
  }
  if (p.lse && threadIdx.x == 0) p.lse[(size_t)t * c.n_head + h] = total > 0.f ? top + logf(total) : -CUDART_INF_F;
}

template <int EL>
cudaError_t attend_as(const AttendParams& p, cudaStream_t st) {
  const dim3 grid(p.rows.T, p.c.n_head);
  if (p.c.hd == 32)
    attend_kernel<EL, 32><<<grid, kWarps * 32, 0, st>>>(p);
  else if (p.c.hd == 64)
    attend_kernel<EL, 64><<<grid, kWarps * 32, 0, st>>>(p);
  else
    attend_kernel<EL, 128><<<grid, kWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend(const AttendParams& p, cudaStream_t st) {
  return p.c.el == 4 ? attend_as<4>(p, st) : attend_as<2>(p, st);
}

}  // namespace dflash
