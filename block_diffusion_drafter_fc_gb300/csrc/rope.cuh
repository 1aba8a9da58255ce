// Shared parts of the kernels that rotate heads: items (two vectors that hold whole
// pairs), angles, and the norm of a head that lies with neighbouring lanes.
#pragma once

#include "cache.cuh"

namespace dflash {
namespace rope {


template <int VB>
struct Vec;
template <>
struct Vec<16> { using T = uint4; };
template <>
struct Vec<8> { using T = uint2; };

template <int EL, int VB>
DF_DEVICE void unpack(const typename Vec<VB>::T& v, float* f) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < VB / 4; ++i) {
    if constexpr (EL == 4) {
      f[i] = __uint_as_float(w[i]);
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <int EL, int VB>
DF_DEVICE typename Vec<VB>::T pack(const float* f) {
  typename Vec<VB>::T v;
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < VB / 4; ++i)
    w[i] = EL == 4 ? __float_as_uint(f[i]) : pack_bf16x2(f[2 * i], f[2 * i + 1]);
  return v;
}

// Turn the pairs of one item in place; cs: the item's (cos, sin), one per pair.
template <int E>
DF_DEVICE void turn(float (&f)[2 * E], const float2* cs, bool interleaved) {
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float2 t = cs[e];
    if (interleaved) {
      const float a = f[2 * e], b = f[2 * e + 1];
      f[2 * e] = a * t.x - b * t.y;
      f[2 * e + 1] = b * t.x + a * t.y;
    } else {
      const float a = f[e], b = f[E + e];
      f[e] = a * t.x - b * t.y;
      f[E + e] = b * t.x + a * t.y;
    }
  }
}
template <int EL, int VB>
DF_DEVICE void turn(typename Vec<VB>::T& v0, typename Vec<VB>::T& v1, const float2* cs, bool interleaved) {
  constexpr int E = VB / EL;
  float f[2 * E];
  unpack<EL, VB>(v0, f);
  unpack<EL, VB>(v1, f + E);
  turn<E>(f, cs, interleaved);
  v0 = pack<EL, VB>(f);
  v1 = pack<EL, VB>(f + E);
}

// Element offsets of item i's two vectors within a head; true for a rotated item.
template <int E>
DF_DEVICE bool item_offsets(const RopeView& r, int i, int& o0, int& o1) {
  const int n_rot = r.rd / (2 * E);
  const bool rot = i < n_rot;
  if (!rot || r.interleaved) {
    o0 = i * 2 * E;
    o1 = o0 + E;
  } else {
    o0 = i * E;
    o1 = r.rd / 2 + o0;
  }
  return rot;
}

DF_DEVICE float2 angle(const RopeView& r, int pos, int j, bool backward) {
  const long long t = (long long)((unsigned long long)(unsigned)pos * r.turns[j]);
  float s, c;
  sincospif((float)t * 0x1p-63f, &s, &c);
  s *= r.mscale;
  return make_float2(c * r.mscale, backward ? -s : s);
}

// Sum over the 2, 4, 8 or 16 neighbouring lanes that hold a head (all lanes of the warp).
DF_DEVICE float head_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// An item's share of its head divided by the head's root mean square, and 1 / that root.
// (Squares and their sum in fp32, in an order that does not depend on the launch.)
template <int E>
DF_DEVICE float norm_head(float (&f)[2 * E], int lanes, float per_dim, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 2 * E; ++e) ss = fmaf(f[e], f[e], ss);
  const float r = rsqrtf(fmaf(head_sum(ss, lanes), per_dim, eps));
#pragma unroll
  for (int e = 0; e < 2 * E; ++e) f[e] *= r;
  return r;
}

}  // namespace rope
}  // namespace dflash
