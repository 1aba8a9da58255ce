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

// A row's (cos, sin), one per pair.  SPREAD: two pairs (16 bytes) of every item, then their
// next two, so that neighbouring lanes read neighbouring words; else items' pairs one after
// another, which meet in the same banks four times but cost an address less (the append of 8192
// rows takes 38.4 us with them, 39.4 spread; the rotation of 16381 rows 52.9 and 51.0).
template <int E, bool SPREAD>
DF_DEVICE int pair_at(int j, int rd) {
  if (!SPREAD) return j;
  const int i = j / E, e = j - i * E;
  return ((e >> 1) * (rd / (2 * E)) + i) * 2 + (e & 1);
}
// Turn the pairs of item i in place; cs: its row's table.
template <int E, bool SPREAD>
DF_DEVICE void turn(float (&f)[2 * E], const float2* cs, int i, const RopeView& r) {
  const float4* pairs = reinterpret_cast<const float4*>(cs) + (SPREAD ? i : i * (E / 2));
  const int step = SPREAD ? r.rd / (2 * E) : 1;
  auto pair = [](float& x, float& y, float c, float s) {
    const float a = x, b = y;
    x = a * c - b * s;
    y = b * c + a * s;
  };
  // (one branch for the item: as a choice of each pair it was made with selects)
  if (r.interleaved) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float4 t = pairs[e / 2 * step];
      pair(f[2 * e], f[2 * e + 1], t.x, t.y);
      pair(f[2 * e + 2], f[2 * e + 3], t.z, t.w);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float4 t = pairs[e / 2 * step];
      pair(f[e], f[E + e], t.x, t.y);
      pair(f[e + 1], f[E + e + 1], t.z, t.w);
    }
  }
}
template <int EL, int VB, bool SPREAD>
DF_DEVICE void turn(typename Vec<VB>::T& v0, typename Vec<VB>::T& v1, const float2* cs, int i, const RopeView& r) {
  constexpr int E = VB / EL;
  float f[2 * E];
  unpack<EL, VB>(v0, f);
  unpack<EL, VB>(v1, f + E);
  turn<E, SPREAD>(f, cs, i, r);
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

// Position of row t of an append (-1: it does nothing) and its slot's row of (layer, k, head 0)
// (-1: not written), by one warp: the row's entry is the number of range starts at or below it
// (ranges ascend), then the page of its slot.  first: report what is bad.
DF_DEVICE void append_row(const AppendParams& p, int t, int lane, bool first, int& pos, long long& dst) {
  const CacheView& c = p.c;
  int below = 0;
  for (int i = lane; i <= p.rows.n_seq; i += 32) below += p.rows.row_start[i] <= t;
  below = __reduce_add_sync(0xffffffffu, below);
  const int s = below - 1;
  pos = -1;
  dst = -1;
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
}
// The same by one lane, of calls of few entries: a block's rows all at once.
DF_DEVICE void append_row_alone(const AppendParams& p, int t, bool first, int& pos, long long& dst) {
  const CacheView& c = p.c;
  int s = -1;
  for (int i = 0; i <= p.rows.n_seq; ++i) s += p.rows.row_start[i] <= t;
  pos = -1;
  dst = -1;
  int lo = 0, n = 0;
  if (s < 0 || s >= p.rows.n_seq || !entry_rows(p.rows, s, lo, n) || t < lo || t >= lo + n) return;
  const int q = entry_sequence(p.rows, s, c.max_seq);
  bool twice = false;
  if (p.rows.seqs)
    for (int i = 0; i < s; ++i) twice |= p.rows.seqs[i] == q;
  const int len = q >= 0 ? c.length[q] : -1;
  const long long at = (long long)len + (p.depth ? p.depth[t] : t - lo);
  const unsigned bad = q < 0 || twice ? DEV_BAD_SEQ : len < 0 ? DEV_BAD_ROWS : at < 0 || at > 0x7fffffffLL ? DEV_BAD_POSITION : 0u;
  if (bad) {
    if (first) set_status(c.status, bad);
    return;
  }
  pos = (int)at;
  const long long slot = (long long)len + (t - lo), idx = slot >> c.ps_log2;
  const int page = idx < c.max_pages ? c.table[(size_t)q * c.max_pages + idx] : -1;
  if (page >= 0 && page < c.n_pages && c.refs[page] <= 1)
    dst = (long long)page_row(c, page, p.layer, 0, 0, (int)(slot & (c.ps - 1)));
  else if (first)
    set_status(c.status, DEV_BAD_PAGE);
}
// Ranges that are no ranges, by one block.
DF_DEVICE void report_ranges(const RowView& rows, unsigned* status) {
  for (int s = threadIdx.x; s < rows.n_seq; s += blockDim.x) {
    int lo, n;
    if (!entry_rows(rows, s, lo, n)) set_status(status, DEV_BAD_ROWS);
  }
}

}  // namespace rope
}  // namespace dflash
