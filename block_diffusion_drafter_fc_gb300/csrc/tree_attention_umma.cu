// Tree attention on the 5th-generation tensor cores (tcgen05), bf16 with heads
// of 64 and 128.
//
// Why not mma.sync: it runs bf16 at 256 products a clock and SM here (ncu on
// the streaming kernel: 32 cycles per m16n8k16 and scheduler, tensor pipe 86%
// busy at 66% of the copy bandwidth with 16-row tiles), a sixteenth of
// tcgen05.mma; the matrix work of a 16-row tile alone (two products, the
// weights split) exceeded the time to read its pages.  tcgen05.mma on a padded
// 128-row tile takes 8 clocks a slot (QK^T and PV, 128 dims), the read of a
// slot at an SM's share of the copy bandwidth 22.
//
// One persistent block per SM walks its range of the call's work (128-slot
// chunks of the tiles of every kv head's query rows; tree_common.cuh) with two
// streams of scores, so that the products of one run under the softmax of the
// other:
//   tile of more than 128 rows (pair): stream i holds rows 128 i .. + 127, both
//     use every chunk;
//   tile of at most 128 rows (split): stream i takes every second chunk, with
//     its own reference, sum and accumulator, joined at the tile's end.  With at
//     most 64 rows, the rows are there twice, in different lanes of the tile, and
//     each copy of a row exponentiates its own half of the slots, its weights for
//     the others zero: the products cost the same, the exponentials spread over
//     all four warps.
// Roles:
//   warps 0..3, 4..7  softmax of stream 0 and 1, a thread per row: S from tensor
//                     memory (tcgen05.ld), reference m and sum l, weights
//                     e^(s - m) back as bf16 over S (the A operand of PV);
//   warp 11           plans the block's segments for all, and loads their Q;
//   warp 8 (a lane)   K and V chunks by TMA into a ring of stages, page by page,
//                     across tiles;
//   warps 9, 10       (a lane each) tcgen05.mma of stream 0 and 1: S_i = Q_i K^T
//                     (both in shared memory), O_i += P_i V (P in tensor memory,
//                     V as it lies: MN-major).  Issuing waits for the pipe (a
//                     product of 16 dims or slots takes some 60 clocks), so an
//                     issuer per stream: one's barriers are under the other's
//                     products.
// Tensor memory: S_0, S_1 (128 columns each), O_0, O_1 (head_dim each): all of it.
// A stream's scores, softmax and PV follow one another; the softmax is done by
// halves of 64 slots, PV of the first under the softmax of the second, and the last
// PV and the next scores are issued together.  The streams of a pair do that in
// turn: otherwise their products interleave in the pipe, and both wait for all of
// them (2047 rows over 8192 slots took 235 us in turn, 262 without; 243 now).  Scores by halves
// too, with a buffer for each, kept both in work all the time, but 64 columns of
// scores cost as much as 128 (both read Q): 261 us.
// The weights are rounded to bf16 for the product with V (their sum is not):
// each is off by at most 2^-8 of itself, independently, which adds as much
// again as the rounding of the result; splitting them as in the streaming
// kernel would cost half of PV more.
// Every mbarrier wait gives up after ~2 s with DFLASH_DEV_TIMEOUT; the block then
// issues nothing more, runs to its end without further waits or arrivals, and
// releases its tensor memory.
#include "internal.h"
#include "tree_common.cuh"

namespace dflash {

using namespace tree;

namespace {

constexpr int kThreads = 384;
constexpr int kChunk = 128, kTile = 256;
// a chunk of a pair costs 3 units, of a split tile 2, a tile 8 besides
constexpr int kWide = 128;
DF_DEVICE Cutting cutting() { return {kTile, kChunk, kWide, 3, 2, 8}; }
constexpr int kMinUnits = 4;   // a block's least share of a call's units
constexpr int kScratch = 32768;   // 32 rows x 32 dims of every softmax warp
constexpr int kProducer = 8, kIssuer = 9;

template <int HD>
struct Lay {
  static constexpr int kHalf = 128 * 128;               // 128 rows x 64 dims, 128-byte swizzle
  static constexpr int kHalves = HD / 64;
  static constexpr int kMat = kHalf * kHalves;          // a Q tile, a K or V chunk
  static constexpr int kOffScratch = 2 * kMat;          // Q tiles first
  static constexpr int kStagesMost = HD == 128 ? 5 : 10;
  static constexpr int kCols = 512;
};

DF_DEVICE uint64_t desc_k(uint32_t a) {   // K-major, 128-byte swizzle, 8-row groups of 1024 bytes
  return ((uint64_t)(a >> 4) & 0x3FFFull) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}
// MN-major, 128-byte swizzle: 64 dims per 128-byte row, the next 64 dims kHalf
// bytes on, the next 8 slots 1024 bytes on.
DF_DEVICE uint64_t desc_mn(uint32_t a, uint32_t next64) {
  return ((uint64_t)(a >> 4) & 0x3FFFull) | ((uint64_t)(next64 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// kind::f16: bf16 A and B, fp32 D, A K-major, B K-major or MN-major.
constexpr uint32_t idesc(int N, bool mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
DF_DEVICE void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
DF_DEVICE void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
DF_DEVICE void commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   su32(b))
               : "memory");
}
DF_DEVICE void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
DF_DEVICE void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
DF_DEVICE void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 columns of the warp's lanes <-> 32 registers
DF_DEVICE void tmem_ld32(uint32_t a, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a));
}
DF_DEVICE void tmem_st32(uint32_t a, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
      "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
      "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]) : "memory");
}
DF_DEVICE void tmem_st16(uint32_t a, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16};" ::"r"(a),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]) : "memory");
}
// Loads done; the loaded registers are operands, so that nothing that reads them can
// be moved ahead of it
DF_DEVICE void wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :: "memory");
}
DF_DEVICE void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
DF_DEVICE void sync_rows() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

DF_DEVICE void prefetch_map(const CUtensorMap* m) { asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory"); }

DF_DEVICE void publish(int* at, int v) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(su32(at)), "r"(v) : "memory");
}
// Wait for copy number `pos` in its stage's barrier.  The stages of a split tile
// alternate between the streams, and copies land in any order, so a stream may
// come to a stage whose last use, the other stream's, has not landed yet: the
// barrier is then two phases behind, which its parity cannot tell from done.  A
// copy that has been issued has no such predecessor.
DF_DEVICE int load_acquire(int* at) {
  int n;
  asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(n) : "r"(su32(at)) : "memory");
  return n;
}
DF_DEVICE bool copy_wait(int* issued, int pos, uint64_t* b, uint32_t par, volatile int* abort, unsigned* status) {
  if (load_acquire(issued) <= pos) {
    const long long t0 = clock64();
    while (load_acquire(issued) <= pos && !*abort)
      if (clock64() - t0 > kWait) {
        *abort = 1;
        set_status(status, DEV_TIMEOUT);
      }
    if (*abort) return false;
  }
  return bar_wait(b, par, abort, status);
}
DF_DEVICE bool copy_there(int* issued, int pos, uint64_t* b, uint32_t par) {
  return load_acquire(issued) > pos && bar_try(b, par);
}

struct UmmaParams {
  CUtensorMap tm;     // pages as [rows of (page, layer, k|v, head)][page_size][hd], boxes of 64 dims
  CUtensorMap tm_q;   // queries as [T][n_head][hd], boxes of 64 dims x a group's heads x nodes: 32 rows
  int q_boxes;        // ... where groups divide 32 heads; else rows are copied piece by piece
  AttendParams a;
  float* part_o;      // [2 blocks][kTile][hd]
  float2* part_ml;    // [2 blocks][kTile]
  Cut* cuts;          // [blocks]
  int stages, box_rows;
  // shared memory of its own for a tile's end (else the tile's Q area): the next
  // tile's Q can then be loaded under it, at the cost of a ring stage
  int scratch;
  uint32_t grp_magic;   // ceil(2^32 / query heads per kv head): quotients of small numbers
};

// Bit j: the row sees slot `slot` + j.  (Plain loads: a dependent launch may start
// before the kernel that writes the mask has ended, which the read-only path excludes.)
DF_DEVICE uint32_t visible(const AttendParams& p, const Entry& x, int node, int slot) {
  const int a = slot - x.len;                    // node index of bit 0
  if (a <= -32) return ~0u;
  const int valid = x.n - a;                     // bits below it are slots of the entry
  uint32_t v;
  if (!p.mask) {
    const int c = node - a + 1;
    v = c >= 32 ? ~0u : c <= 0 ? 0u : (1u << c) - 1u;
  } else {
    const uint32_t* w = p.mask + (size_t)(x.lo + node) * p.words;
    if (a < 0) {
      v = (*w << -a) | ((1u << -a) - 1u);
    } else {
      const int k = a >> 5;
      const uint32_t lo = k < p.words ? w[k] : 0u, hi = k + 1 < p.words ? w[k + 1] : 0u;
      v = __funnelshift_r(lo, hi, a & 31);
    }
  }
  if (valid < 32) v &= valid <= 0 ? 0u : (1u << valid) - 1u;
  return v;
}

// The mask words of the 128 slots from `slot` on, into L1 ahead of their use.
DF_DEVICE void prefetch_mask(const AttendParams& p, const Entry& x, int node, int slot) {
  const int k = max(slot - x.len, 0) >> 5;
  if (k >= p.words) return;
  const uint32_t* w = p.mask + (size_t)(x.lo + node) * p.words;
  asm volatile("prefetch.global.L1 [%0];" ::"l"(w + k));
  asm volatile("prefetch.global.L1 [%0];" ::"l"(w + min(k + 4, p.words - 1)));
}

// Two fp32 operations at a time.
DF_DEVICE uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
DF_DEVICE void unpack2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
DF_DEVICE uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
DF_DEVICE uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Scores that the row does not see become -inf.
DF_DEVICE void hide(uint32_t (&v)[32], uint32_t see) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!(see & (1u << e))) v[e] = 0xff800000u;
}

// One row's share of half a chunk: slots slot0 + col0 .. + 32 NB - 1 of the 64 at
// slot0; scores from tensor memory, weights 2^(s - m) back over them (zeros for
// the rest of the 64), l updated.
//
// m need not be the maximum: any reference that keeps the weights within fp32
// gives the same quotient, as weights, sums and products are all floating point
// (bf16 has fp32's exponents).  m starts at 0, and moves to the largest score
// (with the accumulator rescaled once its products are done: settle()) only when
// all weights so far sum to more than 2^60 or to less than 2^-60.  (An accumulator
// is then below 2^60 times the largest value, four of them from each of 160 blocks
// below 2^70 times: values up to 2^56 stay finite.)  So the maximum - a pass over
// the scores before the first exponential - is not on the path: it took prompts of
// 2047 rows over 8192 slots from 348 to 326 us.  MASKED: the row may not see every
// slot.  `later`: the accumulator holds something.
template <int NB, int HD, bool MASKED, typename F>
DF_DEVICE void softmax_step(const AttendParams& p, const Entry& x, int node, int slot0, int col0, uint32_t tS,
                            uint32_t tO, float scale, bool later, F settle, float& m, float& l) {
  uint32_t w[NB][16];
  float sum;
  for (bool again = false;; again = true) {
    const uint64_t sc2 = pack2(scale, scale), mn2 = pack2(-m, -m);
    uint64_t s2[2] = {0, 0};
    // (all loads at once: one takes some 250 clocks under the products, and a wait
    // is for every load before it)
    uint32_t v[NB][32];
    __syncwarp();
#pragma unroll
    for (int t = 0; t < NB; ++t) tmem_ld32(tS + col0 + 32 * t, v[t]);
    if constexpr (MASKED) {
      uint32_t see[NB];
#pragma unroll
      for (int t = 0; t < NB; ++t) see[t] = visible(p, x, node, slot0 + col0 + 32 * t);
#pragma unroll
      for (int t = 0; t < NB; ++t) wait_ld(v[t]);
#pragma unroll
      for (int t = 0; t < NB; ++t) hide(v[t], see[t]);
    } else {
#pragma unroll
      for (int t = 0; t < NB; ++t) wait_ld(v[t]);
    }
#pragma unroll
    for (int t = 0; t < NB; ++t) {
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        float a0, a1;
        unpack2(fma2(pack2(__uint_as_float(v[t][e]), __uint_as_float(v[t][e + 1])), sc2, mn2), a0, a1);
        a0 = ex2(a0);
        a1 = ex2(a1);
        s2[(e >> 1) & 1] = add2(s2[(e >> 1) & 1], pack2(a0, a1));
        w[t][e / 2] = pack_bf16x2(a0, a1);
      }
    }
    float a0, a1;
    unpack2(add2(s2[0], s2[1]), a0, a1);
    sum = a0 + a1;
    const bool bad = !(l + sum < 0x1p60f) || !(l + sum > 0x1p-60f);
    if (again || !__any_sync(0xffffffffu, bad)) break;
    // ---- a new reference: the larger of the chunk's maximum and the sum so far
    float top = l > 0.f ? m + log2f(l) : -CUDART_INF_F;
#pragma unroll 1
    for (int t = 0; t < NB; ++t) {
      uint32_t o[32];
      __syncwarp();
      tmem_ld32(tS + col0 + 32 * t, o);
      const uint32_t see = MASKED ? visible(p, x, node, slot0 + col0 + 32 * t) : ~0u;
      wait_ld(o);
      hide(o, see);
#pragma unroll
      for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(o[e]) * scale);
    }
    if (!bad || top == -CUDART_INF_F) top = m;   // nothing attended yet: any reference will do
    const float fade = l > 0.f ? ex2(m - top) : 1.f;   // (an empty sum has no scale; m may fall by any amount)
    m = top;
    l *= fade;
    if (later && __any_sync(0xffffffffu, fade != 1.f)) {
      settle();
#pragma unroll 1
      for (int t = 0; t < HD / 32; ++t) {
        uint32_t o[32];
        __syncwarp();
        tmem_ld32(tO + 32 * t, o);
        wait_ld(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fade);
        tmem_st32(tO + 32 * t, o);
      }
    }
  }
  l += sum;
#pragma unroll
  for (int t = 0; t < NB; ++t) tmem_st16(tS + col0 / 2 + 16 * t, w[t]);
  if (NB == 1) {   // the other copy's slots
    const uint32_t z[16] = {};
    tmem_st16(tS + 16 - col0 / 2, z);
  }
  wait_st();
}

// Weights of 32 scores, relative to m (mn2: -m twice); their sums on s2.
DF_DEVICE void weights(const uint32_t (&v)[32], uint64_t sc2, uint64_t mn2, uint64_t (&s2)[2], uint32_t (&w)[16]) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float a0, a1;
    unpack2(fma2(pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sc2, mn2), a0, a1);
    a0 = ex2(a0);
    a1 = ex2(a1);
    s2[(e >> 1) & 1] = add2(s2[(e >> 1) & 1], pack2(a0, a1));
    w[e / 2] = pack_bf16x2(a0, a1);
  }
}

// A chunk whose 128 slots the rows all see, each load under the weights before it.
// Halves of P are stored and told of (told(h)) as they are done; returns the first
// half that is not, because m has to move.
template <typename F>
DF_DEVICE int softmax_chunk(uint32_t tS, float scale, F told, float m, float& l) {
  const uint64_t sc2 = pack2(scale, scale), mn2 = pack2(-m, -m);
  uint32_t v[2][32], n[32], w[2][16];
  __syncwarp();
  tmem_ld32(tS, v[0]);
  wait_ld(v[0]);
  tmem_ld32(tS + 32, v[1]);
  uint64_t s2[2] = {0, 0};
  weights(v[0], sc2, mn2, s2, w[0]);
  wait_ld(v[1]);
  tmem_ld32(tS + 64, n);
  weights(v[1], sc2, mn2, s2, w[1]);
  wait_ld(n);
  float a0, a1;
  unpack2(add2(s2[0], s2[1]), a0, a1);
  float sum = a0 + a1;
  if (__any_sync(0xffffffffu, !(l + sum < 0x1p60f) || !(l + sum > 0x1p-60f))) return 0;
  l += sum;
  tmem_st16(tS, w[0]);
  tmem_st16(tS + 16, w[1]);
  wait_st();
  told(0);
  tmem_ld32(tS + 96, v[0]);
  s2[0] = s2[1] = 0;
  weights(n, sc2, mn2, s2, w[0]);
  wait_ld(v[0]);
  weights(v[0], sc2, mn2, s2, w[1]);
  unpack2(add2(s2[0], s2[1]), a0, a1);
  sum = a0 + a1;
  if (__any_sync(0xffffffffu, !(l + sum < 0x1p60f) || !(l + sum > 0x1p-60f))) return 1;
  l += sum;
  tmem_st16(tS + 64, w[0]);
  tmem_st16(tS + 80, w[1]);
  wait_st();
  told(1);
  return 2;
}

template <int N>
struct Int { static constexpr int value = N; };

// A segment (a run of a tile's chunks), planned by one warp for all: the
// arithmetic that finds it, and its instructions, are paid for once.
struct SegDesc {
  Entry x;
  int kvh, row0, left;   // kv head, first row, rows of the tile
  int node0, h0;         // node and query head of row 0
  int c0, nc;            // first chunk, chunks
  int whole, slot;       // the whole tile; else the slot of its partial rows
};
constexpr int kSegs = 8;

// Segment `seg` has been planned; false: there is none.  All warps get the same
// answer, also after a wait that gave up (they meet in barriers at a tile's end):
// the planning warp, whose own waits are bounded, tells the number of segments in
// any case.
DF_DEVICE bool seg_wait(int* planned, int* total, int seg, volatile int* abort, unsigned* status) {
  const long long t0 = clock64();
  while (true) {
    if (load_acquire(planned) > seg) return true;
    if (load_acquire(total) <= seg) return load_acquire(planned) > seg;
    if (clock64() - t0 > 4 * kWait) {
      *abort = 1;
      set_status(status, DEV_TIMEOUT);
      return false;
    }
  }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1) attend_umma_kernel(const __grid_constant__ UmmaParams p) {
  using Lt = Lay<HD>;
  constexpr int kMat = Lt::kMat, kHalf = Lt::kHalf, kHalves = Lt::kHalves;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int S = p.stages;
  uint8_t* ring = sm + Lt::kOffScratch + p.scratch;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + S * kMat);
  uint64_t* empty = full + S;
  uint64_t* q_full = empty + S;      // [2] the Q of an even (odd) segment is in shared memory
  uint64_t* q_free = q_full + 2;     // [2] Q area i is free
  uint64_t* s_full = q_free + 2;     // [2] S_i computed (and the stream's products before it done)
  uint64_t* p_full = s_full + 2;     // [2][2] half h of P_i stored
  uint64_t* pv_half = p_full + 4;    // [2] the first half of PV of a chunk of stream i is done
  uint64_t* turn = pv_half + 2;      // [2] stream i may issue (of a pair)
  uint64_t* o_full = turn + 2;       // the segment's products are done
  uint64_t* o_free = o_full + 1;     // the segment's O has been read
  long long* s_warp = reinterpret_cast<long long*>(o_free + 1);   // [12]
  long long* s_end = s_warp + 12;
  Entry* s_e = reinterpret_cast<Entry*>(s_end + p.a.rows.n_seq);
  __shared__ SegDesc s_seg[kSegs];
  __shared__ uint32_t s_tmem;
  __shared__ int s_issued;           // copies issued so far
  __shared__ int s_planned, s_total; // segments planned so far; all of them, once known
  __shared__ volatile int s_abort;

  const CacheView& c = p.a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.x;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      bar_init(&full[i], 1);
      bar_init(&empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&q_full[i], 1);
      bar_init(&q_free[i], 8);
      bar_init(&pv_half[i], 1);
      bar_init(&turn[i], 1);
      bar_init(&s_full[i], 1);
      bar_init(&p_full[2 * i], 4);
      bar_init(&p_full[2 * i + 1], 4);
    }
    bar_init(o_full, 2);
    bar_init(o_free, 8);
    s_abort = 0;
    s_issued = 0;
    s_planned = 0;
    s_total = 0x7fffffff;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&s_tmem)),
                 "n"(Lt::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32 * kProducer) {
    prefetch_map(&p.tm);
    if (p.q_boxes) prefetch_map(&p.tm_q);
  }
  pdl_trigger();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;
  // Few entries: warp 11 plans alone, and the roles wait for the launch before this
  // one where their instructions are, which are then there when it ends (together
  // with less to divide: 16 nodes over 2048 slots 16.4 us instead of 17.6).
  const bool few = p.a.rows.n_seq <= 32;
  if (!few) {
    pdl_wait();
    plan_entries(p.a, cutting(), s_e, s_end, s_warp, kThreads, b == 0);
  }

  if (warp >= 8) {
    if (warp == kProducer) {
      // ---------------------------------------------------------------- copies
      pdl_wait();
      const int none = c.n_pages * c.n_layer * 2 * c.n_head_kv;   // past the tensor: reads as zero
      int st = 0, ph = 1, n = 0, stop = 0;   // ring position, parity of its empty barrier, copies issued
      for (int seg = 0; !stop && seg_wait(&s_planned, &s_total, seg, &s_abort, c.status); ++seg) {
        const SegDesc& d = s_seg[seg % kSegs];
        const Entry x = d.x;
        const int32_t* table = c.table + (size_t)x.q * c.max_pages;
        const int last = (x.len + x.n - 1) >> c.ps_log2, head = p.a.layer * 2 * c.n_head_kv + d.kvh;
        const int c0 = d.c0, c1 = c0 + d.nc;
        int base = -64, row = none;             // lane i holds the tensor row of page base + i
        for (int ch = c0; ch < c1 && !stop; ++ch) {
          if (((ch * kChunk + kChunk - 1) >> c.ps_log2) > base + 31) {
            base = (ch * kChunk) >> c.ps_log2;
            row = none;
            if (base + lane <= last) {
              const int t = table[base + lane];
              if (t >= 0 && t < c.n_pages)
                row = t * c.n_layer * 2 * c.n_head_kv + head;
              else
                set_status(c.status, DEV_BAD_PAGE);
            }
          }
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++n) {
            if (lane == 0) {
              stop = !bar_wait(&empty[st], ph, &s_abort, c.status);
              if (!stop) {
                bar_expect(&full[st], kMat);
                publish(&s_issued, n + 1);
              }
            }
            stop = __shfl_sync(0xffffffffu, stop, 0);
            if (stop) break;
            uint8_t* dst = ring + st * kMat;
            for (int i = 0; i < kChunk; i += p.box_rows) {
              const int slot = ch * kChunk + i;
              const int r = __shfl_sync(0xffffffffu, row, ((slot >> c.ps_log2) - base) & 31);
              if (lane == 0)
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                  tma3d(dst + h * kHalf + i * 128, &p.tm, h * 64, slot & (c.ps - 1),
                        r == none ? none : r + kv * c.n_head_kv, &full[st]);
            }
            if (++st == S) {
              st = 0;
              ph ^= 1;
            }
          }
        }
      }
      // no copy may still be landing when the block ends
      if (lane == 0)
        for (int j = max(0, n - S); j < n; ++j) {
          const long long t0 = clock64();
          while (!bar_try(&full[j % S], (uint32_t)((j / S) & 1)) && clock64() - t0 < kWait) {
          }
        }
    } else if (warp < kIssuer + 2) {
      // -------------------------------------------------------------- products
      pdl_wait();
      if (lane == 0) {
        const int i = warp - kIssuer;
        // ring position of the segment's first K chunk, parities, copies before it
        int base = 0, bph = 0, n_p = 0, qb = 0, it = 0, n_t = i ^ 1;
        bool live = true;
        const uint64_t q0 = desc_k(su32(sm)), k0 = desc_k(su32(ring)), v0 = desc_mn(su32(ring), kHalf);
        const uint32_t dS = tmem + i * 128, dO = tmem + 256 + i * HD;
        for (int seg = 0; live && seg_wait(&s_planned, &s_total, seg, &s_abort, c.status); ++seg) {
          const SegDesc& d = s_seg[seg % kSegs];
          const bool pair = d.left > 128;
          const int nc = d.nc, mine = pair ? nc : (nc + 1 - i) >> 1;
          const uint64_t qa = q0 + (uint64_t)((pair ? i : qb) * (kMat >> 4));
          if (!pair) qb ^= 1;
          int st = base, ph = bph, no = it;   // the K chunk's stage, parity, number; its V chunk is the next
          it += 2 * nc;
          // a stage is free once both streams have read it (one, of a split tile)
          auto release = [&](int pos) {
            if (!pair) bar_arrive(&empty[pos]);
            commit(&empty[pos]);
          };
          auto scores = [&]() {
            const uint64_t kb = k0 + (uint64_t)(st * (kMat >> 4));
#pragma unroll
            for (int e = 0; e < HD / 16; ++e) {
              const uint32_t off = ((e >> 2) * kHalf + (e & 3) * 32) >> 4;
              mma_ss(dS, qa + off, kb + off, idesc(128, false), e > 0);
            }
            commit(&s_full[i]);
          };
          // The streams of a pair issue in turn: the pipe serves two issuers by halves,
          // and both streams' softmax would then wait for all products of both.
          auto my_turn = [&]() {
            if (!pair) return true;
            const bool ok = bar_wait(&turn[i], n_t, &s_abort, c.status);
            n_t ^= 1;
            return ok;
          };
          auto pass = [&]() {
            if (pair) bar_arrive(&turn[i ^ 1]);
          };
          if (!pair && i) {
            ring_step(st, ph, 2, S);
            no += 2;
          }
          live = bar_wait(&q_full[seg & 1], (seg >> 1) & 1, &s_abort, c.status);
          if (mine > 0 && live) {
            live = copy_wait(&s_issued, no, &full[st], ph, &s_abort, c.status) && my_turn();
            if (!live) break;
            fence_after();
            scores();
            release(st);
            pass();
          }
          // the last tile's accumulators have been read
          if (seg > 0) live = live && bar_wait(o_free, (seg & 1) ^ 1, &s_abort, c.status);
          for (int k = 0; k < mine && live; ++k) {
            int vs = st, vph = ph;
            ring_step(vs, vph, 1, S);
            ring_step(st, ph, 2, S);
            if (!pair) ring_step(st, ph, 2, S);
            live = copy_wait(&s_issued, no + 1, &full[vs], vph, &s_abort, c.status);
            no += pair ? 2 : 4;
            // with the next K chunk there, its scores follow PV at once
            const bool more = k + 1 < mine, ready = more && copy_there(&s_issued, no, &full[st], ph);
            const uint64_t vb = v0 + (uint64_t)(vs * (kMat >> 4));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              live = live && bar_wait(&p_full[2 * i + h], n_p, &s_abort, c.status) && (!h || my_turn());
              if (!live) break;
              fence_after();
#pragma unroll
              for (int e = 0; e < 4; ++e)   // 16 slots: 2 groups of 1024 bytes
                mma_ts(dO, dS + 64 * h + 8 * e, vb + ((h * 8192 + e * 2048) >> 4), idesc(HD, true), k + h + e > 0);
              if (h == 0) commit(&pv_half[i]);
            }
            if (!live) break;
            n_p ^= 1;
            release(vs);
            if (more) {
              if (!ready) live = copy_wait(&s_issued, no, &full[st], ph, &s_abort, c.status);
              if (!live) break;
              fence_after();
              scores();
              release(st);
            }
            pass();
          }
          if (!live) break;
          commit(o_full);
          const int to = base + 2 * nc;
          bph ^= (to / S) & 1;
          base = to % S;
        }
      }
      __syncwarp();
    } else {
      // ----------------------------------------------------- segments, queries
      pdl_wait();
      if (lane == 0) p.cuts[b] = {0, 0, 0, 0, -1, 0};
      if (few) plan_few(p.a, cutting(), s_e, s_end, b == 0);
      const long long U = s_end[p.a.rows.n_seq - 1];
      // fewer blocks than launched where their shares would get too small
      const int Gr = blocks_used(U, gridDim.x, kMinUnits), grp = p.a.grp;
      const long long ub0 = U > 0 && b < Gr ? range_begin(U, Gr, b) : 0;
      const long long ub1 = U > 0 && b < Gr ? range_begin(U, Gr, b + 1) : 0;
      long long u = ub0;
      int s = ub1 > ub0 ? find_entry(s_end, p.a.rows.n_seq, ub0) : 0, planned = 0;
      bool more = true, live = true;
      int free_par[2] = {1, 1}, qb = 0;
      for (int seg = 0; live; ++seg) {
        // (from the second on) three segments ahead, for the copies (a description's last reader is done
        // when the Q of the fifth segment after it has been loaded)
        while (more && planned < (seg ? seg + 3 : 1)) {
          Segment g;
          more = next_segment(p.a, cutting(), s_e, s_end, u, ub1, s, g);
          if (!more) {
            if (lane == 0) publish(&s_total, planned);
            break;
          }
          const Entry x = s_e[g.s];
          SegDesc& d = s_seg[planned % kSegs];
          const int left = (int)min((long long)x.n * grp - g.row0, (long long)kTile);
          if (lane == 0) {
            d.x = x;
            d.kvh = g.kvh;
            d.row0 = g.row0;
            d.left = left;
            d.node0 = g.row0 ? g.row0 / grp : 0;
            d.h0 = g.row0 - d.node0 * grp;
            d.c0 = g.c0;
            d.nc = g.c1 - g.c0;
            d.whole = g.c0 == 0 && g.c1 == g.nch;
            // partial rows: slot 0 of the block if its range starts in the tile, else 1
            d.slot = 2 * b + (ub0 >= g.u0 ? 0 : 1);
            // the block with a cut tile's first chunk describes it to the join
            if (g.c0 == 0 && !d.whole)
              p.cuts[b] = {x.lo, g.row0, g.kvh, left, block_of(U, Gr, g.u0 + (long long)(g.nch - 1) * g.w), d.slot};
            publish(&s_planned, planned + 1);
          }
          __syncwarp();
          ++planned;
        }
        if (seg >= planned) break;
        // Q: lane q of tile t is row 128 t + q of a pair, row q % per of a split tile
        const SegDesc& d = s_seg[seg % kSegs];
        const int left = d.left;
        const bool pair = left > 128;
        const int per = left > 64 ? 128 : 64;
        for (int y = 0; y < (pair ? 2 : 1); ++y) {
          const int area = pair ? y : qb;
          live = live && bar_wait(&q_free[area], free_par[area], &s_abort, c.status);
          free_par[area] ^= 1;
        }
        if (!live) break;
        if (p.q_boxes) {
          // (groups of 32 rows that do not exist stay as they are: their lanes count
          // for nothing)
          const int groups = (pair ? (left + 31) >> 5 : (left + 31) >> 5 << (per == 64));
          if (lane == 0) {
            bar_expect(&q_full[seg & 1], groups * 4096 * kHalves);
            for (int z = 0; z < (pair ? 8 : 4); ++z) {
              const int r = pair ? 32 * z : 32 * z & (per - 1);
              if (r >= left) continue;
              uint8_t* dst = sm + (pair ? z >> 2 : qb) * kMat + (z & 3) * 4096;
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                tma3d(dst + h * kHalf, &p.tm_q, h * 64, d.kvh * grp, d.x.lo + d.node0 + small_quotient(r, p.grp_magic),
                      &q_full[seg & 1]);
            }
          }
        } else {
          constexpr int kPc = HD / 8, kStep = 32 / kPc;   // 16-byte pieces of a row, rows of a warp's copy
          const int pc = lane & (kPc - 1);
          const char* q_row = p.a.q + (size_t)d.x.lo * p.a.q_ld + (size_t)d.kvh * grp * HD * 2 + pc * 16;
          for (int y = 0; y < (pair ? 2 : 1); ++y) {
            uint8_t* dst0 = sm + (pair ? y : qb) * kMat + (pc >> 3) * kHalf;
#pragma unroll 2
            for (int q = lane / kPc; q < per; q += kStep) {
              const int r = pair ? y * 128 + q : q;
              const bool real = r < left;
              const int x = d.h0 + (real ? r : 0), nd = small_quotient(x, p.grp_magic), h = x - nd * grp;
              const char* src = q_row + (size_t)(d.node0 + nd) * p.a.q_ld + h * HD * 2;
              for (int z = q; z < 128; z += per)   // the row's copies
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 su32(dst0 + z * 128 + (((pc & 7) ^ (z & 7)) << 4))),
                             "l"(src), "r"(real ? 16 : 0)
                             : "memory");
            }
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_async();
          __syncwarp();
          if (lane == 0) bar_arrive(&q_full[seg & 1]);
        }
        if (!pair) qb ^= 1;
        __syncwarp();
      }
      if (lane == 0) publish(&s_total, planned);   // (known already, unless a wait gave up)
      // (a Q that was loaded is a segment's that runs: no copy is in flight at the end)
    }
  } else {
    // ------------------------------------------------------------------ rows
    pdl_wait();
    const int i = warp >> 2, pos = tid & 127;     // stream, lane of the tile
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // the warp's tensor-memory lanes: 32 (warp % 4) << 16
    const uint32_t tS = tmem + i * 128 + lanes, tO = tmem + 256 + i * HD + lanes;
    const float scale = p.a.scale * kLog2e;
    int n_s = 0, qb = 0, it = 0;   // the stream's chunks so far, Q area, copies so far
    bool live = true;   // after a wait that gave up: no more arrivals
    for (int seg = 0;; ++seg) {
      int there = 0;
      if (lane == 0) there = seg_wait(&s_planned, &s_total, seg, &s_abort, c.status);
      if (!__shfl_sync(0xffffffffu, there, 0)) break;
      const SegDesc& d = s_seg[seg % kSegs];
      const int left = d.left, nc = d.nc, ch0 = d.c0, end = d.x.len + d.x.n;
      // the slots that all rows see (of a chain those of its nodes up to the tile's first)
      const int all = d.x.len + (p.a.mask ? 0 : d.node0 + 1);
      const bool pair = left > 128;
      const int rep = left > 64 ? 1 : 2, per = 128 / rep;   // copies of a row, rows
      const int steps = pair ? 2 * nc : nc;
      const int row = pair ? i * 128 + pos : pos & (per - 1);
      const int col0 = rep == 2 ? pos >> 6 << 5 : 0;   // the copy's share of 64 slots: col0 .. col0 + 64 / rep - 1
      const bool real = row < left;
      const int node = real ? d.node0 + small_quotient(d.h0 + row, p.grp_magic) : 0;
      const bool idle = !__any_sync(0xffffffffu, real);   // S and so P are zero, or of no row
      float m = 0.f, l = 0.f;
      // the stream is done with the tile's Q (a pair: its own area, which takes 8
      // arrivals too).  A stream without a chunk says so at the tile's end, when its
      // issuer has seen that Q was there.
      auto free_q = [&]() {
        if (lane == 0 && live) bar_arrive_n(&q_free[pair ? i : qb], pair ? 2 : 1);
      };
      auto step = [&](auto nb, int h, int slot0, bool part, bool later) {
        constexpr int NB = decltype(nb)::value;
        // the stream's products so far are done (those of chunks before this one
        // preceded its scores)
        auto settle = [&]() {
          if (h) live = live && bar_wait(&pv_half[i], n_s & 1, &s_abort, c.status);
          fence_after();
        };
        if (part)
          softmax_step<NB, HD, true>(p.a, d.x, node, slot0, col0, tS + 64 * h, tO, scale, later, settle, m, l);
        else
          softmax_step<NB, HD, false>(p.a, d.x, node, slot0, col0, tS + 64 * h, tO, scale, later, settle, m, l);
      };
      for (int k = i; k < steps; k += 2, ++n_s) {
        const int j = pair ? k >> 1 : k, slot0 = (ch0 + j) * kChunk;
        const bool masked = slot0 + kChunk > all;
        if (masked && real && p.a.mask) prefetch_mask(p.a, d.x, node, slot0);
        if (slot0 + kChunk > end) {
          // slots past the last node may hold anything: 0 x NaN is NaN (of a pair,
          // each stream clears them before its own products)
          const int r = it + 2 * j + 1, st = r % S;
          live = live && copy_wait(&s_issued, r, &full[st], (uint32_t)((r / S) & 1), &s_abort, c.status);
          const int first = max(0, end - slot0);
          for (int e = first * (HD / 8) + pos; e < kChunk * (HD / 8); e += 128) {
            const int q = e / (HD / 8), pc = e - q * (HD / 8);
            *reinterpret_cast<uint4*>(ring + st * kMat + (pc >> 3) * kHalf + q * 128 + (((pc & 7) ^ (q & 7)) << 4)) =
                make_uint4(0, 0, 0, 0);
          }
          fence_async();
        }
        live = live && bar_wait(&s_full[i], n_s & 1, &s_abort, c.status);
        if (p.scratch && k + 2 >= steps) free_q();   // the stream's last scores
        fence_after();
        auto told = [&](int h) {
          fence_before();
          __syncwarp();
          if (lane == 0 && live) bar_arrive(&p_full[2 * i + h]);
        };
        int h = 0;
        if (!idle && rep == 1 && !masked) h = softmax_chunk(tS, scale, told, m, l);
#pragma unroll 1
        for (; h < 2; ++h) {
          if (!idle) {
            const int slot = slot0 + 64 * h;
            if (rep == 1)
              step(Int<2>(), h, slot, slot + 64 > all, k > 1 || h);
            else
              step(Int<1>(), h, slot, slot + 64 > all, k > 1 || h);
          }
          told(h);
        }
      }
      it += 2 * nc;

      // ---- the tile's end
      live = live && bar_wait(o_full, seg & 1, &s_abort, c.status);
      fence_after();
      if (l == 0.f) m = -CUDART_INF_F;   // nothing attended: no reference to others
      const bool whole = d.whole;
      const int slot = d.slot;
      auto out_row = [&](int r, char*& dst, float*& lse) {
        const int y = d.h0 + r, nd = small_quotient(y, p.grp_magic), h = d.kvh * p.a.grp + y - nd * p.a.grp;
        dst = p.a.out + (size_t)(d.x.lo + d.node0 + nd) * p.a.out_ld + (size_t)h * HD * 2;
        lse = p.a.lse ? p.a.lse + (size_t)(d.x.lo + d.node0 + nd) * c.n_head + h : nullptr;
      };
      // Row weights of the accumulators.  A split tile's row lies in both streams'
      // accumulators (the same tensor-memory lane, other columns) and, with copies,
      // in 2 or 4 lanes of each; stream i's warps write half i of its dims.
      float* area = reinterpret_cast<float*>(sm + (p.scratch ? Lt::kOffScratch : qb * kMat));   // 32 KB
      float top = m, sum = l, wa = 1.f, wb = 0.f;
      if (!pair) {
        float2* ml = reinterpret_cast<float2*>(area);   // [stream][lane of the tile]
        ml[tid] = i < steps ? make_float2(m, l) : make_float2(-CUDART_INF_F, 0.f);
        sync_rows();
        top = -CUDART_INF_F;
        sum = 0.f;
        for (int y = row; y < 256; y += per) top = fmaxf(top, ml[y].x);
        const float use = top == -CUDART_INF_F ? 0.f : top;
        for (int y = row; y < 256; y += per) sum += ex2(ml[y].x - use) * ml[y].y;
        wa = ex2(ml[pos].x - use);
        wb = ex2(ml[128 + pos].x - use);
        sync_rows();   // the area is the accumulators' from here on
      }
      if (whole) {
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        wa *= inv;
        wb *= inv;
      }
      char* dst = reinterpret_cast<char*>(p.part_o + ((size_t)slot * kTile + row) * HD);
      if (real) {
        float* lse;
        if (whole) out_row(row, dst, lse);
        if (pair || (i == 0 && pos < per)) {
          if (!whole)
            p.part_ml[(size_t)slot * kTile + row] = make_float2(top, sum);
          else if (lse)
            *lse = sum > 0.f ? (top + log2f(sum)) * kLn2 : -CUDART_INF_F;
        }
      }
      // 32 weighted columns of this thread's row: column d of stream 0's (a pair: of
      // the own) accumulator, and of stream 1's
      const uint32_t tA = pair ? tO : tmem + 256 + lanes;
      auto columns = [&](int d, float (&f)[32]) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(tA + d, v);
        wait_ld(v);
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(v[e]) * wa;
        if (!pair && steps > 1) {   // (an accumulator that was never written may hold anything)
          tmem_ld32(tA + HD + d, v);
          wait_ld(v);
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] += __uint_as_float(v[e]) * wb;
        }
      };
      if (rep == 1) {
        // 32 rows x 32 dims of a warp at a time through its 4 KB of the area, so that
        // rows are written as whole sectors by neighbouring lanes (16-byte pieces of a
        // thread's own row took 10000 clocks a tile)
        float* buf = area + warp * 1024;
        const int last = left - (row - lane), d1 = pair ? HD : HD / 2;   // rows of the warp that exist; its dims
        if (!idle)
#pragma unroll 1
          for (int d0 = 0; d0 < d1; d0 += 32) {
            const int dim = (pair ? 0 : i * (HD / 2)) + d0;
            float f[32];
            columns(dim, f);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<float4*>(buf + lane * 32 + ((q ^ (lane & 7)) << 2)) =
                  make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
            __syncwarp();
            // (loads first, then stores: a branch between them made it 125 clocks a row of four)
            const int q = lane & 7;
            float4 x[8];
            unsigned long long to[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int r = 4 * e + (lane >> 3);
              x[e] = *reinterpret_cast<const float4*>(buf + r * 32 + ((q ^ (r & 7)) << 2));
              to[e] = __shfl_sync(0xffffffffu, (unsigned long long)dst, r);
            }
            if (whole) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (4 * e + (lane >> 3) < last)
                  *reinterpret_cast<uint2*>(to[e] + (dim + 4 * q) * 2) =
                      make_uint2(pack_bf16x2(x[e].x, x[e].y), pack_bf16x2(x[e].z, x[e].w));
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (4 * e + (lane >> 3) < last) *reinterpret_cast<float4*>(to[e] + (dim + 4 * q) * 4) = x[e];
            }
          }
      } else {
        // the copies of a row summed through the area, in one or two passes over the dims
        const int lines = rep * left, line = pos / per * left + row;
        const int D = lines * HD <= 8192 ? HD : HD / 2, ql = __ffs(D) - 3;   // D / 4 = 2^ql
#pragma unroll 1
        for (int p0 = 0; p0 < HD; p0 += D) {
          if (!idle)
#pragma unroll 1
            for (int d0 = i * (D / 2); d0 < (i + 1) * (D / 2); d0 += 32) {
              float f[32];
              columns(p0 + d0, f);
              if (real)
#pragma unroll
                for (int q = 0; q < 8; ++q)
                  *reinterpret_cast<float4*>(area + line * D + d0 + ((q ^ (line & 7)) << 2)) =
                      make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
            }
          sync_rows();
          for (int e0 = tid; e0 < left << ql; e0 += 1024) {   // four at a time
            float4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int y = 0; y < rep; ++y)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int e = e0 + 256 * k, r = e >> ql, q = e - (r << ql), at = y * left + r;
                if (r >= left) continue;
                const float4 f =
                    *reinterpret_cast<const float4*>(area + at * D + (q & ~7) * 4 + (((q & 7) ^ (at & 7)) << 2));
                x[k].x += f.x;
                x[k].y += f.y;
                x[k].z += f.z;
                x[k].w += f.w;
              }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e = e0 + 256 * k, r = e >> ql, dim = p0 + 4 * (e - (r << ql));
              if (r >= left) continue;
              if (whole) {
                char* to;
                float* lse;
                out_row(r, to, lse);
                *reinterpret_cast<uint2*>(to + dim * 2) =
                    make_uint2(pack_bf16x2(x[k].x, x[k].y), pack_bf16x2(x[k].z, x[k].w));
              } else {
                *reinterpret_cast<float4*>(p.part_o + ((size_t)slot * kTile + r) * HD + dim) = x[k];
              }
            }
          }
          if (D < HD) sync_rows();
        }
      }
      // O has been read (and the tile's Q area, if it was the end's memory, is free)
      fence_before();
      __syncwarp();
      if (lane == 0 && live) bar_arrive(o_free);
      if (!p.scratch) fence_async();   // the next Q comes by TMA
      __syncwarp();
      if (!p.scratch || i >= steps) free_q();
      if (!pair) qb ^= 1;
    }
  }

  fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(Lt::kCols) : "memory");
  }
}

template <int HD>
constexpr size_t fixed_smem(int n_seq) {   // without the ring
  return 1024 + Lay<HD>::kOffScratch + 16 * 8 + 12 * 8 + (size_t)n_seq * (sizeof(long long) + sizeof(Entry));
}
constexpr size_t kSmemMost = 227 * 1024 - 512;   // static shared memory aside
// stages of the ring (128 dims: 5, beside the scratch 4, there with 53 entries and more 3)
template <int HD>
constexpr int ring_stages(int n_seq, int scratch) {
  const size_t n = (kSmemMost - fixed_smem<HD>(n_seq) - scratch) / (Lay<HD>::kMat + 16);
  return n > Lay<HD>::kStagesMost ? Lay<HD>::kStagesMost : (int)n;
}
// (a stream's chunk and the next one's keys)
static_assert(ring_stages<128>(kCallSeq, kScratch) >= 3 && ring_stages<64>(kCallSeq, kScratch) >= 3, "ring too short");

// The call's queries as a 3-D tensor (made per call: it names the caller's buffer).
bool q_map(CUtensorMap* m, const AttendParams& a, uint32_t grp) {
  const EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)a.c.hd, (cuuint64_t)a.c.n_head, (cuuint64_t)a.rows.T};
  const cuuint64_t strides[2] = {(cuuint64_t)a.c.hd * 2, (cuuint64_t)a.q_ld};
  const cuuint32_t box[3] = {64, grp, 32 / grp}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<char*>(a.q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD>
cudaError_t umma_as(const AttendParams& a, const AttendWork& w, cudaStream_t st) {
  using Lt = Lay<HD>;
  UmmaParams p;
  p.tm = *w.tm;
  p.a = a;
  p.a.step = trim_step(a, kTile, kChunk);
  const uint32_t grp = a.grp;
  p.q_boxes = 32 % grp == 0;
  if (p.q_boxes && !q_map(&p.tm_q, a, grp)) return cudaErrorInvalidValue;
  p.part_o = w.part_o;
  p.part_ml = w.part_ml;
  p.cuts = w.cuts;
  p.box_rows = a.c.ps < kChunk ? a.c.ps : kChunk;
  // pairs fill both Q areas; split tiles of 128 dims alternate between them and
  // are bound by memory, where the stage counts for more
  const bool pairs = (long long)a.max_tree * a.grp > kWide;
  p.grp_magic = quotient_magic(grp);
  p.scratch = pairs || HD == 64 ? kScratch : 0;
  p.stages = ring_stages<HD>(a.rows.n_seq, p.scratch);
  const size_t smem = fixed_smem<HD>(a.rows.n_seq) + p.scratch + (size_t)p.stages * (Lt::kMat + 16);
  const cudaError_t e = launch_dependent(attend_umma_kernel<HD>, dim3(w.sms), kThreads, smem, st, p);
  if (e != cudaSuccess) return e;
  return launch_join<2, HD>(a, w, kTile, w.sms, st);
}

}  // namespace

cudaError_t configure_attend_umma() {
  const cudaError_t e = cudaFuncSetAttribute(attend_umma_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kSmemMost);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(attend_umma_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMost);
}

cudaError_t launch_attend_umma(const AttendParams& a, const AttendWork& w, cudaStream_t st) {
  return a.c.hd == 64 ? umma_as<64>(a, w, st) : umma_as<128>(a, w, st);
}

}  // namespace dflash
