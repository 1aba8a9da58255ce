// C ABI of the target model's side (include/dflash.h): cache handle, checks,
// rotation table, device-memory layout.  The kernels are in cache.cu, rope.cu
// and tree_attention.cu.
#include "../../include/dflash.h"
#include "cache.h"
#include "internal.h"

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <new>

using namespace dflash;

static_assert(DFLASH_MAX_TREE == kTreeMax && DFLASH_MAX_CALL_SEQ == kCallSeq, "limits of the header");
static_assert(DFLASH_DEV_BAD_POSITION == DEV_BAD_POSITION && DFLASH_DEV_TIMEOUT == DEV_TIMEOUT &&
                  DFLASH_DEV_BAD_ROWS == DEV_BAD_ROWS && DFLASH_DEV_BAD_PAGE == DEV_BAD_PAGE &&
                  DFLASH_DEV_BAD_TREE == DEV_BAD_TREE && DFLASH_DEV_BAD_SEQ == DEV_BAD_SEQ &&
                  DFLASH_DEV_NO_PAGES == DEV_NO_PAGES,
              "status bits of the header");

namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxSeq = 4096;   // rows of the page table

size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct Layout {
  size_t page_bytes;
  size_t table, length, refs, state_bytes;
  size_t status, turns, tickets, free_list, copies, part_o, part_ml, cuts, scratch_bytes;
};

int el_of(const dflash_cache_config& c) { return c.dtype == DFLASH_DTYPE_BF16 ? 2 : 4; }

Layout layout(const dflash_cache_config& c) {
  Layout L{};
  L.page_bytes = (size_t)c.n_pages * c.n_layer * 2 * c.n_head_kv * c.page_size * c.head_dim * el_of(c);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = up(off + bytes);
    return o;
  };
  L.table = take(sizeof(int32_t) * (size_t)c.max_seq * c.max_pages);
  L.length = take(sizeof(int32_t) * (size_t)c.max_seq);
  L.refs = take(sizeof(int32_t) * (size_t)c.n_pages);
  L.state_bytes = off;
  off = 0;
  L.status = take(sizeof(unsigned));
  L.turns = take(sizeof(unsigned long long) * 64);
  L.tickets = take(sizeof(int) * kCallSeq);
  L.free_list = take(sizeof(int32_t) * (size_t)c.n_pages);
  L.copies = take(sizeof(int4) * kCallSeq);
  const size_t parts = attend_part_rows(el_of(c), c.head_dim);
  L.part_o = take(sizeof(float) * parts * c.head_dim);
  L.part_ml = take(sizeof(float2) * parts);
  L.cuts = take(sizeof(Cut) * 2 * kAttendSms);
  L.scratch_bytes = off;
  return L;
}

int validate(const dflash_cache_config* c) {
  if (!c) return DFLASH_ERR_INVALID_ARG;
  if (c->n_layer < 1 || c->n_head < 1 || c->n_head_kv < 1 || c->head_dim < 1 || c->page_size < 1 ||
      c->n_pages < 1 || c->max_seq < 1 || c->max_pages < 1 || c->rotary_dim < 0)
    return DFLASH_ERR_INVALID_ARG;
  if (c->dtype < DFLASH_DTYPE_F32 || c->dtype > DFLASH_DTYPE_FP4_E2M1) return DFLASH_ERR_INVALID_ARG;
  if (c->rope_layout != DFLASH_ROPE_HALF && c->rope_layout != DFLASH_ROPE_INTERLEAVED)
    return DFLASH_ERR_INVALID_ARG;
  if (c->rope_scaling < DFLASH_ROPE_NONE || c->rope_scaling > DFLASH_ROPE_YARN)
    return DFLASH_ERR_INVALID_ARG;
  if (!std::isfinite(c->attn_scale) || c->attn_scale < 0.f || !std::isfinite(c->rope_mscale) || c->rope_mscale < 0.f)
    return DFLASH_ERR_INVALID_ARG;
  if (c->rotary_dim > 0) {
    if (!(c->rope_theta > 1.0) || !std::isfinite(c->rope_theta) || !(c->rope_factor >= 1.f) ||
        !std::isfinite(c->rope_factor))
      return DFLASH_ERR_INVALID_ARG;
    if (c->rope_scaling == DFLASH_ROPE_YARN &&
        (c->rope_orig_positions < 1 || !(c->rope_beta_slow > 0.f) || !std::isfinite(c->rope_beta_fast) ||
         !(c->rope_beta_fast >= c->rope_beta_slow)))
      return DFLASH_ERR_INVALID_ARG;
    if (c->rope_scaling == DFLASH_ROPE_NTK && c->rotary_dim <= 2) return DFLASH_ERR_INVALID_ARG;
  }
  if (c->dtype != DFLASH_DTYPE_F32 && c->dtype != DFLASH_DTYPE_BF16) return DFLASH_ERR_UNSUPPORTED;
  if (c->n_head % c->n_head_kv) return DFLASH_ERR_UNSUPPORTED;
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) return DFLASH_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return DFLASH_ERR_UNSUPPORTED;
  if (c->rotary_dim > c->head_dim || c->rotary_dim % 8) return DFLASH_ERR_UNSUPPORTED;
  // (a tile of slots may reach past the last one: slot numbers stay below 2^31 there too)
  if (c->max_seq > kMaxSeq || (long long)c->max_pages * c->page_size > (1LL << 31) - 1024)
    return DFLASH_ERR_UNSUPPORTED;
  if (c->n_head > 4096 || c->n_layer > 4096) return DFLASH_ERR_UNSUPPORTED;
  if ((long long)c->n_layer * 2 * c->n_head_kv * c->n_pages > 0x7fffffffLL) return DFLASH_ERR_UNSUPPORTED;
  return DFLASH_OK;
}

// Angle per position of pair j, in turns scaled by 2^64 (fp64 on the host).
void rope_turns(const dflash_cache_config& c, unsigned long long (&t)[64]) {
  const double r = c.rotary_dim, F = c.rope_factor, two_pi = 2.0 * M_PI;
  double theta = c.rope_theta;
  if (c.rope_scaling == DFLASH_ROPE_NTK) theta *= std::pow(F, r / (r - 2.0));
  double lo = 0.0, hi = 0.0;
  if (c.rope_scaling == DFLASH_ROPE_YARN) {
    auto dim = [&](double b) { return r * std::log(c.rope_orig_positions / (two_pi * b)) / (2.0 * std::log(theta)); };
    lo = std::max(std::floor(dim(c.rope_beta_fast)), 0.0);
    hi = std::min(std::ceil(dim(c.rope_beta_slow)), r - 1.0);
  }
  for (int j = 0; j < 64; ++j) {
    t[j] = 0;
    if (2 * j >= c.rotary_dim) continue;
    double f = std::pow(theta, -2.0 * j / r);
    if (c.rope_scaling == DFLASH_ROPE_LINEAR) f /= F;
    if (c.rope_scaling == DFLASH_ROPE_YARN) {
      const double w = std::min(std::max((j - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
      f = f * (w / F + 1.0 - w);
    }
    t[j] = (unsigned long long)std::ldexp(f / two_pi, 64);   // f <= 1: below 2^62
  }
}

float rope_mscale(const dflash_cache_config& c) {
  if (c.rope_mscale > 0.f) return c.rope_mscale;
  return c.rope_scaling == DFLASH_ROPE_YARN && c.rope_factor > 1.f
             ? (float)(0.1 * std::log((double)c.rope_factor) + 1.0) : 1.f;
}

}  // namespace

struct dflash_cache {
  dflash_cache_config cfg;
  Layout L;
  CacheView v;
  RopeView rope;
  CUtensorMap tm;
  AttendWork work;
  char* scratch;
  int device;
  char err[512];

  template <typename T>
  T* S(size_t off) const { return reinterpret_cast<T*>(scratch + off); }
};

namespace {

int cuda_fail(dflash_cache* c, cudaError_t e, const char* where) {
  if (c) std::snprintf(c->err, sizeof(c->err), "%s: %s", where, cudaGetErrorString(e));
  return DFLASH_ERR_CUDA;
}

#define DC_CHECK(c, call)                                   \
  do {                                                      \
    cudaError_t e_ = (call);                                \
    if (e_ != cudaSuccess) return cuda_fail(c, e_, #call);  \
  } while (0)

// The handle's device for the duration of a call; clears a stale error of
// earlier unrelated work, so that it is not reported as this call's.
struct OnDevice {
  int was = -1;
  explicit OnDevice(int device) {
    (void)cudaGetLastError();
    int cur = device;
    if (cudaGetDevice(&cur) == cudaSuccess && cur != device && cudaSetDevice(device) == cudaSuccess) was = cur;
  }
  ~OnDevice() {
    if (was >= 0) cudaSetDevice(was);
  }
};

bool bad_area(const void* p, size_t align) {
  return !p || (reinterpret_cast<uintptr_t>(p) & (align - 1));
}

// The pages as a 3-D tensor [rows of (page, layer, k|v, head)][page_size][hd], in
// boxes of up to `rows` slots of one row and 128 bytes (a whole head of 64) of
// each: 64- and 128-byte rows swizzled, rows past the tensor read as zero.
bool page_map(CUtensorMap* m, const CacheView& v, int rows) {
  const EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const uint32_t row_bytes = v.hd * v.el, box_bytes = row_bytes < 128 ? row_bytes : 128;
  const cuuint64_t dims[3] = {(cuuint64_t)v.hd, (cuuint64_t)v.ps,
                              (cuuint64_t)v.n_pages * v.n_layer * 2 * v.n_head_kv};
  const cuuint64_t strides[2] = {row_bytes, (cuuint64_t)row_bytes * v.ps};
  const cuuint32_t box[3] = {box_bytes / v.el, (cuuint32_t)(v.ps < rows ? v.ps : rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, v.el == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, v.pages, dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A [T][heads][head_dim] operand: 16-byte aligned, rows at least a row apart.
bool bad_rows(const dflash_cache* c, const void* p, int64_t stride, int64_t heads) {
  return bad_area(p, 16) || stride < heads * c->cfg.head_dim || (stride * el_of(c->cfg)) % 16;
}

int check_call(const dflash_cache* c, int n_seq, const int32_t* row_start, int T) {
  if (!c || T < 0 || (n_seq > 0 && !row_start)) return DFLASH_ERR_INVALID_ARG;
  if (n_seq < 0 || n_seq > kCallSeq) return DFLASH_ERR_SEQ_RANGE;
  return DFLASH_OK;
}

// Entries of the calls that change the page table: identity entries have to exist.
int check_entries(const dflash_cache* c, int n_seq, const int32_t* seqs, const int32_t* arg) {
  if (!c || (n_seq > 0 && !arg)) return DFLASH_ERR_INVALID_ARG;
  if (n_seq < 0 || n_seq > kCallSeq || (!seqs && n_seq > c->cfg.max_seq)) return DFLASH_ERR_SEQ_RANGE;
  return DFLASH_OK;
}

}  // namespace

int dflash_cache_workspace_size(const dflash_cache_config* cfg, size_t* page_bytes, size_t* state_bytes,
                                size_t* scratch_bytes) {
  const int v = validate(cfg);
  if (v != DFLASH_OK) return v;
  if (!page_bytes || !state_bytes || !scratch_bytes) return DFLASH_ERR_INVALID_ARG;
  const Layout L = layout(*cfg);
  *page_bytes = L.page_bytes;
  *state_bytes = L.state_bytes;
  *scratch_bytes = L.scratch_bytes;
  return DFLASH_OK;
}

int dflash_cache_create(const dflash_cache_config* cfg, void* page_mem, void* state_mem, void* scratch_mem,
                        dflash_cache** out) {
  if (!out) return DFLASH_ERR_INVALID_ARG;
  *out = nullptr;
  const int v = validate(cfg);
  if (v != DFLASH_OK) return v;
  if (bad_area(page_mem, kAlign) || bad_area(state_mem, kAlign) || bad_area(scratch_mem, kAlign))
    return DFLASH_ERR_INVALID_ARG;
  dflash_cache* c = new (std::nothrow) dflash_cache();
  if (!c) return DFLASH_ERR_INVALID_ARG;
  c->cfg = *cfg;
  c->L = layout(*cfg);
  c->scratch = static_cast<char*>(scratch_mem);
  c->err[0] = 0;
  char* state = static_cast<char*>(state_mem);
  CacheView& w = c->v;
  w.pages = static_cast<char*>(page_mem);
  w.table = reinterpret_cast<int32_t*>(state + c->L.table);
  w.length = reinterpret_cast<int32_t*>(state + c->L.length);
  w.refs = reinterpret_cast<int32_t*>(state + c->L.refs);
  w.status = c->S<unsigned>(c->L.status);
  w.n_layer = cfg->n_layer;
  w.n_head = cfg->n_head;
  w.n_head_kv = cfg->n_head_kv;
  w.hd = cfg->head_dim;
  w.ps = cfg->page_size;
  w.ps_log2 = 0;
  while ((1 << w.ps_log2) < w.ps) ++w.ps_log2;
  w.n_pages = cfg->n_pages;
  w.max_seq = cfg->max_seq;
  w.max_pages = cfg->max_pages;
  w.el = el_of(*cfg);
  c->rope = {c->S<unsigned long long>(c->L.turns), cfg->rotary_dim, cfg->rope_layout == DFLASH_ROPE_INTERLEAVED,
             rope_mscale(*cfg)};
  (void)cudaGetLastError();
  // all three areas are memory of one device, which is the handle's
  cudaError_t e = cudaSuccess;
  c->device = -1;
  for (const void* area : {static_cast<const void*>(page_mem), static_cast<const void*>(state_mem),
                           static_cast<const void*>(scratch_mem)}) {
    cudaPointerAttributes at;
    if (e == cudaSuccess) e = cudaPointerGetAttributes(&at, area);
    if (e != cudaSuccess) break;
    if (at.type != cudaMemoryTypeDevice || (c->device >= 0 && at.device != c->device))
      e = cudaErrorInvalidDevicePointer;
    c->device = at.device;
  }
  if (e == cudaSuccess) {
    OnDevice on(c->device);
    unsigned long long turns[64] = {};
    if (cfg->rotary_dim > 0) rope_turns(*cfg, turns);
    // (the areas may be memory that work in flight on some stream still writes: an
    // allocator hands a freed block out again in its own stream's order)
    e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemset(c->scratch, 0, c->L.scratch_bytes);
    if (e == cudaSuccess) e = cudaMemset(w.table, 0xff, sizeof(int32_t) * (size_t)w.max_seq * w.max_pages);
    if (e == cudaSuccess) e = cudaMemset(w.length, 0, sizeof(int32_t) * w.max_seq);
    if (e == cudaSuccess) e = cudaMemset(w.refs, 0, sizeof(int32_t) * w.n_pages);
    if (e == cudaSuccess)
      e = cudaMemcpy(c->S<void>(c->L.turns), turns, sizeof(turns), cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = configure_tree();
    if (e == cudaSuccess) e = configure_attend();
    int sms = 0;
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, c->device);
    if (e == cudaSuccess && !page_map(&c->tm, w, attend_chunk(w.el, w.hd))) e = cudaErrorNotSupported;
    c->work = {&c->tm, c->S<float>(c->L.part_o), c->S<float2>(c->L.part_ml),
               c->S<Cut>(c->L.cuts), std::min(sms, kAttendSms)};
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
  }
  if (e != cudaSuccess) {
    cuda_fail(c, e, "dflash_cache_create");
    std::fprintf(stderr, "dflash_cache_create: %s\n", c->err);
    delete c;
    return DFLASH_ERR_CUDA;
  }
  *out = c;
  return DFLASH_OK;
}

void dflash_cache_destroy(dflash_cache* c) { delete c; }

int dflash_rope(dflash_cache* c, int32_t T, int32_t n_heads, const void* x, int64_t x_stride,
                const int32_t* pos, void* out, int64_t out_stride, int32_t backward, void* stream) {
  if (!c || T < 0 || n_heads < 1) return DFLASH_ERR_INVALID_ARG;
  if (T == 0) return DFLASH_OK;
  if (n_heads > 65535 || bad_rows(c, x, x_stride, n_heads) || bad_rows(c, out, out_stride, n_heads) || !pos)
    return DFLASH_ERR_INVALID_ARG;
  OnDevice on(c->device);
  RopeParams p;
  p.r = c->rope;
  p.T = T;
  p.n_heads = n_heads;
  p.hd = c->v.hd;
  p.el = c->v.el;
  p.x = static_cast<const char*>(x);
  p.out = static_cast<char*>(out);
  p.x_ld = x_stride * p.el;
  p.out_ld = out_stride * p.el;
  p.pos = pos;
  p.backward = backward != 0;
  p.status = c->v.status;
  DC_CHECK(c, launch_rope(p, static_cast<cudaStream_t>(stream)));
  return DFLASH_OK;
}

int dflash_cache_append(dflash_cache* c, int32_t layer, int32_t n_seq, const int32_t* seqs,
                        const int32_t* row_start, int32_t T, const int32_t* depth, const void* q,
                        int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k,
                        int64_t k_stride, const void* v, int64_t v_stride, void* stream) {
  const int rc = check_call(c, n_seq, row_start, T);
  if (rc != DFLASH_OK) return rc;
  if (layer < 0 || layer >= c->cfg.n_layer || !q != !q_out) return DFLASH_ERR_INVALID_ARG;
  if (n_seq == 0 || T == 0) return DFLASH_OK;
  const int hq = c->cfg.n_head, hkv = c->cfg.n_head_kv;
  if (bad_rows(c, k, k_stride, hkv) || bad_rows(c, v, v_stride, hkv)) return DFLASH_ERR_INVALID_ARG;
  if (q && (bad_rows(c, q, q_stride, hq) || bad_rows(c, q_out, q_out_stride, hq))) return DFLASH_ERR_INVALID_ARG;
  OnDevice on(c->device);
  AppendParams p;
  p.c = c->v;
  p.r = c->rope;
  p.rows = {n_seq, seqs, row_start, T};
  p.layer = layer;
  p.depth = depth;
  p.q = static_cast<const char*>(q);
  p.k = static_cast<const char*>(k);
  p.v = static_cast<const char*>(v);
  p.q_out = static_cast<char*>(q_out);
  p.q_ld = q_stride * p.c.el;
  p.q_out_ld = q_out_stride * p.c.el;
  p.k_ld = k_stride * p.c.el;
  p.v_ld = v_stride * p.c.el;
  DC_CHECK(c, launch_append(p, static_cast<cudaStream_t>(stream)));
  return DFLASH_OK;
}

int dflash_tree_mask(dflash_cache* c, int32_t n_seq, const int32_t* row_start, int32_t T,
                     const int32_t* parents, uint32_t* mask, int32_t mask_words, int32_t* depth,
                     void* stream) {
  const int rc = check_call(c, n_seq, row_start, T);
  if (rc != DFLASH_OK) return rc;
  if (mask_words < 1 || mask_words > kTreeMax / 32) return DFLASH_ERR_INVALID_ARG;
  if (n_seq == 0 || T == 0) return DFLASH_OK;
  if (!parents || !mask) return DFLASH_ERR_INVALID_ARG;
  OnDevice on(c->device);
  DC_CHECK(c, launch_tree_mask({n_seq, nullptr, row_start, T}, parents, mask, mask_words, depth,
                               c->v.status, static_cast<cudaStream_t>(stream)));
  return DFLASH_OK;
}

int dflash_tree_attend(dflash_cache* c, int32_t layer, int32_t n_seq, const int32_t* seqs,
                       const int32_t* row_start, int32_t T, int32_t max_tree, const uint32_t* mask,
                       int32_t mask_words, const void* q, int64_t q_stride, void* out, int64_t out_stride,
                       float* lse, void* stream) {
  const int rc = check_call(c, n_seq, row_start, T);
  if (rc != DFLASH_OK) return rc;
  if (layer < 0 || layer >= c->cfg.n_layer || max_tree < 1) return DFLASH_ERR_INVALID_ARG;
  if (mask && (mask_words < 1 || mask_words > kTreeMax / 32 || max_tree > 32 * mask_words))
    return DFLASH_ERR_INVALID_ARG;
  if (n_seq == 0 || T == 0) return DFLASH_OK;
  const int hq = c->cfg.n_head;
  if ((int64_t)T * (hq / c->cfg.n_head_kv) > 0x7fffffff - 1024) return DFLASH_ERR_TOO_MANY_ROWS;
  if (bad_rows(c, q, q_stride, hq) || bad_rows(c, out, out_stride, hq)) return DFLASH_ERR_INVALID_ARG;
  OnDevice on(c->device);
  AttendParams p;
  p.c = c->v;
  p.rows = {n_seq, seqs, row_start, T};
  p.layer = layer;
  p.max_tree = std::min(max_tree, T);
  p.mask = mask;
  p.words = mask_words;
  p.q = static_cast<const char*>(q);
  p.out = static_cast<char*>(out);
  p.q_ld = q_stride * p.c.el;
  p.out_ld = out_stride * p.c.el;
  p.lse = lse;
  p.grp = hq / c->cfg.n_head_kv;
  p.step = 0;
  p.scale = c->cfg.attn_scale != 0.f ? c->cfg.attn_scale : (float)(1.0 / std::sqrt((double)c->cfg.head_dim));
  DC_CHECK(c, launch_attend(p, c->work, static_cast<cudaStream_t>(stream)));
  return DFLASH_OK;
}

int dflash_tree_accept(dflash_cache* c, int32_t n_seq, const int32_t* row_start, int32_t T,
                       const int32_t* parents, const int32_t* tokens, const int32_t* targets,
                       int32_t* path, int32_t max_path, int32_t* n_path, int32_t* id_last, void* stream) {
  const int rc = check_call(c, n_seq, row_start, T);
  if (rc != DFLASH_OK) return rc;
  if (max_path < 1) return DFLASH_ERR_INVALID_ARG;
  if (n_seq == 0) return DFLASH_OK;
  if ((T > 0 && (!parents || !tokens || !targets)) || !path || !n_path || !id_last)
    return DFLASH_ERR_INVALID_ARG;
  OnDevice on(c->device);
  DC_CHECK(c, launch_tree_accept({n_seq, nullptr, row_start, T}, parents, tokens, targets, path, max_path,
                                 n_path, id_last, c->v.status, static_cast<cudaStream_t>(stream)));
  return DFLASH_OK;
}

int dflash_cache_commit(dflash_cache* c, int32_t n_seq, const int32_t* seqs, const int32_t* path,
                        int32_t max_path, const int32_t* n_path, void* stream) {
  const int rc = check_entries(c, n_seq, seqs, n_path);
  if (rc != DFLASH_OK) return rc;
  if (path && (max_path < 1 || max_path > kTreeMax)) return DFLASH_ERR_INVALID_ARG;
  if (n_seq == 0) return DFLASH_OK;
  OnDevice on(c->device);
  DC_CHECK(c, launch_commit(c->v, {n_seq, seqs, nullptr, 0}, path, max_path, n_path,
                            c->S<int>(c->L.tickets), static_cast<cudaStream_t>(stream)));
  return DFLASH_OK;
}

int dflash_cache_reserve(dflash_cache* c, int32_t n_seq, const int32_t* seqs, const int32_t* count,
                         void* stream) {
  const int rc = check_entries(c, n_seq, seqs, count);
  if (rc != DFLASH_OK || n_seq == 0) return rc;
  OnDevice on(c->device);
  DC_CHECK(c, launch_reserve(c->v, {n_seq, seqs, nullptr, 0}, count, c->S<int32_t>(c->L.free_list),
                             c->S<int4>(c->L.copies), static_cast<cudaStream_t>(stream)));
  return DFLASH_OK;
}

int dflash_cache_fork(dflash_cache* c, int32_t n, const int32_t* src, const int32_t* dst, void* stream) {
  if (!c || (n > 0 && (!src || !dst))) return DFLASH_ERR_INVALID_ARG;
  if (n < 0 || n > kCallSeq) return DFLASH_ERR_SEQ_RANGE;
  if (n == 0) return DFLASH_OK;
  OnDevice on(c->device);
  DC_CHECK(c, launch_fork(c->v, n, src, dst, static_cast<cudaStream_t>(stream)));
  return DFLASH_OK;
}

int dflash_cache_trim(dflash_cache* c, int32_t n_seq, const int32_t* seqs, const int32_t* new_len,
                      void* stream) {
  const int rc = check_entries(c, n_seq, seqs, new_len);
  if (rc != DFLASH_OK || n_seq == 0) return rc;
  OnDevice on(c->device);
  DC_CHECK(c, launch_trim(c->v, {n_seq, seqs, nullptr, 0}, new_len, static_cast<cudaStream_t>(stream)));
  return DFLASH_OK;
}

int dflash_cache_read_status(dflash_cache* c, uint32_t* status, void* stream) {
  if (!c || !status) return DFLASH_ERR_INVALID_ARG;
  OnDevice on(c->device);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned v = 0;
  DC_CHECK(c, cudaMemcpyAsync(&v, c->v.status, sizeof(v), cudaMemcpyDeviceToHost, st));
  DC_CHECK(c, cudaMemsetAsync(c->v.status, 0, sizeof(unsigned), st));
  DC_CHECK(c, cudaStreamSynchronize(st));
  *status = v;
  return v ? DFLASH_ERR_DEVICE : DFLASH_OK;
}

const char* dflash_cache_last_error(const dflash_cache* c) { return c ? c->err : ""; }
