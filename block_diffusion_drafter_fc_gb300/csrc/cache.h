// Internal interface of the target model's side: cache pages, trees, rotary
// positions and tree attention (handle and checks: cache_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dflash {

// device status bits (include/dflash.h)
enum : unsigned {
  DEV_BAD_POSITION = 0x2u,
  DEV_TIMEOUT = 0x4u,
  DEV_BAD_ROWS = 0x8u,
  DEV_BAD_PAGE = 0x10u,
  DEV_BAD_TREE = 0x20u,
  DEV_BAD_SEQ = 0x40u,
  DEV_NO_PAGES = 0x80u
};

constexpr int kCallSeq = 1024;   // most entries of one call
constexpr int kTreeMax = 1024;   // most nodes of a tree with a mask

// A cache as every kernel sees it.
struct CacheView {
  char* pages;       // [n_pages][n_layer][2][n_head_kv][page_size][head_dim]
  int32_t* table;    // [max_seq][max_pages]
  int32_t* length;   // [max_seq]
  int32_t* refs;     // [n_pages]
  unsigned* status;
  int n_layer, n_head, n_head_kv, hd;
  int ps, ps_log2;
  int n_pages, max_seq, max_pages;
  int el;            // bytes of an element: 2 (bf16) or 4 (f32)
};

// Rotation angles: turns[j] = 2^64 x (turns of pair j per position), so that
// position x turns modulo 2^64 is the angle's fraction of a turn.
struct RopeView {
  const unsigned long long* turns;
  int rd;            // rotated dims of a head
  int interleaved;
  float mscale;
};

// Rows of a call: T rows, entry s owns row_start[s] .. row_start[s + 1] - 1.
struct RowView {
  int n_seq;
  const int32_t* seqs;   // null: entry s is sequence s
  const int32_t* row_start;
  int T;
};

struct RopeParams {
  RopeView r;
  int T, n_heads, hd, el;
  const char* x;
  char* out;
  int64_t x_ld, out_ld;   // bytes
  const int32_t* pos;
  int backward;
  unsigned* status;
};
cudaError_t launch_rope(const RopeParams& p, cudaStream_t st);

struct AppendParams {
  CacheView c;
  RopeView r;
  RowView rows;
  int layer;
  const int32_t* depth;
  const char *q, *k, *v;   // q null: keys and values alone
  char* q_out;
  int64_t q_ld, q_out_ld, k_ld, v_ld;   // bytes
};
cudaError_t launch_append(const AppendParams& p, cudaStream_t st);

cudaError_t launch_tree_mask(const RowView& rows, const int32_t* parents, uint32_t* mask, int words,
                             int32_t* depth, unsigned* status, cudaStream_t st);
cudaError_t launch_tree_accept(const RowView& rows, const int32_t* parents, const int32_t* tokens,
                               const int32_t* targets, int32_t* path, int max_path, int32_t* n_path,
                               int32_t* id_last, unsigned* status, cudaStream_t st);
cudaError_t configure_tree();

// tickets: [n_seq] counters, zero between launches
cudaError_t launch_commit(const CacheView& c, const RowView& rows, const int32_t* path, int max_path,
                          const int32_t* n_path, int* tickets, cudaStream_t st);
// free_list: [n_pages]; copies: [n_seq] (source page, new page, slots)
cudaError_t launch_reserve(const CacheView& c, const RowView& rows, const int32_t* count,
                           int32_t* free_list, int4* copies, cudaStream_t st);
cudaError_t launch_fork(const CacheView& c, int n, const int32_t* src, const int32_t* dst,
                        cudaStream_t st);
cudaError_t launch_trim(const CacheView& c, const RowView& rows, const int32_t* new_len,
                        cudaStream_t st);

struct AttendParams {
  CacheView c;
  RowView rows;
  int layer, max_tree;
  const uint32_t* mask;
  int words;
  const char* q;
  char* out;
  int64_t q_ld, out_ld;   // bytes
  float* lse;
  float scale;
  int grp;    // query heads per kv head
  int step;   // nodes of a tile where a chain's tiles are cut short (set by the kernels' launchers; 0: never)
};
// What a handle keeps for attention: tensor maps of the pages, scratch for the
// partial rows of tiles that several blocks share, and a description per block
// of the cut tile that begins in it.
struct Cut {
  int lo, row0, kvh, rows;   // first row of the entry; the tile's first row, kv head, rows
  int last, slot;            // its last block (below the block itself: no such tile), the first part's slot
};
constexpr int kAttendSms = 160;        // most SMs a launch uses: 1 (tcgen05) or 2 (streaming) blocks each
struct AttendWork {
  const CUtensorMap* tm;   // boxes of attend_chunk slots
  float* part_o;      // [attend_part_rows][hd]
  float2* part_ml;    // [attend_part_rows]
  Cut* cuts;          // [2 kAttendSms]
  int sms;
};
bool attend_on_umma(int el, int hd);   // tcgen05 kernel, else the streaming kernel
size_t attend_part_rows(int el, int hd);
int attend_chunk(int el, int hd);
cudaError_t configure_attend();
cudaError_t configure_attend_umma();
cudaError_t configure_attend_f32();
cudaError_t launch_attend_f32(const AttendParams& p, const AttendWork& w, cudaStream_t st);
cudaError_t launch_attend_umma(const AttendParams& p, const AttendWork& w, cudaStream_t st);
cudaError_t launch_attend(const AttendParams& p, const AttendWork& w, cudaStream_t st);

}  // namespace dflash
