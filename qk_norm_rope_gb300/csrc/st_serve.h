// Parameter blocks and launchers of the serving kernels: cache append, cached
// attention, tree verification and cache compaction.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>
#include "st_aux.h"
#include "st_common.cuh"

namespace st {

constexpr int kMaxTree = 256;        // nodes of a drafted tree that attention takes
constexpr int kTreeWords = kMaxTree / 32;
constexpr int kMaxVerify = 1024;     // nodes of a drafted tree that the verification takes
constexpr int kMaxGroup = 128;       // query heads per K/V head
constexpr int kMaxClusterVerify = 8;
constexpr int kMaxClusterAttn = 8;

// Ordinary loads, not the read-only path: with programmatic launches a kernel
// may be resident while the one before it still writes what is read here (after
// the dependency wait).
template <class T>
__device__ __forceinline__ T ld_now(const T* p) {
  return *p;
}
__device__ __forceinline__ uint4 ld_v4(const void* p) {  // volatile: stays where it stands among other volatile asm
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// A paged K/V cache: token `pos` of sequence b lies in row pos % page of page
// pages[b][pos / page].
struct PagedKV {
  void* k;
  void* v;
  int dt;                          // element type of both (kDt*)
  int64_t k_sp, k_sr, k_sh;        // element strides of pages, rows and heads
  int64_t v_sp, v_sr, v_sh;
  const int32_t* pages;
  int64_t p_sb, p_sj;              // element strides of the page table
  int n_pages, page, max_pages;
  int page_shift;                  // log2 of page, -1 where it is no power of two
  int Hkv;
};

// Page and row of token `pos` of sequence b; false when the position or the
// table's entry is out of range.
__device__ __forceinline__ bool kv_locate(const PagedKV& c, int b, int64_t pos, int* pg, int* row) {
  if (pos < 0 || pos >= static_cast<int64_t>(c.max_pages) * c.page) return false;
  const unsigned p = static_cast<unsigned>(pos);  // capacity <= 2^30
  const unsigned j = c.page_shift >= 0 ? p >> c.page_shift : p / static_cast<unsigned>(c.page);
  *row = static_cast<int>(p - j * static_cast<unsigned>(c.page));
  *pg = ld_now(c.pages + b * c.p_sb + j * c.p_sj);
  return static_cast<unsigned>(*pg) < static_cast<unsigned>(c.n_pages);
}

// The number of sequence b's T rows that are there.
__device__ __forceinline__ int row_count(const int32_t* counts, int b, int T) {
  return counts ? min(max(ld_now(counts + b), 0), T) : T;
}

struct AppendParams {
  RowTensor q, k, v;               // [B, T, H|Hkv, D]
  const float* wq;
  const float* wk;
  float eps;
  TableParams tab;                 // ids, or cos/sin tables
  unsigned long long turns[kPairs];  // fraction of a turn per position, 2^-64 a unit
  PagedKV kv;
  const int32_t* lens;
  const int32_t* counts;           // or null
  void* qo;                        // rotated q, [B, T, H, D] in the cache's type
  int64_t qo_sb, qo_ss, qo_sh;
  int B, T, H;
  unsigned* status;
};
cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream);

struct CacheAttnParams {
  RowTensor q;                     // rotated q, the cache's type
  PagedKV kv;
  const int32_t* lens;
  const int32_t* counts;           // or null
  const int32_t* parents;          // [B|1, T], or null (a chain)
  int64_t par_sb;
  float scale_log2;
  void* o;
  int64_t o_sb, o_ss, o_sh;
  float* lse;                      // [B, H, T]
  int B, T, H, group;
  float* part;                     // partial results (workspace)
  int splits;                      // SIMT kernel: key ranges over all sequences (0: an item's keys stay together)
  unsigned* status;
  unsigned long long* counters;
  long long wait_budget;
};

// Number of keys of sequence b: its prefix and its new rows, at most what the
// page table has room for.
__device__ __forceinline__ int key_count(const CacheAttnParams& p, int b, int count, int* prefix) {
  const int64_t cap = static_cast<int64_t>(p.kv.max_pages) * p.kv.page;
  const int64_t len = max(ld_now(p.lens + b), 0);
  *prefix = static_cast<int>(min(len, cap));
  return static_cast<int>(min(len + count, cap));
}

// SIMT kernel: items of kSimtRows query rows of one K/V head.
constexpr int kSimtRows = 64, kSimtKeys = 64;
inline int64_t simt_items(int B, int T, int H, int Hkv) {
  return static_cast<int64_t>(B) * Hkv * ((static_cast<int64_t>(T) * (H / Hkv) + kSimtRows - 1) / kSimtRows);
}
cudaError_t launch_cache_attn_simt(const CacheAttnParams& p, cudaStream_t stream);
cudaError_t launch_cache_attn_simt_join(const CacheAttnParams& p, cudaStream_t stream);

// Tensor-core kernel. A group is NT query tiles of 128 rows (tokens x heads of
// one K/V head; NT = 2 where a sequence has more than 128 rows a head), an
// item a (K/V head, sequence, group); its key tiles are dealt out to the CTAs
// in one continuous range each.
struct TcAttnParams {
  CacheAttnParams c;
  CUtensorMap tmap_k, tmap_v;  // cache pages, boxes of 64 columns x box rows
  int k_r_first, v_r_first;    // map dims are (d, row, head, page) instead of (d, head, row, page)
  int box_shift;               // log2 of the rows per box: a power of two that divides the page size, 8..128
  int tpt;                     // tokens per query tile (128 / group)
  int n_groups;                // groups per sequence
  int part_rows;               // rows of a partial result
  int o_wide;                  // 1: o's rows start on 32 bytes
  int ctas;
  int cluster;                 // CTAs per item of the clustered form: 2, 4 or 8; 0: the dealt form
  int cluster_shift;
  struct JoinMeta* meta;       // [ctas], workspace
  float2* part_ml;             // [2 ctas, part_rows] (reference, sum); c.part: [2 ctas, part_rows, D]
};
// Of each CTA: the item whose first inner border is the CTA's beginning. Its
// parts lie in slot0 and then in the slots 2 x of the CTAs x from this one on.
struct JoinMeta {
  int parts, slot0;            // parts = 0: there is no such item
  int h, b, m, cnt;
};
inline int tc_tiles(int T, int group) { return static_cast<int64_t>(T) * group > 128 ? 2 : 1; }
cudaError_t launch_cache_attn_tc(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream);
cudaError_t launch_cache_attn_join(const TcAttnParams& p, int nt, cudaStream_t stream);

struct VerifyParams {
  const void* p;                   // target probabilities [B, T, V]
  const void* q;                   // draft probabilities, or null
  int dt;
  int64_t p_sb, p_st, q_sb, q_st;
  const void* tokens;              // [B, T]
  int tok64;
  int64_t tok_sb, tok_st;
  const int32_t* parents;          // [B|1, T]
  int64_t par_sb;
  const int32_t* counts;           // or null
  const float* u_accept;           // [B, T]
  const float* u_sample;           // [B]
  int32_t* path;                   // [B, T]
  int32_t* n_accepted;             // [B]
  void* next_token;                // [B], the tokens' type
  int B, T, V;
  int cluster;                     // CTAs per sequence
  unsigned* status;
};
cudaError_t launch_tree_verify(const VerifyParams& p, cudaStream_t stream);

struct KeepParams {
  PagedKV kv;
  const int32_t* start;            // [B]
  const int32_t* rows;             // [B, N]
  int64_t r_sb;
  const int32_t* n_rows;           // [B]
  int32_t* lens;                   // [B], out
  int B, N;
  int part_lanes;                  // 16-byte lanes of a row that one CTA moves (4 or 8)
  int wide;                        // 1: CTAs of 1024 threads (part_lanes 8)
  unsigned* status;
};
cudaError_t launch_cache_keep(const KeepParams& p, cudaStream_t stream);

}  // namespace st
