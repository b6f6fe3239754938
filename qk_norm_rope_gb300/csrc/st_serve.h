// Parameter blocks and launchers of the serving kernels: cache append and read,
// cached attention, tree verification and cache compaction.
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

// Element types of a cache of 8 bits (the codes of st_dtype): value = scale of
// the row (a token and K/V head) times what is held.
enum : int { kDtE4M3 = 6, kDtI8 = 7 };
// What a row's largest magnitude is held as.
__host__ __device__ constexpr float top_of(int dt) { return dt == kDtE4M3 ? 448.f : 127.f; }
// Rows whose scale would be below this are held as zeros: its reciprocal, and
// every value's product with it, is a normal number.
constexpr float kMinScale = 7.888609052210118e-31f;  // 2^-100

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

// 32 bytes of a thread in one store, on a 32-byte boundary: whole sectors, in half as
// many instructions of 32 sectors each as with 16-byte stores.
__device__ __forceinline__ void st_v8(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
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
  float* ks;                       // caches of 8 bits: scales [n_pages, Hkv, page], unit stride on page
  float* vs;
  int64_t ks_sp, ks_sh, vs_sp, vs_sh;
};

inline bool held(const PagedKV& kv) { return kv.dt == kDtE4M3 || kv.dt == kDtI8; }

// Four held bytes (the lowest first) as numbers.
template <int DT>
__device__ __forceinline__ void held4(uint32_t w, float (&y)[4]) {
  if constexpr (DT == kDtE4M3) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n}" : "=r"(lo), "=r"(hi) : "r"(w));
    y[0] = f16_lo(lo); y[1] = f16_hi(lo); y[2] = f16_lo(hi); y[3] = f16_hi(hi);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = static_cast<float>(static_cast<int8_t>(w >> (8 * e)));
  }
}

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
  void* qo;                        // rotated q, [B, T, H, D] in v's type (the cache's, unless that is of 8 bits)
  int64_t qo_sb, qo_ss, qo_sh;
  int B, T, H;
  unsigned* status;
};
cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream);

struct CacheAttnParams {
  RowTensor q;                     // rotated q, the cache's type (any with a cache of 8 bits), as o
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
  int window, sinks;               // window > 0: a row at position p sees keys at positions above p - window or below sinks
  const int32_t* shared;           // [1]: tokens that all sequences have in the same pages, or null
  unsigned* status;
  unsigned long long* counters;
  long long wait_budget;
};

// Number of keys of sequence b: its prefix and its new rows, at most what the
// page table has room for.
__device__ __forceinline__ int keys_of(const CacheAttnParams& p, int length, int count, int* prefix) {
  const int64_t cap = static_cast<int64_t>(p.kv.max_pages) * p.kv.page;
  const int64_t len = max(length, 0);
  *prefix = static_cast<int>(min(len, cap));
  return static_cast<int>(min(len + count, cap));
}
__device__ __forceinline__ int key_count(const CacheAttnParams& p, int b, int count, int* prefix) {
  return keys_of(p, ld_now(p.lens + b), count, prefix);
}

// The lowest position in the window of a row at lens[b] + step, at least 0 and
// at most 2^30 (no key lies there). `sinks` aside.
__device__ __forceinline__ int window_low_of(const CacheAttnParams& p, int length, int64_t step) {
  const int64_t low = max(length, 0) + step - p.window + 1;
  return static_cast<int>(min(max(low, int64_t(0)), int64_t(1) << 30));
}
__device__ __forceinline__ int window_low(const CacheAttnParams& p, int b, int64_t step) { return window_low_of(p, ld_now(p.lens + b), step); }
// With a window, how many nodes are above `node` of sequence b's tree (parents
// come before children; anything else ends the walk).
__device__ __forceinline__ int node_depth(const CacheAttnParams& p, int b, int node) {
  int depth = 0;
  while (true) {
    const int up = ld_now(p.parents + b * p.par_sb + node);
    if (up >= node || up < 0) return depth;
    node = up;
    ++depth;
  }
}
// The k-th ancestor of a row of that depth is seen.
__device__ __forceinline__ bool window_sees(const CacheAttnParams& p, int b, int depth, int k) {
  return k < p.window || static_cast<int64_t>(max(ld_now(p.lens + b), 0)) + depth - k < p.sinks;
}
// Keys that a window leaves out, in units of U keys: the first `lead` units and
// those from lead + gap on hold every key that a row whose window begins at
// `low` or higher sees.
struct Gap {
  int lead, gap;
};
template <int U>
__device__ __forceinline__ Gap window_gap(const CacheAttnParams& p, int low, int units) {
  const int lead = min(units, (min(p.sinks, 1 << 30) + U - 1) / U);
  return {lead, max(0, min(low / U, units) - lead)};
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
// Strides of pages, rows and heads of K or V in units of 16 bytes, and of the
// scales' pages and heads in numbers.
struct HeldAt {
  uint32_t sp, sr, sh, sc_sp, sc_sh;
};
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
  HeldAt held_k, held_v;       // 8-bit caches
  int few;                     // 8-bit caches: 1: at most 32 rows, their keys shared by four lane groups
  // Joined by items (a shared prefix, few): parts are [2 ctas, split_rows], then a
  // result of pre_rows or part_rows (few: four times) for each item that one CTA has whole.
  int n_pre;                   // groups of the prefix's rows
  int pre_rows, split_rows;    // rows of such a group, of a split part
  int2* item_meta;             // [items] (parts, slot of the first or -1: whole); null: not by items
  int* p0;                     // [1] tiles of the prefix
};
// Of each CTA: the item whose first inner border is the CTA's beginning. Its
// parts lie in slot0 and then in the slots 2 x of the CTAs x from this one on.
struct JoinMeta {
  int parts, slot0;            // parts = 0: there is no such item
  int h, b, m, cnt;
};
inline int tc_tiles(int64_t T, int group) { return T * group > 128 ? 2 : 1; }
cudaError_t launch_cache_attn_tc(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream);
cudaError_t launch_cache_attn_ext(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream);   // the forms, each in a file of its own
cudaError_t launch_cache_attn_e4m3(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream);
cudaError_t launch_cache_attn_e4m3_ext(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream);
cudaError_t launch_cache_attn_i8(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream);
cudaError_t launch_cache_attn_i8_ext(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream);
cudaError_t launch_cache_attn_join(const TcAttnParams& p, int nt, cudaStream_t stream);

// Rows of a cache into dense tensors [B, T, Hkv, D].
struct ReadParams {
  PagedKV kv;
  const int32_t* start;            // [B]
  const int32_t* counts;           // or null
  void* k;
  void* v;
  int64_t k_sb, k_ss, k_sh, v_sb, v_ss, v_sh;
  int dt;                          // of k and v
  int wide;                        // 1: their rows start on 32 bytes
  int B, T;
  unsigned* status;
};
cudaError_t launch_cache_read(const ReadParams& p, cudaStream_t stream);

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
