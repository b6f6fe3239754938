// The cache's writers: append (RMS norm + rotation of new q/k rows, k' and v
// into their pages) and keep (rows of a sequence move up).
#include <algorithm>
#include <atomic>
#include "st_kernels.h"
#include "st_serve.h"

namespace st {

namespace {

// ------------------------------------------------------------------ append
// Per token and head: y = rotate(x / sqrt(mean x^2 + eps) * w), every product
// in fp32 and one rounding to the cache's type; v is copied. Memory bound:
// each row is read once and written once. A warp is a unit of its own (no
// block barrier): 2 NI rows of one token and of one kind (q, k or v), a
// half-warp (16 lanes x 8 elements) per row, all NI loads of a half-warp in
// flight before the token's (cos, sin) pairs, two per lane, are computed and
// shared through shared memory. Types are template arguments and the kind is
// the warp's: with both decided row by row, the loads of a unit went out one
// after the other and addresses took a third of the instructions (4608-token
// prompts of two samples: 136 us against 83).
constexpr int kAppWarps = 4;

template <int DT>
struct Raw8 {  // eight elements as they lie in memory
  uint4 a, b;  // b: fp32 only
  __device__ __forceinline__ void load(const void* p, int64_t off) {
    if constexpr (DT == kDtF32) {
      a = ld_v4(static_cast<const float*>(p) + off);
      b = ld_v4(static_cast<const float*>(p) + off + 4);
    } else {
      a = ld_v4(static_cast<const uint16_t*>(p) + off);
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t off) const {
    if constexpr (DT == kDtF32) {
      uint4* d = reinterpret_cast<uint4*>(static_cast<float*>(p) + off);
      d[0] = a;
      d[1] = b;
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + off) = a;
    }
  }
  __device__ __forceinline__ void get(float (&y)[8]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (DT == kDtF32) y[e] = __uint_as_float(w[e]);
      else if constexpr (DT == kDtBF16) y[e] = e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
      else y[e] = e & 1 ? f16_hi(w[e >> 1]) : f16_lo(w[e >> 1]);
    }
  }
  __device__ __forceinline__ void set(const float (&y)[8]) {
    if constexpr (DT == kDtF32) {
      a = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
      b = make_uint4(__float_as_uint(y[4]), __float_as_uint(y[5]), __float_as_uint(y[6]), __float_as_uint(y[7]));
    } else {
      a = make_uint4(pack16<DT == kDtF16>(y[0], y[1]), pack16<DT == kDtF16>(y[2], y[3]), pack16<DT == kDtF16>(y[4], y[5]),
                     pack16<DT == kDtF16>(y[6], y[7]));
    }
  }
};

// (cos, sin) of pair `pr` at token (b, t). Integer positions: position times
// the pair's turns per position in 64-bit fixed point, whose low 64 bits are
// the fraction of a turn, exactly reduced however far the position. fp32 positions
// are reduced in fp64 (4608 tokens of two samples, 24 + 24 heads: 81 us against 76).
__device__ __forceinline__ float2 append_pair(const AppendParams& p, int b, int t, int pr) {
  const TableParams& tab = p.tab;
  const int bt = tab.Bt == 1 ? 0 : b;
  float2 cs;
  if (tab.cos) {
    cs.x = table_elem(tab.cos, tab.tab_dtype, bt * tab.c_sb + static_cast<int64_t>(t) * tab.c_ss + (2 * pr) * tab.c_sd);
    cs.y = table_elem(tab.sin, tab.tab_dtype, bt * tab.s_sb + static_cast<int64_t>(t) * tab.s_ss + (2 * pr) * tab.s_sd);
    return cs;
  }
  const int64_t off = bt * tab.i_sb + static_cast<int64_t>(t) * tab.i_ss + tab.axis_of[pr] * tab.i_sa;
  if (tab.ids_f32) return pair_cos_sin(static_cast<double>(static_cast<const float*>(tab.ids)[off]), tab.omega[pr]);
  const long long id = static_cast<const int32_t*>(tab.ids)[off];
  const unsigned long long turn = static_cast<unsigned long long>(id) * p.turns[pr];
  sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &cs.y, &cs.x);  // 2^-31
  return cs;
}

// SRC: type of q and k; DST: of v and the cache. u_q, u_k: units of a token's q
// rows, and of its k (and v) rows.
template <int NI, int SRC, int DST>
__global__ void __launch_bounds__(kAppWarps * 32) append_kernel(const __grid_constant__ AppendParams p, int u_q, int u_k) {
  __shared__ float4 tab[kAppWarps][kPairs / 2];
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kAppWarps + warp;
  const int units = u_q + 2 * u_k;
  const int64_t tok = unit / units;
  if (tok >= static_cast<int64_t>(p.B) * p.T) return;
  const int u = static_cast<int>(unit - tok * units);
  const int kind = u < u_q ? 0 : (u < u_q + u_k ? 1 : 2);  // q, k, v
  const int h0 = (u - (kind == 0 ? 0 : (kind == 1 ? u_q : u_q + u_k))) * 2 * NI + half;
  const int heads = kind == 0 ? p.H : p.kv.Hkv;
  const int b = static_cast<int>(tok / p.T), t = static_cast<int>(tok - static_cast<int64_t>(b) * p.T);
  const bool live = t < row_count(p.counts, b, p.T);
  const int64_t q_off = b * p.qo_sb + t * p.qo_ss + 8 * l;
  if (!live) {  // a padded token: its q' rows are zero, nothing enters the cache
    Raw8<DST> z;
    z.a = z.b = make_uint4(0, 0, 0, 0);
    if (kind == 0)
      for (int h = h0; h < min(h0 + 2 * NI, heads); h += 2) z.store(p.qo, q_off + h * p.qo_sh);
    return;
  }
  // where the rows go: q', or the token's slot of the cache
  void* out = p.qo;
  int64_t o_off = q_off, o_sh = p.qo_sh;
  bool room = true;
  auto find_slot = [&]() {
    int pg = 0, row = 0;
    const int len = ld_now(p.lens + b);
    // a negative length names no position, also where adding t would reach one
    room = len >= 0 && kv_locate(p.kv, b, static_cast<int64_t>(len) + t, &pg, &row);
    if (!room && lane == 0) atomicOr(p.status, kStatusIndex);
    out = kind == 1 ? p.kv.k : p.kv.v;
    o_sh = kind == 1 ? p.kv.k_sh : p.kv.v_sh;
    o_off = kind == 1 ? pg * p.kv.k_sp + row * p.kv.k_sr : pg * p.kv.v_sp + row * p.kv.v_sr;
    o_off += 8 * l;
  };
  if (kind == 2) {
    const int64_t off = b * p.v.sb + t * p.v.ss + 8 * l;
    Raw8<DST> x[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (h0 + 2 * i < heads) x[i].load(p.v.p, off + (h0 + 2 * i) * p.v.sh);
    find_slot();
    if (!room) return;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (h0 + 2 * i < heads) x[i].store(out, o_off + (h0 + 2 * i) * o_sh);
    return;
  }
  const void* src = kind == 0 ? p.q.p : p.k.p;
  const int64_t sh = kind == 0 ? p.q.sh : p.k.sh;
  const int64_t off = (kind == 0 ? b * p.q.sb + t * p.q.ss : b * p.k.sb + t * p.k.ss) + 8 * l;
  Raw8<SRC> x[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int h = min(h0 + 2 * i, heads - 1);  // the shuffles below want every lane
    x[i].load(src, off + h * sh);
  }
  const float4* wp = reinterpret_cast<const float4*>(kind == 0 ? p.wq : p.wk) + 2 * l;
  const float4 wa = ld_now(wp), wb = ld_now(wp + 1);
  if (kind == 1) find_slot();
  const float2 c0 = append_pair(p, b, t, 2 * lane), c1 = append_pair(p, b, t, 2 * lane + 1);
  tab[warp][lane] = make_float4(c0.x, c0.y, c1.x, c1.y);
  __syncwarp();
  const float4 ca = tab[warp][2 * l], cb = tab[warp][2 * l + 1];
  const float2 cs[4] = {{ca.x, ca.y}, {ca.z, ca.w}, {cb.x, cb.y}, {cb.z, cb.w}};
  const float wv[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    float y[8];
    x[i].get(y);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = rsqrtf(ss * (1.0f / kD) + p.eps);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float n0 = y[2 * e] * inv * wv[2 * e], n1 = y[2 * e + 1] * inv * wv[2 * e + 1];
      y[2 * e] = n0 * cs[e].x - n1 * cs[e].y;
      y[2 * e + 1] = n0 * cs[e].y + n1 * cs[e].x;
    }
    Raw8<DST> r;
    r.set(y);
    if (room && h0 + 2 * i < heads) r.store(out, o_off + (h0 + 2 * i) * o_sh);
  }
}

// -------------------------------------------------------------------- keep
// Row start + rows[i] moves to row start + i, rows ascending, so that every
// destination lies at or before its source and a CTA that walks the list in
// order may move in place: the destinations of a chunk are rows that this and
// earlier chunks have read. A CTA owns a column (part_lanes 16-byte lanes of
// one K/V head, of K or of V) of one sequence, so no two CTAs touch the same
// bytes. Memory bound. The addresses of kKeepTable rows at a time are worked
// out ahead of their use into a table in shared memory (list entry -> page
// number -> address is two dependent loads; done row by row in the copy loop it
// held the whole kernel to 1.3 TB/s), and chunks are staged through a ring by
// asynchronous copies, kKeepStages - 1 chunks ahead of the one being written.
// A chunk costs a CTA about a microsecond whatever its size, so that few long
// columns want wide CTAs: moving 28672 rows of 4 sequences of 8 heads takes
// 162 us (5.1 TB/s, reads and writes) with 128 columns of 128 bytes and 1024
// threads, 177 with 256 of 64 bytes and 256 threads, 211 with 128 and 256;
// a path of 8 rows takes 5.2 us with 256 threads and 18 with 1024.
constexpr int kKeepStages = 4;
constexpr int kKeepTable = 1024;
// Shared memory by the call's N (several CTAs per SM where a list is short):
// the ring's chunks, then src and dst byte offsets of one table or two; src < 0:
// the row does not move.
template <int THREADS, int PER>  // PER: 16-byte copies per thread and chunk
struct KeepLay {
  static constexpr int kChunkBytes = THREADS * PER * 16;
  int stages, table, tables;
  __host__ __device__ KeepLay(int N, int part_lanes) {
    const int chunk = THREADS / part_lanes * PER, chunks = (N + chunk - 1) / chunk;
    stages = chunks < 1 ? 1 : (chunks < kKeepStages ? chunks : kKeepStages);
    table = chunks * chunk < kKeepTable ? (chunks < 1 ? chunk : chunks * chunk) : kKeepTable;
    tables = N > kKeepTable ? 2 : 1;
  }
  __host__ __device__ size_t ring() const { return static_cast<size_t>(stages) * kChunkBytes; }
  __host__ __device__ size_t bytes() const { return ring() + static_cast<size_t>(2) * tables * table * 8; }
};

template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) keep_kernel(const __grid_constant__ KeepParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  const KeepLay<THREADS, PER> lay(p.N, p.part_lanes);
  uint4* ring = reinterpret_cast<uint4*>(raw);
  int64_t* t_src = reinterpret_cast<int64_t*>(raw + lay.ring());
  int64_t* t_dst = t_src + lay.tables * lay.table;
  grid_dependency_wait();
  const int b = blockIdx.z, tid = threadIdx.x;
  const int64_t cap = static_cast<int64_t>(p.kv.max_pages) * p.kv.page;
  const int start = ld_now(p.start + b), n_said = ld_now(p.n_rows + b);
  const int n = static_cast<int>(min(static_cast<int64_t>(min(max(n_said, 0), p.N)), max(cap - max(start, 0), int64_t(0))));
  const bool first = blockIdx.x == 0 && blockIdx.y == 0;
  if (first && tid == 0) {
    if (n != n_said || start < 0) atomicOr(p.status, kStatusIndex);
    p.lens[b] = start < 0 ? start : start + n;
  }
  if (start < 0) return;

  const int eb = p.kv.dt == kDtF32 ? 4 : 2;
  const bool is_v = blockIdx.y >= p.kv.Hkv;
  const int h = is_v ? blockIdx.y - p.kv.Hkv : blockIdx.y;
  uint8_t* base = static_cast<uint8_t*>(is_v ? p.kv.v : p.kv.k) + h * (is_v ? p.kv.v_sh : p.kv.k_sh) * eb;
  const int64_t sp = (is_v ? p.kv.v_sp : p.kv.k_sp) * eb, sr = (is_v ? p.kv.v_sr : p.kv.k_sr) * eb;
  const int lanes = p.part_lanes, lane = tid % lanes, row0 = tid / lanes;
  const int rows_pass = THREADS / lanes, chunk = rows_pass * PER;  // chunk divides kKeepTable
  const int64_t col = (static_cast<int64_t>(blockIdx.x) * lanes + lane) * 16;
  const int n_chunks = (n + chunk - 1) / chunk, per_table = lay.table / chunk;
  const int32_t* rows = p.rows + b * p.r_sb;

  auto build = [&](int tb) {  // the table of rows [tb kKeepTable, (tb + 1) kKeepTable)
    constexpr int kPer = (kKeepTable + THREADS - 1) / THREADS;
    int r[kPer], before[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = tb * lay.table + u * THREADS + tid;
      r[u] = i < n ? ld_now(rows + i) : -1;
      before[u] = i < n && i > 0 ? ld_now(rows + i - 1) : -1;
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int e = u * THREADS + tid, i = tb * lay.table + e;
      if (e >= lay.table) break;
      int64_t so = -1, dof = 0;
      if (i < n) {
        int pg, row, pg2, row2;
        const bool ok = r[u] >= i && r[u] > before[u] && kv_locate(p.kv, b, static_cast<int64_t>(start) + r[u], &pg, &row) &&
                        kv_locate(p.kv, b, static_cast<int64_t>(start) + i, &pg2, &row2);
        if (!ok) {
          if (first) atomicOr(p.status, kStatusIndex);
        } else if (r[u] != i) {
          so = pg * sp + row * sr;
          dof = pg2 * sp + row2 * sr;
        }
      }
      t_src[(tb & 1) * lay.table + e] = so;
      t_dst[(tb & 1) * lay.table + e] = dof;
    }
  };
  auto load = [&](int c) {
    if (c < n_chunks) {
      const int64_t* src = t_src + ((c / per_table) & 1) * lay.table + (c % per_table) * chunk + row0;
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int64_t so = src[u * rows_pass];
        if (so >= 0)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(ring + ((c % lay.stages) * PER + u) * THREADS + tid)), "l"(base + so + col) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  build(0);
  __syncthreads();
#pragma unroll 1
  for (int c = 0; c < kKeepStages - 1; ++c) load(c);
#pragma unroll 1
  for (int c = 0; c < n_chunks; ++c) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kKeepStages - 2) : "memory");
    __syncthreads();  // every source of chunk c has been read: its destinations may be written
    const int tb = c / per_table, within = c % per_table;
    const int64_t* src = t_src + (tb & 1) * lay.table + within * chunk + row0;
    const int64_t* dst = t_dst + (tb & 1) * lay.table + within * chunk + row0;
#pragma unroll
    for (int u = 0; u < PER; ++u)
      if (src[u * rows_pass] >= 0) *reinterpret_cast<uint4*>(base + dst[u * rows_pass] + col) = ring[((c % lay.stages) * PER + u) * THREADS + tid];
    // the next table goes where the last one was, which no thread reads any more
    // (chunks ahead stay within it: a table holds at least kKeepStages chunks)
    if (within == 0 && (tb + 1) * per_table < n_chunks) build(tb + 1);
    load(c + kKeepStages - 1);  // its slot was written out in the previous turn
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

}  // namespace

template <int NI, int SRC, int DST>
cudaError_t launch_append_t(const AppendParams& p, cudaStream_t stream) {
  const int u_q = (p.H + 2 * NI - 1) / (2 * NI), u_k = (p.kv.Hkv + 2 * NI - 1) / (2 * NI);
  const int64_t units = static_cast<int64_t>(p.B) * p.T * (u_q + 2 * u_k);
  return launch_chained(append_kernel<NI, SRC, DST>, dim3(static_cast<unsigned>((units + kAppWarps - 1) / kAppWarps)),
                        dim3(kAppWarps * 32), 0, stream, p, u_q, u_k);
}
template <int SRC, int DST>
cudaError_t launch_append_types(const AppendParams& p, cudaStream_t stream) {
  // as many rows per warp as still leave every SM (152) 32 warps: rows in
  // flight hide the reads, warps the rest
  const int64_t rows = static_cast<int64_t>(p.B) * p.T * (p.H + 2 * p.kv.Hkv);
  if (rows >= 152 * 32 * 8) return launch_append_t<4, SRC, DST>(p, stream);
  return launch_append_t<1, SRC, DST>(p, stream);
}

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream) {
  const bool f32 = p.q.dt == kDtF32;
  switch (p.kv.dt) {
    case kDtBF16: return f32 ? launch_append_types<kDtF32, kDtBF16>(p, stream) : launch_append_types<kDtBF16, kDtBF16>(p, stream);
    case kDtF16: return f32 ? launch_append_types<kDtF32, kDtF16>(p, stream) : launch_append_types<kDtF16, kDtF16>(p, stream);
    default: return launch_append_types<kDtF32, kDtF32>(p, stream);
  }
}

template <int THREADS, int PER>
cudaError_t launch_keep_t(const KeepParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  using Lay = KeepLay<THREADS, PER>;
  // the least part_lanes: 4, or 8 in wide CTAs
  static_assert(kKeepTable >= kKeepStages * (THREADS / (THREADS > 256 ? 8 : 4) * PER), "a table holds the chunks ahead");
  cudaError_t e = opt_in_smem(keep_kernel<THREADS, PER>, kKeepStages * Lay::kChunkBytes + 4 * kKeepTable * 8, configured);
  if (e != cudaSuccess) return e;
  const int row_lanes = kD * (p.kv.dt == kDtF32 ? 4 : 2) / 16;
  return launch_chained(keep_kernel<THREADS, PER>, dim3(row_lanes / p.part_lanes, 2 * p.kv.Hkv, p.B), dim3(THREADS),
                        Lay(p.N, p.part_lanes).bytes(), stream, p);
}

cudaError_t launch_cache_keep(const KeepParams& p, cudaStream_t stream) {
  return p.wide ? launch_keep_t<1024, 2>(p, stream) : launch_keep_t<256, 4>(p, stream);
}

}  // namespace st
