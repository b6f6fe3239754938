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
// each row is read once and written once. A row belongs to a half-warp (16
// lanes x 8 elements), a block to `tpb` tokens whose (cos, sin) it computes
// once in shared memory for all of their heads, while the first rows' loads
// are in flight.
constexpr int kAppThreads = 256;
constexpr int kAppBatch = 4;  // rows per half-warp whose loads are issued together

__device__ __forceinline__ void store_chunk8(void* base, int64_t off, int dt, int c, const float (&v)[8]) {
  if (dt == kDtF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + off) + 2 * c;
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off) + c;
    *p = make_uint4(pack_dt(dt, v[0], v[1]), pack_dt(dt, v[2], v[3]), pack_dt(dt, v[4], v[5]), pack_dt(dt, v[6], v[7]));
  }
}

__global__ void __launch_bounds__(kAppThreads) append_kernel(const __grid_constant__ AppendParams p, int hpt) {
  __shared__ float2 tab[4][kPairs];
  __shared__ int loc[4][2];
  grid_dependency_wait();
  const int tpb = (kAppThreads / 16) / hpt;  // tokens per block: 1, 2 or 4
  const int hw = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int slot = hw / hpt, r_first = hw - slot * hpt;
  const int64_t n_tok = static_cast<int64_t>(p.B) * p.T;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * tpb + slot;
  const bool there = tok < n_tok;
  const int b = there ? static_cast<int>(tok / p.T) : 0, t = there ? static_cast<int>(tok - static_cast<int64_t>(b) * p.T) : 0;
  const int Hkv = p.kv.Hkv, n_rows = p.H + 2 * Hkv;
  const bool live = there && t < row_count(p.counts, b, p.T);

  float x[kAppBatch][8];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kAppBatch; ++u) {
      const int r = r0 + u * hpt;
      if (live && r < n_rows) {
        const RowTensor& src = r < p.H ? p.q : (r < p.H + Hkv ? p.k : p.v);
        const int h = r < p.H ? r : (r < p.H + Hkv ? r - p.H : r - p.H - Hkv);
        load_chunk8(src.p, b * src.sb + t * src.ss + h * src.sh, src.dt, l, x[u]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[u][e] = 0.f;
      }
    }
  };
  fetch(r_first);

  // (cos, sin) of the block's tokens: the angle reduced in fp64 so that far
  // positions keep full fp32 accuracy; or entry 2j of the caller's tables
  for (int e = threadIdx.x; e < tpb * kPairs; e += kAppThreads) {
    const int sl = e / kPairs, pr = e % kPairs;
    const int64_t tk = static_cast<int64_t>(blockIdx.x) * tpb + sl;
    float2 cs = make_float2(1.f, 0.f);
    if (tk < n_tok) {
      const int bb = static_cast<int>(tk / p.T), tt = static_cast<int>(tk - static_cast<int64_t>(bb) * p.T);
      const int bt = p.tab.Bt == 1 ? 0 : bb;
      if (p.tab.cos) {
        cs.x = table_elem(p.tab.cos, p.tab.tab_dtype, bt * p.tab.c_sb + static_cast<int64_t>(tt) * p.tab.c_ss + (2 * pr) * p.tab.c_sd);
        cs.y = table_elem(p.tab.sin, p.tab.tab_dtype, bt * p.tab.s_sb + static_cast<int64_t>(tt) * p.tab.s_ss + (2 * pr) * p.tab.s_sd);
      } else {
        const int64_t off = bt * p.tab.i_sb + static_cast<int64_t>(tt) * p.tab.i_ss + p.tab.axis_of[pr] * p.tab.i_sa;
        const double id = p.tab.ids_f32 ? static_cast<double>(static_cast<const float*>(p.tab.ids)[off])
                                        : static_cast<double>(static_cast<const int32_t*>(p.tab.ids)[off]);
        cs = pair_cos_sin(id, p.tab.omega[pr]);
      }
      if (pr == 0) {
        int pg = -1, row = 0;
        if (tt < row_count(p.counts, bb, p.T) &&
            !kv_locate(p.kv, bb, static_cast<int64_t>(__ldg(p.lens + bb)) + tt, &pg, &row)) {
          pg = -1;
          atomicOr(p.status, kStatusIndex);
        }
        loc[sl][0] = pg;
        loc[sl][1] = row;
      }
    }
    tab[sl][pr] = cs;
  }
  __syncthreads();
  if (!there) return;
  if (!live) {  // a padded token: its q' rows are zero, nothing enters the cache
    const float z[8] = {};
    for (int r = r_first; r < p.H; r += hpt) store_chunk8(p.qo, b * p.qo_sb + t * p.qo_ss + r * p.qo_sh, p.kv.dt, l, z);
    return;
  }
  const int pg = loc[slot][0], prow = loc[slot][1];
  const int64_t k_off = pg * p.kv.k_sp + prow * p.kv.k_sr, v_off = pg * p.kv.v_sp + prow * p.kv.v_sr;
  float2 cs[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) cs[e] = tab[slot][4 * l + e];
  float wq[8], wk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    wq[e] = __ldg(p.wq + 8 * l + e);
    wk[e] = __ldg(p.wk + 8 * l + e);
  }
  // the bound is that of the warp's first half: both halves take the shuffles
  for (int r0 = r_first; r0 - (hw & 1) < n_rows; r0 += kAppBatch * hpt) {
    if (r0 != r_first) fetch(r0);
#pragma unroll
    for (int u = 0; u < kAppBatch; ++u) {
      const int r = r0 + u * hpt;
      const bool is_v = r >= p.H + Hkv, is_q = r < p.H;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[u][e], x[u][e], ss);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (r >= n_rows) continue;
      if (!is_v) {
        const float inv = rsqrtf(ss * (1.0f / kD) + p.eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float n0 = x[u][2 * e] * inv * (is_q ? wq[2 * e] : wk[2 * e]);
          const float n1 = x[u][2 * e + 1] * inv * (is_q ? wq[2 * e + 1] : wk[2 * e + 1]);
          x[u][2 * e] = n0 * cs[e].x - n1 * cs[e].y;
          x[u][2 * e + 1] = n0 * cs[e].y + n1 * cs[e].x;
        }
      }
      if (is_q) store_chunk8(p.qo, b * p.qo_sb + t * p.qo_ss + r * p.qo_sh, p.kv.dt, l, x[u]);
      else if (pg >= 0 && !is_v) store_chunk8(p.kv.k, k_off + (r - p.H) * p.kv.k_sh, p.kv.dt, l, x[u]);
      else if (pg >= 0) store_chunk8(p.kv.v, v_off + (r - p.H - Hkv) * p.kv.v_sh, p.kv.dt, l, x[u]);
    }
  }
}

// -------------------------------------------------------------------- keep
// Row start + rows[i] moves to row start + i, rows ascending, so that every
// destination lies at or before its source and a CTA that walks the list in
// order may move in place: the destinations of a chunk are rows that this and
// earlier chunks have read. A CTA owns a column (part_lanes 16-byte lanes of
// one K/V head, of K or of V) of one sequence, so no two CTAs touch the same
// bytes. Memory bound; chunks are staged through a ring of shared memory by
// asynchronous copies, kKeepStages chunks ahead of the one being written.
constexpr int kKeepThreads = 256;
constexpr int kKeepPer = 4;     // 16-byte copies per thread and chunk
constexpr int kKeepStages = 4;
constexpr int kKeepSmem = kKeepStages * kKeepPer * kKeepThreads * 16;

__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const __grid_constant__ KeepParams p) {
  extern __shared__ __align__(16) uint4 ring[];
  grid_dependency_wait();
  const int b = blockIdx.z;
  const int64_t cap = static_cast<int64_t>(p.kv.max_pages) * p.kv.page;
  const int start = __ldg(p.start + b), n_said = __ldg(p.n_rows + b);
  const int n = static_cast<int>(min(static_cast<int64_t>(min(max(n_said, 0), p.N)), max(cap - max(start, 0), int64_t(0))));
  const bool first = blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0;
  if (first) {
    if (n != n_said || start < 0) atomicOr(p.status, kStatusIndex);
    p.lens[b] = start < 0 ? start : start + n;
  }
  if (start < 0) return;

  const int eb = p.kv.dt == kDtF32 ? 4 : 2;
  const bool is_v = blockIdx.y >= p.kv.Hkv;
  const int h = is_v ? blockIdx.y - p.kv.Hkv : blockIdx.y;
  uint8_t* base = static_cast<uint8_t*>(is_v ? p.kv.v : p.kv.k) + h * (is_v ? p.kv.v_sh : p.kv.k_sh) * eb;
  const int64_t sp = (is_v ? p.kv.v_sp : p.kv.k_sp) * eb, sr = (is_v ? p.kv.v_sr : p.kv.k_sr) * eb;
  const int lanes = p.part_lanes, lane = threadIdx.x % lanes;
  const int rows_pass = kKeepThreads / lanes, chunk = rows_pass * kKeepPer;
  const int64_t col = (static_cast<int64_t>(blockIdx.x) * lanes + lane) * 16;
  const int n_chunks = (n + chunk - 1) / chunk;
  const int32_t* rows = p.rows + b * p.r_sb;

  auto load = [&](int c) {
    uint4* st = ring + (c % kKeepStages) * kKeepPer * kKeepThreads + threadIdx.x;
#pragma unroll
    for (int u = 0; u < kKeepPer; ++u) {
      const int i = c * chunk + u * rows_pass + threadIdx.x / lanes;
      if (c < n_chunks && i < n) {
        const int r = __ldg(rows + i);
        int pg, row;
        if (r != i && r > i && kv_locate(p.kv, b, static_cast<int64_t>(start) + r, &pg, &row)) {
          const void* src = base + pg * sp + row * sr + col;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(st + u * kKeepThreads)), "l"(src) : "memory");
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int c = 0; c < kKeepStages - 1; ++c) load(c);
#pragma unroll 1
  for (int c = 0; c < n_chunks; ++c) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kKeepStages - 2) : "memory");
    __syncthreads();  // every source of chunk c has been read: its destinations may be written
    const uint4* st = ring + (c % kKeepStages) * kKeepPer * kKeepThreads + threadIdx.x;
#pragma unroll
    for (int u = 0; u < kKeepPer; ++u) {
      const int i = c * chunk + u * rows_pass + threadIdx.x / lanes;
      if (i < n) {
        const int r = __ldg(rows + i);
        int pg, row, pg2, row2;
        bool bad = r < i || (i > 0 && r <= __ldg(rows + i - 1)) ||
                   !kv_locate(p.kv, b, static_cast<int64_t>(start) + r, &pg2, &row2);
        if (!bad && r != i) {
          if (kv_locate(p.kv, b, static_cast<int64_t>(start) + i, &pg, &row))
            *reinterpret_cast<uint4*>(base + pg * sp + row * sr + col) = st[u * kKeepThreads];
          else bad = true;
        }
        if (bad) atomicOr(p.status, kStatusIndex);
      }
    }
    load(c + kKeepStages - 1);  // its slot was written out in the previous turn
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream) {
  const int n_rows = p.H + 2 * p.kv.Hkv;
  // half-warps per token: as many as it has rows, 16 at most
  const int hpt = n_rows <= 4 ? 4 : (n_rows <= 8 ? 8 : 16);
  const int tpb = 16 / hpt;
  const int64_t blocks = (static_cast<int64_t>(p.B) * p.T + tpb - 1) / tpb;
  return launch_chained(append_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kAppThreads), 0, stream, p, hpt);
}

cudaError_t launch_cache_keep(const KeepParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = opt_in_smem(keep_kernel, kKeepSmem, configured);
  if (e != cudaSuccess) return e;
  const int row_lanes = kD * (p.kv.dt == kDtF32 ? 4 : 2) / 16;
  return launch_chained(keep_kernel, dim3(row_lanes / p.part_lanes, 2 * p.kv.Hkv, p.B), dim3(kKeepThreads), kKeepSmem, stream, p);
}

}  // namespace st
