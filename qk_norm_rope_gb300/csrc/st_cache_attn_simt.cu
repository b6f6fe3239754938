// Cached attention on the CUDA cores: fp32 caches (every product and sum in
// fp32), and 16-bit caches whose pages the tensor-core kernel's boxes do not
// fit (page sizes that are no multiple of 8).
//
// An item is kSimtRows query rows (token x head of the group) of one K/V head
// of one sequence; its keys are walked in tiles of kSimtKeys. Few items are split
// over the keys: the p.splits ranges that there are CTAs for are dealt to the
// sequences by their lengths, which only the device knows (an equal number each
// left the CTAs of short sequences idle). Each CTA leaves (O unnormalised,
// running maximum, sum) in the workspace and a second kernel joins them; without
// a split it writes O and LSE itself.
//
// Bound by the FMA rate and shared memory's: a thread holds 4 x 4 scores and
// 8 x 4 outputs (8 and 12 16-byte reads for 64 and 128 FMAs); with half as many
// rows (2 x 4 and 4 x 4) four trees of 13 nodes after up to 2001 tokens took 47 us
// instead of 37, 34 with packed FMAs, 33 with ranges dealt by length. Those were
// for uneven lengths: 8 single tokens after up to 4000 keys 58 -> 37 us, 30 after
// up to 1000 116 -> 85 us. Long and even ones run at 58% of the FMA rate. The
// weights P take K's place in shared memory once the scores are done, so that
// two CTAs fit on an SM.
#include <algorithm>
#include <atomic>
#include <type_traits>
#include "st_kernels.h"
#include "st_serve.h"

namespace st {

namespace {

constexpr int kR = kSimtRows, kN = kSimtKeys, kThreads = 256;
constexpr int kPad = kD + 4, kPadP = kN + 4;

struct Smem {
  float q[kR][kD];  // read as broadcasts
  union {
    float k[kN][kPad];
    float p[kR][kPadP];
  };
  float v[kN][kD];
  float corr[kR], m[kR], l[kR];
  uint32_t anc[kR][kTreeWords];
  int64_t k_off[2][kN], v_off[2][kN];  // element offsets of a tile's rows, by its parity; < 0: no row
};

// Bit j of the result: node `first + j` is seen from a row whose ancestors
// (itself included) are `anc`.
__device__ __forceinline__ bool tree_sees(const uint32_t* anc, int node) {
  return node < kMaxTree && ((anc[node >> 5] >> (node & 31)) & 1u);
}

// The ranges of sequence b's items, `n` from `first` on among the call's
// p.splits: one, and a share of the others in proportion to the sequence's keys,
// but none shorter than two units of kUnit keys (a token after 100 keys takes
// 13.5 us so, 21 with four units, as a second tile costs more than a part).
struct Ranges {
  int b, first, n;
};
constexpr int kUnit = 16;
constexpr int kMaxRanges = 128;  // of an item: the join goes through them
// By a whole warp: the sequence that range y belongs to (b = -1: none), or, with
// y < 0, the ranges of sequence b.
__device__ Ranges find_ranges(const CacheAttnParams& p, int y, int b) {
  const int lane = threadIdx.x & 31;
  auto units = [&](int i) {
    int prefix;
    return i < p.B ? (key_count(p, i, row_count(p.counts, i, p.T), &prefix) + kUnit - 1) / kUnit : 0;
  };
  const int mine = units(lane);
  long long all = mine;
  for (int i = 32 + lane; i < p.B; i += 32) all += units(i);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) all += __shfl_xor_sync(0xffffffffu, all, x);
  int first = 0;
  for (int base = 0; base < p.B; base += 32) {
    const int u = base == 0 ? mine : units(base + lane);
    const int more = static_cast<int>(min(static_cast<long long>(p.splits - p.B) * u / max(all, 1ll), static_cast<long long>(kMaxRanges - 1)));
    const int n = base + lane < p.B ? 1 + min(more, max(u / 2 - 1, 0)) : 0;
    int upto = n;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, upto, x);
      if (lane >= x) upto += t;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, y >= 0 ? y < first + upto : base + lane == b);
    if (hit != 0) {
      const int at = __ffs(hit) - 1, count = __shfl_sync(0xffffffffu, n, at);
      return {base + at, first + __shfl_sync(0xffffffffu, upto, at) - count, count};
    }
    first += __shfl_sync(0xffffffffu, upto, 31);
  }
  return {-1, 0, 0};
}

__global__ void __launch_bounds__(kThreads, 2) simt_kernel(const __grid_constant__ CacheAttnParams p, int n_rt) {
  extern __shared__ __align__(16) uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>(raw);
  grid_dependency_wait();
  const int tid = threadIdx.x;
  const unsigned it32 = blockIdx.x;  // items are at most 2^30: of a sequence, or (no split) of all
  const int rt = static_cast<int>(it32 % n_rt), hk = static_cast<int>(it32 / n_rt % p.kv.Hkv);
  const Ranges range = p.splits > 0 ? find_ranges(p, blockIdx.y, 0) : Ranges{static_cast<int>(it32 / n_rt / p.kv.Hkv), 0, 1};
  const int b = range.b, split = blockIdx.y - range.first;
  if (b < 0) return;  // short sequences need fewer ranges
  const int G = p.group;
  const int64_t rows = static_cast<int64_t>(p.T) * G;
  const int64_t row0 = static_cast<int64_t>(rt) * kR;
  // row r of the item: token t0 + (g0 + r) / G, head (g0 + r) % G of the group
  const int t0 = static_cast<int>(row0 / G), g0 = static_cast<int>(row0 - static_cast<int64_t>(t0) * G);
  const int n_here = static_cast<int>(min(rows - row0, static_cast<int64_t>(kR)));
  const int cnt = row_count(p.counts, b, p.T);
  int prefix;
  const int keys = key_count(p, b, cnt, &prefix);
  if (tid == 0 && split == 0 && (ld_now(p.lens + b) < 0 || static_cast<int64_t>(ld_now(p.lens + b)) + cnt > keys)) atomicOr(p.status, kStatusIndex);

  // the last key that any row of the item sees
  const int t_last = t0 + (g0 + n_here - 1) / G;
  const int end = p.parents ? keys : min(keys, prefix + min(t_last + 1, cnt));
  const int units = t0 < cnt ? (end + kUnit - 1) / kUnit : 0;
  const int key_lo = static_cast<int>(static_cast<int64_t>(units) * split / range.n) * kUnit;
  const int key_hi = static_cast<int>(static_cast<int64_t>(units) * (split + 1) / range.n) * kUnit;
  const int n_tiles = (key_hi - key_lo + kN - 1) / kN;

  if (tid < kR && p.parents) {  // a walk up from the row's node; parents come before children
    for (int w = 0; w < kTreeWords; ++w) s.anc[tid][w] = 0;
    int node = tid < n_here ? t0 + (g0 + tid) / G : -1;
    if (node >= cnt) node = -1;
    while (node >= 0) {
      s.anc[tid][node >> 5] |= 1u << (node & 31);
      const int up = ld_now(p.parents + b * p.par_sb + node);
      if (up >= node || up < -1) {
        atomicOr(p.status, kStatusIndex);
        break;
      }
      node = up;
    }
  }
  float2 o[8][2];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = make_float2(0.f, 0.f);
  float m_run[4], l_run[4];  // of the thread's score rows: the maximum, and the sum over the thread's own keys
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    m_run[w] = -INFINITY;
    l_run[w] = 0.f;
  }
  const int tr = tid >> 4, tc = tid & 15;   // scores: rows tr + 16 w; keys tc + 16 i
  const int rg = tid >> 5, dg = tid & 31;   // outputs: rows 8 rg + i; dims 4 dg..
  const bool f32 = p.kv.dt == kDtF32;
  auto locate = [&](int jt) {  // the rows of key tile jt
    if (tid < kN && jt < n_tiles) {
      const int j = key_lo + jt * kN + tid;
      int pg, prow;
      int64_t ko = -1, vo = -1;
      if (j < min(keys, key_hi)) {
        if (kv_locate(p.kv, b, j, &pg, &prow)) {
          ko = pg * p.kv.k_sp + prow * p.kv.k_sr + hk * p.kv.k_sh;
          vo = pg * p.kv.v_sp + prow * p.kv.v_sr + hk * p.kv.v_sh;
        } else {
          atomicOr(p.status, kStatusIndex);
        }
      }
      s.k_off[jt & 1][tid] = ko;
      s.v_off[jt & 1][tid] = vo;
    }
  };
  // One of a tile's two operands into shared memory: asynchronous copies of
  // fp32 rows, conversion of 16-bit ones; zeros where there is no row.
  auto fetch = [&](const void* base, const int64_t* off, float* dst, int pad) {
    if (f32) {
#pragma unroll
      for (int u = 0; u < kN * kD / 4 / kThreads; ++u) {
        const int e = u * kThreads + tid, r = e / (kD / 4), c = e % (kD / 4);
        const int64_t o = off[r];
        const float* src = static_cast<const float*>(base) + (o < 0 ? 0 : o) + 4 * c;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst + r * pad + 4 * c)), "l"(o < 0 ? p.q.p : static_cast<const void*>(src)), "r"(o < 0 ? 0 : 16) : "memory");
      }
    } else {
      uint4 x[kN * kD / 8 / kThreads];
#pragma unroll
      for (int u = 0; u < kN * kD / 8 / kThreads; ++u) {
        const int e = u * kThreads + tid, r = e / (kD / 8), c = e % (kD / 8);
        const int64_t o = off[r];
        x[u] = o < 0 ? make_uint4(0, 0, 0, 0) : ld_v4(static_cast<const uint16_t*>(base) + o + 8 * c);
      }
#pragma unroll
      for (int u = 0; u < kN * kD / 8 / kThreads; ++u) {
        const int e = u * kThreads + tid, r = e / (kD / 8), c = e % (kD / 8);
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[2 * i] = p.kv.dt == kDtF16 ? f16_lo(w[i]) : bf16_lo(w[i]);
          y[2 * i + 1] = p.kv.dt == kDtF16 ? f16_hi(w[i]) : bf16_hi(w[i]);
        }
        *reinterpret_cast<float4*>(dst + r * pad + 8 * c) = make_float4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<float4*>(dst + r * pad + 8 * c + 4) = make_float4(y[4], y[5], y[6], y[7]);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  locate(0);
  if (tid < kR) {  // the offsets of the query rows, where the second tile's will be
    const int t = t0 + (g0 + tid) / G, h = hk * G + (g0 + tid) % G;
    s.k_off[1][tid] = tid < n_here && t < cnt ? b * p.q.sb + t * p.q.ss + h * p.q.sh : -1;
  }
  __syncthreads();
  if (n_tiles > 0) {
    fetch(p.q.p, s.k_off[1], &s.q[0][0], kD);
    fetch(p.kv.k, s.k_off[0], &s.k[0][0], kPad);
    fetch(p.kv.v, s.v_off[0], &s.v[0][0], kD);
  }
  for (int jt = 0; jt < n_tiles; ++jt) {
    const int j0 = key_lo + jt * kN, n_units = min(kN, key_hi - j0) / kUnit;  // a range's last tile: only what it has
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // Q and K
    __syncthreads();
    locate(jt + 1);
    float2 acc[4][4];  // even and odd head dims: two products per instruction
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[w][i] = make_float2(0.f, 0.f);
    auto scores = [&](auto count) {  // of the first kUnit * count keys
      constexpr int N = decltype(count)::value;
#pragma unroll 4
      for (int d = 0; d < kD; d += 4) {
        float4 qq[4], kk[N];
#pragma unroll
        for (int w = 0; w < 4; ++w) qq[w] = *reinterpret_cast<const float4*>(&s.q[tr + 16 * w][d]);
#pragma unroll
        for (int i = 0; i < N; ++i) kk[i] = *reinterpret_cast<const float4*>(&s.k[tc + 16 * i][d]);
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int i = 0; i < N; ++i)
            acc[w][i] = __ffma2_rn(make_float2(qq[w].x, qq[w].y), make_float2(kk[i].x, kk[i].y),
                                   __ffma2_rn(make_float2(qq[w].z, qq[w].w), make_float2(kk[i].z, kk[i].w), acc[w][i]));
      }
    };
    if (n_units == 4) scores(std::integral_constant<int, 4>());
    else if (n_units == 3) scores(std::integral_constant<int, 3>());
    else if (n_units == 2) scores(std::integral_constant<int, 2>());
    else scores(std::integral_constant<int, 1>());
    __syncthreads();  // K is read: P takes its place
    const float sl = p.scale_log2;
    float sc[4][4];
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[w][i] = (acc[w][i].x + acc[w][i].y) * sl;
    if (j0 + kN > min(prefix, key_hi)) {  // rows of padding see anything here: they are dropped at the end
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int r = tr + 16 * w, t = t0 + (g0 + r) / G;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = j0 + tc + 16 * i, node = j - prefix;
          const bool sees = j < min(keys, key_hi) && (node < 0 || (p.parents ? tree_sees(s.anc[r], node) : node <= t));
          if (!sees) sc[w][i] = -INFINITY;
        }
      }
    }
    float mt[4], sum[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) mt[w] = fmaxf(fmaxf(sc[w][0], sc[w][1]), fmaxf(sc[w][2], sc[w][3]));
#pragma unroll
    for (int x = 8; x > 0; x >>= 1)
#pragma unroll
      for (int w = 0; w < 4; ++w) mt[w] = fmaxf(mt[w], __shfl_xor_sync(0xffffffffu, mt[w], x));
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int r = tr + 16 * w;
      const float m_new = fmaxf(m_run[w], mt[w]), m_use = m_new == -INFINITY ? 0.f : m_new;
      if (tc == 0) s.corr[r] = ex2(m_run[w] - m_use);  // 0 while the row has seen nothing
      l_run[w] *= ex2(m_run[w] - m_use);
      m_run[w] = m_new;
      sum[w] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = ex2(sc[w][i] - m_use);
        s.p[r][tc + 16 * i] = e;
        sum[w] += e;
      }
      l_run[w] += sum[w];  // this lane's keys
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");  // V
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float corr = s.corr[8 * rg + i];
      o[i][0] = make_float2(o[i][0].x * corr, o[i][0].y * corr);
      o[i][1] = make_float2(o[i][1].x * corr, o[i][1].y * corr);
    }
#pragma unroll 2
    for (int k = 0; k < kUnit * n_units; k += 4) {
      float4 vv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) vv[u] = *reinterpret_cast<const float4*>(&s.v[k + u][4 * dg]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 pp = *reinterpret_cast<const float4*>(&s.p[8 * rg + i][k]);
        const float pw[4] = {pp.x, pp.y, pp.z, pp.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 pp2 = make_float2(pw[u], pw[u]);
          o[i][0] = __ffma2_rn(pp2, make_float2(vv[u].x, vv[u].y), o[i][0]);
          o[i][1] = __ffma2_rn(pp2, make_float2(vv[u].z, vv[u].w), o[i][1]);
        }
      }
    }
    __syncthreads();
    if (jt + 1 < n_tiles) {
      fetch(p.kv.k, s.k_off[(jt + 1) & 1], &s.k[0][0], kPad);
      fetch(p.kv.v, s.v_off[(jt + 1) & 1], &s.v[0][0], kD);
    }
  }
#pragma unroll
  for (int w = 0; w < 4; ++w) {
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) l_run[w] += __shfl_xor_sync(0xffffffffu, l_run[w], x);
    const int r = tr + 16 * w;
    const bool there = r < n_here && t0 + (g0 + r) / G < cnt;  // padding: nothing seen
    if (tc == 0) {
      s.m[r] = there ? m_run[w] : -INFINITY;
      s.l[r] = there ? l_run[w] : 0.f;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 8 * rg + i;
    if (r >= n_here) continue;
    if (p.splits > 0) {
      const int64_t slot = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kR + r;
      *reinterpret_cast<float4*>(p.part + slot * kD + 4 * dg) = make_float4(o[i][0].x, o[i][0].y, o[i][1].x, o[i][1].y);
      if (dg == 0) {
        float2* ml = reinterpret_cast<float2*>(p.part + static_cast<int64_t>(gridDim.x) * gridDim.y * kR * kD);
        ml[slot] = make_float2(s.m[r], s.l[r]);
      }
      continue;
    }
    const float l = s.l[r], inv = l == 0.f ? 0.f : 1.f / l;
    const int t = t0 + (g0 + r) / G, h = hk * G + (g0 + r) % G;
    const int64_t off = b * p.o_sb + t * p.o_ss + h * p.o_sh + 4 * dg;
    if (p.kv.dt == kDtF32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.o) + off) = make_float4(o[i][0].x * inv, o[i][0].y * inv, o[i][1].x * inv, o[i][1].y * inv);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + off) =
          make_uint2(pack_dt(p.kv.dt, o[i][0].x * inv, o[i][0].y * inv), pack_dt(p.kv.dt, o[i][1].x * inv, o[i][1].y * inv));
    if (dg == 0) p.lse[(static_cast<int64_t>(b) * p.H + h) * p.T + t] = l == 0.f ? -INFINITY : (s.m[r] + log2f(l)) * kLn2;
  }
}

// W warps per query row, 1 or 8: each brings every W-th range's part to their
// common maximum, four in flight, and the first one the warps' results.
template <int W>
__global__ void __launch_bounds__(256) simt_join_kernel(const __grid_constant__ CacheAttnParams p, int n_rt, int64_t items) {
  __shared__ float4 so[W][kD / 4];
  __shared__ float2 sml[W];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * 8 + warp) / W;
  const int64_t item = w / kR;
  const int r = static_cast<int>(w % kR), part0 = warp % W;
  if (item >= items) return;  // with W = 8 these hold for the whole block
  const int rt = static_cast<int>(item % n_rt), hk = static_cast<int>(item / n_rt % p.kv.Hkv);
  const int b = static_cast<int>(item / n_rt / p.kv.Hkv);
  const int64_t row = static_cast<int64_t>(rt) * kR + r;
  if (row >= static_cast<int64_t>(p.T) * p.group) return;
  const Ranges range = find_ranges(p, -1, b);
  const int64_t per_seq = static_cast<int64_t>(n_rt) * p.kv.Hkv, step = per_seq * kR;  // items; rows from a range to the next
  const float2* ml = reinterpret_cast<const float2*>(p.part + per_seq * p.splits * kR * kD);
  const int64_t slot0 = (range.first * per_seq + item % per_seq) * kR + r;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto merge = [&](const float2 (&x)[4], const float4 (&y)[4]) {
    const float top = fmaxf(fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x)), m), use = top == -INFINITY ? 0.f : top;
    const float f0 = ex2(m - use);
    m = top;
    l *= f0;
    o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float f = ex2(x[u].x - use);
      l = fmaf(f, x[u].y, l);
      o = make_float4(fmaf(f, y[u].x, o.x), fmaf(f, y[u].y, o.y), fmaf(f, y[u].z, o.z), fmaf(f, y[u].w, o.w));
    }
  };
  for (int s0 = part0; s0 < range.n; s0 += 4 * W) {
    float2 x[4];
    float4 y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = s0 + u * W;
      const int64_t slot = slot0 + min(i, range.n - 1) * step;  // no branch around a load
      x[u] = ml[slot];
      y[u] = reinterpret_cast<const float4*>(p.part + slot * kD)[lane];
      if (i >= range.n) x[u] = make_float2(-INFINITY, 0.f);
    }
    merge(x, y);
  }
  if constexpr (W > 1) {
    so[warp][lane] = o;
    if (lane == 0) sml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp > 0) return;
    m = -INFINITY;
    l = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s0 = 0; s0 < W; s0 += 4) {
      const float2 x[4] = {sml[s0], sml[s0 + 1], sml[s0 + 2], sml[s0 + 3]};
      const float4 y[4] = {so[s0][lane], so[s0 + 1][lane], so[s0 + 2][lane], so[s0 + 3][lane]};
      merge(x, y);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int t = static_cast<int>(row / p.group), h = hk * p.group + static_cast<int>(row % p.group);
  const int64_t off = b * p.o_sb + t * p.o_ss + h * p.o_sh + 4 * lane;
  if (p.kv.dt == kDtF32)
    *reinterpret_cast<float4*>(static_cast<float*>(p.o) + off) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + off) =
        make_uint2(pack_dt(p.kv.dt, o.x * inv, o.y * inv), pack_dt(p.kv.dt, o.z * inv, o.w * inv));
  if (lane == 0) p.lse[(static_cast<int64_t>(b) * p.H + h) * p.T + t] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

cudaError_t launch_cache_attn_simt(const CacheAttnParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = opt_in_smem(simt_kernel, sizeof(Smem), configured);
  if (e != cudaSuccess) return e;
  const int n_rt = static_cast<int>((static_cast<int64_t>(p.T) * p.group + kR - 1) / kR);
  const int64_t items = simt_items(p.splits > 0 ? 1 : p.B, p.T, p.H, p.kv.Hkv);
  return launch_chained(simt_kernel, dim3(static_cast<unsigned>(items), std::max(p.splits, 1)), dim3(kThreads), sizeof(Smem), stream, p, n_rt);
}

cudaError_t launch_cache_attn_simt_join(const CacheAttnParams& p, cudaStream_t stream) {
  const int n_rt = static_cast<int>((static_cast<int64_t>(p.T) * p.group + kR - 1) / kR);
  const int64_t items = simt_items(p.B, p.T, p.H, p.kv.Hkv);
  // several warps a row where its parts are many: with one, 125 parts took 27 us
  // more than one (10 us in all with eight)
  const int warps = p.splits > 4 * p.B ? 8 : 1;
  return launch_chained(warps == 8 ? simt_join_kernel<8> : simt_join_kernel<1>, dim3(static_cast<unsigned>((items * kR * warps + 7) / 8)),
                        dim3(256), 0, stream, p, n_rt, items);
}

}  // namespace st
