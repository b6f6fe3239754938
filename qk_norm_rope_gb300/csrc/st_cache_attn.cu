// Cached attention on the tensor cores: the plain forms over 16-bit caches, and
// the kernels that join the parts of any form. (The kernel itself and what bounds
// it: st_cache_attn.cuh.)
#include "st_cache_attn.cuh"

namespace st {

namespace {

// Joins the parts of an item whose tiles several CTAs held: block (x, y) looks
// at the border before CTA x + 1 and, if it is an item's first inner border,
// at rows kJoinRows y .. of that item. A warp takes a row, a lane four columns; U
// parts are in flight: many where there are few rows (a decoding step, whose
// items are spread over many CTAs), few and more warps per SM where there are
// many rows.
constexpr int kJoinRows = 16;
template <int U>
__global__ void __launch_bounds__(256, U > 4 ? 2 : 6) join_kernel(const __grid_constant__ TcAttnParams P, int nt) {
  grid_dependency_wait();
  const CacheAttnParams& c = P.c;
  const int cta = blockIdx.x + 1;
  const JoinMeta me = P.meta[cta];
  if (me.parts == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tile_rows = P.tpt * c.group;
  for (int r = blockIdx.y * kJoinRows + warp; r < min((static_cast<int>(blockIdx.y) + 1) * kJoinRows, P.part_rows); r += 8) {
    const int ti = r / tile_rows, rr = r - ti * tile_rows;
    const int t = (me.m * nt + ti) * P.tpt + rr / c.group, h = me.h * c.group + rr % c.group;
    if (t >= me.cnt) continue;
    // the running maximum and sum over the parts
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < me.parts; i0 += U) {
      float2 x[U];
      float4 y[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u;
        x[u] = make_float2(-INFINITY, 0.f);
        y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < me.parts) {  // the same for the whole block
          const int64_t row = (i == 0 ? me.slot0 : 2 * static_cast<int64_t>(cta - 1 + i)) * P.part_rows + r;
          x[u] = P.part_ml[row];
          y[u] = reinterpret_cast<const float4*>(c.part + row * kD)[lane];
        }
      }
      float top = m;
#pragma unroll
      for (int u = 0; u < U; ++u) top = fmaxf(top, x[u].x);
      const float use = top == -INFINITY ? 0.f : top, f0 = ex2(m - use);
      m = top;
      l *= f0;
      o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = ex2(x[u].x - use);
        l = fmaf(f, x[u].y, l);
        o.x = fmaf(f, y[u].x, o.x);
        o.y = fmaf(f, y[u].y, o.y);
        o.z = fmaf(f, y[u].z, o.z);
        o.w = fmaf(f, y[u].w, o.w);
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t off = me.b * c.o_sb + static_cast<int64_t>(t) * c.o_ss + static_cast<int64_t>(h) * c.o_sh + 4 * lane;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c.o) + off) =
        make_uint2(pack_dt(c.q.dt, o.x * inv, o.y * inv), pack_dt(c.q.dt, o.z * inv, o.w * inv));
    if (lane == 0) c.lse[(static_cast<int64_t>(me.b) * c.H + h) * c.T + t] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// By items (a shared prefix, FEW): a row's results over the prefix's tiles and over
// its own keys come together, each whole or in the parts that CTAs left of it, these
// in four copies with FEW. W warps take a row, a lane four columns; four parts are in
// flight for each, and the first warp brings the warps' results together. (One token
// of 8 K/V heads after 30000 keys in 8 bits has 76 parts a row.)
template <int W>
__global__ void __launch_bounds__(256) join_items_kernel(const __grid_constant__ TcAttnParams P, int nt) {
  __shared__ float4 so[W][kD / 4];
  __shared__ float2 sml[W];
  grid_dependency_wait();
  const CacheAttnParams& c = P.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % W;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 8 + warp) / W;
  if (row >= static_cast<int64_t>(c.B) * c.T * c.H) return;  // with W = 8 these hold for the whole block
  const int64_t tok = row / c.H;  // at most 2^30
  const int hq = static_cast<int>(row - tok * c.H), b = static_cast<int>(tok / c.T), t = static_cast<int>(tok - static_cast<int64_t>(b) * c.T);
  const int h = hq / c.group, g = hq - h * c.group, tpg = P.tpt * nt, im = t / tpg, pm = static_cast<int>(tok / tpg);
  // everything that says where the parts are in one round trip
  const int cnt = row_count(c.counts, b, c.T), len = ld_now(c.lens + b), p0 = c.shared ? ld_now(P.p0) : 0;
  const int2 own = P.item_meta[item_index(P, h, b, im)], pre = c.shared ? P.item_meta[item_index(P, h, -1, pm)] : make_int2(0, 0);
  if (t >= cnt) return;  // the attention kernel wrote it
  // the prefix's parts come first, then those of the row's own keys (no tiles: what is
  // said of them is of another call)
  const int copies = P.few ? 4 : 1, n_pre = p0 > 0 ? pre.x : 0;
  const int n = n_pre + (item_from<true>(P, nt, im, p0, len, cnt).n > 0 ? own.x * copies : 0);
  auto place = [&](const int2& meta, int m, int ib, int i, int copy, int r) {
    const int64_t first = meta.y < 0 ? whole_part(P, h, ib, m) : static_cast<int64_t>(meta.y) * P.split_rows;
    return (i == 0 ? first : 2 * (static_cast<int64_t>(meta.y >> 1) + i) * P.split_rows) + copy * P.part_rows + r;
  };
  // rows in their items: tiles of tpt tokens follow one another without gaps
  const int own_r = (t - im * tpg) * c.group + g, pre_r = (static_cast<int>(tok) - pm * tpg) * c.group + g;
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
  for (int i0 = 4 * part; i0 < n; i0 += 4 * W) {
    float2 x[4];
    float4 y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int v = min(i0 + u, n - 1), w = v - n_pre;
      const int64_t at = w < 0 ? place(pre, pm, -1, v, 0, pre_r)
                               : place(own, im, b, copies == 4 ? w >> 2 : w, copies == 4 ? w & 3 : 0, own_r);
      x[u] = P.part_ml[at];
      y[u] = reinterpret_cast<const float4*>(c.part + at * kD)[lane];
      if (i0 + u >= n) x[u] = make_float2(-INFINITY, 0.f);
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
    for (int w = 0; w < W; w += 4) {
      const float2 x[4] = {sml[w], sml[w + 1], sml[w + 2], sml[w + 3]};
      const float4 y[4] = {so[w][lane], so[w + 1][lane], so[w + 2][lane], so[w + 3][lane]};
      merge(x, y);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t off = b * c.o_sb + static_cast<int64_t>(t) * c.o_ss + static_cast<int64_t>(hq) * c.o_sh + 4 * lane;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c.o) + off) = make_uint2(pack_dt(c.q.dt, o.x * inv, o.y * inv), pack_dt(c.q.dt, o.z * inv, o.w * inv));
  if (lane == 0) c.lse[(static_cast<int64_t>(b) * c.H + hq) * c.T + t] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

cudaError_t launch_cache_attn_tc(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream) {
  const bool ext = p.c.window > 0 || p.c.shared;
  if (p.c.kv.dt == kDtE4M3) return ext ? launch_cache_attn_e4m3_ext(p, nt, f16, stream) : launch_cache_attn_e4m3(p, nt, f16, stream);
  if (p.c.kv.dt == kDtI8) return ext ? launch_cache_attn_i8_ext(p, nt, f16, stream) : launch_cache_attn_i8(p, nt, f16, stream);
  if (ext) return launch_cache_attn_ext(p, nt, f16, stream);
  return launch_form<0, false>(p, nt, f16, stream);
}

cudaError_t launch_cache_attn_join(const TcAttnParams& p, int nt, cudaStream_t stream) {
  if (p.item_meta) {
    const int64_t rows = static_cast<int64_t>(p.c.B) * p.c.T * p.c.H;
    // eight warps a row where all blocks then run at once and have several parts each
    // (one token of 8 K/V heads after 240000 keys 25 us with one warp and 10 with eight,
    // 512 rows 10.6 and 8.7, 1024 rows 9.4 and 11.8, 4608 rows 10 and 25)
    const int warps = rows <= 768 ? 8 : 1;
    return launch_chained(warps == 8 ? join_items_kernel<8> : join_items_kernel<1>, dim3(static_cast<unsigned>((rows * warps + 7) / 8)), dim3(256),
                          0, stream, p, nt);
  }
  // few rows, or few items, whose parts are then many
  const bool deep = p.part_rows <= 32 || static_cast<int64_t>(p.c.B) * p.c.kv.Hkv * p.n_groups * 4 <= p.ctas;
  return launch_chained(deep ? join_kernel<16> : join_kernel<4>, dim3(p.ctas - 1, (p.part_rows + kJoinRows - 1) / kJoinRows), dim3(256), 0, stream, p, nt);
}

}  // namespace st
