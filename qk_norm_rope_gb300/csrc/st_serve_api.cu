// C-ABI host layer of the serving calls: argument checks, workspace sizes and
// launches. Nothing here allocates device memory or synchronises a stream.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "st_host.h"
#include "st_kernels.h"
#include "st_serve.h"

namespace {

using namespace st;

constexpr unsigned kRowTypes = bit(ST_BF16) | bit(ST_F16) | bit(ST_F32), kHeldTypes = bit(ST_E4M3) | bit(ST_I8);
static_assert(static_cast<int>(ST_E4M3) == kDtE4M3 && static_cast<int>(ST_I8) == kDtI8, "type codes");
constexpr int kSmCount = 152;

// A contiguous int32 or fp32 vector [B].
st_status check_flat(const st_tensor* t, const char* name, int64_t B, int dtype) {
  if (!t) return fail(ST_ERR_INVALID_ARG, "%s is NULL", name);
  if (t->ndim != 1 || t->shape[0] != B) return fail(ST_ERR_SHAPE, "%s must be [%lld]", name, (long long)B);
  if (t->dtype != dtype) return fail(ST_ERR_DTYPE, "%s must be %s", name, dtype == ST_I32 ? "int32" : "fp32");
  if (B > 0 && !t->data) return fail(ST_ERR_INVALID_ARG, "%s data is NULL", name);
  if (B > 1 && t->stride[0] != 1) return fail(ST_ERR_ALIGN, "%s must be contiguous", name);
  if (reinterpret_cast<uintptr_t>(t->data) & 3u) return fail(ST_ERR_ALIGN, "%s data pointer is not 4-byte aligned", name);
  return ST_OK;
}

// A two-dimensional int32 (or fp32, or int64) tensor [B (or 1), n] with unit
// stride on n; *sb is its batch stride (0 when shared).
st_status check_rows(const st_tensor* t, const char* name, int64_t B, int64_t n, bool one, int dtype, int64_t* sb) {
  if (!t) return fail(ST_ERR_INVALID_ARG, "%s is NULL", name);
  if (t->ndim != 2 || !(t->shape[0] == B || (one && t->shape[0] == 1)) || t->shape[1] != n)
    return fail(ST_ERR_SHAPE, "%s must be [%lld%s, %lld]", name, (long long)B, one ? "|1" : "", (long long)n);
  if (t->dtype != dtype) return fail(ST_ERR_DTYPE, "%s must be %s", name, dtype == ST_I32 ? "int32" : "fp32");
  if (t->shape[0] * n > 0 && !t->data) return fail(ST_ERR_INVALID_ARG, "%s data is NULL", name);
  if (n > 1 && t->stride[1] != 1) return fail(ST_ERR_ALIGN, "%s must have unit stride on its last dim", name);
  if (reinterpret_cast<uintptr_t>(t->data) & 3u) return fail(ST_ERR_ALIGN, "%s data pointer is not 4-byte aligned", name);
  *sb = t->shape[0] > 1 ? t->stride[0] : 0;
  return ST_OK;
}

// Rows that are written: none may stand for several.
st_status check_own_rows(const st_tensor* t, const char* name) {
  if (t->shape[0] * t->shape[1] * t->shape[2] == 0) return ST_OK;
  for (int a = 0; a < 3; ++a)
    if (t->shape[a] > 1 && t->stride[a] <= 0) return fail(ST_ERR_ALIGN, "%s must not be expanded (stride[%d]=%lld)", name, a, (long long)t->stride[a]);
  return ST_OK;
}

// The scales of K or V of a cache of 8 bits.
st_status check_scales(const st_tensor* t, const char* name, int n, int Hkv, int page, float** p, int64_t* sp, int64_t* sh) {
  if (!t) return fail(ST_ERR_INVALID_ARG, "%s is NULL: a cache of 8 bits needs its scales", name);
  if (t->ndim != 3 || t->shape[0] != n || t->shape[1] != Hkv || t->shape[2] != page)
    return fail(ST_ERR_SHAPE, "%s must be [N_pages, H_kv, page] = [%d, %d, %d]", name, n, Hkv, page);
  if (t->dtype != ST_F32) return fail(ST_ERR_DTYPE, "%s must be fp32", name);
  if (static_cast<int64_t>(n) * Hkv > 0 && !t->data) return fail(ST_ERR_INVALID_ARG, "%s data is NULL", name);
  if (page > 1 && t->stride[2] != 1) return fail(ST_ERR_ALIGN, "%s must have unit stride on page", name);
  if (reinterpret_cast<uintptr_t>(t->data) & 3u) return fail(ST_ERR_ALIGN, "%s data pointer is not 4-byte aligned", name);
  if ((n > 1 && t->stride[0] <= 0) || (Hkv > 1 && t->stride[1] <= 0)) return fail(ST_ERR_ALIGN, "%s must not be expanded", name);
  *p = static_cast<float*>(t->data);
  *sp = n > 1 ? t->stride[0] : 0;
  *sh = Hkv > 1 ? t->stride[1] : 0;
  return ST_OK;
}

// B < 0: the page table's own batch size is taken. sc: the scales of a cache of
// 8 bits, or NULL.
st_status check_cache(const st_kv_cache* c, const st_kv_scales* sc, int64_t B, PagedKV* out, const char* who) {
  if (!c || !c->k || !c->v || !c->pages) return fail(ST_ERR_INVALID_ARG, "%s: the cache needs k, v and pages", who);
  const st_tensor *k = c->k, *pt = c->pages;
  if (k->ndim != 4) return fail(ST_ERR_SHAPE, "cache.k must be 4-D [N_pages, page, H_kv, D]");
  for (int a = 0; a < 3; ++a)
    if (k->shape[a] < 0 || k->shape[a] > (a == 2 ? 32767 : (1ll << 30))) return fail(ST_ERR_SHAPE, "cache.k sizes out of range");
  if (k->shape[3] != kD) return fail(ST_ERR_UNSUPPORTED, "head dimension %lld is not supported (this build handles D=128)", (long long)k->shape[3]);
  if (k->shape[1] < 1) return fail(ST_ERR_SHAPE, "cache pages must hold at least one row");
  RowTensor rk, rv;
  const int n = static_cast<int>(k->shape[0]), page = static_cast<int>(k->shape[1]), H = static_cast<int>(k->shape[2]);
  st_status st;
  if ((st = check_bshd(k, "cache.k", n, page, H, kD, sc ? kRowTypes | kHeldTypes : kRowTypes, &rk)) != ST_OK) return st;
  if ((st = check_bshd(c->v, "cache.v", n, page, H, kD, bit(k->dtype), &rv)) != ST_OK) return st;
  if ((st = check_own_rows(k, "cache.k")) != ST_OK) return st;
  if ((st = check_own_rows(c->v, "cache.v")) != ST_OK) return st;
  if (pt->ndim != 2 || (B >= 0 && pt->shape[0] != B)) return fail(ST_ERR_SHAPE, "cache.pages must be [%lld, max_pages]", (long long)B);
  if (pt->shape[0] < 0 || pt->shape[0] > 65535 || pt->shape[1] < 0) return fail(ST_ERR_SHAPE, "cache.pages sizes out of range");
  if (pt->dtype != ST_I32) return fail(ST_ERR_DTYPE, "cache.pages must be int32");
  if (pt->shape[0] * pt->shape[1] > 0 && !pt->data) return fail(ST_ERR_INVALID_ARG, "cache.pages data is NULL");
  if (pt->shape[1] > 1 && pt->stride[1] != 1) return fail(ST_ERR_ALIGN, "cache.pages must have unit stride on its last dim");
  if (reinterpret_cast<uintptr_t>(pt->data) & 3u) return fail(ST_ERR_ALIGN, "cache.pages data pointer is not 4-byte aligned");
  if (pt->shape[1] > (1ll << 30) / page) return fail(ST_ERR_SHAPE, "cache.pages: max_pages * page must be at most 2^30");
  memset(out, 0, sizeof(*out));
  out->k = k->data;
  out->v = c->v->data;
  out->dt = k->dtype;
  out->k_sp = rk.sb; out->k_sr = rk.ss; out->k_sh = rk.sh;
  out->v_sp = rv.sb; out->v_sr = rv.ss; out->v_sh = rv.sh;
  out->pages = static_cast<const int32_t*>(pt->data);
  out->p_sb = pt->shape[0] > 1 ? pt->stride[0] : 0;
  out->p_sj = 1;
  out->n_pages = n;
  out->page = page;
  out->page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (page == 1 << i) out->page_shift = i;
  out->max_pages = static_cast<int>(pt->shape[1]);
  out->Hkv = H;
  if (!sc) return ST_OK;
  if (!(bit(k->dtype) & kHeldTypes)) return fail(ST_ERR_INVALID_ARG, "%s: scales belong to a cache of 8 bits", who);
  if ((st = check_scales(sc->k, "k_scale", n, H, page, &out->ks, &out->ks_sp, &out->ks_sh)) != ST_OK) return st;
  return check_scales(sc->v, "v_scale", n, H, page, &out->vs, &out->vs_sp, &out->vs_sh);
}

// Sizes of a new-rows tensor [B, T, H, D].
st_status check_new_rows(const st_tensor* q, const char* name, int* B, int* T, int* H) {
  if (!q) return fail(ST_ERR_INVALID_ARG, "%s is NULL", name);
  if (q->ndim != 4) return fail(ST_ERR_SHAPE, "%s must be 4-D [B,T,H,D], got ndim=%d", name, q->ndim);
  if (q->shape[3] != kD) return fail(ST_ERR_UNSUPPORTED, "head dimension %lld is not supported (this build handles D=128)", (long long)q->shape[3]);
  if (q->shape[0] < 0 || q->shape[0] > 65535 || q->shape[1] < 0 || q->shape[1] > (1ll << 30) || q->shape[2] < 0 || q->shape[2] > 65535)
    return fail(ST_ERR_SHAPE, "%s sizes out of range", name);
  *B = static_cast<int>(q->shape[0]);
  *T = static_cast<int>(q->shape[1]);
  *H = static_cast<int>(q->shape[2]);
  return ST_OK;
}

st_status check_heads(int H, int Hkv) {
  if (H == 0 ? Hkv != 0 : (Hkv < 1 || H % Hkv != 0))
    return fail(ST_ERR_SHAPE, "the cache has %d heads: the K/V head count must divide H=%d", Hkv, H);
  return ST_OK;
}

st_status check_counts(const st_tensor* t, int B, const int32_t** out) {
  *out = nullptr;
  if (!t) return ST_OK;
  st_status st = check_flat(t, "counts", B, ST_I32);
  if (st == ST_OK) *out = static_cast<const int32_t*>(t->data);
  return st;
}

struct AttnPlan {
  TcAttnParams tc;        // c: the parameters of either kernel
  bool tensor = false;    // the tensor-core kernel
  int nt = 1;
  size_t bytes = 0, off_ml = 0, off_meta = 0, off_p0 = 0;
};

// Strides for 32-bit places of rows and scales; false where these do not fit.
bool held_at(const PagedKV& kv, TcAttnParams* t) {
  const int64_t n = kv.n_pages - 1, r = kv.page - 1, h = kv.Hkv - 1, most = (1ll << 32) - 2;
  if ((n * kv.k_sp + r * kv.k_sr + h * kv.k_sh) / 16 > most || (n * kv.v_sp + r * kv.v_sr + h * kv.v_sh) / 16 > most ||
      n * kv.ks_sp + h * kv.ks_sh + r > most || n * kv.vs_sp + h * kv.vs_sh + r > most)
    return false;
  auto u = [](int64_t x) { return static_cast<uint32_t>(x); };
  t->held_k = {u(kv.k_sp / 16), u(kv.k_sr / 16), u(kv.k_sh / 16), u(kv.ks_sp), u(kv.ks_sh)};
  t->held_v = {u(kv.v_sp / 16), u(kv.v_sr / 16), u(kv.v_sh / 16), u(kv.vs_sp), u(kv.vs_sh)};
  return true;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

st_status plan_attn(const st_tensor* q, const st_kv_cache* cache, const st_cache_attn_opts* opts, const st_tensor* parents, AttnPlan* P) {
  memset(&P->tc, 0, sizeof(P->tc));
  CacheAttnParams& p = P->tc.c;
  st_status st;
  if ((st = check_new_rows(q, "q_rot", &p.B, &p.T, &p.H)) != ST_OK) return st;
  if ((st = check_cache(cache, opts ? opts->scales : nullptr, p.B, &p.kv, "st_cache_attn")) != ST_OK) return st;
  if ((st = check_bshd(q, "q_rot", p.B, p.T, p.H, kD, held(p.kv) ? kRowTypes : bit(p.kv.dt), &p.q)) != ST_OK) return st;
  if ((st = check_heads(p.H, p.kv.Hkv)) != ST_OK) return st;
  p.group = p.kv.Hkv > 0 ? p.H / p.kv.Hkv : 1;
  if (p.group > kMaxGroup) return fail(ST_ERR_UNSUPPORTED, "%d query heads per K/V head: at most %d are supported", p.group, kMaxGroup);
  if (parents) {
    if ((st = check_rows(parents, "parents", p.B, p.T, true, ST_I32, &p.par_sb)) != ST_OK) return st;
    if (p.T > kMaxTree) return fail(ST_ERR_UNSUPPORTED, "a tree of %d nodes: at most %d are supported", p.T, kMaxTree);
    p.parents = static_cast<const int32_t*>(parents->data);
  }
  if (opts) {
    if (opts->window < 0 || opts->sinks < 0) return fail(ST_ERR_INVALID_ARG, "window and sinks must be at least 0");
    p.window = opts->window;
    p.sinks = opts->window > 0 ? opts->sinks : 0;
    if (opts->shared) {
      if ((st = check_flat(opts->shared, "shared", 1, ST_I32)) != ST_OK) return st;
      // with a window a sequence has few keys, and the rows see different ones
      if (p.window == 0) p.shared = static_cast<const int32_t*>(opts->shared->data);
    }
  }
  P->bytes = 256;
  if (static_cast<int64_t>(p.B) * p.T * p.H == 0) return ST_OK;
  // The tensor-core kernel takes every 16-bit cache whose pages are whole TMA
  // boxes (at least one 8-row swizzle atom), and caches of 8 bits whose K and V
  // span at most 64 GB each; fp32 rows and what is left take the CUDA cores.
  P->tensor = p.kv.dt != ST_F32 && (held(p.kv) ? held_at(p.kv, &P->tc) : p.kv.page % 8 == 0) && p.kv.n_pages > 0 && p.kv.max_pages > 0 &&
              p.q.dt != ST_F32;
  if (P->tensor) {
    TcAttnParams& t = P->tc;
    P->nt = tc_tiles(p.T, p.group);
    // A shared prefix's rows are the whole batch's: two tiles of them for each K/V
    // tile, unless that leaves the sequences' own tiles nearly empty (half of one
    // tile's rows, over 8 bits those of the form for few rows, where a tile's
    // conversion counts for more). 16384 to 32768 shared tokens, up to 2000 more: 72
    // rows of a sequence 132 us with one tile and 129 with two, over e4m3 189 and 166;
    // 36 rows 134 and 147, 195 and 182; 16 rows 86 and 101, 116 and 124.
    const int64_t own_rows = static_cast<int64_t>(p.T) * p.group;
    if (p.shared && P->nt == 1 && own_rows >= (held(p.kv) ? 33 : 64)) P->nt = tc_tiles(static_cast<int64_t>(p.B) * p.T, p.group);
    t.box_shift = 3;
    while ((1 << t.box_shift) < kTile && p.kv.page % (2 << t.box_shift) == 0) ++t.box_shift;
    t.tpt = kTile / p.group;
    const int64_t tpg = static_cast<int64_t>(t.tpt) * P->nt;
    t.n_groups = static_cast<int>((p.T + tpg - 1) / tpg);
    t.part_rows = static_cast<int>(std::min<int64_t>(p.T, tpg)) * p.group;
    int64_t cap_tiles = (static_cast<int64_t>(p.kv.max_pages) * p.kv.page + kTile - 1) / kTile;
    // a window's tiles: the first tokens', the window's and its rows', one for the window's edge
    if (p.window > 0)
      cap_tiles = std::min(cap_tiles, (static_cast<int64_t>(p.sinks) + kTile - 1) / kTile +
                                          (static_cast<int64_t>(p.window) + std::min<int64_t>(p.T, p.parents ? p.T : tpg) + kTile - 1) / kTile + 1);
    int64_t items = static_cast<int64_t>(p.B) * p.kv.Hkv * t.n_groups;
    t.few = held(p.kv) && t.part_rows <= 32;
    t.split_rows = t.part_rows * (t.few ? 4 : 1);
    if (p.shared) {
      const int64_t tokens = static_cast<int64_t>(p.B) * p.T;
      if (tokens > (1ll << 30)) return fail(ST_ERR_SHAPE, "too many query rows");
      t.n_pre = static_cast<int>((tokens + tpg - 1) / tpg);
      t.pre_rows = static_cast<int>(std::min<int64_t>(tokens, tpg)) * p.group;
      t.split_rows = std::max(t.pre_rows, t.split_rows);
      items += static_cast<int64_t>(p.kv.Hkv) * t.n_pre;
    }
    if (items > (1ll << 40) || static_cast<int64_t>(p.B) * t.n_groups + t.n_pre > (1ll << 30)) return fail(ST_ERR_SHAPE, "too many query rows");
    // The clustered form: as many CTAs per item as let all clusters run at once
    // (15 clusters of 8 such CTAs, 36 of 4, 76 of 2 fit the GPU; 16 of 8 took
    // two turns: 18.3 us against 11.0 with 4). Its shares are even per item
    // instead of over the call: up to room * (1 / cluster - mean * items / SMs)
    // key tiles more for a CTA (mean: the mean length over the room, taken as 1
    // for one sequence and 1/2 for a batch, whose lengths differ: the lengths are on
    // the device, so a table with room for far more than they need is dealt, 777
    // keys with room for 16384 or more 11.5 us, 8 sequences of up to 1000 16.9);
    // it saves the scan for the beginning and the join, as much as about 8 tiles.
    // One token, 8 K/V heads: 777 keys 10.5 us dealt, 7.1 clustered; 8000 keys 17.9 and
    // 14.4; 16000 keys 18.8 and 22.3; 8 sequences of up to 1000 keys 16.6 and
    // 10.9, of up to 8000 keys 36 and 43.
    // With more than 128 rows a head the join is the larger part: as much as 16
    // tiles (a tree of 61 nodes, 32 / 8 heads: 1000 keys 22 us dealt, 15.6
    // clustered; 8000 keys 41 and 26; 32000 keys 61 and 69).
    t.cluster = 0;
    {
      const int cl = items <= 15 ? 8 : (items <= 36 ? 4 : (items <= 76 ? 2 : 1));
      static_assert(kMaxClusterAttn == 8, "the largest cluster");
      const int64_t mean = p.B == 1 ? 2 : 1, saved = P->nt == 1 ? 16 : 32;  // halves of the room; of tiles
      if (cl > 1 && !p.shared && cap_tiles * (2 * kSmCount - mean * items * cl) <= saved * cl * kSmCount) t.cluster = cl;
    }
    if (t.cluster > 0) {
      t.ctas = static_cast<int>(items) * t.cluster;
      t.cluster_shift = t.cluster == 8 ? 3 : t.cluster / 2;
      return ST_OK;  // no workspace
    }
    t.ctas = static_cast<int>(items >= kSmCount ? kSmCount : std::min<int64_t>(kSmCount, items * cap_tiles));
    if (p.shared || t.few) {
      const int64_t own = items - static_cast<int64_t>(p.kv.Hkv) * t.n_pre;
      const size_t rows = static_cast<size_t>(2) * t.ctas * t.split_rows + static_cast<size_t>(items - own) * t.pre_rows + static_cast<size_t>(own) * t.part_rows * (t.few ? 4 : 1);
      size_t off = align256(rows * kD * sizeof(float));
      P->off_ml = off;
      off = align256(off + rows * sizeof(float2));
      P->off_meta = off;
      P->off_p0 = align256(off + items * sizeof(int2));
      P->bytes = P->off_p0 + 256;
      return ST_OK;
    }
    // a CTA leaves at most two parts: one at each end of its range
    size_t off = align256(static_cast<size_t>(2) * t.ctas * t.part_rows * kD * sizeof(float));
    P->off_ml = off;
    off = align256(off + static_cast<size_t>(2) * t.ctas * t.part_rows * sizeof(float2));
    P->off_meta = off;
    P->bytes = align256(off + t.ctas * sizeof(JoinMeta));
    return ST_OK;
  }
  const int64_t items = simt_items(p.B, p.T, p.H, p.kv.Hkv);
  if (items > (1ll << 30)) return fail(ST_ERR_SHAPE, "too many query rows");
  const int64_t tiles = (static_cast<int64_t>(p.kv.max_pages) * p.kv.page + kSimtKeys - 1) / kSimtKeys;
  // few items: as many key ranges as give two CTAs per SM (what fits), dealt to
  // the sequences by their lengths (fp32, 8 K/V heads, single tokens after 2000
  // keys each: 19 sequences 234 us with their two ranges each, 20 without 449)
  if (2 * kSmCount / items >= 2 && tiles > 1) {
    const int64_t per_seq = items / p.B;
    p.splits = static_cast<int>(2 * kSmCount / per_seq);
    P->bytes = static_cast<size_t>(per_seq) * p.splits * kSimtRows * (kD + 2) * sizeof(float);
  }
  return ST_OK;
}

}  // namespace

extern "C" {

st_status st_cache_append(const st_tensor* q, const st_tensor* k, const st_tensor* v, const st_tensor* q_norm_w,
                          const st_tensor* k_norm_w, float eps, const st_rope* rope, const st_kv_cache* cache,
                          const st_tensor* lens, const st_tensor* counts, st_tensor* q_rot, void* stream_) {
  return st_cache_append_held(q, k, v, q_norm_w, k_norm_w, eps, rope, cache, nullptr, lens, counts, q_rot, stream_);
}

st_status st_cache_append_held(const st_tensor* q, const st_tensor* k, const st_tensor* v, const st_tensor* q_norm_w,
                               const st_tensor* k_norm_w, float eps, const st_rope* rope, const st_kv_cache* cache,
                               const st_kv_scales* scales, const st_tensor* lens, const st_tensor* counts, st_tensor* q_rot,
                               void* stream_) {
  clear_error();
  AppendParams p;
  memset(&p, 0, sizeof(p));
  st_status st;
  if ((st = check_new_rows(q, "q", &p.B, &p.T, &p.H)) != ST_OK) return st;
  if ((st = check_cache(cache, scales, p.B, &p.kv, "st_cache_append")) != ST_OK) return st;
  if ((st = check_heads(p.H, p.kv.Hkv)) != ST_OK) return st;
  // the type of v and q': the cache's, with one of 8 bits any
  const unsigned row = held(p.kv) ? kRowTypes : bit(p.kv.dt);
  if ((st = check_bshd(v, "v", p.B, p.T, p.kv.Hkv, kD, row, &p.v)) != ST_OK) return st;
  const unsigned qk = bit(v->dtype) | bit(ST_F32);
  if ((st = check_bshd(q, "q", p.B, p.T, p.H, kD, qk, &p.q)) != ST_OK) return st;
  if ((st = check_bshd(k, "k", p.B, p.T, p.kv.Hkv, kD, qk, &p.k)) != ST_OK) return st;
  if (q->dtype != k->dtype) return fail(ST_ERR_DTYPE, "q and k must have the same dtype");
  if ((st = check_vec(q_norm_w, "q_norm_w", kD)) != ST_OK) return st;
  if ((st = check_vec(k_norm_w, "k_norm_w", kD)) != ST_OK) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(ST_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!rope) return fail(ST_ERR_INVALID_ARG, "rope is NULL");
  if (rope->ids_k || rope->cos_k || rope->sin_k)
    return fail(ST_ERR_INVALID_ARG, "rope: the new rows of q and k share one rotation (no ids_k, cos_k or sin_k)");
  Ids ids{};
  if (rope->cos || rope->sin) {
    if (rope->ids) return fail(ST_ERR_INVALID_ARG, "rope: give either ids or cos/sin tables, not both");
    if ((st = check_tables(rope->cos, rope->sin, "rope.cos/sin", p.B, p.T, &ids)) != ST_OK) return st;
  } else {
    if ((st = check_axes(rope, kD)) != ST_OK) return st;
    if ((st = check_ids(rope->ids, "rope.ids", p.B, p.T, rope->n_axes, &ids)) != ST_OK) return st;
  }
  if ((st = check_flat(lens, "lens", p.B, ST_I32)) != ST_OK) return st;
  if ((st = check_counts(counts, p.B, &p.counts)) != ST_OK) return st;
  RowTensor ro;
  if ((st = check_bshd(q_rot, "q_rot", p.B, p.T, p.H, kD, bit(v->dtype), &ro)) != ST_OK) return st;
  if ((st = check_own_rows(q_rot, "q_rot")) != ST_OK) return st;
  const int64_t tokens = static_cast<int64_t>(p.B) * p.T;
  if (tokens > (1ll << 30) || tokens * (p.H + 2 * p.kv.Hkv) > (1ll << 32)) return fail(ST_ERR_SHAPE, "too many new rows");
  if (tokens * p.H == 0) return ST_OK;
  Dev dev;
  if ((st = device_globals(&dev)) != ST_OK) return st;
  if (ids.table) {
    fill_table(ids, rope, nullptr, nullptr, nullptr, &p.tab);
  } else {
    // the pairs' frequencies depend on the widths and theta alone, which a
    // model never changes: a thread keeps its last ones (64 powers a call
    // otherwise)
    struct Freq {
      int n = 0, axes[8];
      double theta;
      TableParams tab;
      unsigned long long turns[kPairs];
    };
    static thread_local Freq f;
    if (f.n != rope->n_axes || f.theta != rope->theta || memcmp(f.axes, rope->axes_dim, sizeof(int) * f.n) != 0) {
      f.n = 0;
      fill_table(ids, rope, nullptr, nullptr, nullptr, &f.tab);
      for (int j = 0; j < kPairs; ++j) {
        const double turn = f.tab.omega[j] * 0.15915494309189535;  // 1 / (2 pi)
        f.turns[j] = static_cast<unsigned long long>((turn - std::floor(turn)) * 18446744073709551616.0);
      }
      memcpy(f.axes, rope->axes_dim, sizeof(int) * rope->n_axes);
      f.theta = rope->theta;
      f.n = rope->n_axes;
    }
    memcpy(p.tab.omega, f.tab.omega, sizeof(p.tab.omega));
    memcpy(p.tab.axis_of, f.tab.axis_of, sizeof(p.tab.axis_of));
    memcpy(p.turns, f.turns, sizeof(p.turns));
    fill_ids(ids, &p.tab);
  }
  p.wq = static_cast<const float*>(q_norm_w->data);
  p.wk = static_cast<const float*>(k_norm_w->data);
  p.eps = eps;
  p.lens = static_cast<const int32_t*>(lens->data);
  p.qo = q_rot->data;
  p.qo_sb = ro.sb; p.qo_ss = ro.ss; p.qo_sh = ro.sh;
  p.status = dev.status;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return cuda_check(launch_counted(ST_K_CACHE_APPEND, stream, [&] { return launch_cache_append(p, stream); }),
                    "cache append launch");
}

size_t st_cache_attn_workspace_size(const st_tensor* q_rot, const st_kv_cache* cache, const st_tensor* parents) {
  return st_cache_attn_opt_workspace_size(q_rot, cache, nullptr, parents);
}

size_t st_cache_attn_opt_workspace_size(const st_tensor* q_rot, const st_kv_cache* cache, const st_cache_attn_opts* opts,
                                        const st_tensor* parents) {
  clear_error();
  AttnPlan P;
  if (plan_attn(q_rot, cache, opts, parents, &P) != ST_OK) return 0;
  return P.bytes;
}

st_status st_cache_attn(const st_tensor* q_rot, const st_kv_cache* cache, const st_tensor* lens, const st_tensor* counts,
                        const st_tensor* parents, float scale, st_tensor* o, st_tensor* lse, void* workspace,
                        size_t workspace_bytes, void* stream_) {
  return st_cache_attn_opt(q_rot, cache, nullptr, lens, counts, parents, scale, o, lse, workspace, workspace_bytes, stream_);
}

st_status st_cache_attn_opt(const st_tensor* q_rot, const st_kv_cache* cache, const st_cache_attn_opts* opts, const st_tensor* lens,
                            const st_tensor* counts, const st_tensor* parents, float scale, st_tensor* o, st_tensor* lse,
                            void* workspace, size_t workspace_bytes, void* stream_) {
  clear_error();
  AttnPlan P;
  st_status st = plan_attn(q_rot, cache, opts, parents, &P);
  if (st != ST_OK) return st;
  CacheAttnParams& p = P.tc.c;
  if ((st = check_flat(lens, "lens", p.B, ST_I32)) != ST_OK) return st;
  if ((st = check_counts(counts, p.B, &p.counts)) != ST_OK) return st;
  if (!std::isfinite(scale)) return fail(ST_ERR_INVALID_ARG, "scale must be finite");
  RowTensor ro;
  if ((st = check_bshd(o, "o", p.B, p.T, p.H, kD, bit(p.q.dt), &ro)) != ST_OK) return st;
  if ((st = check_own_rows(o, "o")) != ST_OK) return st;
  if (static_cast<int64_t>(p.B) * p.T * p.H > 0 && o->data == q_rot->data)
    return fail(ST_ERR_INVALID_ARG, "o must not be q_rot: its rows are read until the call ends");
  if (!lse || lse->ndim != 3 || lse->shape[0] != p.B || lse->shape[1] != p.H || lse->shape[2] != p.T)
    return fail(ST_ERR_SHAPE, "lse must be [B,H,T] = [%d,%d,%d]", p.B, p.H, p.T);
  if (lse->dtype != ST_F32) return fail(ST_ERR_DTYPE, "lse must be fp32");
  const int64_t rows = static_cast<int64_t>(p.B) * p.T * p.H;
  if (rows > 0 && (!lse->data || (p.T > 1 && lse->stride[2] != 1) || (p.H > 1 && lse->stride[1] != p.T) ||
                   (p.B > 1 && lse->stride[0] != static_cast<int64_t>(p.H) * p.T)))
    return fail(ST_ERR_ALIGN, "lse must be contiguous");
  if (workspace_bytes < P.bytes)
    return fail(ST_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu required", workspace_bytes, P.bytes);
  if (!workspace) return fail(ST_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return fail(ST_ERR_ALIGN, "workspace must be 256-byte aligned");
  if (rows == 0) return ST_OK;
  Dev dev;
  if ((st = device_globals(&dev)) != ST_OK) return st;
  p.lens = static_cast<const int32_t*>(lens->data);
  const float sc = scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(kD));
  p.scale_log2 = sc * kLog2e;
  p.o = o->data;
  p.o_sb = ro.sb; p.o_ss = ro.ss; p.o_sh = ro.sh;
  p.lse = static_cast<float*>(lse->data);
  p.part = static_cast<float*>(workspace);
  p.status = dev.status;
  p.counters = dev.counters;
  p.wait_budget = wait_budget();
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (P.tensor) {
    TcAttnParams& t = P.tc;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    t.part_ml = reinterpret_cast<float2*>(ws + P.off_ml);
    t.meta = reinterpret_cast<JoinMeta*>(ws + P.off_meta);
    t.item_meta = P.off_p0 > 0 ? reinterpret_cast<int2*>(ws + P.off_meta) : nullptr;  // by items
    t.p0 = reinterpret_cast<int*>(ws + P.off_p0);
    t.o_wide = (reinterpret_cast<uintptr_t>(p.o) & 31u) == 0 && p.o_sb % 16 == 0 && p.o_ss % 16 == 0 && p.o_sh % 16 == 0;
    if (!held(p.kv) && (st = encode_rows_map(cache->k, &t.tmap_k, &t.k_r_first, 1 << t.box_shift)) != ST_OK) return st;
    if (!held(p.kv) && (st = encode_rows_map(cache->v, &t.tmap_v, &t.v_r_first, 1 << t.box_shift)) != ST_OK) return st;
    if ((st = cuda_check(launch_counted(ST_K_CACHE_ATTN, stream, [&] { return launch_cache_attn_tc(t, P.nt, p.q.dt == ST_F16, stream); }),
                         "cached attention launch")) != ST_OK)
      return st;
    if (t.cluster > 0) return ST_OK;
    return cuda_check(launch_counted(ST_K_CACHE_JOIN, stream, [&] { return launch_cache_attn_join(t, P.nt, stream); }),
                      "cached attention join launch");
  }
  if ((st = cuda_check(launch_counted(ST_K_CACHE_ATTN, stream, [&] { return launch_cache_attn_simt(p, stream); }),
                       "cached attention launch")) != ST_OK)
    return st;
  if (p.splits == 0) return ST_OK;
  return cuda_check(launch_counted(ST_K_CACHE_JOIN, stream, [&] { return launch_cache_attn_simt_join(p, stream); }),
                    "cached attention join launch");
}

st_status st_tree_verify(const st_tensor* target, const st_tensor* draft, const st_tensor* tokens, const st_tensor* parents,
                         const st_tensor* counts, const st_tensor* u_accept, const st_tensor* u_sample, st_tensor* path,
                         st_tensor* n_accepted, st_tensor* next_token, void* stream_) {
  clear_error();
  VerifyParams p;
  memset(&p, 0, sizeof(p));
  st_status st;
  if (!target) return fail(ST_ERR_INVALID_ARG, "target_probs is NULL");
  if (target->ndim != 3) return fail(ST_ERR_SHAPE, "target_probs must be 3-D [B, T, V]");
  const int64_t B = target->shape[0], T = target->shape[1], V = target->shape[2];
  if (B < 0 || B > 65535 || T < 0 || V < 0 || V > (1ll << 30)) return fail(ST_ERR_SHAPE, "target_probs sizes out of range");
  if (T > kMaxVerify) return fail(ST_ERR_UNSUPPORTED, "a tree of %lld nodes: at most %d are supported", (long long)T, kMaxVerify);
  if (T < 1 || V < 1) return fail(ST_ERR_SHAPE, "target_probs needs at least the root's row and one token");
  for (const st_tensor* t : {target, draft}) {
    if (!t) continue;
    const char* name = t == target ? "target_probs" : "draft_probs";
    if (t->ndim != 3 || t->shape[0] != B || t->shape[1] != T || t->shape[2] != V)
      return fail(ST_ERR_SHAPE, "%s must be [%lld, %lld, %lld]", name, (long long)B, (long long)T, (long long)V);
    if (t->dtype != ST_F32 && t->dtype != ST_BF16 && t->dtype != ST_F16) return fail(ST_ERR_DTYPE, "%s must be fp32, bf16 or fp16", name);
    if (t->dtype != target->dtype) return fail(ST_ERR_DTYPE, "target_probs and draft_probs must have the same dtype");
    if (B > 0 && !t->data) return fail(ST_ERR_INVALID_ARG, "%s data is NULL", name);
    if (V > 1 && t->stride[2] != 1) return fail(ST_ERR_ALIGN, "%s must have unit stride on V", name);
    if (reinterpret_cast<uintptr_t>(t->data) % elem_bytes(t->dtype)) return fail(ST_ERR_ALIGN, "%s data pointer is not aligned to its elements", name);
  }
  if (!tokens) return fail(ST_ERR_INVALID_ARG, "tokens is NULL");
  if (tokens->ndim != 2 || tokens->shape[0] != B || tokens->shape[1] != T) return fail(ST_ERR_SHAPE, "tokens must be [%lld, %lld]", (long long)B, (long long)T);
  if (tokens->dtype != ST_I32 && tokens->dtype != ST_I64) return fail(ST_ERR_DTYPE, "tokens must be int32 or int64");
  if (B > 0 && !tokens->data) return fail(ST_ERR_INVALID_ARG, "tokens data is NULL");
  p.tok64 = tokens->dtype == ST_I64;
  if (reinterpret_cast<uintptr_t>(tokens->data) % (p.tok64 ? 8 : 4)) return fail(ST_ERR_ALIGN, "tokens data pointer is not aligned to its elements");
  if ((st = check_rows(parents, "parents", B, T, true, ST_I32, &p.par_sb)) != ST_OK) return st;
  if ((st = check_counts(counts, static_cast<int>(B), &p.counts)) != ST_OK) return st;
  int64_t sb;
  if ((st = check_rows(u_accept, "u_accept", B, T, false, ST_F32, &sb)) != ST_OK) return st;
  if (B > 1 && sb != T) return fail(ST_ERR_ALIGN, "u_accept must be contiguous");
  if ((st = check_flat(u_sample, "u_sample", B, ST_F32)) != ST_OK) return st;
  if ((st = check_rows(path, "path", B, T, false, ST_I32, &sb)) != ST_OK) return st;
  if (B > 1 && sb != T) return fail(ST_ERR_ALIGN, "path must be contiguous");
  if ((st = check_flat(n_accepted, "n_accepted", B, ST_I32)) != ST_OK) return st;
  if (!next_token) return fail(ST_ERR_INVALID_ARG, "next_token is NULL");
  if (next_token->ndim != 1 || next_token->shape[0] != B) return fail(ST_ERR_SHAPE, "next_token must be [%lld]", (long long)B);
  if (next_token->dtype != tokens->dtype) return fail(ST_ERR_DTYPE, "next_token must have the dtype of tokens");
  if (B > 0 && !next_token->data) return fail(ST_ERR_INVALID_ARG, "next_token data is NULL");
  if (B > 1 && next_token->stride[0] != 1) return fail(ST_ERR_ALIGN, "next_token must be contiguous");
  if (reinterpret_cast<uintptr_t>(next_token->data) % (p.tok64 ? 8 : 4)) return fail(ST_ERR_ALIGN, "next_token data pointer is not aligned to its elements");
  if (B == 0) return ST_OK;
  Dev dev;
  if ((st = device_globals(&dev)) != ST_OK) return st;
  p.p = target->data;
  p.q = draft ? draft->data : nullptr;
  p.dt = target->dtype;
  p.p_sb = B > 1 ? target->stride[0] : 0;
  p.p_st = T > 1 ? target->stride[1] : 0;
  if (draft) {
    p.q_sb = B > 1 ? draft->stride[0] : 0;
    p.q_st = T > 1 ? draft->stride[1] : 0;
  }
  p.tokens = tokens->data;
  p.tok_sb = B > 1 ? tokens->stride[0] : 0;
  p.tok_st = T > 1 ? tokens->stride[1] : 0;
  p.parents = static_cast<const int32_t*>(parents->data);
  p.u_accept = static_cast<const float*>(u_accept->data);
  p.u_sample = static_cast<const float*>(u_sample->data);
  p.path = static_cast<int32_t*>(path->data);
  p.n_accepted = static_cast<int32_t*>(n_accepted->data);
  p.next_token = next_token->data;
  p.B = static_cast<int>(B);
  p.T = static_cast<int>(T);
  p.V = static_cast<int>(V);
  // CTAs per sequence: as many as the SMs have room for, each with some work
  p.cluster = 1;
  while (p.cluster < kMaxClusterVerify && B * p.cluster < 2 * kSmCount && V > 2048 * p.cluster) p.cluster *= 2;
  p.status = dev.status;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return cuda_check(launch_counted(ST_K_VERIFY, stream, [&] { return launch_tree_verify(p, stream); }), "tree verification launch");
}

st_status st_cache_keep(const st_kv_cache* cache, const st_tensor* start, const st_tensor* rows, const st_tensor* n_rows,
                        st_tensor* lens, void* stream_) {
  return st_cache_keep_held(cache, nullptr, start, rows, n_rows, lens, stream_);
}

st_status st_cache_keep_held(const st_kv_cache* cache, const st_kv_scales* scales, const st_tensor* start, const st_tensor* rows,
                             const st_tensor* n_rows, st_tensor* lens, void* stream_) {
  clear_error();
  KeepParams p;
  memset(&p, 0, sizeof(p));
  st_status st;
  if ((st = check_cache(cache, scales, -1, &p.kv, "st_cache_keep")) != ST_OK) return st;
  p.B = static_cast<int>(cache->pages->shape[0]);
  if (!rows || rows->ndim != 2 || rows->shape[1] < 0 || rows->shape[1] > (1ll << 30)) return fail(ST_ERR_SHAPE, "rows must be [%d, N]", p.B);
  if ((st = check_flat(start, "start", p.B, ST_I32)) != ST_OK) return st;
  if ((st = check_rows(rows, "rows", p.B, rows->shape[1], false, ST_I32, &p.r_sb)) != ST_OK) return st;
  if ((st = check_flat(n_rows, "n_rows", p.B, ST_I32)) != ST_OK) return st;
  if ((st = check_flat(lens, "lens", p.B, ST_I32)) != ST_OK) return st;
  p.N = static_cast<int>(rows->shape[1]);
  if (p.B == 0) return ST_OK;
  // CTAs read start, n_rows and rows while one writes lens
  const uintptr_t l0 = reinterpret_cast<uintptr_t>(lens->data), l1 = l0 + 4 * static_cast<uintptr_t>(p.B);
  auto overlaps = [&](const void* d, int64_t n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(d);
    return n > 0 && a < l1 && l0 < a + 4 * static_cast<uintptr_t>(n);
  };
  if (overlaps(start->data, p.B) || overlaps(n_rows->data, p.B) ||
      overlaps(rows->data, p.N > 0 ? (p.B - 1) * std::max<int64_t>(p.r_sb, 0) + p.N : 0))
    return fail(ST_ERR_INVALID_ARG, "lens may not overlap start, n_rows or rows");
  if (p.kv.Hkv < 1) return fail(ST_ERR_SHAPE, "the cache has no heads");
  Dev dev;
  if ((st = device_globals(&dev)) != ST_OK) return st;
  p.start = static_cast<const int32_t*>(start->data);
  p.rows = static_cast<const int32_t*>(rows->data);
  p.n_rows = static_cast<const int32_t*>(n_rows->data);
  p.lens = static_cast<int32_t*>(lens->data);
  // columns of 128 bytes; where there are fewer of them than SMs, long lists
  // take wide CTAs and short ones narrower columns
  const int64_t chains = static_cast<int64_t>(p.B) * 2 * p.kv.Hkv * (kD * elem_bytes(p.kv.dt) / 128);
  p.wide = chains < kSmCount && p.N > 2048;
  p.part_lanes = p.wide || chains >= kSmCount ? 8 : 4;
  p.status = dev.status;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return cuda_check(launch_counted(ST_K_CACHE_KEEP, stream, [&] { return launch_cache_keep(p, stream); }), "cache keep launch");
}

st_status st_cache_read(const st_kv_cache* cache, const st_kv_scales* scales, const st_tensor* start, const st_tensor* counts,
                        st_tensor* k, st_tensor* v, void* stream_) {
  clear_error();
  ReadParams p;
  memset(&p, 0, sizeof(p));
  st_status st;
  if ((st = check_cache(cache, scales, -1, &p.kv, "st_cache_read")) != ST_OK) return st;
  p.B = static_cast<int>(cache->pages->shape[0]);
  if (!k || !v) return fail(ST_ERR_INVALID_ARG, "%s is NULL", k ? "v" : "k");
  if (k->ndim != 4) return fail(ST_ERR_SHAPE, "k must be 4-D [B,T,H_kv,D], got ndim=%d", k->ndim);
  if (k->shape[1] < 0 || k->shape[1] > (1ll << 30)) return fail(ST_ERR_SHAPE, "k sizes out of range");
  p.T = static_cast<int>(k->shape[1]);
  RowTensor rk, rv;
  if ((st = check_bshd(k, "k", p.B, p.T, p.kv.Hkv, kD, held(p.kv) ? kRowTypes : bit(p.kv.dt), &rk)) != ST_OK) return st;
  if ((st = check_bshd(v, "v", p.B, p.T, p.kv.Hkv, kD, bit(k->dtype), &rv)) != ST_OK) return st;
  if ((st = check_own_rows(k, "k")) != ST_OK) return st;
  if ((st = check_own_rows(v, "v")) != ST_OK) return st;
  if ((st = check_flat(start, "start", p.B, ST_I32)) != ST_OK) return st;
  if ((st = check_counts(counts, p.B, &p.counts)) != ST_OK) return st;
  const int64_t tokens = static_cast<int64_t>(p.B) * p.T;
  if (tokens > (1ll << 30) || tokens * 2 * p.kv.Hkv > (1ll << 32)) return fail(ST_ERR_SHAPE, "too many rows");
  if (tokens * p.kv.Hkv == 0) return ST_OK;
  Dev dev;
  if ((st = device_globals(&dev)) != ST_OK) return st;
  p.start = static_cast<const int32_t*>(start->data);
  p.k = k->data;
  p.v = v->data;
  p.k_sb = rk.sb; p.k_ss = rk.ss; p.k_sh = rk.sh;
  p.v_sb = rv.sb; p.v_ss = rv.ss; p.v_sh = rv.sh;
  p.dt = k->dtype;
  const int per32 = 32 / static_cast<int>(elem_bytes(p.dt));
  auto wide = [&](const void* x, int64_t sb, int64_t ss, int64_t sh) {
    return (reinterpret_cast<uintptr_t>(x) & 31u) == 0 && sb % per32 == 0 && ss % per32 == 0 && sh % per32 == 0;
  };
  p.wide = wide(p.k, p.k_sb, p.k_ss, p.k_sh) && wide(p.v, p.v_sb, p.v_ss, p.v_sh);
  p.status = dev.status;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return cuda_check(launch_counted(ST_K_CACHE_KEEP, stream, [&] { return launch_cache_read(p, stream); }), "cache read launch");
}

}  // extern "C"
