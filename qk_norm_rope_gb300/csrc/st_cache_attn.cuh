// Cached attention on the tensor cores (caches of 16 and of 8 bits): tcgen05
// QK^T and PV with TMEM accumulators over pages gathered by TMA, online base-2
// softmax, split over the keys and joined. The kernel's template: each of its
// forms is instantiated in a file of its own.
//
// Work: an item is a (K/V head, sequence, group of NT 128-row query tiles); a
// tile's rows are tokens x the query heads of the K/V head, so that one read of
// K and V serves the whole group of heads. The items' key tiles (128 keys),
// laid end to end, are dealt out as one continuous range per CTA: the lengths
// live on the device, and this way any mix of lengths loads every SM alike. A
// CTA that holds all of an item's tiles writes O and LSE; else it leaves
// (O unnormalised, reference, sum) in the workspace, at most one such part at
// each end of its range, and the join kernel puts them together.
//
// Few items with short caches (CL, below): instead of the deal, a cluster of
// CTAs per item shares its key tiles out evenly and joins its parts through
// distributed shared memory, which saves the scan for the range's beginning
// and the second launch.
//
// EXT, windows: an item's key tiles are the first tokens' and, behind a gap, those
// from the first row's window on; each row masks by its own window. Boxes of keys
// that no row of the item sees are not fetched.
// EXT, a shared prefix: its whole tiles are items of their own (b = -1), whose
// rows are the tokens of all sequences, laid end to end; the sequences' items begin
// behind them. Every piece leaves its result in the workspace, the prefix's and
// the own keys' are joined row by row.
//
// KV, caches of 8 bits: fp16 holds e4m3's and int8's numbers exactly, so the held
// values are the operands, as fp16, and the scales enter in fp32: K's multiply the
// scores, V's the weights P before these are rounded. bf16 rows of q come to fp16
// by a power of two of their own (what is lost is 2^-39 of the row's largest
// element or less). Four warps each bring K's and V's bytes into shared memory and
// turn them into the 16-bit operand tiles; a thread fetches just the 16-byte pieces
// that it converts later, by asynchronous copies, so that nothing is handed over in
// between, and pages may be of any size. (With TMA boxes their issue set the pace:
// 64-key stages of 16-row boxes took the TMA warp 2900 cycles a tile.) Half the
// bytes are read for each key; all else has half the time of the 16-bit form.
//
// FEW (KV, at most 32 rows of one query tile: decoding): a thread per row left
// seven of eight warps idle and 128 scores of a tile to one after the other. The
// rows are put into all four lane groups of the tile (the MMA has room for 128) and
// each warp takes a quarter of the tile's keys, its weights of the others being
// zero; every group has sums and accumulators of its own, which are joined at the
// end like parts of the keys.
//
// Roles (512 threads, KV: 576; one CTA per SM):
//   warps 0-7   softmax, two groups of four warps; thread = query row = TMEM lane
//   warps 8-11  Q rows of the next item into shared memory; KV: K's conversion, and
//               four more warps V's and the Q rows
//   then        tcgen05.mma issue for slot 0 (one thread; TMEM allocation); TMA of K
//               boxes, one lane per box, and of V boxes (KV: neither); tcgen05.mma
//               issue for slot 1
// TMEM: S0 | S1 | O0 | O1, 128 fp32 columns each; P (16-bit) overwrites the
// first half of its S and feeds PV from TMEM. The stream of score tiles
// alternates between the two halves ("slots"): with NT = 2 a slot is a query
// tile, with NT = 1 (decoding: few rows, bound by the reading of K and V) the
// slots take alternate key tiles with accumulators of their own, which are
// merged at the end; either way one slot's softmax runs under the other's
// MMAs. A slot's scores run one tile ahead of its PV, across the borders of
// items.
#pragma once
#include <atomic>
#include <type_traits>
#include "st_kernels.h"
#include "st_serve.h"

namespace st {

namespace {

constexpr int kSoftWarps = 8, kWarpQ0 = 8, kQWarps = 4;
template <bool HELD>
struct Roles {
  static constexpr int kWarpMma = HELD ? 16 : 12, kWarpK = HELD ? 99 : 13, kWarpV = HELD ? 99 : 14;  // the last warp: the second slot's MMAs
  static constexpr int kWarps = HELD ? 18 : 16, kThreads = kWarps * 32;
};
// Registers per thread of the 16-bit form: its softmax threads hold a row of 128
// scores. 256 * 184 + 256 * 72 = 512 * 128. KV reads the scores from TMEM twice
// instead and has 96 everywhere (five warps on one of the SM's four register files).
constexpr int kRegsSoft = 184, kRegsRest = 72;
constexpr float kRescale = 8.0f;  // O is rescaled when the running maximum grows by more than this (base 2)
// How far the reference stays below the running maximum (base 2). fp16 weights
// end at 2^-25 of 1, and a long row's many small ones would leave PV but stay in
// the sum; with the maximum's at 2^7, at most 2^15 while the reference lags,
// they end 2^-32 below it. bf16 has fp32's range.
template <bool F16>
constexpr float kLift = F16 ? 7.0f : 0.0f;

constexpr int kPlaceBytes = 80;

template <int NT, bool HELD = false>
struct Lay {  // shared memory, offsets from a 1024-byte aligned base
  // With NT = 1 a stage belongs to one slot for good (even counts): a slot's
  // thread waits for every phase of the stages that it uses, and a wait on
  // parity says nothing where phases went by unseen.
  static constexpr int KS = NT == 1 || HELD ? 2 : 3, VS = NT == 1 && !HELD ? 4 : 2;
  // Stages of scales. Nothing says when one is free: those of tile n + 2 (NT = 2: n + 1)
  // are fetched while tile n is converted, whose place was free after the scores of
  // n - 2 (K; V: the products of n - 2), which were issued after the products of n - 4
  // (n - 3), whose weights were there. So 6 (4) do; NT = 1 takes a power of two.
  static constexpr int SS = HELD ? (NT == 1 ? 8 : 4) : 0;
  // stages of bytes, of K and of V each, and their keys: 48 KB where reading bounds
  static constexpr int RS = HELD ? 3 : 0, kRawRows = NT == 1 ? 64 : 32;
  static constexpr uint32_t kRawBytes = kRawRows * kD;
  static_assert(NT == 2 || (KS % 2 == 0 && VS % 2 == 0 && SS % 2 == 0), "stages of one slot");
  static constexpr uint32_t q = 0, k = NT * kTileBytes, v = k + KS * kTileBytes, raw = v + VS * kTileBytes, bar = raw + 2 * RS * kRawBytes;
  static constexpr uint32_t ml = bar + 512;          // [2][128] (reference, sum), NT = 1
  static constexpr uint32_t sc = ml + (NT == 1 ? 2 * 128 * 8 : 0);  // [SS] Scales
  static constexpr uint32_t walk = sc + SS * 1040;   // HELD: places of the roles' walks
  static constexpr uint32_t lens = walk + (HELD ? (2 * Roles<true>::kWarps - kSoftWarps) * kPlaceBytes : 0);
  static constexpr uint32_t qs = lens + (HELD ? 144 : 0);  // HELD: [2][NT][128] the rows' factors, by the parity of the piece
  static constexpr uint32_t bytes = qs + (HELD ? 2 * NT * 128 * 4 : 0);
  enum { QFull = 0, QEmpty, KFull, KEmpty = KFull + KS, VFull = KEmpty + KS, VEmpty = VFull + VS, SFull = VEmpty + VS,
         PFull = SFull + 2, OFull = PFull + 2, MlFull, ORead = MlFull + 2, Drain = ORead + 2, ScFull = Drain + 2, Num = ScFull + SS };
};
static_assert(Lay<1>::bytes <= 232448 && Lay<2>::bytes <= 232448, "shared memory");
static_assert(Lay<1, true>::bytes <= 232448 && Lay<2, true>::bytes <= 232448, "shared memory");
static_assert(Lay<1>::Num * 8 + 128 <= 512 && Lay<2>::Num * 8 + 128 <= 512, "barrier area");
static_assert(Lay<1, true>::Num * 8 + 128 <= 512 && Lay<2, true>::Num * 8 + 128 <= 512, "barrier area");

// The scales of a key tile; those of keys that no row sees are 0. ends: log2 of V's
// largest, and minus that of its least but 0, of the keys that each of four warps fetched.
struct Scales {
  float k[kTile], v[kTile];
  __half2 ends[4];
};
static_assert(sizeof(Scales) == 1040, "layout");
// V's scales are good in this range (base 2): between its ends a row's sum, in
// units of them, may shrink by 2^-100, and a share of it above 2^-26 stays in ex2's
// range.
constexpr float kTopRange = 50.f;
// Where V's scales in a tile differ by more than this (base 2), a row's reference goes
// by its own largest product of a weight and a scale. Else the largest scale stands for
// all: a row whose keys have lesser ones has its largest weight at 2^-1 or above.
constexpr float kTopSpread = 8.f;

__device__ __forceinline__ constexpr uint32_t kofs(int kk) { return (kk >> 2) * kHalfBytes + (kk & 3) * 32; }
__device__ __forceinline__ constexpr uint32_t mofs(int kk) { return kk * 2048; }

// Asynchronous 16-byte copy into shared memory; zeros when !there.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// The same of one fp32 number.
__device__ __forceinline__ void cp_async4(void* dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 4 : 0) : "memory");
}

struct Item {
  int prefix, keys, cnt, n;  // n: key tiles
  // EXT: tiles from `lead` on lie `gap` tiles further on; keys below `low`, first
  // tokens aside, are in no row's window
  int lead, gap, low;
};
// An item of a sequence of that length (of the cache) and number of rows.
template <bool EXT>
__device__ __forceinline__ Item item_from(const TcAttnParams& p, int nt, int m, int p0, int len, int cnt) {
  Item it;
  it.lead = it.gap = it.low = 0;
  it.cnt = cnt;
  it.keys = keys_of(p.c, len, cnt, &it.prefix);
  const int64_t t0 = static_cast<int64_t>(m) * nt * p.tpt;
  if (t0 >= it.cnt) {
    it.n = 0;
  } else {
    // a chain's last row of the group sees no further than itself
    const int64_t end = p.c.parents ? it.keys : min(static_cast<int64_t>(it.keys), it.prefix + t0 + nt * p.tpt);
    it.n = static_cast<int>((end + kTile - 1) / kTile);
    if constexpr (EXT) {
      if (p.c.window > 0) {
        it.low = window_low_of(p.c, len, p.c.parents ? 0 : t0);
        const Gap g = window_gap<kTile>(p.c, it.low, it.n);
        it.lead = g.lead;
        // (a length beyond the table leaves no key in the window: one tile, all masked,
        // gives the rows their zeros)
        it.gap = g.gap == it.n ? it.n - 1 : g.gap;
      } else {
        it.gap = min(p0, it.n);
      }
      it.n -= it.gap;
    }
  }
  return it;
}
// b < 0: the shared prefix, p0 tiles.
template <bool EXT>
__device__ __forceinline__ Item item_of(const TcAttnParams& p, int nt, int b, int m, int p0) {
  if (EXT && b < 0) {
    Item it;
    it.lead = it.gap = it.low = 0;
    it.cnt = p.c.B * p.c.T;
    it.prefix = it.keys = p0 * kTile;
    it.n = p0;
    return it;
  }
  const int cnt = row_count(p.c.counts, b, p.c.T);
  return item_from<EXT>(p, nt, m, p0, ld_now(p.c.lens + b), cnt);
}
// Lengths of sequences that a CTA comes to, in shared memory: from memory they are
// two round trips at each piece, for every role (64 tokens of short sequences: 10 us
// a piece with them, and with the rows' factors read from q by the softmax).
constexpr int kLens = 16;
struct Lens {
  int b0, len[kLens], cnt[kLens];
};
// The first key of the item's kt-th tile.
template <bool EXT>
__device__ __forceinline__ int tile_key(const Item& it, int kt) {
  return (EXT && kt >= it.lead ? kt + it.gap : kt) * kTile;
}

// What an item costs beyond its key tiles, in tiles: its rows' way in and its results'
// way out hold the pipeline up. The deal goes by the sum, so that no CTA gets the
// short items of many sequences while another has one long one. Measured from 0 to 10:
// 22 trees of 40 nodes, 41 keys of their own each after 7349 shared tokens in bf16
// 263 us with 0, 141 with 2 to 4, 148 with 7; 64 tokens after up to 8191 keys in e4m3
// 167, 160 with 4, 163 with 7; 64 tokens, 1000 keys of their own after 16384 shared ones
// in bf16 96, 86 with 2 and 3, 101 with 7, in e4m3 101, 107 with 2, 121 with 4 (a tile
// of the prefix has 128 rows and takes longer there than one of a single token's).
// The plain 16-bit forms, older, are dealt by tiles alone.
template <int NT, bool CL, int KV, bool EXT>
constexpr int kItemCost = CL || (KV == 0 && !EXT) ? 0 : (NT == 2 || !EXT ? 4 : (KV == 0 ? 3 : 2));

// A CTA's walk over its range: pieces of items. An item's range is its cost and then
// its tiles.
template <bool EXT>
struct Walk {
  int h, b, m, off;
  long long left;
  int p0;  // tiles of the shared prefix
  // the present piece
  int ph, pb, pm, kt0, kt1;
  Item it;
  __device__ __forceinline__ void advance(const TcAttnParams& p) {
    off = 0;
    if (++m == (EXT && b < 0 ? p.n_pre : p.n_groups)) {
      m = 0;
      if (++b == p.c.B) {
        b = EXT && p0 > 0 ? -1 : 0;
        ++h;
      }
    }
  }
  // a range that is one piece of the item (h, b, m, it)
  __device__ __forceinline__ void alone(int t0, int t1) {
    left = t1 - t0;
    ph = h;
    pb = b;
    pm = m;
    kt0 = t0;
    kt1 = t1;
  }
  template <bool ONE>
  __device__ __forceinline__ bool next(const TcAttnParams& p, int nt, int cost, const Lens* lens = nullptr) {
    if (left <= 0) return false;
    if constexpr (ONE) {
      left = 0;
      return true;
    }
    while (true) {
      int i = kLens;
      if (lens && b >= 0) {
        i = b - lens->b0;
        if (i < 0) i += p.c.B;
      }
      it = i < kLens ? item_from<EXT>(p, nt, m, p0, lens->len[i], lens->cnt[i]) : item_of<EXT>(p, nt, b, m, p0);
      if (it.n > 0 && off < it.n + cost) break;
      advance(p);
      if (h >= p.c.kv.Hkv) {  // lengths that changed under the kernel: no tiles are left
        left = 0;
        return false;
      }
    }
    ph = h;
    pb = b;
    pm = m;
    const int end = static_cast<int>(min(static_cast<long long>(it.n) + cost, off + left));
    kt0 = max(off - cost, 0);
    kt1 = end - cost;
    left -= end - off;
    off = end;
    if (off == it.n + cost) advance(p);
    return kt1 > kt0;  // else the range ends before the item's first tile
  }
  __device__ __forceinline__ bool whole() const { return kt0 == 0 && kt1 == it.n; }
  // HELD: what the walk goes on from lies in shared memory between pieces, and the
  // step is a function of its own (below).
  struct Place {
    int h, b, m, off;
    long long left;
    int p0, ph, pb, pm, kt0, kt1;
    Item it;
  };
  __device__ __forceinline__ void save(Place* at) const { *at = {h, b, m, off, left, p0, 0, 0, 0, 0, 0, {}}; }
  __device__ __forceinline__ void take(const Place* at) {
    ph = at->ph;
    pb = at->pb;
    pm = at->pm;
    kt0 = at->kt0;
    kt1 = at->kt1;
    it = at->it;
  }
};
// The next piece of the walk at `at`, by one thread. Inlined into every role, with
// the rest unrolled, it made a kernel of 197 KB, which the instruction cache did
// not hold: every role was held up by its own instructions (64 tokens after up to
// 8191 keys in e4m3 253 us).
template <bool EXT>
__device__ __noinline__ bool next_piece_of(const TcAttnParams& p, int nt, int cost, typename Walk<EXT>::Place* at, const Lens* lens) {
  Walk<EXT> w;
  w.h = at->h;
  w.b = at->b;
  w.m = at->m;
  w.off = at->off;
  w.left = at->left;
  w.p0 = at->p0;
  if (!w.template next<false>(p, nt, cost, lens)) return false;
  *at = {w.h, w.b, w.m, w.off, w.left, w.p0, w.ph, w.pb, w.pm, w.kt0, w.kt1, w.it};
  return true;
}

// The deal: CTA x has [first(x), first(x + 1)) of the call's tiles (and items' costs),
// shares that differ by one at most. 32-bit division where the numbers allow it.
struct Deal {
  long long total, share;
  int ctas, extra;
  __device__ __forceinline__ void make(long long tiles, int most) {
    total = tiles;
    ctas = static_cast<int>(min(static_cast<long long>(most), tiles));
    share = ctas == 0 ? 0 : div(tiles, ctas);
    extra = static_cast<int>(tiles - share * ctas);
  }
  static __device__ __forceinline__ long long div(long long a, long long b) {
    if (((a | b) >> 31) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
  }
  __device__ __forceinline__ long long first(int x) const { return x * share + min(x, extra); }
  // the CTA that has tile t
  __device__ __forceinline__ int holder(long long t) const {
    const long long big = (share + 1) * extra;
    return static_cast<int>(t < big ? div(t, share + 1) : extra + div(t - big, share));
  }
};

struct Start {  // found by the block, read by every role
  int h, b, m, off;
  long long left;
  int p0, pre_b;           // EXT: tiles of the shared prefix, the sequence whose pages hold it
  long long first, total;  // joined by items: where the range begins, the call's sum
};

// The shared prefix: whole tiles of what the least of the sequences that have
// rows reaches, and the first of these sequences.
template <int W>  // warps
__device__ __forceinline__ void find_shared(const TcAttnParams& p, int* scratch, Start* st) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int least = 0x7fffffff, first = 0x7fffffff;
  for (int b = tid; b < p.c.B; b += W * 32)
    if (row_count(p.c.counts, b, p.c.T) > 0) {
      least = min(least, max(ld_now(p.c.lens + b), 0));
      first = min(first, b);
    }
  least = __reduce_min_sync(0xffffffffu, least);
  first = __reduce_min_sync(0xffffffffu, first);
  if (lane == 0) {
    scratch[warp] = least;
    scratch[W + warp] = first;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < W; ++w) {
      least = min(least, scratch[w]);
      first = min(first, scratch[W + w]);
    }
    const int cap = p.c.kv.max_pages * p.c.kv.page;  // at most 2^30
    st->p0 = first == 0x7fffffff ? 0 : min(min(max(ld_now(p.c.shared), 0), least), cap) / kTile;
    st->pre_b = first;
    if (blockIdx.x == 0) *p.p0 = st->p0;
  }
  __syncthreads();
}

// Where the CTA's range begins: every thread sums the key tiles of a run of
// (sequence, group) pairs (the shared prefix's groups first), a block scan places
// the runs.
template <bool EXT, int W, bool ITEMS>  // ITEMS: the call may join by items
__device__ __forceinline__ void find_start(const TcAttnParams& p, int nt, int cost, long long* scan, Start* st) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int p0 = 0;
  if constexpr (EXT) {
    if (p.c.shared) {
      find_shared<W>(p, reinterpret_cast<int*>(scan), st);
      p0 = st->p0;
    }
  }
  const int pre = p0 > 0 ? p.n_pre : 0, pairs = pre + p.c.B * p.n_groups;  // at most 2^30
  const int per = (pairs + W * 32 - 1) / (W * 32), lo = min(pairs, tid * per), hi = min(pairs, lo + per);
  int b0, m0;
  if (EXT && lo < pre) {
    b0 = -1;
    m0 = lo;
  } else {
    b0 = p.n_groups == 1 ? lo - pre : (lo - pre) / p.n_groups;
    m0 = lo - pre - b0 * p.n_groups;
  }
  long long sum = 0;
  for (int e = lo, b = b0, m = m0; e < hi; ++e) {
    const Item it = item_of<EXT>(p, nt, b, m, p0);
    sum += it.n > 0 ? it.n + cost : 0;
    if (m == 0 && b >= 0 && blockIdx.x == 0 && (ld_now(p.c.lens + b) < 0 || static_cast<int64_t>(ld_now(p.c.lens + b)) + it.cnt > it.keys))
      atomicOr(p.c.status, kStatusIndex);
    if (++m == (EXT && b < 0 ? pre : p.n_groups)) {
      m = 0;
      ++b;
    }
  }
  long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) scan[warp] = inc;
  if (tid == 0) {
    st->left = 0;
    // a CTA behind the last range has nothing of an earlier kernel's here (the plain
    // 16-bit forms look at no more than `left` there)
    if constexpr (ITEMS) st->h = st->b = st->m = st->off = 0;
  }
  __syncthreads();
  long long before = 0, one = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += scan[w];
    one += scan[w];
  }
  Deal d;
  d.make(one * p.c.kv.Hkv, p.ctas);
  if constexpr (ITEMS) {
    if (tid == 0) {
      st->first = blockIdx.x < d.ctas ? d.first(blockIdx.x) : 0;
      st->total = d.total;
    }
  }
  if (blockIdx.x < d.ctas) {
    const long long s0 = d.first(blockIdx.x);
    const int h = static_cast<int>(Deal::div(s0, one));
    long long rem = s0 - h * one - (before + inc - sum);
    if (rem >= 0 && rem < sum) {  // one thread
      for (int e = lo, b = b0, m = m0; e < hi; ++e) {
        const Item it = item_of<EXT>(p, nt, b, m, p0);
        const int all = it.n > 0 ? it.n + cost : 0;
        if (rem < all) {
          st->h = h;
          st->b = b;
          st->m = m;
          st->off = static_cast<int>(rem);
          st->left = d.first(blockIdx.x + 1) - s0;
          if (ITEMS && p.item_meta) break;
          // for the join: is this border the first inside of its item, and
          // who has the item's tiles?
          JoinMeta meta{0, 0, h, b, m, it.cnt};
          const long long item = s0 - rem;
          if (rem > cost && d.first(blockIdx.x - 1) <= item + cost) {
            meta.parts = d.holder(item + all - 1) - static_cast<int>(blockIdx.x) + 2;
            meta.slot0 = 2 * (static_cast<int>(blockIdx.x) - 1) + (d.first(blockIdx.x - 1) >= item ? 0 : 1);
          }
          p.meta[blockIdx.x] = meta;
          break;
        }
        rem -= all;
        if (++m == (EXT && b < 0 ? pre : p.n_groups)) {
          m = 0;
          ++b;
        }
      }
    }
  } else if (tid == 0 && !(ITEMS && p.item_meta)) {
    p.meta[blockIdx.x].parts = 0;
  }
  __syncthreads();
}

template <bool F16, int K0, int K1>  // of the eight K-steps of 16 head dims
__device__ __forceinline__ void issue_s(uint32_t tS, uint64_t dQ, uint64_t dK) {
  constexpr uint32_t idesc = idesc16(F16, 128, 128, 0, 0);
#pragma unroll
  for (int kk = K0; kk < K1; ++kk) mma_ss(tS, sdesc_add(dQ, kofs(kk)), sdesc_add(dK, kofs(kk)), idesc, kk > 0);
}
template <bool F16>
__device__ __forceinline__ void issue_pv(uint32_t tO, uint32_t tP, uint64_t dV, bool acc) {
  constexpr uint32_t idesc = idesc16(F16, 128, 128, 0, 1);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) mma_ts(tO, tP + kk * 8, sdesc_add(dV, mofs(kk)), idesc, acc || kk > 0);
}

// Bits of the keys [j0, j0 + 32) that row (token t, ancestors anc) sees.
template <bool TREE>
__device__ __forceinline__ uint32_t key_bits(int j0, const Item& it, int t, const uint32_t (&anc)[kTreeWords]) {
  const int n0 = j0 - it.prefix;  // node of bit 0
  uint32_t w;
  if constexpr (TREE) {
    if (n0 <= -32) w = ~0u;
    else if (n0 < 0) w = (~0u >> (32 + n0)) | (anc[0] << (-n0));
    else {
      uint32_t a = 0, c = 0;
#pragma unroll
      for (int i = 0; i < kTreeWords; ++i) {
        if (i == (n0 >> 5)) a = anc[i];
        if (i == (n0 >> 5) + 1) c = anc[i];
      }
      w = __funnelshift_r(a, c, n0 & 31);
    }
  } else {
    const int k = t + 1 - n0;  // that many of the 32 are seen
    w = k >= 32 ? ~0u : (k <= 0 ? 0u : (1u << k) - 1u);
  }
  const int in = it.keys - j0;
  return in >= 32 ? w : (in <= 0 ? 0u : w & ((1u << in) - 1u));
}

// Bits of the keys [j0, j0 + 32) that lie in the window from `low` on or among
// the first tokens; TREE: or from `prefix` on (a tree's nodes were chosen by their
// depth).
template <bool TREE>
__device__ __forceinline__ uint32_t window_bits(int j0, int low, int sinks, int prefix) {
  auto from = [](int d) { return d <= 0 ? ~0u : (d >= 32 ? 0u : ~0u << d); };  // bits d ..
  uint32_t w = from(low - j0) | ~from(min(sinks, 1 << 30) - j0);
  if constexpr (TREE) w |= from(prefix - j0);
  return w;
}

// Softmax of one 128 x 128 score tile, a thread's row: running reference and
// sum, P into the first 64 columns; O is rescaled where the reference moved.
template <bool F16, bool MASK>
__device__ __forceinline__ void softmax_tile(uint32_t tS, uint32_t tO, float sc, const uint32_t (&mb)[4], bool first,
                                             float& m_run, float& l_run) {
  uint32_t x[4][32];  // the whole row: TMEM is read once
#pragma unroll
  for (int i = 0; i < 4; ++i) tmem_ld32_issue(tS + 32 * i, x[i]);
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    tmem_ld_wait32(x[i]);
    if constexpr (MASK) {
#pragma unroll
      for (int t = 0; t < 32; ++t)
        if (!((mb[i] >> t) & 1u)) x[i][t] = 0xff800000u;
    }
#pragma unroll
    for (int t = 0; t < 32; t += 4) {
      m0 = fmax3(m0, __uint_as_float(x[i][t]), __uint_as_float(x[i][t + 1]));
      m1 = fmax3(m1, __uint_as_float(x[i][t + 2]), __uint_as_float(x[i][t + 3]));
    }
  }
  const float mt = fmaf(fmaxf(m0, m1), sc, -kLift<F16>);
  float corr = 1.f;
  if (mt > m_run + kRescale || (m_run == -INFINITY && mt > -INFINITY)) {
    corr = ex2(m_run - mt);  // 0 when m_run is -inf
    m_run = mt;
  }
  const float m_use = m_run == -INFINITY ? 0.f : m_run;
  const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-m_use, -m_use);
  float2 ls = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t pw[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const float2 y = __ffma2_rn(make_float2(__uint_as_float(x[i][2 * t]), __uint_as_float(x[i][2 * t + 1])), sc2, nm2);
      const float p0 = ex2(y.x), p1 = ex2(y.y);
      ls = __fadd2_rn(ls, make_float2(p0, p1));
      pw[t] = pack16<F16>(p0, p1);
    }
    tmem_st16(tS + 16 * i, pw);
  }
  l_run = l_run * corr + (ls.x + ls.y);
  if (!first && __any_sync(0xffffffffu, corr != 1.f)) {  // warp-uniform: tcgen05.ld/st are collective
#pragma unroll 1
    for (int q4 = 0; q4 < 4; ++q4) {
      uint32_t r32[32];
      tmem_ld32(tO + 32 * q4, r32);
#pragma unroll
      for (int t = 0; t < 32; ++t) r32[t] = __float_as_uint(__uint_as_float(r32[t]) * corr);
      tmem_st32(tO + 32 * q4, r32);
    }
  }
  tmem_st_wait();
}

// The same over a cache of 8 bits, in chunks of 32 keys (FEW: a warp has one, and its
// weights of the others are zero). Scores are s ks sc: ks the key's scale, sc the row's
// factor. The weights are rounded as P vs, vs V's scale, and so that they end at 2^15
// the reference has log2 of the tile's largest vs added to it; sums and accumulators
// alike are in its units. (Only where the tile's vs are of about one size. Else the
// largest may be that of a key which the row does not see, or hardly, and its weights
// would end below fp16's range: with 2^32 between them the row read as zeros. There the
// reference is the largest sum of a score and its key's log2 vs, found in a pass of its
// own: where every tile takes it, 64 tokens after up to 8191 keys in e4m3 201 us instead
// of 154, 2048 after 16384 1090 instead of 670.) There are no registers for a row of
// 128 scores: they go back to TMEM, scaled and masked, while the maximum is found, and
// come again for the weights, which take the place of scores that have been read.
// (Scaled and masked a second time instead 2048 tokens after 16384 took 926 us over
// e4m3, so 755: the reads of the scales from shared memory stand in line with the MMAs'
// operands.)
template <int N>
__device__ __forceinline__ void scale_chunk(uint32_t (&x)[N], const float* ks) {
#pragma unroll
  for (int t = 0; t < N; t += 4) {
    const float4 k4 = *reinterpret_cast<const float4*>(ks + t);
    const float2 a = __fmul2_rn(make_float2(__uint_as_float(x[t]), __uint_as_float(x[t + 1])), make_float2(k4.x, k4.y));
    const float2 b = __fmul2_rn(make_float2(__uint_as_float(x[t + 2]), __uint_as_float(x[t + 3])), make_float2(k4.z, k4.w));
    x[t] = __float_as_uint(a.x);
    x[t + 1] = __float_as_uint(a.y);
    x[t + 2] = __float_as_uint(b.x);
    x[t + 3] = __float_as_uint(b.y);
  }
}
__device__ __forceinline__ void mask_chunk(uint32_t (&x)[32], uint32_t mb) {
#pragma unroll
  for (int t = 0; t < 32; ++t)
    if (!((mb >> t) & 1u)) x[t] = 0xff800000u;
}
template <int N>
__device__ __forceinline__ float max_chunk(const uint32_t (&x)[N]) {
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
  for (int t = 0; t < N; t += 4) {
    m0 = fmax3(m0, __uint_as_float(x[t]), __uint_as_float(x[t + 1]));
    m1 = fmax3(m1, __uint_as_float(x[t + 2]), __uint_as_float(x[t + 3]));
  }
  return fmaxf(m0, m1);
}
// The weights of N keys into their N / 2 columns of P; their sum before V's scales.
template <int N>
__device__ __forceinline__ float2 weigh_chunk(uint32_t tP, const uint32_t (&x)[N], const float* vs, float sc, float m_use, float2 ls) {
  const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-m_use, -m_use);
  uint32_t pw[N / 2];
#pragma unroll
  for (int t = 0; t < N / 2; t += 2) {
    const float4 v4 = *reinterpret_cast<const float4*>(vs + 2 * t);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 y = __ffma2_rn(make_float2(__uint_as_float(x[2 * (t + e)]), __uint_as_float(x[2 * (t + e) + 1])), sc2, nm2);
      const float2 p = make_float2(ex2(y.x), ex2(y.y));
      ls = __fadd2_rn(ls, p);
      const float2 w = __fmul2_rn(p, e == 0 ? make_float2(v4.x, v4.y) : make_float2(v4.z, v4.w));
      pw[t + e] = pack16<true>(w.x, w.y);
    }
  }
  if constexpr (N == 32) tmem_st16(tP, pw);
  else tmem_st8(tP, pw);
  return ls;
}
// The largest sum of a scaled score and log2 of its key's vs over n chunks of scores in
// TMEM (vs within the range in which these are good; one of 0 counts as its lower end).
// A function of its own: inlined, the kernel's size cost 13% where no tile comes here
// (256 tokens of short sequences in e4m3 158 us, 177; so 163).
__device__ __noinline__ float max_product(uint32_t tS, const float* vs, int n, float sc) {
  float m = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < 2 * n; ++i) {
    uint32_t x[16];
    tmem_ld16_issue(tS + 16 * i, x);
    tmem_ld_wait16(x);
#pragma unroll
    for (int t = 0; t < 16; t += 4) {
      const float4 v4 = *reinterpret_cast<const float4*>(vs + 16 * i + t);
      const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        m = fmaxf(m, fmaf(__uint_as_float(x[t + e]), sc, fminf(fmaxf(__log2f(fabsf(v[e])), -kTopRange), kTopRange)));
    }
  }
  return m;
}
// The eight runs of 16 columns from tS on, each on its way from TMEM while f works on
// the one before it.
template <class F>
__device__ __forceinline__ void for_halves(uint32_t tS, F&& f) {
  uint32_t a[16], b[16];
  tmem_ld16_issue(tS, a);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    tmem_ld_wait16(a);
    tmem_ld16_issue(tS + 16 * i + 16, b);
    f(a, i);
    tmem_ld_wait16(b);
    if (i < 6) tmem_ld16_issue(tS + 16 * i + 32, a);
    f(b, i + 1);
  }
}
// bits(i): the keys of chunk i that the row sees, where a mask is needed. With two
// query tiles a softmax thread's own time is what bounds (2048 tokens after 16384
// 755 us rolled, 689 by halves), with one the kernel's size and its registers (64
// tokens after up to 8191 keys 181 and 186 us, by halves in both passes several times
// that).
template <int NT, class Bits>
__device__ __forceinline__ void softmax_held(uint32_t tS, uint32_t tO, float sc, const Scales& scales, bool mask, Bits&& bits, bool few, int quarter,
                                             bool first, float& m_run, float& l_run) {
  uint32_t x[32];
  const int c0 = few ? quarter : 0, c1 = few ? quarter + 1 : 4;
  float top = -INFINITY;
  if (NT == 2 && !mask) {
    for_halves(tS, [&](uint32_t (&y)[16], int i) {
      scale_chunk(y, scales.k + 16 * i);
      top = fmaxf(top, max_chunk(y));
      tmem_st16(tS + 16 * i, y);
    });
  } else {
#pragma unroll 1
    for (int i = c0; i < c1; ++i) {  // rolled, here and below, for the instruction cache
      tmem_ld32(tS + 32 * i, x);
      scale_chunk(x, scales.k + 32 * i);
      if (mask) mask_chunk(x, bits(i));
      top = fmaxf(top, max_chunk(x));
      if (!few) tmem_st32(tS + 32 * i, x);
    }
  }
  if (!few) tmem_st_wait();
  const uint4 ew = *reinterpret_cast<const uint4*>(scales.ends);
  const __half2 e01 = __hmax2(*reinterpret_cast<const __half2*>(&ew.x), *reinterpret_cast<const __half2*>(&ew.y));
  const __half2 ends = __hmax2(e01, __hmax2(*reinterpret_cast<const __half2*>(&ew.z), *reinterpret_cast<const __half2*>(&ew.w)));
  const float v_top = __low2float(ends);
  float mt = fmaf(top, sc, v_top - kLift<true>);
  if (v_top + __high2float(ends) > kTopSpread) {  // the same for all threads
    if (few) {
      tmem_st32(tS + 32 * c0, x);
      tmem_st_wait();
    }
    mt = max_product(tS + 32 * c0, scales.v + 32 * c0, c1 - c0, sc) - kLift<true>;
    if (few) tmem_ld32(tS + 32 * c0, x);
  }
  float corr = 1.f;
  if (mt > m_run + kRescale || (m_run == -INFINITY && mt > -INFINITY)) {
    corr = ex2(m_run - mt);  // 0 when m_run is -inf
    m_run = mt;
  }
  const float m_use = m_run == -INFINITY ? 0.f : m_run;
  float2 ls = make_float2(0.f, 0.f);
  if constexpr (NT == 2) {
    for_halves(tS, [&](const uint32_t (&y)[16], int i) { ls = weigh_chunk(tS + 8 * i, y, scales.v + 16 * i, sc, m_use, ls); });
  } else {
#pragma unroll 1
    for (int i = c0; i < c1; ++i) {
      if (!few) tmem_ld32(tS + 32 * i, x);  // else they are still here
      ls = weigh_chunk(tS + 16 * i, x, scales.v + 32 * i, sc, m_use, ls);
    }
    if (few) {
      const uint32_t none[16] = {};
#pragma unroll 1
      for (int i = 1; i < 4; ++i) tmem_st16(tS + 16 * ((quarter + i) & 3), none);
    }
  }
  l_run = l_run * corr + (ls.x + ls.y);
  if (!first && __any_sync(0xffffffffu, corr != 1.f)) {  // warp-uniform: tcgen05.ld/st are collective
#pragma unroll 1
    for (int q4 = 0; q4 < 4; ++q4) {
      tmem_ld32(tO + 32 * q4, x);
#pragma unroll
      for (int t = 0; t < 32; ++t) x[t] = __float_as_uint(__uint_as_float(x[t]) * corr);
      tmem_st32(tO + 32 * q4, x);
    }
  }
  tmem_st_wait();
}

// The exponent e for which a bf16 row whose largest magnitude has the bits `top`
// goes into fp16 as x 2^e: the largest becomes 2^14 to 2^15, elements down to
// 2^-39 of it keep half a step of 2^-25 (zeros, infinity and NaN: 0).
__device__ __forceinline__ int row_shift(uint32_t top) {
  const int e = static_cast<int>(top >> 7);  // of a bf16 number
  return e == 0 || e == 255 ? 0 : min(14 + 127 - e, 126);
}
// Largest magnitude of eight bf16 elements, as bits.
__device__ __forceinline__ uint32_t top_bits(const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) top = max(top, max((w[e] >> 16) & 0x7fffu, w[e] & 0x7fffu));
  return top;
}
__device__ __forceinline__ uint4 to_f16(const uint4& x, float f) {
  return make_uint4(pack_f16(bf16_lo(x.x) * f, bf16_hi(x.x) * f), pack_f16(bf16_lo(x.y) * f, bf16_hi(x.y) * f),
                    pack_f16(bf16_lo(x.z) * f, bf16_hi(x.z) * f), pack_f16(bf16_lo(x.w) * f, bf16_hi(x.w) * f));
}

// Two held bytes each (of the halves of w) as fp16 pairs.
template <int KV>
__device__ __forceinline__ void held_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (KV == kDtE4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n}" : "=r"(lo), "=r"(hi) : "r"(w));
  } else {
    // the byte plus 128 in the low bits of 1024: 1152 too much
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), off), y = __hsub2(*reinterpret_cast<__half2*>(&b), off);
    lo = *reinterpret_cast<uint32_t*>(&x);
    hi = *reinterpret_cast<uint32_t*>(&y);
  }
}

// Columns [32 q4, 32 q4 + 32) of a row: fp32 into a part, or 16 bits into the
// result (`wide`: its rows start on 32 bytes).
__device__ __forceinline__ void store_part32(float* row, int q4, const float (&y)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(y[8 * i + e]);
    st_v8(row + 32 * q4 + 8 * i, w);
  }
}
template <bool F16>
__device__ __forceinline__ void store_out32(void* o, int64_t off, bool wide, int q4, const float (&y)[32]) {
  uint16_t* row = static_cast<uint16_t*>(o) + off + 32 * q4;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = pack16<F16>(y[16 * i + 2 * e], y[16 * i + 2 * e + 1]);
    if (wide) {
      st_v8(row + 16 * i, w);
    } else {
      reinterpret_cast<uint4*>(row + 16 * i)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(row + 16 * i)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

// Reads of a peer CTA's shared memory (cluster addresses from mapa).
__device__ __forceinline__ float4 ld_peer_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_peer_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// The page and row of a TMA lane's box of key tile kt: lane = (64-column half,
// box of keys).
struct Box {
  bool mine;  // the lane has a box, and keys lie in it
  int pg, row;
};
template <bool EXT>
__device__ __forceinline__ Box find_box(const TcAttnParams& P, const Walk<EXT>& wk, int kt, int lane, int pre_b) {
  const int nb = kTile >> P.box_shift, j = tile_key<EXT>(wk.it, kt) + ((lane & (nb - 1)) << P.box_shift);
  Box b;
  b.mine = lane < 2 * nb && j < wk.it.keys;
  if constexpr (EXT) b.mine = b.mine && (j + (1 << P.box_shift) > wk.it.low || j < P.c.sinks);
  b.pg = b.row = 0;
  if (b.mine && !kv_locate(P.c.kv, EXT && wk.pb < 0 ? pre_b : wk.pb, j, &b.pg, &b.row)) atomicOr(P.c.status, kStatusIndex);  // reads as zeros
  return b;
}

// Of a row of an item: the sequence and its token (the prefix's rows go through
// all sequences).
struct RowAt {
  int b, t;
};
template <bool EXT>
__device__ __forceinline__ RowAt row_at(const TcAttnParams& P, int b, int t) {
  if (EXT && b < 0) {
    const int s = static_cast<int>(static_cast<unsigned>(t) / static_cast<unsigned>(P.c.T));
    return {s, t - s * P.c.T};
  }
  return {b, t};
}

// Q rows of the present piece into shared memory, by N threads.
template <int NT, bool EXT, int N>
__device__ __forceinline__ void load_q(const TcAttnParams& P, const Walk<EXT>& wk, uint8_t* sm, int qt) {
  const CacheAttnParams& c = P.c;
  const int G = c.group;
#pragma unroll 1
  for (int ti = 0; ti < NT; ++ti) {
    const int t0 = (wk.pm * NT + ti) * P.tpt;
    const int nv = max(0, min(P.tpt, wk.it.cnt - t0)) * G;     // rows that are there
    const int fill = ((nv + 31) & ~31) * 16;                   // whole warps of rows: zeros behind them
    uint8_t* tile = sm + ti * kTileBytes;
    for (int e = qt; e < fill; e += N) {
      const int row = e >> 4, ch = e & 15, rr = row < nv ? row : 0;
      const RowAt at = row_at<EXT>(P, wk.pb, t0 + rr / G);
      const int h = wk.ph * G + rr % G;
      cp_async16(tile + (ch >> 3) * kHalfBytes + sw128_off(row, ch & 7),
                 static_cast<const uint16_t*>(c.q.p) + at.b * c.q.sb + at.t * c.q.ss + h * c.q.sh + 8 * ch, row < nv);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  fence_proxy_async_smem();
}
// The same over caches of 8 bits, as fp16 and by way of registers (16 lanes have a
// row, and other copies of theirs stay in flight). few: every 32 rows of the tile
// are the same ones. The first 32 rows are read before the wait for the tile; qs:
// the rows' factors.
template <int NT, bool F16, bool EXT, int N, class Wait>
__device__ __forceinline__ bool load_q_held(const TcAttnParams& P, const Walk<EXT>& wk, uint8_t* sm, float* qs, int qt, bool few, Wait&& wait) {
  const CacheAttnParams& c = P.c;
  const int G = c.group;
  static_assert(N * 4 == 512, "32 rows a turn");
  const uint32_t inv = (65536u + G - 1) / G;  // row / G = row inv / 2^16 for rows below 256
  bool first = true;
#pragma unroll 1
  for (int r0 = 0; r0 < NT * kTile; r0 += 32) {
    const int ti = r0 / kTile, in0 = r0 - ti * kTile, t0 = (wk.pm * NT + ti) * P.tpt;
    const int nv = max(0, min(P.tpt, wk.it.cnt - t0)) * G;
    if (in0 >= nv && !first) continue;
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int row = in0 + ((qt + u * N) >> 4);
      const uint32_t tok = (row * inv) >> 16;
      x[u] = make_uint4(0, 0, 0, 0);
      if (row < nv) {
        const RowAt at = row_at<EXT>(P, wk.pb, t0 + tok);
        x[u] = ld_v4(static_cast<const uint16_t*>(c.q.p) + at.b * c.q.sb + at.t * c.q.ss + (wk.ph * G + row - tok * G) * c.q.sh + 8 * (qt & 15));
      }
    }
    if (first && !wait()) return false;
    first = false;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int row = in0 + ((qt + u * N) >> 4), ch = qt & 15;
      uint4 y = x[u];
      if constexpr (!F16) {
        uint32_t top = top_bits(y);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int shift = row_shift(top);
        y = to_f16(y, __int_as_float((shift + 127) << 23));
        if (ch == 0) qs[ti * 128 + row] = c.scale_log2 * __int_as_float((127 - shift) << 23);
      }
      uint8_t* at = sm + ti * kTileBytes + (ch >> 3) * kHalfBytes + sw128_off(row, ch & 7);
      *reinterpret_cast<uint4*>(at) = y;
      if (few) {
#pragma unroll
        for (int i = 1; i < 4; ++i) *reinterpret_cast<uint4*>(at + i * 32 * 128) = y;
      }
    }
  }
  fence_proxy_async_smem();
  return true;
}

// A part in shared memory: NT x 128 rows of 128 floats over the K stages (and
// on over the V stages), the 16-byte chunks of a row permuted so that neither a
// thread per row (writing) nor a warp per row (reading) meets bank conflicts;
// behind them (reference, sum) of the rows.
__device__ __forceinline__ uint32_t stage_off(int row, int chunk) { return row * 512u + ((chunk ^ (row & 31)) << 4); }
__device__ __forceinline__ void stage_chunk32(uint8_t* base, int row, int q4, const float (&y)[32]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    *reinterpret_cast<float4*>(base + stage_off(row, 8 * q4 + e)) = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
}

// The place of an item in the list of the call's items, and, where one CTA has
// all of its tiles, of its result's first row (calls that join by items).
__device__ __forceinline__ int64_t item_index(const TcAttnParams& p, int h, int b, int m) {
  if (b < 0) return static_cast<int64_t>(h) * p.n_pre + m;
  return static_cast<int64_t>(p.c.kv.Hkv) * p.n_pre + (static_cast<int64_t>(h) * p.c.B + b) * p.n_groups + m;
}
__device__ __forceinline__ int64_t whole_part(const TcAttnParams& p, int h, int b, int m) {
  const int64_t first = 2 * static_cast<int64_t>(p.ctas) * p.split_rows, pre = static_cast<int64_t>(p.c.kv.Hkv) * p.n_pre, i = item_index(p, h, b, m);
  return b < 0 ? first + i * p.pre_rows : first + pre * p.pre_rows + (i - pre) * p.part_rows * (p.few ? 4 : 1);
}

// F16: the type of q and o (and of a 16-bit cache). KV: 0, kDtE4M3 or kDtI8.
template <int NT, bool F16, bool TREE, bool CL, int KV, bool EXT>
__global__ void __launch_bounds__(Roles<KV != 0>::kThreads, 1) tc_kernel(const __grid_constant__ TcAttnParams P) {
  constexpr bool HELD = KV != 0, OP16 = F16 || HELD;  // fp16 operands
  using L = Lay<NT, HELD>;
  constexpr int kCost = kItemCost<NT, CL, KV, EXT>;
  constexpr int kWarpMma = Roles<HELD>::kWarpMma, kWarpK = Roles<HELD>::kWarpK, kWarpV = Roles<HELD>::kWarpV, kTcWarps = Roles<HELD>::kWarps;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  const CacheAttnParams& c = P.c;
  if (smem_u32(sm) & 1023u) {
    if (threadIdx.x == 0) atomicOr(c.status, kStatusLayout);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bar);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + L::Num);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  int* pipe_lock = reinterpret_cast<int*>(tslot + 2);  // held by the slot that is issuing MMAs
  Start* start = reinterpret_cast<Start*>(tslot + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane_id = tid & 31;
  const long long budget = c.wait_budget;

  if (warp == kWarpMma) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(&bars[L::QFull], kQWarps * 32);
    mbar_init(&bars[L::QEmpty], 2);
    if constexpr (HELD)
      for (int s = 0; s < L::SS; ++s) mbar_init(&bars[L::ScFull + s], 2 * kQWarps);
    for (int s = 0; s < L::KS; ++s) {
      mbar_init(&bars[L::KFull + s], HELD ? kQWarps * 32 : 1);
      mbar_init(&bars[L::KEmpty + s], NT);  // NT = 1: a tile is one slot's
    }
    for (int s = 0; s < L::VS; ++s) {
      mbar_init(&bars[L::VFull + s], HELD ? kQWarps * 32 : 1);
      mbar_init(&bars[L::VEmpty + s], NT);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars[L::SFull + s], 1);
      mbar_init(&bars[L::PFull + s], 128);
      mbar_init(&bars[L::MlFull + s], 128);
      mbar_init(&bars[L::ORead + s], 128);
      mbar_init(&bars[L::Drain + s], 1);
    }
    mbar_init(&bars[L::OFull], 2);
    *abort_flag = 0;
    *pipe_lock = 0;
    fence_mbar_init();
  }
  if (!HELD && tid == kWarpK * 32) tma_prefetch_desc(&P.tmap_k);
  if (!HELD && tid == kWarpV * 32) tma_prefetch_desc(&P.tmap_v);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  grid_dependency_wait();  // what came before touches no global memory
  Walk<EXT> wk;  // with CL every role finds its way alone from here on
  wk.p0 = 0;
  int pre_b = 0;
  if constexpr (CL) {
    // grid (cluster x K/V heads, sequences x groups)
    const int rank = static_cast<int>(cluster_rank());
    wk.h = blockIdx.x >> P.cluster_shift;
    wk.b = blockIdx.y;
    wk.m = 0;
    if (P.n_groups > 1) {
      wk.b = blockIdx.y / P.n_groups;
      wk.m = blockIdx.y - wk.b * P.n_groups;
    }
    wk.it = item_of<EXT>(P, NT, wk.b, wk.m, 0);
    wk.alone((wk.it.n * rank) >> P.cluster_shift, (wk.it.n * (rank + 1)) >> P.cluster_shift);
    if (tid == 0 && rank == 0 && wk.h == 0 && wk.m == 0 &&
        (ld_now(c.lens + wk.b) < 0 || static_cast<int64_t>(ld_now(c.lens + wk.b)) + wk.it.cnt > wk.it.keys))
      atomicOr(c.status, kStatusIndex);
  } else {
    // the scan's scratch lies in the Q tile, which is written later
    find_start<EXT, kTcWarps, EXT || HELD>(P, NT, kCost, reinterpret_cast<long long*>(sm + L::q), start);
    wk.h = start->h;
    wk.b = start->b;
    wk.m = start->m;
    wk.off = start->off;
    wk.left = start->left;
    if (EXT && c.shared) {
      wk.p0 = start->p0;
      pre_b = start->pre_b;
    }
  }
  const bool by_items = (EXT || HELD) && !CL && P.item_meta;  // every result is joined
  using Place = typename Walk<EXT>::Place;
  static_assert(sizeof(Place) == kPlaceBytes, "layout");
  // HELD: this warp's place, and behind all of them a second one of each warp that
  // is no softmax warp
  Place* place = reinterpret_cast<Place*>(sm + L::walk) + warp;
  constexpr int kSecond = kTcWarps - kSoftWarps;
  Lens* lens = reinterpret_cast<Lens*>(sm + L::lens);
  static_assert(sizeof(Lens) <= 144, "layout");
  if constexpr (HELD && !CL) {
    const int b0 = max(wk.b, 0);
    if (tid < kLens) {
      const int b = (b0 + tid) % c.B;
      lens->len[tid] = ld_now(c.lens + b);
      lens->cnt[tid] = row_count(c.counts, b, c.T);
      lens->b0 = b0;
    }
    __syncthreads();
    if (lane_id == 0) {
      wk.save(place);
      if (warp >= kSoftWarps) wk.save(place + kSecond);
    }
    __syncwarp();
  }
  // the next piece of walk `w` (second: the warp's other walk)
  auto next_piece = [&](Walk<EXT>& w, auto warp_wide, bool second) -> bool {
    if constexpr (HELD && !CL) {
      Place* at = place + (second ? kSecond : 0);
      bool more = false;
      if constexpr (decltype(warp_wide)::value) {
        __syncwarp();  // every lane has what it wants of the last piece
        if (lane_id == 0) more = next_piece_of<EXT>(P, NT, kCost, at, lens);
        __syncwarp();  // the place is read by all (a shuffle orders no memory)
        more = __shfl_sync(0xffffffffu, more, 0);
      } else {
        more = next_piece_of<EXT>(P, NT, kCost, at, lens);
      }
      if (more) w.take(at);
      return more;
    } else {
      return w.template next<CL>(P, NT, kCost);
    }
  };
  constexpr std::true_type all_lanes;
  constexpr std::false_type one_lane;
  const int G = c.group, tile_rows = P.tpt * G;
  float2* part_ml = reinterpret_cast<float2*>(sm + L::k + NT * 65536);  // CL
  static_assert(NT * (65536 + 1024) <= (L::KS + L::VS) * kTileBytes + 2 * L::RS * L::kRawBytes, "a part fits over the stages");

  if (warp < kSoftWarps) {
    // -------------------------------------------------------------- softmax
    if constexpr (!HELD) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    // padding rows (a cache without room for keys is not this kernel's)
    if (c.counts) {
      for (int b = CL ? blockIdx.y * gridDim.x + blockIdx.x : blockIdx.x; b < c.B; b += CL ? gridDim.x * gridDim.y : gridDim.x) {
        const int t0 = row_count(c.counts, b, c.T);
        for (int64_t e = tid; e < static_cast<int64_t>(c.T - t0) * c.H * 16; e += kSoftWarps * 32) {
          const int64_t row = e >> 4;
          const int t = t0 + static_cast<int>(row / c.H), h = static_cast<int>(row % c.H);
          reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.o) + b * c.o_sb + t * c.o_ss + h * c.o_sh)[e & 15] = make_uint4(0, 0, 0, 0);
          if ((e & 15) == 0) c.lse[(static_cast<int64_t>(b) * c.H + h) * c.T + t] = -INFINITY;
        }
      }
    }
    const int slot = warp >> 2;
    const int r = (warp & 3) * 32 + lane_id;
    const uint32_t lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + slot * 128 + lane, tO = tmem + 256 + slot * 128 + lane;
    const int r_few = r & 31;  // FEW: the row, of which this warp has a quarter of the keys
    const bool call_few = HELD && NT == 1 && P.few;
    int rt = r / G, rg = r - rt * G;
    const float sc = c.scale_log2;
    long long g = 0;    // score tiles before the present piece
    int vc = 0;         // key tiles before the present piece
    int n_piece = 0;
    bool ok = true, at_start = true;
    const long long range_end = by_items ? start->first + start->left : 0;
    while (ok && next_piece(wk, all_lanes, false)) {
      const int steps = (wk.kt1 - wk.kt0) * NT;
      const bool few = call_few && wk.pb >= 0;
      if constexpr (HELD && NT == 1) {
        const int rr = few ? r_few : r;
        rt = rr / G;
        rg = rr - rt * G;
      }
      const int t = (wk.pm * NT + (NT == 2 ? slot : 0)) * P.tpt + rt;
      const bool valid = (few ? r_few : r) < tile_rows && t < wk.it.cnt;
      const bool act = __any_sync(0xffffffffu, valid);  // this warp has rows
      uint32_t anc[kTreeWords] = {};
      int low = 0, low_last = 0;  // where the row's window begins, and the last of the warp's
      if (TREE && valid && (tile_key<EXT>(wk.it, wk.kt1 - 1) + kTile > wk.it.prefix || (EXT && c.window > 0))) {
        int node = t, depth = 0, k = 0;
        if (EXT && c.window > 0) {
          depth = node_depth(c, wk.pb, t);
          low = window_low(c, wk.pb, depth);
        }
        while (node >= 0) {
          const bool sees = !EXT || c.window == 0 || window_sees(c, wk.pb, depth, k++);
#pragma unroll
          for (int i = 0; i < kTreeWords; ++i)
            if (sees && i == (node >> 5)) anc[i] |= 1u << (node & 31);
          const int up = ld_now(c.parents + wk.pb * c.par_sb + node);
          if (up >= node || up < -1) {
            atomicOr(c.status, kStatusIndex);
            break;
          }
          node = up;
        }
      }
      if (EXT && c.window > 0) {
        if (!TREE && valid) low = window_low(c, wk.pb, t);
        low_last = __reduce_max_sync(0xffffffffu, low);
      }
      float row_sc = sc;
      float m_run = -INFINITY, l_run = 0.f;
      bool first = true;
      for (int j = static_cast<int>((slot ^ g) & 1); j < steps; j += 2) {
        const int kt = wk.kt0 + (NT == 2 ? j >> 1 : j), j0 = tile_key<EXT>(wk.it, kt);
        const long long gg = g + j;
        const int sc_at = NT == 2 ? vc + kt - wk.kt0 : static_cast<int>(gg);  // HELD: the tile, counted by the CTA
        if constexpr (HELD) {  // the scales are there first
          if (!(ok = wait_bar_warp(&bars[L::ScFull + sc_at % L::SS], (sc_at / L::SS) & 1, abort_flag, budget))) break;
        }
        if (!(ok = wait_bar_warp(&bars[L::SFull + slot], (gg >> 1) & 1, abort_flag, budget))) break;
        const Scales& scales = reinterpret_cast<const Scales*>(sm + L::sc)[HELD ? sc_at % (HELD ? L::SS : 1) : 0];
        // the row's factor: its way into shared memory ends before its warps say that
        // the piece's first scales are there, and the next but one comes after this
        // slot's weights
        if (HELD && !F16 && first && valid) row_sc = reinterpret_cast<const float*>(sm + L::qs)[((n_piece & 1) * NT + (NT == 2 ? slot : 0)) * 128 + (few ? r_few : r)];
        tc_fence_after();
        if (act) {
          // the first node that the warp's first token does not see
          const int open = TREE ? wk.it.prefix : wk.it.prefix + __shfl_sync(0xffffffffu, t, 0) + 1;
          bool all = j0 + kTile <= min(open, wk.it.keys);
          if constexpr (EXT) all = all && (c.window == 0 || j0 >= low_last || j0 + kTile <= c.sinks);
          if constexpr (HELD) {
            softmax_held<NT>(tS, tO, row_sc, scales, !all, [&](int i) {
              uint32_t w = valid ? key_bits<TREE>(j0 + 32 * i, wk.it, t, anc) : 0u;
              if (EXT && c.window > 0) w &= window_bits<TREE>(j0 + 32 * i, low, c.sinks, wk.it.prefix);
              return w;
            }, few, warp & 3, first, m_run, l_run);
          } else if (all) {
            const uint32_t mb[4] = {~0u, ~0u, ~0u, ~0u};
            softmax_tile<F16, false>(tS, tO, sc, mb, first, m_run, l_run);
          } else {
            uint32_t mb[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              mb[w] = valid ? key_bits<TREE>(j0 + 32 * w, wk.it, t, anc) : 0u;
              if (EXT && c.window > 0) mb[w] &= window_bits<TREE>(j0 + 32 * w, low, c.sinks, wk.it.prefix);
            }
            softmax_tile<F16, true>(tS, tO, sc, mb, first, m_run, l_run);
          }
        }
        first = false;
        if (!HELD && (j0 + kTile > wk.it.keys || (EXT && j0 < wk.it.low && j0 + kTile > c.sinks))) {
          // rows of V behind the last key (or before every window) hold anything:
          // zero weights do not silence infinities and NaN, zeros do (with NT = 2
          // both slots write the same zeros: neither waits for the other)
          const int st = (vc + kt - wk.kt0) % L::VS;
          if (!(ok = wait_bar_warp(&bars[L::VFull + st], ((vc + kt - wk.kt0) / L::VS) & 1, abort_flag, budget))) break;
          if (j0 + r >= wk.it.keys || (EXT && j0 + r < wk.it.low && j0 + r >= c.sinks)) zero_row(sm + L::v + st * kTileBytes, r);
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(&bars[L::PFull + slot]);
      }
      if (!ok) break;
      // ---- the piece's result
      const int h = wk.ph * G + rg;
      const bool whole = wk.whole() && !by_items;
      const int64_t pslot = 2 * static_cast<int64_t>(blockIdx.x) + (at_start ? 0 : 1);
      at_start = false;
      int64_t prow0 = pslot * P.part_rows;  // the part's first row
      if constexpr ((EXT || HELD) && !CL) {
        if (by_items) {
          prow0 = pslot * P.split_rows;
          if (wk.whole()) prow0 = whole_part(P, wk.ph, wk.pb, wk.pm);
          if (tid == 0 && wk.kt0 == 0) {
            int2 meta = make_int2(1, -1);
            if (!wk.whole()) {
              Deal d;
              d.make(start->total, P.ctas);
              // where the item ends: as far behind the piece as it has tiles behind it
              const long long end = range_end - (HELD ? place->left : wk.left) + wk.it.n - wk.kt1;
              meta = make_int2(d.holder(end - 1) - static_cast<int>(blockIdx.x) + 1, static_cast<int>(pslot));
            }
            P.item_meta[item_index(P, wk.ph, wk.pb, wk.pm)] = meta;
          }
        }
      }
      if (!(ok = wait_bar_warp(&bars[L::OFull], n_piece & 1, abort_flag, budget))) break;
      tc_fence_after();
      if constexpr (NT == 2) {
        if (act) {
          const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
          const int64_t ooff = wk.pb * c.o_sb + static_cast<int64_t>(t) * c.o_ss + static_cast<int64_t>(h) * c.o_sh;
          const int64_t prow = prow0 + slot * tile_rows + r;
#pragma unroll 1
          for (int q4 = 0; q4 < 4; ++q4) {
            uint32_t r32[32];
            tmem_ld32(tO + 32 * q4, r32);
            float y[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(r32[e]) * (whole && !CL ? inv : 1.f);
            if constexpr (CL) {
              stage_chunk32(sm + L::k, slot * 128 + r, q4, y);
              continue;
            }
            if (valid && whole) store_out32<F16>(c.o, ooff, P.o_wide != 0, q4, y);
            else if (valid) store_part32(c.part + prow * kD, q4, y);
          }
          if (CL) part_ml[slot * 128 + r] = make_float2(m_run, l_run);
          if (!CL && valid) {
            if (whole) c.lse[(static_cast<int64_t>(wk.pb) * c.H + h) * c.T + t] = l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * kLn2;
            else P.part_ml[prow] = make_float2(m_run, l_run);
          }
        }
      } else {
        // the two slots' accumulators come together: this group takes 64 columns
        float2* ml = reinterpret_cast<float2*>(sm + L::ml);
        ml[slot * 128 + r] = make_float2(m_run, l_run);
        mbar_arrive(&bars[L::MlFull + slot]);
        if (!(ok = wait_bar_warp(&bars[L::MlFull + (slot ^ 1)], n_piece & 1, abort_flag, budget))) break;
        if (act) {
          const float2 other = ml[(slot ^ 1) * 128 + r];
          const float m = fmaxf(m_run, other.x), m_use = m == -INFINITY ? 0.f : m;
          const float f0 = ex2(m_run - m_use), f1 = ex2(other.x - m_use);
          const float l = f0 * l_run + f1 * other.y, inv = whole && !CL ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
          const bool mine = steps > 1 || (g & 1) == slot, theirs = steps > 1 || (g & 1) != slot;
          const int64_t ooff = wk.pb * c.o_sb + static_cast<int64_t>(t) * c.o_ss + static_cast<int64_t>(h) * c.o_sh;
          const int64_t prow = prow0 + (few ? (warp & 3) * P.part_rows + r_few : r);
          const uint32_t tOther = tmem + 256 + (slot ^ 1) * 128 + lane;
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            const int q4 = 2 * slot + q;
            uint32_t a[32], d[32];
            float y[32];
            tmem_ld32_issue(tO + 32 * q4, a);
            tmem_ld32_issue(tOther + 32 * q4, d);
            tmem_ld_wait32(a);
            tmem_ld_wait32(d);
#pragma unroll
            for (int e = 0; e < 32; ++e) {  // a slot without tiles holds anything
              const float v0 = mine ? __uint_as_float(a[e]) : 0.f, v1 = theirs ? __uint_as_float(d[e]) : 0.f;
              y[e] = fmaf(v1, f1, v0 * f0) * inv;
            }
            if constexpr (CL) {
              stage_chunk32(sm + L::k, r, q4, y);
              continue;
            }
            if (valid && whole) store_out32<F16>(c.o, ooff, P.o_wide != 0, q4, y);
            else if (valid) store_part32(c.part + prow * kD, q4, y);
          }
          if (CL && slot == 0) part_ml[r] = make_float2(m, l);
          if (!CL && valid && slot == 0) {
            if (whole) c.lse[(static_cast<int64_t>(wk.pb) * c.H + h) * c.T + t] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            else P.part_ml[prow] = make_float2(m, l);
          }
        }
        // neither accumulator is overwritten before both groups have read it
        tc_fence_before();
        mbar_arrive(&bars[L::ORead + slot]);
        if (!(ok = wait_bar_warp(&bars[L::ORead + (slot ^ 1)], n_piece & 1, abort_flag, budget))) break;
      }
      tc_fence_before();
      g += steps;
      vc += wk.kt1 - wk.kt0;
      ++n_piece;
    }
    if (CL && n_piece == 0 && (NT == 2 || slot == 0)) part_ml[(NT == 2 ? slot * 128 : 0) + r] = make_float2(-INFINITY, 0.f);
  } else if (warp < kWarpMma) {
    // ---------------------------------------------------------------- Q rows
    if constexpr (!HELD) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    const int qt = tid - kWarpQ0 * 32;
    int n_piece = 0;
    if constexpr (HELD) {
      // ------------------------------------------------- bytes into operands
      const bool is_v = warp >= kWarpQ0 + kQWarps;
      constexpr int kParts = kTile / L::kRawRows, kU = L::kRawRows / 16;  // stages of a tile, a thread's pieces of a stage
      const PagedKV& kv = c.kv;
      const int gw = warp & 3;
      // A lane has 16 columns (cg) of the rows r0 + 16 u. Eight lanes write two
      // rows' 64 columns of one half of the operand tile, whose swizzles differ: no
      // bank twice. (In the ring a thread's pieces lie anywhere: it alone reads them.)
      const int half = (lane_id >> 3) & 1, cg = 4 * half + (lane_id & 3), r_in = ((lane_id >> 4) << 1) | ((lane_id >> 2) & 1), r0 = 4 * gw + r_in;
      uint64_t* full = &bars[is_v ? L::VFull : L::KFull];
      uint64_t* empty = &bars[is_v ? L::VEmpty : L::KEmpty];
      uint8_t* tiles = sm + (is_v ? L::v : L::k);
      static_assert(L::KS == L::VS, "one count");
      uint8_t* raw = sm + L::raw + (is_v ? L::RS : 0) * L::kRawBytes + (gw * 32 + lane_id) * 16;  // + 2048 u
      // places in 32 bits: of rows in units of 16 bytes, of scales in numbers (the
      // host has seen that they fit)
      const HeldAt at = is_v ? P.held_v : P.held_k;
      const uint8_t* base = static_cast<const uint8_t*>(is_v ? kv.v : kv.k) + 16 * cg;
      const float* sc_base = is_v ? kv.vs : kv.ks;
      constexpr uint32_t kNowhere = ~0u;
      // ---- the stream of fetches, RS stages ahead of the conversion. A
      // lane looks up the place of one of its warp's 32 rows of a tile, a tile ahead
      // of the fetch, and has that row's scale.
      const int my_row = 4 * gw + (lane_id & 3) + 16 * (lane_id >> 2);
      Walk<EXT> wl = wk;
      bool l_have = false, l_in = false;
      int lt = 0, l_left = 0, l_pg = 0;
      uint32_t l_off = 0, l_sc = 0;  // the row's place in its page
      const int32_t* l_pages = nullptr;
      auto look_on = [&]() {  // the next piece
        l_have = next_piece(wl, all_lanes, true);
        lt = wl.kt0;
        l_left = wl.kt1 - wl.kt0;
        l_pages = kv.pages + (EXT && wl.pb < 0 ? pre_b : wl.pb) * kv.p_sb;
      };
      auto look = [&]() {  // the next tile
        const int j = tile_key<EXT>(wl.it, lt++) + my_row;
        l_in = j < wl.it.keys && (!EXT || j >= wl.it.low || j < c.sinks);  // (keys lie within the table)
        if (l_in) {
          const int page = kv.page_shift >= 0 ? j >> kv.page_shift : j / kv.page, row = j - page * kv.page;
          l_pg = ld_now(l_pages + page);
          l_off = row * at.sr + wl.ph * at.sh;
          l_sc = row + wl.ph * at.sc_sh;
        }
        if (--l_left == 0) look_on();
      };
      look_on();
      bool there = l_have;  // a tile was looked up
      if (there) look();
      int i_tile = 0;
      bool i_have = false;
      uint32_t off = kNowhere;  // of the lane's row
      auto fetch = [&](int i_part, uint8_t* dst) {
        if (i_part == 0) {
          i_have = there;
          if (there) {
            off = kNowhere;
            uint32_t sc_at = 0;
            if (l_in && static_cast<unsigned>(l_pg) >= static_cast<unsigned>(kv.n_pages)) {
              atomicOr(c.status, kStatusIndex);  // reads as zeros
            } else if (l_in) {
              off = l_pg * at.sp + l_off;
              sc_at = l_pg * at.sc_sp + l_sc;
            }
            there = l_have;
            if (there) look();
            const int st = i_tile % L::SS;
            Scales& s = reinterpret_cast<Scales*>(sm + L::sc)[st];
            cp_async4(is_v ? &s.v[my_row] : &s.k[my_row], sc_base + sc_at, off != kNowhere);
            ++i_tile;
          }
        }
        if (i_have) {
          uint32_t o[kU];
#pragma unroll
          for (int u = 0; u < kU; ++u) o[u] = __shfl_sync(0xffffffffu, off, r_in + 4 * (i_part * kU + u));
#pragma unroll
          for (int u = 0; u < kU; ++u) cp_async16(dst + u * 2048, base + (o[u] == kNowhere ? 0u : o[u]) * static_cast<uint64_t>(16), o[u] != kNowhere);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      // ---- the conversion. Columns 16 cg .. + 16 are chunks 2 cg and 2 cg + 1; rows
      // r0 + 16 u have the swizzle of r0.
      const uint32_t at0 = half * kHalfBytes + sw128_off(r0, 2 * (lane_id & 3)), at1 = half * kHalfBytes + sw128_off(r0, 2 * (lane_id & 3) + 1);
      bool ok = true;
      int left = 0, n = 0, slot = 0;  // left: tiles of the present piece
#pragma unroll
      for (int i = 0; i < L::RS; ++i) fetch(i % kParts, raw + i * L::kRawBytes);
#pragma unroll 1
      while (ok) {
        if (left == 0) {
          if (!next_piece(wk, all_lanes, false)) break;
          left = wk.kt1 - wk.kt0;
          if (is_v) {
            // its rows, once the last one's scores are done: V's warps bring them, whose tiles
            // are wanted after K's (K's warps: 256 tokens of short sequences 160 us, so 156)
            const bool q_few = NT == 1 && P.few && wk.pb >= 0;
            float* qs = reinterpret_cast<float*>(sm + L::qs) + (n_piece & 1) * NT * 128;
            if (!load_q_held<NT, F16, EXT, kQWarps * 32>(P, wk, sm + L::q, qs, qt & 127, q_few, [&]() -> bool {
                  return n_piece == 0 || wait_bar_warp(&bars[L::QEmpty], (n_piece - 1) & 1, abort_flag, budget);
                }))
              break;
            mbar_arrive(&bars[L::QFull]);
            ++n_piece;
          }
        }
        const int op = n % L::KS;
        uint8_t* dst = tiles + op * kTileBytes;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          asm volatile("cp.async.wait_group %0;" ::"n"(HELD ? L::RS - 1 : 0) : "memory");
          if (part == 0) {
            const int st = n % L::SS;
            Scales& s = reinterpret_cast<Scales*>(sm + L::sc)[st];
            if (is_v) {
              const float v = fabsf(s.v[my_row]);  // 0: not seen, or a row of zeros
              const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, v == v ? __float_as_uint(v) : 0u));
              const float low = __uint_as_float(__reduce_min_sync(0xffffffffu, v > 0.f ? __float_as_uint(v) : 0x7f800000u));
              // any numbers near them do; no key but zeros: -50 and -50
              if (lane_id == 0)
                s.ends[gw] = __floats2half2_rn(fminf(fmaxf(__log2f(top), -kTopRange), kTopRange), fminf(fmaxf(-__log2f(low), -kTopRange), kTopRange));
            }
            __syncwarp();
            if (lane_id == 0) mbar_arrive(&bars[L::ScFull + st]);
            if (n >= L::KS && !(ok = wait_bar_warp(&empty[op], ((n / L::KS) - 1) & 1, abort_flag, budget))) break;
          }
          uint8_t* src = raw + slot * L::kRawBytes;
          uint4 x[kU];  // all reads before the first write: the compiler keeps their order
#pragma unroll
          for (int u = 0; u < kU; ++u) x[u] = *reinterpret_cast<const uint4*>(src + u * 2048);
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            uint4 a, b;
            held_f16<KV>(x[u].x, a.x, a.y);
            held_f16<KV>(x[u].y, a.z, a.w);
            held_f16<KV>(x[u].z, b.x, b.y);
            held_f16<KV>(x[u].w, b.z, b.w);
            *reinterpret_cast<uint4*>(dst + at0 + (part * kU + u) * 16 * 128) = a;
            *reinterpret_cast<uint4*>(dst + at1 + (part * kU + u) * 16 * 128) = b;
          }
          fetch((part + L::RS) % kParts, src);  // into the stage that has just been read, by this thread
          slot = slot == L::RS - 1 ? 0 : slot + 1;
        }
        if (!ok) break;
        fence_proxy_async_smem();
        mbar_arrive(&full[op]);
        ++n;
        --left;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
      while (wk.template next<CL>(P, NT, kCost)) {
        if (n_piece > 0 && !wait_bar_warp(&bars[L::QEmpty], (n_piece - 1) & 1, abort_flag, budget)) break;
        load_q<NT, EXT, kQWarps * 32>(P, wk, sm + L::q, qt);
        mbar_arrive(&bars[L::QFull]);
        ++n_piece;
      }
    }
  } else {
    if constexpr (!HELD) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (!HELD && (warp == kWarpK || warp == kWarpV)) {
      // ------------------------------------------------------- TMA of K and V
      const bool is_k = warp == kWarpK;
      const int stages = is_k ? L::KS : L::VS;
      uint64_t* full = &bars[is_k ? L::KFull : L::VFull];
      uint64_t* empty = &bars[is_k ? L::KEmpty : L::VEmpty];
      const CUtensorMap* map = is_k ? &P.tmap_k : &P.tmap_v;
      const bool r_first = (is_k ? P.k_r_first : P.v_r_first) != 0;
      uint8_t* ring = sm + (is_k ? L::k : L::v);
      const int half = lane_id >> (7 - P.box_shift), x = half * 64;  // a lane per box: two halves of 128 / box
      const uint32_t dst = half * kHalfBytes + ((lane_id & ((kTile >> P.box_shift) - 1)) << P.box_shift) * 128;
      int n = 0;
      bool ok = true, have = wk.template next<CL>(P, NT, kCost);
      int kt = wk.kt0;
      Box box{false, 0, 0};
      if (have) box = find_box<EXT>(P, wk, kt, lane_id, pre_b);
      while (ok && have) {
        const int st = n % stages;
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, box.mine));
        if (n >= stages && !(ok = wait_bar_warp(&empty[st], ((n / stages) - 1) & 1, abort_flag, budget))) break;
        if (lane_id == 0) mbar_arrive_expect_tx(&full[st], (boxes << P.box_shift) * 128);
        __syncwarp();
        if (box.mine)
          tma_load_4d(ring + st * kTileBytes + dst, map, &full[st], x, r_first ? box.row : wk.ph, r_first ? wk.ph : box.row, box.pg);
        // the next tile's pages are looked up while its stage is in use
        if (++kt == wk.kt1) {
          have = wk.template next<CL>(P, NT, kCost);
          kt = wk.kt0;
        }
        if (have) box = find_box<EXT>(P, wk, kt, lane_id, pre_b);
        ++n;
      }
      // every issued load lands before the CTA exits
      for (int m = max(0, n - stages); m < n; ++m) mbar_wait(&full[m % stages], (m / stages) & 1, budget);
    } else if (lane_id == 0) {
      // ------------------------------------------------------------ MMA issue
      // one thread per slot: its waits run under the other's MMAs
      const int slot = warp == kWarpMma ? 0 : 1;
      const uint32_t tS = tmem + slot * 128, tO = tmem + 256 + slot * 128;
      const uint64_t dQ = sdesc_sw128(smem_u32(sm + L::q) + (NT == 2 ? slot * kTileBytes : 0), 16, 1024);
      const uint64_t dK0 = sdesc_sw128(smem_u32(sm + L::k), 16, 1024);
      const uint64_t dV0 = sdesc_sw128(smem_u32(sm + L::v), kHalfBytes, 1024);
      // the scores' stream runs one of the slot's tiles ahead of PV's, each with
      // a walk of its own; kn counts key tiles over all pieces
      Walk<EXT> ws = wk;
      bool ok = true, issued = false;
      int s_left = 0, s_kn = 0, s_next = 0, s_piece = -1, p_left = 0, p_kn = 0, p_next = 0, p_done = 0, p_piece = 0;
      // Enters the next piece: its first key tile and its number of tiles for
      // this slot (none, where NT = 1 and its only tile is the other slot's).
      auto enter = [&](Walk<EXT>& w, bool second, int& kn, int& next, int& left) -> bool {
        if (!next_piece(w, one_lane, second)) return false;
        const int tiles = w.kt1 - w.kt0;
        // NT = 1: the slots take alternate tiles of the whole stream
        const int skip = NT == 2 ? 0 : (slot ^ next) & 1;
        kn = next + skip;
        left = NT == 2 ? tiles : (tiles - skip + 1) / 2;
        next += tiles;
        return true;
      };
      bool more = true;
      // makes the slot's next score tile ready to be issued, if any is left
      auto find_scores = [&]() -> bool {
        while (s_left == 0) {
          if (!enter(ws, true, s_kn, s_next, s_left)) {
            more = false;
            return true;
          }
          ++s_piece;
          if (!wait_bar(&bars[L::QFull], s_piece & 1, abort_flag, budget)) return false;
          if (s_left == 0) mma_commit(&bars[L::QEmpty]);  // a piece of one tile, the other slot's
        }
        return wait_bar(&bars[L::KFull + s_kn % L::KS], (s_kn / L::KS) & 1, abort_flag, budget);
      };
      constexpr int kHold = 6;  // K-steps of the scores under the lock (8: 468 us, 6 and 7: 459, 4: 464, 2: 481, 0: 514)
      auto scores = [&](auto&& release) {
        issue_s<OP16, 0, kHold>(tS, dQ, sdesc_add(dK0, (s_kn % L::KS) * kTileBytes));
        release();
        issue_s<OP16, kHold, 8>(tS, dQ, sdesc_add(dK0, (s_kn % L::KS) * kTileBytes));
        issued = true;
        mma_commit(&bars[L::SFull + slot]);
        mma_commit(&bars[L::KEmpty + s_kn % L::KS]);
        s_kn += NT == 2 ? 1 : 2;
        if (--s_left == 0) mma_commit(&bars[L::QEmpty]);
      };
      // NT = 2: a slot's PV and next scores enter the tensor pipe as one batch:
      // two threads' MMAs taken in turns end together, and the slots' softmax
      // then runs side by side with the tensor pipe idle (2048-token chunk after
      // 16384 tokens: 563 us without the lock, 459 with it).
      // The lock is let go before the last MMAs, so that it has changed hands
      // when the pipe has done them.
      auto batch = [&](auto&& issue) -> bool {
        if constexpr (NT == 1) {
          tc_fence_after();
          issue([] {});
          return true;
        }
        const long long t0 = clock64();
        while (atomicCAS(pipe_lock, 0, 1) != 0) {
          if (*abort_flag || clock64() - t0 > budget) {
            *abort_flag = 1;
            return false;
          }
        }
        tc_fence_after();
        issue([&] {
          __threadfence_block();
          atomicExch(pipe_lock, 0);
        });
        return true;
      };
      ok = find_scores() && (!more || batch(scores));
      while (ok && enter(wk, false, p_kn, p_next, p_left)) {
        for (int i = 0; i < p_left; ++i, ++p_done) {
          const bool same = s_left > 0;  // the next scores are of the same piece: Q is there
          if (same && !(ok = find_scores())) break;
          if (!(ok = wait_bar(&bars[L::VFull + p_kn % L::VS], (p_kn / L::VS) & 1, abort_flag, budget))) break;
          if (!(ok = wait_bar(&bars[L::PFull + slot], p_done & 1, abort_flag, budget))) break;
          ok = batch([&](auto&& release) {
            issue_pv<OP16>(tO, tS, sdesc_add(dV0, (p_kn % L::VS) * kTileBytes), i > 0);
            mma_commit(&bars[L::VEmpty + p_kn % L::VS]);
            if (i + 1 == p_left) mma_commit(&bars[L::OFull]);
            if (same) scores(release);
            else release();
          });
          if (!ok) break;
          p_kn += NT == 2 ? 1 : 2;
          if (!same && more && !(ok = find_scores() && (!more || batch(scores)))) break;
        }
        if (!ok) break;
        if (p_left == 0) {
          // nothing of this piece is this slot's: its arrival must not fall
          // into the phase of the piece before, which the other slot may be at
          if (p_piece > 0 && !(ok = wait_bar(&bars[L::OFull], (p_piece - 1) & 1, abort_flag, budget))) break;
          mma_commit(&bars[L::OFull]);
        }
        ++p_piece;
      }
      if (issued && !ok) {
        // every MMA of this thread done before anyone frees TMEM or shared memory
        mma_commit(&bars[L::Drain + slot]);
        const long long t0 = clock64();
        while (!mbar_try_wait(&bars[L::Drain + slot], 0) && clock64() - t0 < budget) {
        }
      }
    }
  }

  __syncwarp();
  if (*abort_flag && tid == 0) {
    atomicOr(c.status, kStatusTimeout);
    atomicAdd(c.counters + kCtrTimeouts, 1ull);
  }
  tc_fence_before();
  if constexpr (CL) {
    if constexpr (HELD && NT == 1) {
      // FEW: the four groups' results become one
      if (P.few && warp < kSoftWarps) {
        named_bar(1, kSoftWarps * 32);
        const int there = max(0, min(P.tpt, wk.it.cnt - wk.m * P.tpt)) * G;
        for (int e = warp; e < there; e += kSoftWarps) {
          float2 x[4];
          float4 y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = part_ml[32 * i + e];
            y[i] = *reinterpret_cast<const float4*>(sm + L::k + stage_off(32 * i + e, lane_id));
          }
          const float top = fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x)), use = top == -INFINITY ? 0.f : top;
          float l = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (x[i].x == -INFINITY) continue;
            const float f = ex2(x[i].x - use);
            l = fmaf(f, x[i].y, l);
            o = make_float4(fmaf(f, y[i].x, o.x), fmaf(f, y[i].y, o.y), fmaf(f, y[i].z, o.z), fmaf(f, y[i].w, o.w));
          }
          __syncwarp();
          *reinterpret_cast<float4*>(sm + L::k + stage_off(e, lane_id)) = o;
          if (lane_id == 0) part_ml[e] = make_float2(top, l);
        }
        __syncwarp();
      }
    }
    cluster_sync();  // every CTA's part is in place
    const int rank = static_cast<int>(cluster_rank()), m = wk.m, b = wk.b, h = wk.h;
    const int there = max(0, min(NT * P.tpt, wk.it.cnt - m * NT * P.tpt)) * G;  // rows, tile after tile
    for (int e = (warp << P.cluster_shift) + rank; e < there; e += kTcWarps << P.cluster_shift) {
      const int r = NT == 2 && e >= tile_rows ? 128 + e - tile_rows : e;  // in the part
      float2 x[kMaxClusterAttn];
      float4 y[kMaxClusterAttn];
#pragma unroll
      for (int i = 0; i < kMaxClusterAttn; ++i) {
        x[i] = make_float2(-INFINITY, 0.f);
        y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < P.cluster) {
          x[i] = ld_peer_f2(mapa_shared(smem_u32(part_ml + r), i));
          y[i] = ld_peer_f4(mapa_shared(smem_u32(sm + L::k) + stage_off(r, lane_id), i));
        }
      }
      float top = -INFINITY, l = 0.f;
#pragma unroll
      for (int i = 0; i < kMaxClusterAttn; ++i) top = fmaxf(top, x[i].x);
      const float use = top == -INFINITY ? 0.f : top;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kMaxClusterAttn; ++i) {
        if (x[i].x == -INFINITY) continue;  // a CTA without tiles left nothing there
        const float f = ex2(x[i].x - use);
        l = fmaf(f, x[i].y, l);
        o = make_float4(fmaf(f, y[i].x, o.x), fmaf(f, y[i].y, o.y), fmaf(f, y[i].z, o.z), fmaf(f, y[i].w, o.w));
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int t = m * NT * P.tpt + e / G, hq = h * G + e % G;
      const int64_t off = b * c.o_sb + static_cast<int64_t>(t) * c.o_ss + static_cast<int64_t>(hq) * c.o_sh + 4 * lane_id;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c.o) + off) =
          make_uint2(pack16<F16>(o.x * inv, o.y * inv), pack16<F16>(o.z * inv, o.w * inv));
      if (lane_id == 0) c.lse[(static_cast<int64_t>(b) * c.H + hq) * c.T + t] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
    }
    __syncwarp();
    // no CTA leaves while a peer reads its part (nothing is published here: a
    // releasing arrival would wait for the results' way to memory)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

template <int NT, bool F16, bool TREE, bool CL, int KV, bool EXT>
cudaError_t launch_t(const TcAttnParams& p, cudaStream_t stream) {
  auto kern = tc_kernel<NT, F16, TREE, CL, KV, EXT>;
  constexpr uint32_t bytes = Lay<NT, KV != 0>::bytes;
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = opt_in_smem(kern, bytes, configured);
  if (e != cudaSuccess) return e;
  if constexpr (CL) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.cluster * p.c.kv.Hkv, p.c.B * p.n_groups);
    cfg.blockDim = dim3(Roles<KV != 0>::kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
  }
  return launch_chained(kern, dim3(p.ctas), dim3(Roles<KV != 0>::kThreads), bytes, stream, p);
}
template <int NT, bool CL, int KV, bool EXT>
cudaError_t launch_nt(const TcAttnParams& p, bool f16, cudaStream_t stream) {
  if (p.c.parents) return f16 ? launch_t<NT, true, true, CL, KV, EXT>(p, stream) : launch_t<NT, false, true, CL, KV, EXT>(p, stream);
  return f16 ? launch_t<NT, true, false, CL, KV, EXT>(p, stream) : launch_t<NT, false, false, CL, KV, EXT>(p, stream);
}
template <int KV, bool EXT>
cudaError_t launch_form(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream) {
  if (p.cluster > 0) return nt == 2 ? launch_nt<2, true, KV, EXT>(p, f16, stream) : launch_nt<1, true, KV, EXT>(p, f16, stream);
  return nt == 2 ? launch_nt<2, false, KV, EXT>(p, f16, stream) : launch_nt<1, false, KV, EXT>(p, f16, stream);
}

}  // namespace

}  // namespace st
