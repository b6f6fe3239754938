// Cached attention on the tensor cores (bf16 and fp16 caches): tcgen05 QK^T
// and PV with TMEM accumulators over pages gathered by TMA, online base-2
// softmax, split over the keys and joined.
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
// Roles (512 threads, one CTA per SM):
//   warps 0-7   softmax, two groups of four warps; thread = query row = TMEM lane
//   warps 8-11  Q rows of the next item into shared memory
//   warp 12/15  tcgen05.mma issue for slot 0 / 1 (one thread each); TMEM allocation
//   warp 13/14  TMA of K / V boxes, one lane per box
// TMEM: S0 | S1 | O0 | O1, 128 fp32 columns each; P (16-bit) overwrites the
// first half of its S and feeds PV from TMEM. The stream of score tiles
// alternates between the two halves ("slots"): with NT = 2 a slot is a query
// tile, with NT = 1 (decoding: few rows, bound by the reading of K and V) the
// slots take alternate key tiles with accumulators of their own, which are
// merged at the end; either way one slot's softmax runs under the other's
// MMAs. A slot's scores run one tile ahead of its PV, across the borders of
// items.
#include <atomic>
#include "st_kernels.h"
#include "st_serve.h"

namespace st {

namespace {

constexpr int kSoftWarps = 8, kWarpQ0 = 8, kQWarps = 4, kWarpMma = 12, kWarpK = 13, kWarpV = 14;  // warp 15: the second slot's MMAs
constexpr int kTcWarps = 16, kTcThreads = kTcWarps * 32;
// Registers per thread: the softmax threads hold a row of 128 scores. 256 * 184 + 256 * 72 = 512 * 128.
constexpr int kRegsSoft = 184, kRegsRest = 72;
constexpr float kRescale = 8.0f;  // O is rescaled when the running maximum grows by more than this (base 2)
// How far the reference stays below the running maximum (base 2). fp16 weights
// end at 2^-25 of 1, and a long row's many small ones would leave PV but stay in
// the sum; with the maximum's at 2^7, at most 2^15 while the reference lags,
// they end 2^-32 below it. bf16 has fp32's range.
template <bool F16>
constexpr float kLift = F16 ? 7.0f : 0.0f;

template <int NT>
struct Lay {  // shared memory, offsets from a 1024-byte aligned base
  // With NT = 1 a stage belongs to one slot for good (even counts): a slot's
  // thread waits for every phase of the stages that it uses, and a wait on
  // parity says nothing where phases went by unseen.
  static constexpr int KS = NT == 1 ? 2 : 3, VS = NT == 1 ? 4 : 2;
  static_assert(NT == 2 || (KS % 2 == 0 && VS % 2 == 0), "stages of one slot");
  static constexpr uint32_t q = 0, k = NT * kTileBytes, v = k + KS * kTileBytes, bar = v + VS * kTileBytes;
  static constexpr uint32_t ml = bar + 512;          // [2][128] (reference, sum), NT = 1
  static constexpr uint32_t bytes = ml + (NT == 1 ? 2 * 128 * 8 : 0);
  enum { QFull = 0, QEmpty, KFull, KEmpty = KFull + KS, VFull = KEmpty + KS, VEmpty = VFull + VS, SFull = VEmpty + VS,
         PFull = SFull + 2, OFull = PFull + 2, MlFull, ORead = MlFull + 2, Drain = ORead + 2, Num = Drain + 2 };
};
static_assert(Lay<1>::bytes <= 232448 && Lay<2>::bytes <= 232448, "shared memory");
static_assert(Lay<1>::Num * 8 + 128 <= 512 && Lay<2>::Num * 8 + 128 <= 512, "barrier area");

__device__ __forceinline__ constexpr uint32_t kofs(int kk) { return (kk >> 2) * kHalfBytes + (kk & 3) * 32; }
__device__ __forceinline__ constexpr uint32_t mofs(int kk) { return kk * 2048; }

// Asynchronous 16-byte copy into shared memory; zeros when !there.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}

struct Item {
  int prefix, keys, cnt, n;  // n: key tiles
};
__device__ __forceinline__ Item item_of(const TcAttnParams& p, int nt, int b, int m) {
  Item it;
  it.cnt = row_count(p.c.counts, b, p.c.T);
  it.keys = key_count(p.c, b, it.cnt, &it.prefix);
  const int64_t t0 = static_cast<int64_t>(m) * nt * p.tpt;
  if (t0 >= it.cnt) {
    it.n = 0;
  } else {
    // a chain's last row of the group sees no further than itself
    const int64_t end = p.c.parents ? it.keys : min(static_cast<int64_t>(it.keys), it.prefix + t0 + nt * p.tpt);
    it.n = static_cast<int>((end + kTile - 1) / kTile);
  }
  return it;
}

// A CTA's walk over its range: pieces of items.
struct Walk {
  int h, b, m, off;
  long long left;
  // the present piece
  int ph, pb, pm, kt0, kt1;
  Item it;
  __device__ __forceinline__ void advance(const TcAttnParams& p) {
    off = 0;
    if (++m == p.n_groups) {
      m = 0;
      if (++b == p.c.B) {
        b = 0;
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
  __device__ __forceinline__ bool next(const TcAttnParams& p, int nt) {
    if (left <= 0) return false;
    if constexpr (ONE) {
      left = 0;
      return true;
    }
    while (true) {
      it = item_of(p, nt, b, m);
      if (off < it.n) break;
      advance(p);
      if (h >= p.c.kv.Hkv) {  // lengths that changed under the kernel: no tiles are left
        left = 0;
        return false;
      }
    }
    ph = h;
    pb = b;
    pm = m;
    kt0 = off;
    kt1 = static_cast<int>(min(static_cast<long long>(it.n), off + left));
    left -= kt1 - kt0;
    off = kt1;
    if (off == it.n) advance(p);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return kt0 == 0 && kt1 == it.n; }
};

// The deal: CTA x has the tiles [first(x), first(x + 1)) of the call's, shares
// that differ by one at most. 32-bit division where the numbers allow it.
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
};

// Where the CTA's range begins: every thread sums the key tiles of a run of
// (sequence, group) pairs, a block scan places the runs.
__device__ __forceinline__ void find_start(const TcAttnParams& p, int nt, long long* scan, Start* st) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pairs = p.c.B * p.n_groups;  // at most 2^30
  const int per = (pairs + kTcThreads - 1) / kTcThreads, lo = min(pairs, tid * per), hi = min(pairs, lo + per);
  const int b0 = p.n_groups == 1 ? lo : lo / p.n_groups, m0 = lo - b0 * p.n_groups;
  long long sum = 0;
  for (int e = lo, b = b0, m = m0; e < hi; ++e) {
    const Item it = item_of(p, nt, b, m);
    sum += it.n;
    if (m == 0 && blockIdx.x == 0 && (ld_now(p.c.lens + b) < 0 || static_cast<int64_t>(ld_now(p.c.lens + b)) + it.cnt > it.keys))
      atomicOr(p.c.status, kStatusIndex);
    if (++m == p.n_groups) {
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
  if (tid == 0) st->left = 0;
  __syncthreads();
  long long before = 0, one = 0;
#pragma unroll
  for (int w = 0; w < kTcWarps; ++w) {
    if (w < warp) before += scan[w];
    one += scan[w];
  }
  Deal d;
  d.make(one * p.c.kv.Hkv, p.ctas);
  if (blockIdx.x < d.ctas) {
    const long long s0 = d.first(blockIdx.x);
    const int h = static_cast<int>(Deal::div(s0, one));
    long long rem = s0 - h * one - (before + inc - sum);
    if (rem >= 0 && rem < sum) {  // one thread
      for (int e = lo, b = b0, m = m0; e < hi; ++e) {
        const Item it = item_of(p, nt, b, m);
        if (rem < it.n) {
          st->h = h;
          st->b = b;
          st->m = m;
          st->off = static_cast<int>(rem);
          st->left = d.first(blockIdx.x + 1) - s0;
          // for the join: is this border the first inside of its item, and
          // who has the item's tiles?
          JoinMeta meta{0, 0, h, b, m, it.cnt};
          const long long item = s0 - rem;
          if (rem > 0 && d.first(blockIdx.x - 1) <= item) {
            meta.parts = d.holder(item + it.n - 1) - static_cast<int>(blockIdx.x) + 2;
            meta.slot0 = 2 * (static_cast<int>(blockIdx.x) - 1) + (d.first(blockIdx.x - 1) == item ? 0 : 1);
          }
          p.meta[blockIdx.x] = meta;
          break;
        }
        rem -= it.n;
        if (++m == p.n_groups) {
          m = 0;
          ++b;
        }
      }
    }
  } else if (tid == 0) {
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

// 32 bytes of a thread in one store: a thread per row writes whole sectors, in
// half as many instructions of 32 sectors each as with 16-byte stores.
__device__ __forceinline__ void st_v8(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
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
__device__ __forceinline__ Box find_box(const TcAttnParams& P, const Walk& wk, int kt, int lane) {
  const int nb = kTile >> P.box_shift, j = kt * kTile + ((lane & (nb - 1)) << P.box_shift);
  Box b;
  b.mine = lane < 2 * nb && j < wk.it.keys;
  b.pg = b.row = 0;
  if (b.mine && !kv_locate(P.c.kv, wk.pb, j, &b.pg, &b.row)) atomicOr(P.c.status, kStatusIndex);  // reads as zeros
  return b;
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

template <int NT, bool F16, bool TREE, bool CL>
__global__ void __launch_bounds__(kTcThreads, 1) tc_kernel(const __grid_constant__ TcAttnParams P) {
  using L = Lay<NT>;
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
    for (int s = 0; s < L::KS; ++s) {
      mbar_init(&bars[L::KFull + s], 1);
      mbar_init(&bars[L::KEmpty + s], NT);  // NT = 1: a tile is one slot's
    }
    for (int s = 0; s < L::VS; ++s) {
      mbar_init(&bars[L::VFull + s], 1);
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
  if (tid == kWarpK * 32) tma_prefetch_desc(&P.tmap_k);
  if (tid == kWarpV * 32) tma_prefetch_desc(&P.tmap_v);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  grid_dependency_wait();  // what came before touches no global memory
  Walk wk;  // with CL every role finds its way alone from here on
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
    wk.it = item_of(P, NT, wk.b, wk.m);
    wk.alone((wk.it.n * rank) >> P.cluster_shift, (wk.it.n * (rank + 1)) >> P.cluster_shift);
    if (tid == 0 && rank == 0 && wk.h == 0 && wk.m == 0 &&
        (ld_now(c.lens + wk.b) < 0 || static_cast<int64_t>(ld_now(c.lens + wk.b)) + wk.it.cnt > wk.it.keys))
      atomicOr(c.status, kStatusIndex);
  } else {
    // the scan's scratch lies in the Q tile, which is written later
    find_start(P, NT, reinterpret_cast<long long*>(sm + L::q), start);
    wk.h = start->h;
    wk.b = start->b;
    wk.m = start->m;
    wk.off = start->off;
    wk.left = start->left;
  }
  const int G = c.group, tile_rows = P.tpt * G;
  float2* part_ml = reinterpret_cast<float2*>(sm + L::k + NT * 65536);  // CL
  static_assert(NT * (65536 + 1024) <= (L::KS + L::VS) * kTileBytes, "a part fits over the K and V stages");

  if (warp < kSoftWarps) {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
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
    const int rt = r / G, rg = r - rt * G;
    const float sc = c.scale_log2;
    long long g = 0;    // score tiles before the present piece
    int vc = 0;         // key tiles before the present piece
    int n_piece = 0;
    bool ok = true, at_start = true;
    while (ok && wk.next<CL>(P, NT)) {
      const int steps = (wk.kt1 - wk.kt0) * NT;
      const int t = (wk.pm * NT + (NT == 2 ? slot : 0)) * P.tpt + rt;
      const bool valid = r < tile_rows && t < wk.it.cnt;
      const bool act = __any_sync(0xffffffffu, valid);  // this warp has rows
      uint32_t anc[kTreeWords] = {};
      if (TREE && valid && wk.kt1 * kTile > wk.it.prefix) {
        int node = t;
        while (node >= 0) {
#pragma unroll
          for (int i = 0; i < kTreeWords; ++i)
            if (i == (node >> 5)) anc[i] |= 1u << (node & 31);
          const int up = ld_now(c.parents + wk.pb * c.par_sb + node);
          if (up >= node || up < -1) {
            atomicOr(c.status, kStatusIndex);
            break;
          }
          node = up;
        }
      }
      float m_run = -INFINITY, l_run = 0.f;
      bool first = true;
      for (int j = static_cast<int>((slot ^ g) & 1); j < steps; j += 2) {
        const int kt = wk.kt0 + (NT == 2 ? j >> 1 : j), j0 = kt * kTile;
        const long long gg = g + j;
        if (!(ok = wait_bar_warp(&bars[L::SFull + slot], (gg >> 1) & 1, abort_flag, budget))) break;
        tc_fence_after();
        if (act) {
          // the first node that the warp's first token does not see
          const int open = TREE ? wk.it.prefix : wk.it.prefix + __shfl_sync(0xffffffffu, t, 0) + 1;
          if (j0 + kTile <= min(open, wk.it.keys)) {
            const uint32_t mb[4] = {~0u, ~0u, ~0u, ~0u};
            softmax_tile<F16, false>(tS, tO, sc, mb, first, m_run, l_run);
          } else {
            uint32_t mb[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) mb[w] = valid ? key_bits<TREE>(j0 + 32 * w, wk.it, t, anc) : 0u;
            softmax_tile<F16, true>(tS, tO, sc, mb, first, m_run, l_run);
          }
        }
        first = false;
        if (j0 + kTile > wk.it.keys) {
          // rows of V behind the last key hold anything: zero weights do not
          // silence infinities and NaN, zeros do (with NT = 2 both slots write
          // the same zeros: neither waits for the other)
          const int st = (vc + kt - wk.kt0) % L::VS;
          if (!(ok = wait_bar_warp(&bars[L::VFull + st], ((vc + kt - wk.kt0) / L::VS) & 1, abort_flag, budget))) break;
          if (j0 + r >= wk.it.keys) zero_row(sm + L::v + st * kTileBytes, r);
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(&bars[L::PFull + slot]);
      }
      if (!ok) break;
      // ---- the piece's result
      const int h = wk.ph * G + rg;
      const bool whole = wk.whole();
      const int64_t pslot = 2 * static_cast<int64_t>(blockIdx.x) + (at_start ? 0 : 1);
      at_start = false;
      if (!(ok = wait_bar_warp(&bars[L::OFull], n_piece & 1, abort_flag, budget))) break;
      tc_fence_after();
      if constexpr (NT == 2) {
        if (act) {
          const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
          const int64_t ooff = wk.pb * c.o_sb + static_cast<int64_t>(t) * c.o_ss + static_cast<int64_t>(h) * c.o_sh;
          const int64_t prow = pslot * P.part_rows + slot * tile_rows + r;
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
          const int64_t prow = pslot * P.part_rows + r;
          const uint32_t tOther = tmem + 256 + (slot ^ 1) * 128 + lane;
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            const int q4 = 2 * slot + q;
            uint32_t a[32], d[32];
            float y[32];
            tmem_ld32(tO + 32 * q4, a);
            tmem_ld32(tOther + 32 * q4, d);
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
  } else if (warp < kWarpQ0 + kQWarps) {
    // ---------------------------------------------------------------- Q rows
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    const int qt = tid - kWarpQ0 * 32;
    int n_piece = 0;
    while (wk.next<CL>(P, NT)) {
      if (n_piece > 0 && !wait_bar_warp(&bars[L::QEmpty], (n_piece - 1) & 1, abort_flag, budget)) break;
#pragma unroll 1
      for (int ti = 0; ti < NT; ++ti) {
        const int t0 = (wk.pm * NT + ti) * P.tpt;
        const int nv = max(0, min(P.tpt, wk.it.cnt - t0)) * G;     // rows that are there
        const int fill = ((nv + 31) & ~31) * 16;                   // whole warps of rows: zeros behind them
        uint8_t* tile = sm + L::q + ti * kTileBytes;
        for (int e = qt; e < fill; e += kQWarps * 32) {
          const int row = e >> 4, ch = e & 15, rr = row < nv ? row : 0;
          const int tt = t0 + rr / G, h = wk.ph * G + rr % G;
          cp_async16(tile + (ch >> 3) * kHalfBytes + sw128_off(row, ch & 7),
                     static_cast<const uint16_t*>(c.q.p) + wk.pb * c.q.sb + tt * c.q.ss + h * c.q.sh + 8 * ch, row < nv);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      mbar_arrive(&bars[L::QFull]);
      ++n_piece;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == kWarpK || warp == kWarpV) {
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
      bool ok = true, have = wk.next<CL>(P, NT);
      int kt = wk.kt0;
      Box box{false, 0, 0};
      if (have) box = find_box(P, wk, kt, lane_id);
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
          have = wk.next<CL>(P, NT);
          kt = wk.kt0;
        }
        if (have) box = find_box(P, wk, kt, lane_id);
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
      Walk ws = wk;
      bool ok = true, issued = false;
      int s_left = 0, s_kn = 0, s_next = 0, s_piece = -1, p_left = 0, p_kn = 0, p_next = 0, p_done = 0, p_piece = 0;
      // Enters the next piece: its first key tile and its number of tiles for
      // this slot (none, where NT = 1 and its only tile is the other slot's).
      auto enter = [&](Walk& w, int& kn, int& next, int& left) -> bool {
        if (!w.next<CL>(P, NT)) return false;
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
          if (!enter(ws, s_kn, s_next, s_left)) {
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
        issue_s<F16, 0, kHold>(tS, dQ, sdesc_add(dK0, (s_kn % L::KS) * kTileBytes));
        release();
        issue_s<F16, kHold, 8>(tS, dQ, sdesc_add(dK0, (s_kn % L::KS) * kTileBytes));
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
      while (ok && enter(wk, p_kn, p_next, p_left)) {
        for (int i = 0; i < p_left; ++i, ++p_done) {
          const bool same = s_left > 0;  // the next scores are of the same piece: Q is there
          if (same && !(ok = find_scores())) break;
          if (!(ok = wait_bar(&bars[L::VFull + p_kn % L::VS], (p_kn / L::VS) & 1, abort_flag, budget))) break;
          if (!(ok = wait_bar(&bars[L::PFull + slot], p_done & 1, abort_flag, budget))) break;
          ok = batch([&](auto&& release) {
            issue_pv<F16>(tO, tS, sdesc_add(dV0, (p_kn % L::VS) * kTileBytes), i > 0);
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
        make_uint2(pack_dt(c.kv.dt, o.x * inv, o.y * inv), pack_dt(c.kv.dt, o.z * inv, o.w * inv));
    if (lane == 0) c.lse[(static_cast<int64_t>(me.b) * c.H + h) * c.T + t] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

template <int NT, bool F16, bool TREE, bool CL>
cudaError_t launch_t(const TcAttnParams& p, cudaStream_t stream) {
  auto kern = tc_kernel<NT, F16, TREE, CL>;
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = opt_in_smem(kern, Lay<NT>::bytes, configured);
  if (e != cudaSuccess) return e;
  if constexpr (CL) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.cluster * p.c.kv.Hkv, p.c.B * p.n_groups);
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = Lay<NT>::bytes;
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
  return launch_chained(kern, dim3(p.ctas), dim3(kTcThreads), Lay<NT>::bytes, stream, p);
}
template <int NT, bool CL>
cudaError_t launch_nt(const TcAttnParams& p, bool f16, cudaStream_t stream) {
  if (p.c.parents) return f16 ? launch_t<NT, true, true, CL>(p, stream) : launch_t<NT, false, true, CL>(p, stream);
  return f16 ? launch_t<NT, true, false, CL>(p, stream) : launch_t<NT, false, false, CL>(p, stream);
}

}  // namespace

cudaError_t launch_cache_attn_tc(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream) {
  if (p.cluster > 0) return nt == 2 ? launch_nt<2, true>(p, f16, stream) : launch_nt<1, true>(p, f16, stream);
  return nt == 2 ? launch_nt<2, false>(p, f16, stream) : launch_nt<1, false>(p, f16, stream);
}

cudaError_t launch_cache_attn_join(const TcAttnParams& p, int nt, cudaStream_t stream) {
  // few rows, or few items, whose parts are then many
  const bool deep = p.part_rows <= 32 || static_cast<int64_t>(p.c.B) * p.c.kv.Hkv * p.n_groups * 4 <= p.ctas;
  return launch_chained(deep ? join_kernel<16> : join_kernel<4>, dim3(p.ctas - 1, (p.part_rows + kJoinRows - 1) / kJoinRows), dim3(256), 0, stream, p, nt);
}

}  // namespace st
