// Verification of drafted trees by speculative rejection sampling.
//
// Node 0 is the root (already part of the sequence). At the present node with
// target distribution p and draft distribution q its children are tried in
// index order, with residual weights
//   w_0 = p,  C_0 = 1,  a_0 = 0;   child with token x is accepted when
//   u q(x) C_k < w_k(x);  after a rejection
//   a_{k+1} = a_k + C_k,  w_{k+1}(v) = max(p(v) - a_{k+1} q(v), 0),
//   C_{k+1} = sum_v w_{k+1}(v)
// (w_k / C_k is the normalised residual distribution after k rejections: the
// normalising factors are folded into a). Without draft probabilities q is
// one-hot at the child's token: a rejection removes the token, C_{k+1} = C_k -
// p(x). When every child was rejected, or there is none, the next token is
// drawn from w by inverse CDF: the first v whose running sum exceeds
// u_sample * sum w.
//
// Weights are held as integers, 2^-43 a unit (rounded to nearest), and summed
// in integer arithmetic: sums do not depend on their order, so a row may be
// split over any number of threads and CTAs and the drawn token is the same. A
// running sum over V tokens is off by V 2^-44 at most, by about 2^-36 over 2^17
// tokens, whose roundings are independent. What is left of a row whose draft is
// close to its target sums to far less than 1, and loses its small weights in
// that unit: after a sum below 2^-12 (finish_small) the rest of the sequence is
// done with exact weights and a unit that goes by the sum.
//
// The walk is latency, the residual sums and the draw read two rows of V. One
// cluster of CTAs serves a sequence: each CTA gathers every node's two
// probabilities at once, walks redundantly (the same integers in every CTA),
// owns a slice of V in the sums, and exchanges its slice's total through
// distributed shared memory.
//
// 32 trees of 61 nodes over 131072 tokens in fp32 take 18 to 23 us (six sets of
// inputs) by the rejections of the longest walk: 7 for a walk without
// rejections (launch, gather, one sum of p, the draw), 2 for a first rejection's
// sum (a = 1), 5 for each further one and for the draw behind it; 16-bit
// probabilities take as long. The busiest SMs issue half of the time (about 45
// instructions for two weights of p - a q); the rest are waits for loads, the
// cluster's barriers and the walk. What was slower: the next batch's loads ahead
// of a batch's sums, in registers (spills, 26) or through shared memory (21); 512
// threads (25).
#include <type_traits>
#include "st_kernels.h"
#include "st_serve.h"

namespace st {

namespace {

constexpr int kVerThreads = 256;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kBatches = 64;    // batches of a warp's slice whose sums are kept for the draw (further ones are read again)
constexpr int kRowBatch = 16;  // rows of 32 probabilities whose loads are issued together
constexpr float kUnit = 1.0f / 8796093022208.0f;       // 2^-43, the unit of a weight
constexpr unsigned long long kOne = 8796093022208ull;  // 1 in it

// The type is the kernel's template argument: a branch on it per element would
// keep the loads of a batch from being issued together (60000 cycles for a sum
// that takes 2500).
template <int DT>
__device__ __forceinline__ float prob(const void* p, int64_t e) {
  float v;
  if constexpr (DT == kDtF32) v = ld_now(static_cast<const float*>(p) + e);
  else if constexpr (DT == kDtBF16) v = __bfloat162float(ld_now(static_cast<const __nv_bfloat16*>(p) + e));
  else v = __half2float(ld_now(static_cast<const __half*>(p) + e));
  return __saturatef(v);  // [0, 1]; NaN: 0
}
// Four neighbours that start on four elements, in one load.
template <int DT>
__device__ __forceinline__ void prob4(const void* p, int64_t e, float* v) {
  if constexpr (DT == kDtF32) {
    const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
    v[0] = __saturatef(x.x), v[1] = __saturatef(x.y), v[2] = __saturatef(x.z), v[3] = __saturatef(x.w);
  } else {
    const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + e);
    const uint32_t w[2] = {x.x, x.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float2 y;
      if constexpr (DT == kDtBF16) y = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      else y = __half22float2(__halves2half2(__ushort_as_half(static_cast<unsigned short>(w[i])), __ushort_as_half(static_cast<unsigned short>(w[i] >> 16))));
      v[2 * i] = __saturatef(y.x), v[2 * i + 1] = __saturatef(y.y);
    }
  }
}
// A value in [-1, 1] as two integer limbs of 21 and 22 bits, value =
// (hi 2^22 + lo) 2^-43 rounded to nearest. Adding 1.5 * 2^(23 - b) leaves the
// multiple of 2^-b in the low significand bits; what it rounded off is exact
// and goes through the same step (a 64-bit conversion per element, or shifts,
// cost twice the instructions of the rest of the sum).
constexpr float kHi = 1.5f * 4.0f;                    // 1.5 * 2^(23 - 21)
constexpr float kLo = 1.5f * 9.5367431640625e-7f;     // 1.5 * 2^(23 - 43)
struct Limbs {  // of two values, modulo 2^32; kHi's and kLo's own bits are still in them
  uint32_t hi, lo;
};
__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 less(float2 x, float2 y) { return __ffma2_rn(y, pair(-1.f), x); }  // x - y, without negating y first
__device__ __forceinline__ Limbs limbs(float2 v, float2 tail) {  // of v + tail, |tail| <= 2^-23; both values added up
  const float2 t = __fadd2_rn(v, pair(kHi));
  const float2 rem = __fadd2_rn(less(v, __fadd2_rn(t, pair(-kHi))), tail);
  const float2 l = __fadd2_rn(rem, pair(kLo));
  return {__float_as_uint(t.x) + __float_as_uint(t.y), __float_as_uint(l.x) + __float_as_uint(l.y)};
}
// The limbs of max(p - a q, 0). a = 0 and a = 1 (before and after the first
// rejection) need no product; else a = ah + al and the product is s with the
// error r. For s <= p the difference d of p and s has the error (p - d) - s
// exactly; for p < s <= 2 p it is exact, and that term 0; beyond it is below
// -s/2 and its sign stands whatever the error.
struct Scale {
  float ah, al;
};
// A sum in two floats. (fp64 arithmetic would serve, at a hundredth of the rate:
// a wave of it in every warp costs 1 us a turn.)
__device__ __forceinline__ Scale split(unsigned long long x) {
  const float h = __ull2float_rn(x);
  const long long rest = static_cast<long long>(x - __float2ull_rn(h));
  return {h * kUnit, __ll2float_rn(rest) * kUnit};
}
template <int A>  // 0: a = 0; 1: a = 1; 2: any a
__device__ __forceinline__ Limbs weight(float2 p, float2 q, Scale a) {
  if constexpr (A == 0) return limbs(p, pair(0.f));
  if constexpr (A == 1) {
    const float2 s = make_float2(fminf(p.x, q.x), fminf(p.y, q.y));
    const float2 d = less(p, s);
    return limbs(d, less(less(p, d), s));
  }
  const float2 ns = __fmul2_rn(q, pair(-a.ah)), r = __ffma2_rn(q, pair(a.ah), ns);
  float2 d = __fadd2_rn(p, ns);
  float2 e = __ffma2_rn(q, pair(-a.al), less(__fadd2_rn(less(p, d), ns), r));
  const float2 x = __fadd2_rn(d, e);
  d = make_float2(x.x > 0.f ? d.x : 0.f, x.y > 0.f ? d.y : 0.f);
  e = make_float2(x.x > 0.f ? e.x : 0.f, x.y > 0.f ? e.y : 0.f);
  return limbs(d, e);
}
// u q C < max(p - a q, 0), the acceptance of a child with siblings rejected
// before: both sides in two floats, the differences of their parts added up.
__device__ __forceinline__ bool accepts(float u, float p, float q, Scale a, Scale c) {
  const float s = __fmul_rn(a.ah, q), d = __fsub_rn(p, s);
  const float e = __fmaf_rn(-a.al, q, __fsub_rn(__fsub_rn(__fsub_rn(p, d), s), __fmaf_rn(a.ah, q, -s)));
  const float t = __fmul_rn(u, q), t2 = __fmaf_rn(u, q, -t), w = __fmul_rn(t, c.ah);
  const float w2 = __fadd_rn(__fmaf_rn(t, c.ah, -w), __fmaf_rn(t, c.al, __fmul_rn(t2, c.ah)));
  return __fadd_rn(d, e) > 0.f && __fadd_rn(__fsub_rn(w, d), __fsub_rn(w2, e)) < 0.f;
}
constexpr uint32_t kPairHi = 2u * 0x40c00000u, kPairLo = 2u * 0x35c00000u;  // kHi's and kLo's bits, twice
__device__ __forceinline__ unsigned long long whole(uint32_t hi, uint32_t lo) {
  return static_cast<unsigned long long>(static_cast<long long>(static_cast<int>(hi)) * 4194304 + static_cast<int>(lo));
}
__device__ __forceinline__ unsigned long long fix(float v) {
  const Limbs x = limbs(make_float2(v, 0.f), make_float2(0.f, 0.f));
  return whole(x.hi - kPairHi, x.lo - kPairLo);
}
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

struct VerState {
  int par[kMaxVerify], tok[kMaxVerify];
  float pp[kMaxVerify], qq[kMaxVerify], uu[kMaxVerify];
  bool first_yes[kMaxVerify];    // accepted when no sibling was rejected before it
  int path[kMaxVerify];
  unsigned long long warp_tot[kVerWarps];
  unsigned long long batch_tot[kVerWarps][kBatches];
  unsigned long long cta_tot[2][kMaxClusterVerify];  // by the parity of the exchange
  int rejected[kMaxVerify];      // of the node where the walk ended, without draft probabilities
};

// The tokens of a warp's slice of V, rounded up to whole rows of 32.
__device__ __forceinline__ int slice_of(int V, int C) { return ((V + C * kVerWarps - 1) / (C * kVerWarps) + 31) & ~31; }
// The next child of `cur` behind node `from`, or cnt; by a whole warp.
__device__ __forceinline__ int next_child(const VerState& s, int cur, int from, int cnt) {
  const int lane = threadIdx.x & 31;
  for (int base = from + 1; base < cnt; base += 32) {
    const int i = base + lane;
    const unsigned m = __ballot_sync(0xffffffffu, i < cnt && s.par[i] == cur);
    if (m) return base + __ffs(m) - 1;
  }
  return cnt;
}
// floor(u_sample * total): the draw takes the first token whose running sum is above it.
__device__ __forceinline__ unsigned long long draw_at(const VerifyParams& P, int b, unsigned long long total) {
  const float us = fminf(fmaxf(ld_now(P.u_sample + b), 0.f), 1.f);
  // u in 2^-64 units (below 1), so that the result is below total
  const unsigned long long u64 = us >= 1.f ? ~0ull : __double2ull_rz(static_cast<double>(us) * 18446744073709551616.0);
  return __umul64hi(u64, total);
}
__device__ __forceinline__ void put_token(const VerifyParams& P, int b, int token) {
  if (P.tok64) static_cast<long long*>(P.next_token)[b] = token;
  else static_cast<int32_t*>(P.next_token)[b] = token;
}

// ------------------------------------------------------ residuals of small sums
// The rest of a sequence's walk and its draw once a residual has summed to less
// than kSmall units, from the present node's first child on: what the ordinary
// sums rounded off weighs in such a residual. Weights are to the last bit that
// fp64 gives, in the unit 2^-(43 + shift), with shift raised until the sum has
// kEnough units or nothing is left; a raise leaves room for what was rounded off
// before, V / 2 units. Residuals only shrink from one rejection to the next, so a
// node's shift stays good. A function of its own and plain code, as few sequences
// need it (a first residual below 2^-12 means that less than one guess in 4096 was
// rejected): built into the ordinary passes it cost all of them 6 to 8%, as it is
// 0.15 us of a chain's 5.9. 24 sequences over 131072 tokens take 45 us with
// one such rejection and 75 more with each further one (fp64), 13 with ordinary
// residuals.
constexpr unsigned long long kSmall = 1ull << 31, kEnough = 1ull << 50;
constexpr int kFineBatch = 8;
constexpr int kShiftFirst = -16, kShiftMost = 125;   // rows of any sum up to 2^30; 2^-168: fp32's smallest number is 2^-149
constexpr int kRoom = 59;                            // a CTA's and the row's sums stay below 2^59
constexpr unsigned long long kAnyLeft = 1ull << 60;  // in a CTA's total: it has weights above 0

// `n` nodes being accepted, the last of them `cur`; without draft probabilities
// its children are done with and n_rej tokens removed. The small sum was `found`,
// at `found_a`. `parity`: of the next exchange. Returns the accepted nodes and
// writes the token.
template <int DT>
__device__ __noinline__ int finish_small(const VerifyParams& P, VerState& s, int b, int rank, int cnt, int cur, int n, int n_rej,
                                         unsigned long long found_a, unsigned long long found, int parity) {
  const int C = P.cluster, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, V = P.V, sub = slice_of(V, C);
  const bool drafted = P.q != nullptr;
  const int64_t lo = static_cast<int64_t>(rank * kVerWarps + warp) * sub, end = min(lo + sub, static_cast<int64_t>(V));  // the warp's slice
  const int found_at = cur, found_rej = n_rej;
  double a = 0.0, c = 1.0;
  int shift = kShiftFirst;
  auto raise = [&](unsigned long long total) {  // for a sum of `total` units
    shift = min(shift + kRoom - (64 - __clzll(static_cast<long long>(total + V / 2 + 1))), kShiftMost);
  };
  // tokens v0 + 32 u of the row of node `cur`, their loads in flight together, in
  // units. Returns whether any is above 0. a = 0 and a = 1 need no fp64: p - min(p, q)
  // is a float and its error.
  auto batch = [&](int64_t v0, unsigned long long (&x)[kFineBatch]) {
    const int64_t pe = b * P.p_sb + cur * P.p_st, qe = b * P.q_sb + cur * P.q_st;
    const bool with_q = drafted && a != 0.0, plain = shift <= 80 && (!with_q || a == 1.0);
    float pv[kFineBatch], qv[kFineBatch];
#pragma unroll
    for (int u = 0; u < kFineBatch; ++u) {
      const int64_t v = min(v0 + 32 * u, end - 1);
      pv[u] = prob<DT>(P.p, pe + v);
      qv[u] = with_q ? prob<DT>(P.q, qe + v) : 0.f;
    }
    for (int r = 0; r < n_rej; ++r) {
      const int64_t gone = s.tok[s.rejected[r]] - v0;
#pragma unroll
      for (int u = 0; u < kFineBatch; ++u)
        if (gone == 32 * u) pv[u] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < kFineBatch; ++u)
      if (v0 + 32 * u >= end) pv[u] = 0.f;  // weighs nothing, whatever q
    bool any = false;
    if (plain) {
      const float scale = scalbnf(1.f, 43 + shift);
#pragma unroll
      for (int u = 0; u < kFineBatch; ++u) {
        const float m = fminf(pv[u], qv[u]), d = __fsub_rn(pv[u], m), e = __fsub_rn(__fsub_rn(pv[u], d), m);
        x[u] = __float2ull_rn(d * scale) + static_cast<unsigned long long>(__float2ll_rn(e * scale));
        any |= d > 0.f;
      }
    } else {
      const double scale = scalbn(1.0, 43 + shift);
#pragma unroll
      for (int u = 0; u < kFineBatch; ++u) {
        const double w = fmax(fma(-a, static_cast<double>(qv[u]), static_cast<double>(pv[u])), 0.0);
        x[u] = static_cast<unsigned long long>(__double2ll_rn(w * scale));
        any |= w > 0.0;
      }
    }
    return any;
  };
  // the sum over the row of node `cur`; the warps' totals stay in s.warp_tot, the CTAs' in s.cta_tot[parity ^ 1]
  auto sum_row = [&]() -> unsigned long long {
    if (shift == kShiftFirst && cur == found_at && n_rej == found_rej && a == static_cast<double>(found_a) * kUnit) {  // that very sum
      shift = 0;
      raise(found);
    }
    while (true) {
      unsigned long long acc = 0;
      bool any = false;
      for (int64_t v0 = lo + lane; v0 < end; v0 += 32 * kFineBatch) {
        unsigned long long x[kFineBatch];
        any |= batch(v0, x);
#pragma unroll
        for (int u = 0; u < kFineBatch; ++u) acc += x[u];
      }
      acc = warp_sum(acc);
      if (lane == 0) s.warp_tot[warp] = acc;
      any = __syncthreads_or(any) != 0;
      unsigned long long cta = any ? kAnyLeft : 0;
      for (int w = 0; w < kVerWarps; ++w) cta += s.warp_tot[w];
      if (C == 1) {
        if (tid == 0) s.cta_tot[parity][0] = cta;
        __syncthreads();
      } else {
        if (tid < C) st_cluster_u64(mapa_shared(smem_u32(&s.cta_tot[parity][rank]), tid), cta);
        cluster_sync();
      }
      unsigned long long total = 0;
      for (int r = 0; r < C; ++r) total += s.cta_tot[parity][r];
      const bool left = total >= kAnyLeft;
      total &= kAnyLeft - 1;
      parity ^= 1;
      if (total >= kEnough || !left || shift >= kShiftMost) return total;
      raise(total);
    }
  };
  for (int i = drafted ? next_child(s, cur, cur, cnt) : cnt; i < cnt;) {
    const double px = s.pp[i], qx = s.qq[i];
    const bool yes = static_cast<double>(s.uu[i]) * qx * c < fmax(fma(-a, qx, px), 0.0);
    const int last = i;
    if (yes) {
      if (tid == 0) s.path[n] = i;
      cur = i;
      ++n;
      a = 0.0;
      c = 1.0;
      shift = kShiftFirst;
    } else {
      a += c;
    }
    i = next_child(s, cur, last, cnt);
    if (!yes && i < cnt) {
      const unsigned long long total = sum_row();  // which may raise the shift
      c = scalbn(static_cast<double>(total), -43 - shift);
    }
  }
  unsigned long long total = sum_row();
  if (total == 0) {  // p <= a q everywhere: the target's own distribution
    a = 0.0;
    shift = kShiftFirst;
    n_rej = 0;
    total = sum_row();
  }
  if (total == 0) {
    if (rank == 0 && tid == 0) put_token(P, b, -1);
    return n;
  }
  const unsigned long long thr = draw_at(P, b, total);
  unsigned long long run = 0;
  for (int r = 0; r < rank; ++r) run += s.cta_tot[parity ^ 1][r] & (kAnyLeft - 1);
  for (int w = 0; w < warp; ++w) run += s.warp_tot[w];
  if (thr < run || thr >= run + s.warp_tot[warp]) return n;
  // one warp of the cluster: 32 tokens at a time
  for (int64_t v0 = lo; v0 < end && thr >= run; v0 += 32 * kFineBatch) {
    unsigned long long y[kFineBatch];
    batch(v0 + lane, y);
#pragma unroll
    for (int u = 0; u < kFineBatch; ++u) {
      unsigned long long inc = y[u];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
      }
      if (thr >= run + inc - y[u] && thr < run + inc) put_token(P, b, static_cast<int>(v0) + 32 * u + lane);  // one thread
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  return n;
}

template <int DT>
__global__ void __launch_bounds__(kVerThreads, 2) verify_kernel(const __grid_constant__ VerifyParams P) {
  __shared__ VerState s;
  grid_dependency_wait();
  const int C = P.cluster, rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int b = blockIdx.x / C, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cnt = row_count(P.counts, b, P.T);
  const int V = P.V;
  const bool drafted = P.q != nullptr;

  for (int i = tid; i < cnt; i += kVerThreads) {
    const int64_t te = b * P.tok_sb + i * P.tok_st;
    const int64_t t64 = P.tok64 ? ld_now(static_cast<const long long*>(P.tokens) + te) : ld_now(static_cast<const int32_t*>(P.tokens) + te);
    const int par = ld_now(P.parents + b * P.par_sb + i);
    const bool ok = i > 0 && par >= 0 && par < i && t64 >= 0 && t64 < V;
    // the root has no parent; -1 stands for a node that nothing leads to
    if (!ok && (i > 0 ? (par >= i || par < -1 || t64 < 0 || t64 >= V) : par >= 0) && rank == 0) atomicOr(P.status, kStatusIndex);
    const int x = ok ? static_cast<int>(t64) : 0;
    s.par[i] = ok ? par : -2;
    s.tok[i] = x;
    s.pp[i] = ok ? prob<DT>(P.p, b * P.p_sb + par * P.p_st + x) : 0.f;
    s.qq[i] = ok && drafted ? prob<DT>(P.q, b * P.q_sb + par * P.q_st + x) : 1.f;
    s.uu[i] = ok ? ld_now(P.u_accept + static_cast<int64_t>(b) * P.T + i) : 0.f;
    s.first_yes[i] = static_cast<double>(s.uu[i]) * s.qq[i] < static_cast<double>(s.pp[i]);
  }
  if (tid == 0) s.path[0] = 0;
  // also: every CTA of the cluster runs before another writes into its memory
  if (C > 1) cluster_sync();
  else __syncthreads();

  // slice of V of this CTA, and of each warp of it
  const int sub = slice_of(V, C);
  const int64_t lo64 = static_cast<int64_t>(rank * kVerWarps + warp) * sub;
  const int w_lo = static_cast<int>(min(lo64, static_cast<int64_t>(V))), w_hi = static_cast<int>(min(lo64 + sub, static_cast<int64_t>(V)));
  int parity = 0;

  // kRowBatch x 32 probabilities from v0 on, all loads in flight together; a
  // whole batch takes constant offsets from one address, and four tokens per
  // load where its rows allow it (sums do not care which thread has which)
  auto load_rows = [&](int64_t pe, int64_t qe, bool wide, int v0, auto with_q, float (&pv)[kRowBatch], float (&qv)[kRowBatch]) {
    constexpr bool Q = decltype(with_q)::value;
    if (v0 + 32 * kRowBatch <= w_hi && wide) {
#pragma unroll
      for (int u = 0; u < kRowBatch; u += 4) {
        prob4<DT>(P.p, pe + v0 + 4 * lane + 32 * u, pv + u);
        if (Q) prob4<DT>(P.q, qe + v0 + 4 * lane + 32 * u, qv + u);
      }
      return;
    }
    if (v0 + 32 * kRowBatch <= w_hi) {
#pragma unroll
      for (int u = 0; u < kRowBatch; ++u) {
        pv[u] = prob<DT>(P.p, pe + v0 + lane + 32 * u);
        qv[u] = Q ? prob<DT>(P.q, qe + v0 + lane + 32 * u) : 0.f;
      }
      return;
    }
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) {
      const int v = min(v0 + 32 * u + lane, w_hi - 1);  // no branch around a load
      pv[u] = prob<DT>(P.p, pe + v);
      qv[u] = Q ? prob<DT>(P.q, qe + v) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u)
      if (v0 + 32 * u + lane >= w_hi) pv[u] = 0.f;  // weighs nothing, whatever q
  };

  // sum over V of the residual weights of node `cur` at `a`, less the removed
  // tokens; leaves the warps' totals in s.warp_tot and the CTAs' in s.cta_tot
  auto sum_row = [&](int cur, unsigned long long a, int removed, bool keep) -> unsigned long long {
    const int64_t pe = b * P.p_sb + cur * P.p_st, qe = b * P.q_sb + cur * P.q_st;
    unsigned long long acc = 0;
    constexpr int kSize = DT == kDtF32 ? 4 : 2;
    const bool wide = ((reinterpret_cast<uintptr_t>(P.p) + pe * kSize) | (drafted ? reinterpret_cast<uintptr_t>(P.q) + qe * kSize : 0)) % (4 * kSize) == 0;
    const Scale sc = split(a);
    auto pass = [&](auto kind) {
      constexpr int A = decltype(kind)::value;
      for (int v0 = w_lo; v0 < w_hi; v0 += 32 * kRowBatch) {
        float pv[kRowBatch], qv[kRowBatch];
        load_rows(pe, qe, wide, v0, std::integral_constant<bool, A != 0>(), pv, qv);
        uint32_t hi = 0, lo = 0;  // modulo 2^32: the sums of 16 limbs are far below it
#pragma unroll
        for (int u = 0; u < kRowBatch; u += 2) {
          const Limbs x = weight<A>(make_float2(pv[u], pv[u + 1]), make_float2(qv[u], qv[u + 1]), sc);
          hi += x.hi;
          lo += x.lo;
        }
        unsigned long long part = whole(hi - kRowBatch / 2 * kPairHi, lo - kRowBatch / 2 * kPairLo);
        if (keep) {  // the batches' own sums, where the draw will look
          const int batch = (v0 - w_lo) / (32 * kRowBatch);
          if (batch < kBatches) {
            part = warp_sum(part);
            if (lane == 0) s.batch_tot[warp][batch] = part;
            if (lane != 0) part = 0;
          }
        }
        acc += part;
      }
    };
    if (!drafted || a == 0) pass(std::integral_constant<int, 0>());
    else if (a == kOne) pass(std::integral_constant<int, 1>());
    else pass(std::integral_constant<int, 2>());
    acc = warp_sum(acc);
    if (lane == 0) s.warp_tot[warp] = acc;
    __syncthreads();
    if (removed > 0) {
      for (int r = tid; r < removed; r += kVerThreads) {
        const int x = s.tok[s.rejected[r]], w = x / sub - rank * kVerWarps;
        if (w >= 0 && w < kVerWarps) {
          const unsigned long long f = 0ull - fix(s.pp[s.rejected[r]]);
          atomicAdd(&s.warp_tot[w], f);
          const int batch = x % sub / (32 * kRowBatch);
          if (keep && batch < kBatches) atomicAdd(&s.batch_tot[w][batch], f);
        }
      }
      __syncthreads();
    }
    unsigned long long cta = 0;
    for (int w = 0; w < kVerWarps; ++w) cta += s.warp_tot[w];
    if (C == 1) {
      if (tid == 0) s.cta_tot[parity][0] = cta;
      __syncthreads();
    } else {
      if (tid < C) st_cluster_u64(mapa_shared(smem_u32(&s.cta_tot[parity][rank]), tid), cta);
      cluster_sync();
    }
    unsigned long long total = 0;
    for (int r = 0; r < C; ++r) total += s.cta_tot[parity][r];
    return total;
  };

  // the walk, by every warp for itself
  int cur = 0, n = cnt > 0 ? 1 : 0, n_rej = 0;
  unsigned long long a = 0, c = kOne;  // a and C, in 2^-43
  double left = 1.0;                   // C without draft probabilities
  // a child of `cur` before node i has i's token
  auto tried = [&](int i) {
    bool again = false;
    for (int base = 0; base < i; base += 32) again |= base + lane < i && s.par[base + lane] == cur && s.tok[base + lane] == s.tok[i];
    return __any_sync(0xffffffffu, again) != 0;
  };
  bool small = false;                  // a residual's sum was too small for the unit
  int i = next_child(s, cur, 0, cnt);
  while (i < cnt) {
    const float u = s.uu[i], px = s.pp[i], qx = s.qq[i];
    const bool again = !drafted && n_rej > 0 && tried(i);  // a token that was already removed here
    bool yes;
    if (drafted)
      yes = a == 0 ? s.first_yes[i] : accepts(u, px, qx, split(a), split(c));
    else
      yes = !again && (n_rej == 0 ? s.first_yes[i] : static_cast<double>(u) * left < static_cast<double>(px));
    const int last = i;
    if (yes) {
      cur = i;
      if (tid == 0) s.path[n] = i;
      ++n;
      a = 0;
      c = kOne;
      left = 1.0;
      n_rej = 0;
      i = next_child(s, cur, last, cnt);
      continue;
    }
    i = next_child(s, cur, last, cnt);
    if (drafted) {
      a += c;
      if (i < cnt) {  // the next sibling needs the residual's sum
        c = sum_row(cur, a, 0, false);
        parity ^= 1;
        if ((small = c < kSmall)) break;
      }
    } else if (!again) {
      left -= px;
      if (tid == 0) s.rejected[n_rej] = last;
      ++n_rej;
    }
  }

  // the draw
  if (cnt > 0) {
    unsigned long long total = c;
    if (!small) {
      total = sum_row(cur, a, n_rej, true);
      if ((small = total < kSmall)) parity ^= 1;
    }
    if (small) {
      n = finish_small<DT>(P, s, b, rank, cnt, cur, n, n_rej, a, total, parity);
    } else {
      const unsigned long long thr = draw_at(P, b, total);
      unsigned long long run = 0;
      for (int r = 0; r < rank; ++r) run += s.cta_tot[parity][r];
      if (thr >= run && thr < run + s.cta_tot[parity][rank]) {  // one CTA of the cluster
        const int64_t pe = b * P.p_sb + cur * P.p_st, qe = b * P.q_sb + cur * P.q_st;
        const Scale sc = split(a);
        // the slice, then the batch, that holds it, by their sums
        int w = 0;
        while (w < kVerWarps - 1 && run + s.warp_tot[w] <= thr) run += s.warp_tot[w++];
        const int64_t lo = static_cast<int64_t>(rank * kVerWarps + w) * sub;
        const int end = static_cast<int>(min(lo + sub, static_cast<int64_t>(V)));
        int v0 = static_cast<int>(min(lo, static_cast<int64_t>(V)));
        for (int k = 0; k < kBatches && v0 < end && run + s.batch_tot[w][k] <= thr; ++k, v0 += 32 * kRowBatch) run += s.batch_tot[w][k];
        __syncthreads();  // warp_tot serves the scans below
        // two neighbours per thread: a batch at a time, usually one
        auto find = [&](auto kind) {
          constexpr int A = decltype(kind)::value;
          static_assert(32 * kRowBatch == 2 * kVerThreads, "two tokens per thread");
          for (bool found = false; v0 < end && !found; v0 += 32 * kRowBatch) {
            unsigned long long x[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int e = v0 + 2 * tid + u, i = min(e, end - 1);
              const Limbs y = weight<A>(make_float2(prob<DT>(P.p, pe + i), 0.f), make_float2(A != 0 ? prob<DT>(P.q, qe + i) : 0.f, 0.f), sc);
              x[u] = e < end ? whole(y.hi - kPairHi, y.lo - kPairLo) : 0ull;
              if (A == 0)
                for (int r = 0; r < n_rej; ++r)
                  if (s.tok[s.rejected[r]] == e) x[u] = 0;
            }
            unsigned long long inc = x[0] + x[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const unsigned long long t = __shfl_up_sync(0xffffffffu, inc, o);
              if (lane >= o) inc += t;
            }
            if (lane == 31) s.warp_tot[warp] = inc;
            __syncthreads();
            unsigned long long at = run + inc - x[0] - x[1], all = 0;
            for (int i = 0; i < kVerWarps; ++i) {
              if (i < warp) at += s.warp_tot[i];
              all += s.warp_tot[i];
            }
            if (thr >= at && thr < at + x[0] + x[1]) {  // one thread
              put_token(P, b, v0 + 2 * tid + (thr < at + x[0] ? 0 : 1));
            }
            found = thr < run + all;
            run += all;
            __syncthreads();
          }
        };
        if (!drafted || a == 0) find(std::integral_constant<int, 0>());
        else if (a == kOne) find(std::integral_constant<int, 1>());
        else find(std::integral_constant<int, 2>());
      }
    }
  } else if (rank == 0 && tid == 0) {
    put_token(P, b, -1);
  }
  if (rank == 0) {
    for (int i = tid; i < P.T; i += kVerThreads) P.path[static_cast<int64_t>(b) * P.T + i] = i < n ? s.path[i] : -1;
    if (tid == 0) P.n_accepted[b] = n;
  }
}

}  // namespace

cudaError_t launch_tree_verify(const VerifyParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.cluster);
  cfg.blockDim = dim3(kVerThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  switch (p.dt) {
    case kDtF32: return cudaLaunchKernelEx(&cfg, verify_kernel<kDtF32>, p);
    case kDtBF16: return cudaLaunchKernelEx(&cfg, verify_kernel<kDtBF16>, p);
    default: return cudaLaunchKernelEx(&cfg, verify_kernel<kDtF16>, p);
  }
}

}  // namespace st
