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
// running sum over 2^17 tokens is off by about 2^-37 of the total.
//
// The walk is latency, the residual sums and the draw read two rows of V. One
// cluster of CTAs serves a sequence: each CTA gathers every node's two
// probabilities at once, walks redundantly (the same integers in every CTA),
// owns a slice of V in the sums, and exchanges its slice's total through
// distributed shared memory.
#include <type_traits>
#include "st_kernels.h"
#include "st_serve.h"

namespace st {

namespace {

constexpr int kVerThreads = 256;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kRowBatch = 16;  // rows of 32 probabilities whose loads are issued together
constexpr double kUnit = 1.0 / 8796093022208.0;  // 2^-43, the unit of a weight

// The type is the kernel's template argument: a branch on it per element would
// keep the loads of a batch from being issued together (60000 cycles for a sum
// that takes 2500).
template <int DT>
__device__ __forceinline__ float prob(const void* p, int64_t e) {
  float v;
  if constexpr (DT == kDtF32) v = __ldg(static_cast<const float*>(p) + e);
  else if constexpr (DT == kDtBF16) v = __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + e));
  else v = __half2float(__ldg(static_cast<const __half*>(p) + e));
  return __saturatef(v);  // [0, 1]; NaN: 0
}
// A value in [-1, 1] as two integer limbs of 21 and 22 bits, value =
// (hi 2^22 + lo) 2^-43 rounded to nearest. Adding 1.5 * 2^(23 - b) leaves the
// multiple of 2^-b in the low significand bits; what it rounded off is exact
// and goes through the same step (a 64-bit conversion per element, or shifts,
// cost twice the instructions of the rest of the sum).
constexpr float kHi = 1.5f * 4.0f;                    // 1.5 * 2^(23 - 21)
constexpr float kLo = 1.5f * 9.5367431640625e-7f;     // 1.5 * 2^(23 - 43)
struct Limbs {
  int hi, lo;
};
__device__ __forceinline__ Limbs limbs(float v, float tail = 0.f) {  // of v + tail, |tail| <= 2^-23
  const float t = __fadd_rn(v, kHi);
  const float rem = __fadd_rn(__fsub_rn(v, __fsub_rn(t, kHi)), tail);
  Limbs r;
  r.hi = __float_as_int(t) - __float_as_int(kHi);
  r.lo = __float_as_int(__fadd_rn(rem, kLo)) - __float_as_int(kLo);
  return r;
}
// The limbs of max(p - a q, 0). a = 0 and a = 1 (before and after the first
// rejection) need no product; else a = ah + al and the product is carried with
// its rounding error.
struct Scale {
  float ah, al;
};
template <int A>  // 0: a = 0; 1: a = 1; 2: any a
__device__ __forceinline__ Limbs weight(float p, float q, Scale a) {
  if constexpr (A == 0) return limbs(p);
  Limbs r{0, 0};
  if constexpr (A == 1) {
    const Limbs x = limbs(p), y = limbs(q);
    if (p > q) {
      r.hi = x.hi - y.hi;
      r.lo = x.lo - y.lo;
    }
  } else {
    const float sh = __fmul_rn(a.ah, q), sl = __fmaf_rn(a.al, q, __fmaf_rn(a.ah, q, -sh));
    const float d = __fsub_rn(p, sh), bb = __fsub_rn(p, d);          // d + e = p - sh exactly
    const float e = __fsub_rn(__fsub_rn(bb, sh), sl) + __fsub_rn(p, __fadd_rn(d, bb));
    if (__fadd_rn(d, e) > 0.f && d <= 1.f) r = limbs(d, e);
  }
  return r;
}
__device__ __forceinline__ unsigned long long whole(int hi, int lo) {
  return static_cast<unsigned long long>((static_cast<long long>(hi) << 22) + lo);
}
__device__ __forceinline__ unsigned long long fix(float v) {
  const Limbs x = limbs(v);
  return whole(x.hi, x.lo);
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
  unsigned long long cta_tot[2][kMaxClusterVerify];  // by the parity of the exchange
  int rejected[kMaxVerify];
  int n_rejected;
  int cur, n_path, more;         // more: a rejected child has a sibling left
  double a;
};

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
    const int64_t t64 = P.tok64 ? __ldg(static_cast<const long long*>(P.tokens) + te) : __ldg(static_cast<const int32_t*>(P.tokens) + te);
    const int par = __ldg(P.parents + b * P.par_sb + i);
    const bool ok = i > 0 && par >= 0 && par < i && t64 >= 0 && t64 < V;
    // the root has no parent; -1 stands for a node that nothing leads to
    if (!ok && (i > 0 ? (par >= i || par < -1 || t64 < 0 || t64 >= V) : par >= 0) && rank == 0) atomicOr(P.status, kStatusIndex);
    const int x = ok ? static_cast<int>(t64) : 0;
    s.par[i] = ok ? par : -2;
    s.tok[i] = x;
    s.pp[i] = ok ? prob<DT>(P.p, b * P.p_sb + par * P.p_st + x) : 0.f;
    s.qq[i] = ok && drafted ? prob<DT>(P.q, b * P.q_sb + par * P.q_st + x) : 1.f;
    s.uu[i] = ok ? __ldg(P.u_accept + static_cast<int64_t>(b) * P.T + i) : 0.f;
    s.first_yes[i] = static_cast<double>(s.uu[i]) * s.qq[i] < static_cast<double>(s.pp[i]);
  }
  if (tid == 0) {
    s.cur = 0;
    s.n_path = cnt > 0 ? 1 : 0;
    s.path[0] = 0;
    s.n_rejected = 0;
  }
  // also: every CTA of the cluster runs before another writes into its memory
  if (C > 1) cluster_sync();
  else __syncthreads();

  // slice of V of this CTA, and of each warp of it
  const int sub = ((V + C * kVerWarps - 1) / (C * kVerWarps) + 31) & ~31;
  const int64_t lo64 = static_cast<int64_t>(rank * kVerWarps + warp) * sub;
  const int w_lo = static_cast<int>(min(lo64, static_cast<int64_t>(V))), w_hi = static_cast<int>(min(lo64 + sub, static_cast<int64_t>(V)));
  int parity = 0;

  // kRowBatch x 32 probabilities from v0 on, all loads in flight together
  auto load_rows = [&](int64_t pe, int64_t qe, int v0, bool with_q, float (&pv)[kRowBatch], float (&qv)[kRowBatch]) {
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) {
      const int v = min(v0 + 32 * u + lane, w_hi - 1);  // no branch around a load
      pv[u] = prob<DT>(P.p, pe + v);
      qv[u] = with_q ? prob<DT>(P.q, qe + v) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u)
      if (v0 + 32 * u + lane >= w_hi) pv[u] = 0.f;  // weighs nothing, whatever q
  };
  // sum over V of the residual weights of node `cur` at `a`, less the removed
  // tokens; leaves the warps' totals in s.warp_tot and the CTAs' in s.cta_tot
  auto sum_row = [&](int cur, double a, bool removed) -> unsigned long long {
    const int64_t pe = b * P.p_sb + cur * P.p_st, qe = b * P.q_sb + cur * P.q_st;
    unsigned long long acc = 0;
    const Scale sc{static_cast<float>(a), static_cast<float>(a - static_cast<float>(a))};
    auto pass = [&](auto kind) {
      constexpr int A = decltype(kind)::value;
      for (int v0 = w_lo; v0 < w_hi; v0 += 32 * kRowBatch) {
        float pv[kRowBatch], qv[kRowBatch];
        load_rows(pe, qe, v0, A != 0, pv, qv);
        int hi = 0, lo = 0;
#pragma unroll
        for (int u = 0; u < kRowBatch; ++u) {
          const Limbs x = weight<A>(pv[u], qv[u], sc);
          hi += x.hi;
          lo += x.lo;
        }
        acc += whole(hi, lo);
      }
    };
    if (!drafted || a == 0.0) pass(std::integral_constant<int, 0>());
    else if (a == 1.0) pass(std::integral_constant<int, 1>());
    else pass(std::integral_constant<int, 2>());
    acc = warp_sum(acc);
    if (lane == 0) s.warp_tot[warp] = acc;
    __syncthreads();
    if (removed) {
      for (int r = tid; r < s.n_rejected; r += kVerThreads) {
        const int x = s.tok[s.rejected[r]], w = x / sub - rank * kVerWarps;
        if (w >= 0 && w < kVerWarps) atomicAdd(&s.warp_tot[w], 0ull - fix(s.pp[s.rejected[r]]));
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

  int last = 0;                       // warp 0: the last child tried
  double a = 0.0, c = 1.0;            // warp 0
  while (cnt > 0) {  // every turn tries further nodes: at most cnt turns
    if (warp == 0) {
      int cur = s.cur, n = s.n_path, n_rej = s.n_rejected, more = 0;
      // the next child of `cur` behind node `from`, or cnt
      auto next_child = [&](int from) {
        for (int base = from + 1; base < cnt; base += 32) {
          const int i = base + lane;
          const unsigned m = __ballot_sync(0xffffffffu, i < cnt && s.par[i] == cur);
          if (m) return base + __ffs(m) - 1;
        }
        return cnt;
      };
      int i = next_child(last);
      while (i < cnt) {
        const float u = s.uu[i], px = s.pp[i], qx = s.qq[i];
        bool yes;
        bool again = false;  // a token that was already removed here
        if (drafted) {
          yes = a == 0.0 ? s.first_yes[i]
                         : static_cast<double>(u) * qx * c < fmax(static_cast<double>(px) - a * qx, 0.0);
        } else {
          for (int r0 = 0; r0 < n_rej; r0 += 32)
            again |= __any_sync(0xffffffffu, r0 + lane < n_rej && s.tok[s.rejected[min(r0 + lane, n_rej - 1)]] == s.tok[i]);
          yes = !again && (n_rej == 0 ? s.first_yes[i] : static_cast<double>(u) * c < static_cast<double>(px));
        }
        last = i;
        if (yes) {
          cur = i;
          if (lane == 0) s.path[n] = i;
          ++n;
          a = 0.0;
          c = 1.0;
          n_rej = 0;
          i = next_child(last);
          continue;
        }
        i = next_child(last);
        if (drafted) {
          a += c;
          if (i < cnt) {  // the next sibling needs the residual's sum
            more = 1;
            break;
          }
        } else if (!again) {
          c -= px;
          if (lane == 0) s.rejected[n_rej] = last;
          ++n_rej;
          __syncwarp();
        }
      }
      __syncwarp();
      if (lane == 0) {
        s.cur = cur;
        s.n_path = n;
        s.n_rejected = drafted ? 0 : n_rej;
        s.a = a;
        s.more = more;
      }
    }
    __syncthreads();
    if (!s.more) break;
    const unsigned long long total = sum_row(s.cur, s.a, false);
    parity ^= 1;
    if (warp == 0) c = static_cast<double>(total) * kUnit;
    __syncthreads();
  }

  // the draw
  if (cnt > 0) {
    const int cur = s.cur;
    double aa = s.a;
    bool removed = s.n_rejected > 0;
    unsigned long long total = sum_row(cur, aa, removed);
    if (total == 0) {  // p <= a q everywhere: the target's own distribution
      parity ^= 1;
      aa = 0.0;
      removed = false;
      __syncthreads();
      total = sum_row(cur, 0.0, false);
    }
    if (total > 0) {
      const float us = fminf(fmaxf(__ldg(P.u_sample + b), 0.f), 1.f);
      // u in 2^-64 units (below 1), so that thr = floor(u * total) < total
      const unsigned long long u64 = us >= 1.f ? ~0ull : __double2ull_rz(static_cast<double>(us) * 18446744073709551616.0);
      const unsigned long long thr = __umul64hi(u64, total);
      unsigned long long before = 0;
      for (int r = 0; r < rank; ++r) before += s.cta_tot[parity][r];
      for (int w = 0; w < warp; ++w) before += s.warp_tot[w];
      const unsigned long long mine = s.warp_tot[warp];
      if (thr >= before && thr < before + mine) {  // one warp of the cluster
        const int64_t pe = b * P.p_sb + cur * P.p_st, qe = b * P.q_sb + cur * P.q_st;
        const bool with_q = drafted && aa != 0.0;
        const Scale sc{static_cast<float>(aa), static_cast<float>(aa - static_cast<float>(aa))};
        unsigned long long run = before;
        int found = -1;
        for (int v0 = w_lo; v0 < w_hi && found < 0; v0 += 32 * kRowBatch) {
          float pv[kRowBatch], qv[kRowBatch];
          load_rows(pe, qe, v0, with_q, pv, qv);
          unsigned long long w[kRowBatch];
#pragma unroll
          for (int u = 0; u < kRowBatch; ++u) {
            const Limbs x = !with_q ? weight<0>(pv[u], 0.f, sc) : aa == 1.0 ? weight<1>(pv[u], qv[u], sc) : weight<2>(pv[u], qv[u], sc);
            w[u] = whole(x.hi, x.lo);
            if (removed)
              for (int r = 0; r < s.n_rejected; ++r)
                if (s.tok[s.rejected[r]] == v0 + 32 * u + lane) w[u] = 0;
          }
          unsigned long long all = 0;
#pragma unroll
          for (int u = 0; u < kRowBatch; ++u) all += w[u];
          all = warp_sum(all);
          if (run + all <= thr) {  // not in this batch
            run += all;
            continue;
          }
#pragma unroll
          for (int u = 0; u < kRowBatch; ++u) {
            const unsigned long long sum = warp_sum(w[u]);
            if (found < 0 && run + sum > thr) {  // uniform: the row of 32 that holds it
              unsigned long long inc = w[u];
#pragma unroll
              for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long t = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += t;
              }
              found = v0 + 32 * u + __ffs(__ballot_sync(0xffffffffu, run + inc > thr)) - 1;
            }
            run += sum;
          }
        }
        if (lane == 0) {
          if (P.tok64) static_cast<long long*>(P.next_token)[b] = found;
          else static_cast<int32_t*>(P.next_token)[b] = found;
        }
      }
    } else if (rank == 0 && tid == 0) {
      if (P.tok64) static_cast<long long*>(P.next_token)[b] = -1;
      else static_cast<int32_t*>(P.next_token)[b] = -1;
    }
  } else if (rank == 0 && tid == 0) {
    if (P.tok64) static_cast<long long*>(P.next_token)[b] = -1;
    else static_cast<int32_t*>(P.next_token)[b] = -1;
  }
  if (rank == 0) {
    const int n = s.n_path;
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
