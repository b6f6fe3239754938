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
// Weights are held as integers, 2^-52 a unit, and summed in 64-bit integer
// arithmetic: sums do not depend on their order, so a row may be split over
// any number of threads and CTAs and the drawn token is the same. The fp32
// probabilities enter exactly down to 2^-29, truncated at 2^-52 below.
//
// The walk is latency, the residual sums and the draw read two rows of V. One
// cluster of CTAs serves a sequence: each CTA gathers every node's two
// probabilities at once, walks redundantly (the same integers in every CTA),
// owns a slice of V in the sums, and exchanges its slice's total through
// distributed shared memory.
#include "st_kernels.h"
#include "st_serve.h"

namespace st {

namespace {

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr unsigned long long kOne = 1ull << 52;
constexpr double kUnit = 1.0 / 4503599627370496.0;  // 2^-52

__device__ __forceinline__ float prob(const void* p, int dt, int64_t e) {
  float v;
  if (dt == kDtF32) v = __ldg(static_cast<const float*>(p) + e);
  else if (dt == kDtBF16) v = __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + e));
  else v = __half2float(__ldg(static_cast<const __half*>(p) + e));
  return fminf(fmaxf(v, 0.f), 1.f);  // NaN: 0
}
__device__ __forceinline__ unsigned long long fix(float v) { return __float2ull_rz(v * 4503599627370496.0f); }
// a * q, a with 52 fractional bits
__device__ __forceinline__ unsigned long long mul_fix(unsigned long long a, unsigned long long q) {
  return __umul64hi(a << 1, q << 11);
}
__device__ __forceinline__ unsigned long long residual(unsigned long long p, unsigned long long a, unsigned long long q) {
  const unsigned long long s = mul_fix(a, q);
  return p > s ? p - s : 0ull;
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
  int path[kMaxVerify];
  unsigned long long warp_tot[kVerWarps];
  unsigned long long cta_tot[2][kMaxClusterVerify];  // by the parity of the exchange
  int rejected[kMaxVerify];
  int n_rejected;
  int cur, n_path, more;         // more: a rejected child has a sibling left
  unsigned long long a;
};

__global__ void __launch_bounds__(kVerThreads) verify_kernel(const __grid_constant__ VerifyParams P) {
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
    s.pp[i] = ok ? prob(P.p, P.dt, b * P.p_sb + par * P.p_st + x) : 0.f;
    s.qq[i] = ok && drafted ? prob(P.q, P.dt, b * P.q_sb + par * P.q_st + x) : 1.f;
    s.uu[i] = ok ? __ldg(P.u_accept + static_cast<int64_t>(b) * P.T + i) : 0.f;
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

  // sum over V of the residual weights of node `cur` at `a`, less the removed
  // tokens; leaves the warps' totals in s.warp_tot and the CTAs' in s.cta_tot
  auto sum_row = [&](int cur, unsigned long long a, bool removed) -> unsigned long long {
    const int64_t pe = b * P.p_sb + cur * P.p_st, qe = b * P.q_sb + cur * P.q_st;
    unsigned long long acc = 0;
    const bool with_q = drafted && a != 0;
    for (int v0 = w_lo; v0 < w_hi; v0 += 32 * 8) {
      float pv[8], qv[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int v = v0 + 32 * u + lane;
        pv[u] = v < w_hi ? prob(P.p, P.dt, pe + v) : 0.f;
        qv[u] = with_q && v < w_hi ? prob(P.q, P.dt, qe + v) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) acc += with_q ? residual(fix(pv[u]), a, fix(qv[u])) : fix(pv[u]);
    }
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
  unsigned long long a = 0, c = kOne; // warp 0
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
          if (a == 0) yes = static_cast<double>(u) * qx < static_cast<double>(px);
          else yes = static_cast<double>(u) * qx * (static_cast<double>(c) * kUnit) < static_cast<double>(residual(fix(px), a, fix(qx))) * kUnit;
        } else {
          for (int r0 = 0; r0 < n_rej; r0 += 32)
            again |= __any_sync(0xffffffffu, r0 + lane < n_rej && s.tok[s.rejected[min(r0 + lane, n_rej - 1)]] == s.tok[i]);
          yes = !again && static_cast<double>(u) * (static_cast<double>(c) * kUnit) < static_cast<double>(px);
        }
        last = i;
        if (yes) {
          cur = i;
          if (lane == 0) s.path[n] = i;
          ++n;
          a = 0;
          c = kOne;
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
          const unsigned long long f = fix(px);
          c = c > f ? c - f : 0ull;
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
    if (warp == 0) c = total;
    __syncthreads();
  }

  // the draw
  if (cnt > 0) {
    const int cur = s.cur;
    unsigned long long aa = s.a;
    bool removed = s.n_rejected > 0;
    unsigned long long total = sum_row(cur, aa, removed);
    if (total == 0) {  // p <= a q everywhere: the target's own distribution
      parity ^= 1;
      aa = 0;
      removed = false;
      __syncthreads();
      total = sum_row(cur, 0, false);
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
        const bool with_q = drafted && aa != 0;
        unsigned long long run = before;
        int found = -1;
        for (int v0 = w_lo; v0 < w_hi && found < 0; v0 += 32 * 8) {
          float pv[8], qv[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int v = v0 + 32 * u + lane;
            pv[u] = v < w_hi ? prob(P.p, P.dt, pe + v) : 0.f;
            qv[u] = with_q && v < w_hi ? prob(P.q, P.dt, qe + v) : 0.f;
          }
#pragma unroll 1
          for (int u = 0; u < 8 && found < 0; ++u) {
            const int v = v0 + 32 * u + lane;
            float pu = 0.f, qu = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k == u) {
                pu = pv[k];
                qu = qv[k];
              }
            unsigned long long w = with_q ? residual(fix(pu), aa, fix(qu)) : fix(pu);
            if (removed)
              for (int r = 0; r < s.n_rejected; ++r)
                if (s.tok[s.rejected[r]] == v) w = 0;
            unsigned long long inc = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const unsigned long long t = __shfl_up_sync(0xffffffffu, inc, o);
              if (lane >= o) inc += t;
            }
            const unsigned m = __ballot_sync(0xffffffffu, run + inc > thr);
            if (m) found = v0 + 32 * u + __ffs(m) - 1;
            run += __shfl_sync(0xffffffffu, inc, 31);
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
  return cudaLaunchKernelEx(&cfg, verify_kernel, p);
}

}  // namespace st
