// Verification of drafted tokens against the target's probabilities from given random numbers
// (kda_draft_verify).
//
// Row b takes its drafts in order while u q(x) < p(x), then samples one token: from max(p - q, 0)
// at the first refusal, from p after the last draft. The sampling weights are integers,
// floor(clamp(., 0, 1) 2^40), so their sums are exact and the answer does not depend on the order
// in which they are added: the vocabulary can be cut over as many warps as the row needs.
//
// What bounds it: two rows of the vocabulary are read once (8 bytes per entry in fp32), so many
// rows are HBM-bound and few rows are bound by latency: the drafts' probabilities (two dependent
// loads), the stream, and the search for the threshold. A cluster of CTAs takes a row. Every warp
// decides the drafts by itself (lane j looks at draft j), sums one contiguous stretch of the
// vocabulary, and the stretches' sums are exchanged through distributed shared memory; the warp
// whose stretch holds the threshold reads it again (from L2) and finds the token.
#include "kda_internal.cuh"
#include "kda_fp8.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

constexpr int kMaxCluster = 8;
// floor(clamp(y, 0, 1) * 2^40), 0 for NaN, by shifting the significand: y = m 2^(e - 150) with m
// below 2^24, so the weight is m 2^7 2^32 shifted right by 149 - e (at most 63, which leaves 0).
// (The conversion instruction to 64-bit integers runs on the fp64 pipe and bounded the kernel:
// 97 us against 87 on 256 rows of 131072 entries, before the vector loads.)
__device__ __forceinline__ uint64_t weight_of(float y) {
  const uint32_t b = __float_as_uint(__saturatef(y));
  const uint32_t m = ((b & 0x7fffffu) | 0x800000u) << 7;
  return ((uint64_t)m << 32) >> min(149u - (b >> 23), 63u);
}

__device__ __forceinline__ uint64_t warp_sum_u64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What a row samples from: p, minus q where q is given, with the entry `hot` left out.
template <class T>
struct Source {
  const T* p;
  const T* q;
  int hot;
};

// N entries from r + i on: one vector load (N > 1: r + i 16-byte aligned) or one element.
template <int N, class T>
__device__ __forceinline__ void load_n(const T* r, float* x) {
  if constexpr (N == 1) x[0] = ld_elem(r, 0);
  else Vec16<T>::unpack(__ldcs(reinterpret_cast<const uint4*>(r)), x);
}

// A group is kUnroll rows of 32 N consecutive entries; lane l holds entries i + l N .. of each
// row u (i the group's first entry), as their weights. kEdge: entries from `end` on weigh nothing.
template <int N>
struct Group {
  static constexpr int kUnroll = N == 1 ? 8 : (N == 4 ? 4 : 2);
  static constexpr int kSize = kUnroll * 32 * N;
};
template <int N, bool kEdge, class T, class F>
__device__ __forceinline__ void each_weight(const Source<T>& s, int i, int end, int lane, F f) {
  using G = Group<N>;
  float pv[G::kUnroll][N], qv[G::kUnroll][N];
#pragma unroll
  for (int u = 0; u < G::kUnroll; ++u)
#pragma unroll
    for (int k = 0; k < N; ++k) pv[u][k] = qv[u][k] = 0.0f;
#pragma unroll
  for (int u = 0; u < G::kUnroll; ++u) {
    const int at = i + (u * 32 + lane) * N;
    if (!kEdge || at + N <= end) {
      load_n<N>(s.p + at, pv[u]);
    } else if (N > 1) {
      for (int k = 0; k < N; ++k)
        if (at + k < end) pv[u][k] = ld_elem(s.p, at + k);
    }
  }
  if (s.q) {
#pragma unroll
    for (int u = 0; u < G::kUnroll; ++u) {
      const int at = i + (u * 32 + lane) * N;
      if (!kEdge || at + N <= end) {
        load_n<N>(s.q + at, qv[u]);
      } else if (N > 1) {
        for (int k = 0; k < N; ++k)
          if (at + k < end) qv[u][k] = ld_elem(s.q, at + k);
      }
    }
  }
  const bool hot_here = s.hot >= i && s.hot < i + G::kSize;
#pragma unroll
  for (int u = 0; u < G::kUnroll; ++u) {
    uint64_t w[N];
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = weight_of(pv[u][k] - qv[u][k]);
    if (hot_here) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (i + (u * 32 + lane) * N + k == s.hot) w[k] = 0;
    }
    f(u, w);
  }
}

// Sum of the weights of [i0, i1), over the warp.
template <int N, class T>
__device__ __forceinline__ uint64_t sum_weights(const Source<T>& s, int i0, int i1, int lane) {
  uint64_t sum = 0;
  auto add = [&](int, const uint64_t* w) {
#pragma unroll
    for (int k = 0; k < N; ++k) sum += w[k];
  };
  int i = i0;
  for (; i + Group<N>::kSize <= i1; i += Group<N>::kSize) each_weight<N, false>(s, i, i1, lane, add);
  if (i < i1) each_weight<N, true>(s, i, i1, lane, add);
  return warp_sum_u64(sum);
}

// First entry of [i0, i1) at which `before` plus the weights up to it exceeds limit (-1: none).
template <int N, class T>
__device__ __forceinline__ int find_weight(const Source<T>& s, int i0, int i1, int lane,
                                           uint64_t before, uint64_t limit) {
  int tok = -1;
  for (int i = i0; i < i1 && tok < 0; i += Group<N>::kSize)
    each_weight<N, true>(s, i, i1, lane, [&](int u, const uint64_t* w) {
      uint64_t mine = 0;
#pragma unroll
      for (int k = 0; k < N; ++k) mine += w[k];
      uint64_t upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const unsigned over = __ballot_sync(0xffffffffu, before + upto > limit);
      if (tok < 0 && over) {
        const int l = __ffs(over) - 1;
        uint64_t c = before + (upto - mine);
        int k = 0;
        for (; k < N - 1; ++k) {
          c += w[k];
          if (c > limit) break;
        }
        tok = i + (u * 32 + l) * N + __shfl_sync(0xffffffffu, k, l);
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    });
  return tok;
}

template <class T, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, kWarps == 4 ? 8 : 1)
verify_kernel(const VerifyParams p, int cluster) {
  __shared__ uint64_t part[2][kWarps];
  __shared__ uint64_t all[kMaxCluster * kWarps];
  const int b = blockIdx.x / cluster, rank = blockIdx.x - b * cluster;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int V = p.vocab, W = p.window;
  const T* target = (const T*)p.target + (int64_t)b * (W + 1) * p.target_stride;
  const T* draft = (const T*)p.draft + (int64_t)b * W * p.draft_stride;

  // the drafts that are taken: lane j decides draft j
  int len = p.lens ? p.lens[b] : W;
  const bool pad = len < 0;
  len = len > W ? W : len;
  int x = 0;
  bool bad = false, take = false;
  if (lane < len) {
    x = p.drafts[(int64_t)b * W + lane];
    bad = x < 0 || x >= V;
    if (!bad) {
      const float px = ld_elem(target, lane * p.target_stride + x);
      const float qx = p.draft ? ld_elem(draft, lane * p.draft_stride + x) : 1.0f;
      take = __fmul_rn(p.ua[(int64_t)b * W + lane], qx) < px;
    }
  }
  const int n = __ffs(__ballot_sync(0xffffffffu, !take)) - 1;  // lanes from len on do not take
  const bool bad_n = __shfl_sync(0xffffffffu, bad, n);
  const int x_n = __shfl_sync(0xffffffffu, x, n);
  const bool sub = n < len && !bad_n;
  if (bad_n && rank == 0 && threadIdx.x == 0 && p.status)
    atomicOr(p.status, KDA_STATUS_BAD_TOKEN);

  Source<T> src;
  src.p = target + n * p.target_stride;
  src.q = sub && p.draft ? draft + n * p.draft_stride : nullptr;
  src.hot = sub && !p.draft ? x_n : -1;
  const float u = pad ? 0.0f : p.us[b];
  const uint64_t u24 = u > 0.0f ? (uint64_t)(fminf(u, 0.99999994f) * 16777216.0f) : 0;

  // this warp's stretch of the vocabulary
  const int chunks = cluster * kWarps;
  const int per = ((V + chunks - 1) / chunks + 7) & ~7;  // keeps the stretches' alignment
  const int mine = rank * kWarps + warp;
  const int i0 = min(V, mine * per), i1 = min(V, i0 + per);
  // whole vectors where both rows start on 16 bytes (a vocabulary of whole vectors), else elements
  constexpr int kVec = Vec16<T>::N;
  const bool vec = (((uintptr_t)src.p | (uintptr_t)src.q) & 15) == 0;
  int tok = -1;
  bool owner = rank == 0 && warp == 0;  // writes the sampled token
  if (!pad) {
    for (int round = 0; round < 2; ++round) {
      const uint64_t sum = vec ? sum_weights<kVec>(src, i0, i1, lane)
                               : sum_weights<1>(src, i0, i1, lane);
      if (lane == 0) part[round][warp] = sum;
      // all stretches' sums, from every CTA of the cluster
      if (cluster > 1) ptx::cluster_sync();
      else __syncthreads();
      for (int i = threadIdx.x; i < chunks; i += kWarps * 32) {
        const uint64_t* from = &part[round][i % kWarps];
        all[i] = cluster > 1 ? ptx::ld_cluster_u64(from, i / kWarps) : *from;
      }
      __syncthreads();
      // the other CTAs' sums are read: they may leave (or write them again) once all are here
      if (cluster > 1) ptx::cluster_arrive();
      uint64_t total = 0, before = 0;
      for (int i = lane; i < chunks; i += 32) {
        total += all[i];
        if (i < mine) before += all[i];
      }
      total = warp_sum_u64(total);
      before = warp_sum_u64(before);
      if (total == 0) {
        if (!sub || round == 1) break;
        src.q = nullptr;
        src.hot = -1;
        if (cluster > 1) ptx::cluster_wait();
        else __syncthreads();  // all[] is written again
        continue;
      }
      const uint64_t limit = __umul64hi(total, u24 << 40);
      owner = before <= limit && limit < before + sum;
      if (owner)
        tok = vec ? find_weight<kVec>(src, i0, i1, lane, before, limit)
                  : find_weight<1>(src, i0, i1, lane, before, limit);
      break;
    }
  }

  if (owner && lane == 0 && !pad) p.tokens[(int64_t)b * (W + 1) + n] = tok;
  if (rank == 0 && warp == 0) {
    const int taken = pad ? 0 : n;
    if (lane <= W && (pad || lane != n))
      p.tokens[(int64_t)b * (W + 1) + lane] = lane < taken ? x : -1;
    if (lane == 0) {
      p.n_accepted[b] = taken;
      if (p.resume) p.resume[b] = pad ? -1 : p.slots[(int64_t)b * (W + 1) + n];
    }
  }
  if (!pad && cluster > 1) {
    __syncwarp();
    ptx::cluster_wait();
  }
}

template <class T, int kWarps>
kda_status launch_t(const VerifyParams& p, int cluster, cudaStream_t s) {
  while (cluster > 1 && (int64_t)p.vocab < (int64_t)cluster * kWarps * 32) cluster >>= 1;
  if ((int64_t)p.batch * cluster > 0x7fffffffLL) cluster = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.batch * (unsigned)cluster);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, verify_kernel<T, kWarps>, p, cluster);
  count_launches(1);
  return check_launch("kda_draft_verify");
}

template <class T>
kda_status dispatch(const VerifyParams& p, cudaStream_t s) {
  // Few rows (up to two large CTAs per SM): as many warps per row as a cluster has, so that each
  // stretch is short: 4 us less than one CTA a row for 4 rows of 32003 entries (a call takes 8.2).
  // Many rows: small CTAs, whose loads cover each other's waits: 55 us on 256 rows of 131072 entries
  // (4.9 TB/s, 72% of the copy rate) against 84 with 16 warps; clusters of 4 or 2 are 10-60% slower.
  if (p.batch <= 38) return launch_t<T, 16>(p, kMaxCluster, s);
  return launch_t<T, 4>(p, kMaxCluster, s);
}

}  // namespace

kda_status launch_verify(const VerifyParams& p, kda_dtype dt, cudaStream_t s) {
  return dt == KDA_BF16 ? dispatch<__nv_bfloat16>(p, s) : dispatch<float>(p, s);
}

}  // namespace kda
