// Verification of drafted tokens against the target's probabilities from given random numbers
// (kda_draft_verify).
//
// Row b takes its drafts in order while u q(x) < p(x), then samples one token: from max(p - q, 0)
// at the first refusal, from p after the last draft. The sampling weights are integers,
// floor(clamp(., 0, 1) 2^40), so their sums are exact and the answer does not depend on the order
// in which they are added.
//
// One CTA per row: every thread sums the weights of its stretch of the vocabulary, the stretch
// that holds the threshold is found from the partial sums, and its owner walks it again.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 1024;

// floor(clamp(y, 0, 1) * 2^40), 0 for NaN. The product is exact.
__device__ __forceinline__ uint64_t weight_of(float y) {
  return __float2ull_rd(fminf(fmaxf(y, 0.0f), 1.0f) * 1099511627776.0f);
}

template <class T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyParams p) {
  __shared__ uint64_t part[kThreads];
  __shared__ int s_tok;
  const int b = blockIdx.x, V = p.vocab, W = p.window;
  int len = p.lens ? p.lens[b] : W;
  const bool pad = len < 0;
  len = len > W ? W : len;
  int n = 0;
  bool bad = false;
  for (; n < len; ++n) {
    const int x = p.drafts[(int64_t)b * W + n];
    bad = x < 0 || x >= V;
    if (bad) break;
    const float px = ld_elem((const T*)p.target, ((int64_t)b * (W + 1) + n) * p.target_stride + x);
    const float qx =
        p.draft ? ld_elem((const T*)p.draft, ((int64_t)b * W + n) * p.draft_stride + x) : 1.0f;
    if (!(__fmul_rn(p.ua[(int64_t)b * W + n], qx) < px)) break;
  }
  if (pad) n = 0;
  int tok = -1;
  if (!pad) {
    if (bad && threadIdx.x == 0 && p.status) atomicOr(p.status, KDA_STATUS_BAD_TOKEN);
    const T* pr = (const T*)p.target + ((int64_t)b * (W + 1) + n) * p.target_stride;
    bool sub = n < len && !bad;
    const T* qr = sub && p.draft ? (const T*)p.draft + ((int64_t)b * W + n) * p.draft_stride
                                 : nullptr;
    const int hot = sub && !p.draft ? p.drafts[(int64_t)b * W + n] : -1;
    const int per = (V + kThreads - 1) / kThreads;
    const int i0 = threadIdx.x * per, i1 = min(V, i0 + per);
    const float u = p.us[b];
    const uint64_t u24 = u > 0.0f ? (uint64_t)(fminf(u, 0.99999994f) * 16777216.0f) : 0;
    if (threadIdx.x == 0) s_tok = -1;
    for (int round = 0; round < 2; ++round) {
      auto weight = [&](int i) {
        float y = ld_elem(pr, i);
        if (round == 0 && qr) y -= ld_elem(qr, i);
        return round == 0 && i == hot ? 0ull : weight_of(y);
      };
      uint64_t sum = 0;
      for (int i = i0; i < i1; ++i) sum += weight(i);
      part[threadIdx.x] = sum;
      __syncthreads();
      uint64_t total = 0, before = 0;
      for (int t = 0; t < kThreads; ++t) {
        if (t == (int)threadIdx.x) before = total;
        total += part[t];
      }
      const uint64_t limit = __umul64hi(total, u24 << 40);
      if (before <= limit && limit < before + sum) {
        uint64_t c = before;
        int i = i0;
        for (; i < i1; ++i) {
          c += weight(i);
          if (c > limit) break;
        }
        s_tok = i;
      }
      __syncthreads();
      if (total > 0) break;
      if (!sub) break;
    }
    tok = s_tok;
  }
  for (int j = threadIdx.x; j <= W; j += kThreads)
    p.tokens[(int64_t)b * (W + 1) + j] =
        pad || j > n ? -1 : (j == n ? tok : p.drafts[(int64_t)b * W + j]);
  if (threadIdx.x == 0) {
    p.n_accepted[b] = n;
    if (p.resume) p.resume[b] = pad ? -1 : p.slots[(int64_t)b * (W + 1) + n];
  }
}

}  // namespace

kda_status launch_verify(const VerifyParams& p, kda_dtype dt, cudaStream_t s) {
  if (dt == KDA_BF16)
    verify_kernel<__nv_bfloat16><<<(unsigned)p.batch, kThreads, 0, s>>>(p);
  else
    verify_kernel<float><<<(unsigned)p.batch, kThreads, 0, s>>>(p);
  count_launches(1);
  return check_launch("kda_draft_verify");
}

}  // namespace kda
