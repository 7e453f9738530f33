// Attention of one decoded token, or of a verify window, over the paged 8-bit cache
// (kda_cache_attention): o = sum_t softmax_t(scale q . k_t) v_t in one pass over the cache with
// the running maximum and sum of the softmax.
//
// One CTA per (query token, query head). Each of its warps walks every eighth key with its own
// running maximum m, sum l and weighted sum of values (the lanes share the head's channels), and
// the warps' results are joined at the end: o = sum_w e^{m_w - m} acc_w / sum_w e^{m_w - m} l_w.
#include "kda_internal.cuh"
#include "kda_fp8.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;

template <int N>
__device__ __forceinline__ void load_codes(const uint8_t* p, float* f) {
  uint32_t w;
  if constexpr (N == 4) w = *reinterpret_cast<const uint32_t*>(p);
  else w = *reinterpret_cast<const uint16_t*>(p);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 a = f32x2_from_f16x2(f16x2_from_e4m3((w >> (16 * i)) & 0xffffu));
    f[2 * i] = a.x;
    f[2 * i + 1] = a.y;
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kWarps * 32) attn_kernel(const CacheAttnParams p) {
  constexpr int N = D / 32;  // channels per lane
  __shared__ float acc_s[kWarps][D], m_s[kWarps], l_s[kWarps];
  const int hq = blockIdx.x % p.Hq, tok = blockIdx.x / p.Hq;
  const int b = tok / p.window, j = tok - b * p.window;
  const int h = hq / (p.Hq / p.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t n = 0;  // keys this query sees
  if (p.start[b] >= 0 && (!p.lens || j < p.lens[b])) {
    n = (int64_t)p.start[b] + j + 1;
    const int64_t top = (int64_t)p.max_pages * kPage;
    if (n > top) {
      if (threadIdx.x == 0 && hq == 0 && p.status) atomicOr(p.status, KDA_STATUS_BAD_PAGE);
      n = top;
    }
  }
  float q[N], acc[N], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = ld_elem((const T*)p.q, ((int64_t)tok * p.Hq + hq) * D + lane * N + i) * p.scale;
    acc[i] = 0.0f;
  }
  for (int64_t t = warp; t < n; t += kWarps) {
    const int64_t page = p.table[(int64_t)b * p.max_pages + t / kPage];
    if (page < 0) continue;
    if (page >= p.n_pages) {
      if (lane == 0 && p.status) atomicOr(p.status, KDA_STATUS_BAD_PAGE);
      continue;
    }
    const int64_t slice = page * p.Hkv + h;
    const int64_t at = (slice * kPage + t % kPage) * D + lane * N;
    float f[N], s = 0.0f;
    load_codes<N>(p.kc + at, f);
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(q[i], f[i], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= p.ks[slice];
    const float mn = fmaxf(m, s);
    const float c = mn == -INFINITY ? 0.0f : expf(m - mn);
    const float e = mn == -INFINITY ? 0.0f : expf(s - mn);
    m = mn;
    l = l * c + e;
    load_codes<N>(p.vc + at, f);
    const float ev = e * p.vs[slice];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = acc[i] * c + ev * f[i];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) acc_s[warp][lane * N + i] = acc[i];
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w]);
  float c[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    c[w] = m_s[w] == -INFINITY ? 0.0f : expf(m_s[w] - top);
    sum += c[w] * l_s[w];
  }
  for (int i = threadIdx.x; i < D; i += kWarps * 32) {
    float o = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (c[w] != 0.0f) o += c[w] * acc_s[w][i];
    st_elem((T*)p.o, ((int64_t)tok * p.Hq + hq) * D + i, sum == 0.0f ? 0.0f : o / sum);
  }
}

template <class T, int D>
kda_status launch_t(const CacheAttnParams& p, cudaStream_t s) {
  attn_kernel<T, D><<<(unsigned)(p.batch * p.window * p.Hq), kWarps * 32, 0, s>>>(p);
  count_launches(1);
  return check_launch("kda_cache_attention");
}

}  // namespace

size_t cache_attn_workspace_bytes(int, int, int, int, int) { return 0; }

kda_status launch_cache_attn(const CacheAttnParams& p, kda_dtype dt, int d, cudaStream_t s) {
  if (dt == KDA_BF16)
    return d == 128 ? launch_t<__nv_bfloat16, 128>(p, s) : launch_t<__nv_bfloat16, 64>(p, s);
  return d == 128 ? launch_t<float, 128>(p, s) : launch_t<float, 64>(p, s);
}

}  // namespace kda
