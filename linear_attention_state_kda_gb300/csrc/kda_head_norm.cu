// Norms of queries and keys for each head, with the position rotation in the same pass
// (kda_head_norm_rope).
//
// For a (token, head) row x in R^d: y = x / sqrt(mean(x^2) + eps) * w (sum for the 2-norm), then
// (a, b) -> (a cos - b sin, b cos + a sin) on the rotated pairs. Everything is fp32; the row is
// rounded to its type once, after the rotation.
//
// The pass reads and writes each row once (2 d elements) for some 10 operations per element, so
// it is HBM-bound. A row is held by d * sizeof(T) / 16 consecutive lanes, 16 bytes each, so its
// sum of squares is a few shuffles and a half-split pair's partner one more; the 16-byte chunks
// never straddle the halves because rot_dim is a multiple of 16. A warp takes kHeads heads of
// one token, so that the token's cosines and sines are loaded once into registers for all of
// them, and issues every row load before it reduces the first.
#include "kda_internal.cuh"
#include "kda_fp8.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4;
constexpr int kUnroll = 4;  // row loads in flight per lane

// N floats from a 4 N-byte aligned address.
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float* x) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
      x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    }
  } else {
    const float2 v = __ldg(reinterpret_cast<const float2*>(p));
    x[0] = v.x; x[1] = v.y;
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kWarps * 32, 8)
head_norm_kernel(const HeadNormParams p, int q_groups, int groups) {
  constexpr int N = Vec16<T>::N;
  constexpr int LPR = D / N;        // lanes per row
  constexpr int RPW = 32 / LPR;     // rows a warp loads at once
  constexpr int HEADS = RPW * kUnroll;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const int64_t tok = item / groups;
  if (tok >= p.tokens) return;
  const int group = (int)(item - tok * groups);
  const HeadNormSide& s = group < q_groups ? p.q : p.k;
  const int h0 = (group < q_groups ? group : group - q_groups) * HEADS + sub;
  const int e0 = l * N;  // first channel of this lane
  int64_t pos = tok;
  if (p.rot && p.positions) pos = __ldg(p.positions + tok);

  const T* xr = (const T*)s.x + tok * s.x_stride + h0 * D + e0;
  uint4 raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    raw[u] = make_uint4(0u, 0u, 0u, 0u);
    if (h0 + u * RPW < s.H) raw[u] = __ldcs(reinterpret_cast<const uint4*>(xr + u * RPW * D));
  }

  // y_i = r (x_i a_i + x_partner b_i): weights and rotation in two factors per channel, the same
  // for all heads. A channel that is not rotated is its own partner, with b = 0.
  const int half = p.rot / 2;
  const bool inter = (p.flags & KDA_ROPE_INTERLEAVED) != 0;
  bool rotate = e0 < p.rot;
  if (rotate && (pos < 0 || pos >= p.n_pos)) {
    if (group == 0 && lane == 0 && p.status) atomicOr(p.status, KDA_STATUS_BAD_POSITION);
    rotate = false;
  }
  float a[N], b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a[i] = 1.0f;
    b[i] = 0.0f;
  }
  if (rotate) {
    const float* row = p.cos_sin + pos * p.rot;
    if (inter) {
      float c2[N / 2], s2[N / 2];
      load_floats<N / 2>(row + e0 / 2, c2);
      load_floats<N / 2>(row + half + e0 / 2, s2);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        a[2 * i] = a[2 * i + 1] = c2[i];
        b[2 * i + 1] = s2[i];
        b[2 * i] = -s2[i];
      }
    } else {
      const int i0 = e0 < half ? e0 : e0 - half;
      load_floats<N>(row + i0, a);
      load_floats<N>(row + half + i0, b);
      if (e0 < half) {
#pragma unroll
        for (int i = 0; i < N; ++i) b[i] = -b[i];
      }
    }
  }
  // the chunk that holds the partners of a half-split pair
  const int step = inter || !rotate ? 0 : (e0 < half ? half : -half);
  const int partner = lane + step / N;
  if (s.w) {
    float w[N];
    load_floats<N>(s.w + e0, w);
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] *= w[i];
    if (!inter) load_floats<N>(s.w + e0 + step, w);
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] *= inter ? w[i ^ 1] : w[i];
  }

#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    float x[N], y[N];
    Vec16<T>::unpack(raw[u], x);
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(((p.flags & KDA_NORM_L2) ? ss : ss * (1.0f / D)) + p.eps);
    if (p.rot && !inter) {
      uint4 o;
      o.x = __shfl_sync(0xffffffffu, raw[u].x, partner);
      o.y = __shfl_sync(0xffffffffu, raw[u].y, partner);
      o.z = __shfl_sync(0xffffffffu, raw[u].z, partner);
      o.w = __shfl_sync(0xffffffffu, raw[u].w, partner);
      Vec16<T>::unpack(o, y);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = rotate ? x[i ^ 1] : x[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = fmaf(x[i], a[i], y[i] * b[i]) * r;
    const int h = h0 + u * RPW;
    if (h < s.H) {
      T* out = (T*)s.out + tok * s.out_stride + h * D + e0;
      __stcs(reinterpret_cast<uint4*>(out), Vec16<T>::pack(x));
    }
  }
}

template <class T, int D>
kda_status launch_t(const HeadNormParams& p, cudaStream_t s) {
  constexpr int HEADS = 32 / (D / Vec16<T>::N) * kUnroll;
  const int q_groups = (p.q.H + HEADS - 1) / HEADS;
  const int groups = q_groups + (p.k.H + HEADS - 1) / HEADS;
  const int64_t blocks = ((int64_t)p.tokens * groups + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL)
    return set_error(KDA_ERR_INVALID_ARG, "kda_head_norm_rope: too many tokens x heads");
  head_norm_kernel<T, D><<<(unsigned)blocks, kWarps * 32, 0, s>>>(p, q_groups, groups);
  count_launches(1);
  return check_launch("kda_head_norm_rope");
}

}  // namespace

kda_status launch_head_norm(const HeadNormParams& p, kda_dtype dt, int d, cudaStream_t s) {
  if (dt == KDA_BF16)
    return d == 128 ? launch_t<__nv_bfloat16, 128>(p, s) : launch_t<__nv_bfloat16, 64>(p, s);
  return d == 128 ? launch_t<float, 128>(p, s) : launch_t<float, 64>(p, s);
}

}  // namespace kda
