// Norms of queries and keys for each head, with the position rotation in the same pass
// (kda_head_norm_rope).
//
// For a (token, head) row x in R^d: y = x / sqrt(mean(x^2) + eps) * w (sum for the 2-norm), then
// (a, b) -> (a cos - b sin, b cos + a sin) on the rotated pairs. Everything is fp32; the row is
// rounded to its type once, after the rotation.
//
// The pass reads and writes each row once (2 d elements) for some 10 operations per element, so
// it is HBM-bound as long as those are few instructions. A row is held by d * sizeof(T) / 16
// consecutive lanes, 16 bytes each, as two 8-byte chunks that hold both channels of every pair:
// channels c .. and rot/2 + c .. for the half-split rotation, two adjacent chunks for the
// interleaved one and for channels that are not rotated (the chunks never straddle the halves
// because rot_dim is a multiple of 16). So a lane needs each angle once, and no shuffles but the
// sum of squares'. Weights and rotation are two factors per channel, y_u = r (u w_u cos - v w_v sin),
// y_v = r (v w_v cos + u w_u sin), computed once for the heads of a token that a warp takes, and
// applied with packed fp32 operations. Every row load is issued before the first is reduced: 57.5 us
// for 16384 tokens of 32 + 8 heads at d = 128, 6.0 TB/s, 88% of the copy rate. (In a run in which it
// took 55: four rows a lane instead of eight 57, two 62. 16-byte chunks with the partner's fetched by
// shuffles took 67, with twice the instructions; a persistent grid that loads a token ahead measured
// the same as that.)
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4;
constexpr int kUnroll = 8;  // rows in flight per lane

// Two fp32 values in one register pair, and the packed operations on them.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// N (2 or 4) floats from a 4 N-byte aligned address.
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float* x) {
  if constexpr (N == 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
    const float2 v = __ldg(reinterpret_cast<const float2*>(p));
    x[0] = v.x; x[1] = v.y;
  }
}

// 8 bytes of a row as fp32 values (4 bf16 or 2 fp32), and back.
__device__ __forceinline__ void widen(const uint2& r, float (&x)[4]) {
  x[0] = __uint_as_float(r.x << 16); x[1] = __uint_as_float(r.x & 0xffff0000u);
  x[2] = __uint_as_float(r.y << 16); x[3] = __uint_as_float(r.y & 0xffff0000u);
}
__device__ __forceinline__ void widen(const uint2& r, float (&x)[2]) {
  x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint2 narrow(const float (&x)[4]) {
  return make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
}
__device__ __forceinline__ uint2 narrow(const float (&x)[2]) {
  return make_uint2(__float_as_uint(x[0]), __float_as_uint(x[1]));
}

template <class T, int D, bool kInter>
__global__ void __launch_bounds__(kWarps * 32, 6)
head_norm_kernel(const HeadNormParams p, int q_groups, int groups) {
  constexpr int CH = 8 / sizeof(T);      // channels of a chunk, and pairs of a lane
  constexpr int LPR = D / (2 * CH);      // lanes per row
  constexpr int RPW = 32 / LPR;          // rows a warp loads at once
  constexpr int HEADS = RPW * kUnroll;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const int64_t tok = item / groups;
  if (tok >= p.tokens) return;
  const int group = (int)(item - tok * groups);
  const HeadNormSide& s = group < q_groups ? p.q : p.k;
  const int h0 = (group < q_groups ? group : group - q_groups) * HEADS + sub;
  int64_t pos = tok;
  if (p.rot && p.positions) pos = __ldg(p.positions + tok);

  // the lane's two chunks
  const int half = p.rot / 2;
  bool rotate = 2 * CH * l < p.rot;
  int c0 = !kInter && rotate ? CH * l : 2 * CH * l;
  int c1 = !kInter && rotate ? half + CH * l : 2 * CH * l + CH;
  const T* xr = (const T*)s.x + tok * s.x_stride + h0 * D;
  uint2 raw[kUnroll][2];
  auto load = [&]() {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      raw[u][0] = raw[u][1] = make_uint2(0u, 0u);
      if (h0 + u * RPW < s.H) {
        raw[u][0] = __ldcs(reinterpret_cast<const uint2*>(xr + u * RPW * D + c0));
        raw[u][1] = __ldcs(reinterpret_cast<const uint2*>(xr + u * RPW * D + c1));
      }
    }
  };
  load();

  if (p.rot && (pos < 0 || pos >= p.n_pos)) {
    // not rotated: as without a table, to the order of the sum
    if (group == 0 && lane == 0 && p.status) atomicOr(p.status, KDA_STATUS_BAD_POSITION);
    rotate = false;
    c0 = 2 * CH * l;
    c1 = c0 + CH;
    load();
  }
  // Pairs: (chunk 0's k-th, chunk 1's k-th) channel, or adjacent channels when interleaved. The
  // weights in the same order, then the four factors.
  float wu[CH], wv[CH], cs[CH], sn[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    wu[k] = wv[k] = cs[k] = 1.0f;
    sn[k] = 0.0f;
  }
  if (s.w) {
    float a[CH], b[CH];
    load_floats<CH>(s.w + c0, a);
    load_floats<CH>(s.w + c1, b);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      wu[k] = kInter ? (2 * k < CH ? a[2 * k % CH] : b[2 * k % CH]) : a[k];
      wv[k] = kInter ? (2 * k < CH ? a[(2 * k + 1) % CH] : b[(2 * k + 1) % CH]) : b[k];
    }
  }
  if (rotate) {
    const float* row = p.cos_sin + pos * p.rot + (kInter ? c0 / 2 : c0);
    load_floats<CH>(row, cs);
    load_floats<CH>(row + half, sn);
  }
  f32x2 uc[CH / 2], us[CH / 2], vc[CH / 2], vs[CH / 2];
#pragma unroll
  for (int k = 0; k < CH / 2; ++k) {
    const f32x2 c = pack2(cs[2 * k], cs[2 * k + 1]), n = pack2(sn[2 * k], sn[2 * k + 1]);
    const f32x2 a = pack2(wu[2 * k], wu[2 * k + 1]), b = pack2(wv[2 * k], wv[2 * k + 1]);
    uc[k] = mul2(a, c);
    us[k] = mul2(a, n);
    vc[k] = mul2(b, c);
    vs[k] = mul2(b, pack2(-sn[2 * k], -sn[2 * k + 1]));
  }

#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    float a[CH], b[CH];
    widen(raw[u][0], a);
    widen(raw[u][1], b);
    f32x2 x[CH / 2], y[CH / 2], q2 = 0ull;  // u's and v's of the pairs
#pragma unroll
    for (int k = 0; k < CH / 2; ++k) {
      if (kInter) {
        const float* f = 4 * k < CH ? a : b;
        constexpr int M = CH - 1;
        x[k] = CH == 2 ? pack2(a[0], b[0]) : pack2(f[4 * k & M], f[(4 * k + 2) & M]);
        y[k] = CH == 2 ? pack2(a[1], b[1]) : pack2(f[(4 * k + 1) & M], f[(4 * k + 3) & M]);
      } else {
        x[k] = pack2(a[2 * k], a[2 * k + 1]);
        y[k] = pack2(b[2 * k], b[2 * k + 1]);
      }
      q2 = fma2(x[k], x[k], q2);
      q2 = fma2(y[k], y[k], q2);
    }
    const float2 q = unpack2(q2);
    float ss = q.x + q.y;
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(((p.flags & KDA_NORM_L2) ? ss : ss * (1.0f / D)) + p.eps);
    const f32x2 r2 = pack2(r, r);
#pragma unroll
    for (int k = 0; k < CH / 2; ++k) {
      f32x2 yu = mul2(x[k], uc[k]), yv = mul2(y[k], vc[k]);
      if (rotate) {  // a channel that is not rotated is not touched by another one's infinity
        yu = fma2(y[k], vs[k], yu);
        yv = fma2(x[k], us[k], yv);
      }
      x[k] = mul2(yu, r2);
      y[k] = mul2(yv, r2);
    }
#pragma unroll
    for (int k = 0; k < CH / 2; ++k) {
      const float2 e = unpack2(x[k]), f = unpack2(y[k]);
      if (kInter) {
        float* g = 4 * k < CH ? a : b;
        constexpr int M = CH - 1;
        if (CH == 2) {
          a[0] = e.x; a[1] = f.x; b[0] = e.y; b[1] = f.y;
        } else {
          g[4 * k & M] = e.x; g[(4 * k + 1) & M] = f.x;
          g[(4 * k + 2) & M] = e.y; g[(4 * k + 3) & M] = f.y;
        }
      } else {
        a[2 * k] = e.x; a[2 * k + 1] = e.y;
        b[2 * k] = f.x; b[2 * k + 1] = f.y;
      }
    }
    if (h0 + u * RPW < s.H) {
      T* out = (T*)s.out + tok * s.out_stride + (h0 + u * RPW) * D;
      __stcs(reinterpret_cast<uint2*>(out + c0), narrow(a));
      __stcs(reinterpret_cast<uint2*>(out + c1), narrow(b));
    }
  }
}

template <class T, int D>
kda_status launch_t(const HeadNormParams& p, cudaStream_t s) {
  constexpr int HEADS = 32 / (D * (int)sizeof(T) / 16) * kUnroll;
  const int q_groups = (p.q.H + HEADS - 1) / HEADS;
  const int groups = q_groups + (p.k.H + HEADS - 1) / HEADS;
  const int64_t blocks = ((int64_t)p.tokens * groups + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL)
    return set_error(KDA_ERR_INVALID_ARG, "kda_head_norm_rope: too many tokens x heads");
  if (p.flags & KDA_ROPE_INTERLEAVED)
    head_norm_kernel<T, D, true><<<(unsigned)blocks, kWarps * 32, 0, s>>>(p, q_groups, groups);
  else
    head_norm_kernel<T, D, false><<<(unsigned)blocks, kWarps * 32, 0, s>>>(p, q_groups, groups);
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
