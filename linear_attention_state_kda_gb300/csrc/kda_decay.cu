// Linear attention with one decay per head,
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,
// for tokens and verify windows over the slot-addressed state pool, and, on CUDA cores, for
// fp32 prompts in chunks. (Prompts in bf16 run on the tensor cores, kda_decay_tc.cu.)
#include "kda_decay.cuh"
#include "kda_fp8.cuh"

namespace kda {
namespace {

using namespace decay;

// ---------------------------------------------------------------- windows
//
// HBM-bound: a state is read once and stored once per token. As in the KDA decode kernel a CTA
// owns 64 columns of one (row, head)'s state in registers: 8 warps own D/8 rows each, a lane two
// columns, so that every warp moves 256-byte row segments. A column evolves on its own; the only
// exchange is the sum over the key channels in o, one barrier a token (two sets of partial sums
// take turns). 256 rows x 32 heads of 128, one token each: 161 us, 6.7 TB/s; 96 x 32 with windows of
// 4, every state kept: 153 us, 6.6 TB/s; 3 rows x 8 heads 4.9 us, which is latency.
constexpr int kWarps = 8;
constexpr int kCols = 64;

template <int D, class T>
__global__ void __launch_bounds__(kWarps * 32, 4) decay_window_kernel(const DecayParams p) {
  constexpr int NSPLIT = D / kCols;
  constexpr int RPW = D / kWarps;
  const int part = blockIdx.x % NSPLIT;
  const int bh = blockIdx.x / NSPLIT;
  const int b = bh / p.H, h = bh - b * p.H;
  const int hk = h / (p.H / p.Hk);
  const int W = p.window;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = warp * RPW, c0 = lane * 2, cg = part * kCols + c0;

  extern __shared__ float win[];  // [W][D] q, k; [W][64] v; [W] decays
  float* s_q = win;
  float* s_k = s_q + W * D;
  float* s_v = s_k + W * D;
  float* s_a = s_v + W * kCols;
  __shared__ float red[2][kWarps][kCols];

  const int64_t tok0 = (int64_t)b * W;
  T* o = (T*)p.o;
  const int slot = p.read_slots[b];
  if (slot < 0 || (int64_t)slot >= p.n_slots) {
    if ((int64_t)slot >= p.n_slots && threadIdx.x == 0 && h == 0 && part == 0 && p.status)
      atomicOr(p.status, KDA_STATUS_BAD_SLOT);
    for (int i = threadIdx.x; i < W * kCols; i += blockDim.x)
      st_elem(o, ((tok0 + i / kCols) * p.H + h) * D + part * kCols + i % kCols, 0.0f);
    return;
  }
  const float* S = p.pool + ((int64_t)slot * p.H + h) * (int64_t)(D * D);
  float2 st[RPW];
#pragma unroll
  for (int i = 0; i < RPW; ++i)
    st[i] = __ldcs(reinterpret_cast<const float2*>(S + (int64_t)(r0 + i) * D + cg));

  const T *q = (const T*)p.q + (int64_t)hk * D, *k = (const T*)p.k + (int64_t)hk * D,
          *v = (const T*)p.v + (int64_t)h * D + part * kCols;
  for (int i = threadIdx.x; i < W * D; i += blockDim.x) {
    const int64_t t = tok0 + i / D;
    s_q[i] = ld_elem(q, t * p.qs + i % D);
    s_k[i] = ld_elem(k, t * p.ks + i % D);
  }
  for (int i = threadIdx.x; i < W * kCols; i += blockDim.x)
    s_v[i] = ld_elem(v, (tok0 + i / kCols) * p.vs + i % kCols);
  for (int j = threadIdx.x; j < W; j += blockDim.x) s_a[j] = expf(p.g[(tok0 + j) * p.gs + h]);
  __syncthreads();

  for (int j = 0; j < W; ++j) {
    const float* kr = s_k + j * D + r0;
    const float* qr = s_q + j * D + r0;
    const float a = s_a[j], v0 = s_v[j * kCols + c0], v1 = s_v[j * kCols + c0 + 1];
    float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      st[i].x = fmaf(kr[i], v0, st[i].x * a);
      st[i].y = fmaf(kr[i], v1, st[i].y * a);
      y0 = fmaf(qr[i], st[i].x, y0);
      y1 = fmaf(qr[i], st[i].y, y1);
    }
    *reinterpret_cast<float2*>(&red[j & 1][warp][c0]) = make_float2(y0, y1);
    const int ws = p.write_slots[tok0 + j];
    if ((int64_t)ws >= p.n_slots) {
      if (threadIdx.x == 0 && h == 0 && part == 0 && p.status)
        atomicOr(p.status, KDA_STATUS_BAD_SLOT);
    } else if (ws >= 0) {
      float* out = p.pool + ((int64_t)ws * p.H + h) * (int64_t)(D * D);
#pragma unroll
      for (int i = 0; i < RPW; ++i)
        __stcs(reinterpret_cast<float2*>(out + (int64_t)(r0 + i) * D + cg), st[i]);
    }
    __syncthreads();
    if (threadIdx.x < kCols) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += red[j & 1][w][threadIdx.x];
      st_elem(o, ((tok0 + j) * p.H + h) * D + part * kCols + threadIdx.x, p.scale * s);
    }
  }
}

template <int D, class T>
kda_status launch_window_t(const DecayParams& p, cudaStream_t s) {
  const size_t smem = (size_t)p.window * (2 * D + kCols + 1) * sizeof(float);
  const dim3 grid((unsigned)p.batch * (unsigned)p.H * (unsigned)(D / kCols));
  decay_window_kernel<D, T><<<grid, kWarps * 32, smem, s>>>(p);
  count_launches(1);
  return check_launch("kda_decay_window");
}

// ---------------------------------------------------------------- prompts on CUDA cores
//
// fp32 throughout. A CTA walks one segment of one head for 64 value columns in chunks of 32
// tokens. With gamma the running sum of g in the chunk,
//     o_i = e^{gamma_i} scale S^T q_i + sum_{j <= i} e^{gamma_i - gamma_j} scale (q_i . k_j) v_j
//     S'  = e^{gamma_C} S + sum_j e^{gamma_C - gamma_j} k_j v_j^T
// The state is in registers (D/16 x 4 a thread), copied to shared memory for the first sum. Bound by
// the fp32 units and, nearly as much, by shared memory: 5 prompts up to 1301 tokens x 6 heads of 64
// 49 us, 8192 x 16 of 128 606 us, 13 T multiply-adds/s in both passes (740 us with the rows asked for
// only when they were needed).
constexpr int kC = 32;
constexpr int kSimtThreads = 256;

template <int D>
struct SimtShape {
  static constexpr int DP = D + 4, VP = kCols + 4, PP = kC + 1;
  static constexpr int floats = 2 * kC * DP + kC * VP + D * VP + kC * PP;
};

template <int D, bool kStates>
__global__ void __launch_bounds__(kSimtThreads, D == 64 ? 4 : 2)
decay_chunk_kernel(const DecayParams p, int seg, float* added, float* added_log) {
  using S = SimtShape<D>;
  using T = float;
  constexpr int RPT = D / 16;
  extern __shared__ float smem[];
  float* sq = smem;
  float* sk = sq + kC * S::DP;
  float* sv = sk + kC * S::DP;
  float* ss = sv + kC * S::VP;
  float* sp = ss + D * S::VP;
  __shared__ float2 gam[kC];
  __shared__ float s_in[kC], s_out[kC];  // e^gamma_i, e^(gamma_C - gamma_i)
  __shared__ float s_total;

  const int h = blockIdx.y, col0 = blockIdx.z * kCols, tid = threadIdx.x;
  Segment x;
  if (!find_segment<kStates>(p, seg, blockIdx.x, tid & 31, tid == 0 && h == 0 && blockIdx.z == 0, x))
    return;
  const int hk = h / (p.H / p.Hk);
  const int ty = tid >> 4, tx = tid & 15;
  const int r0 = ty * RPT, c0 = col0 + tx * 4;

  float st[RPT][4];
  const float* entry = nullptr;
  if (!kStates)
    entry = !x.first ? added + ((int64_t)(x.place - 1) * p.H + h) * (D * D)
            : p.init ? p.init + ((int64_t)x.seq * p.H + h) * (D * D) : nullptr;
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (entry) f = *reinterpret_cast<const float4*>(entry + (int64_t)(r0 + i) * D + c0);
    st[i][0] = f.x; st[i][1] = f.y; st[i][2] = f.z; st[i][3] = f.w;
  }
  float2 log_sum = make_float2(0.0f, 0.0f);  // thread 0

  const T *q = (const T*)p.q + (int64_t)hk * D, *k = (const T*)p.k + (int64_t)hk * D,
          *v = (const T*)p.v + (int64_t)h * D + col0;
  // a chunk's rows, zeros past its end, are asked for while the chunk before is worked on
  constexpr int NK = kC * (D / 4) / kSimtThreads, NV = kC * (kCols / 4) / kSimtThreads;
  float4 fq[NK], fk[NK], fv[NV];
  auto ask = [&](int64_t t0) {
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      const int i = tid + j * kSimtThreads, t = i / (D / 4), c = (i % (D / 4)) * 4;
      fq[j] = fk[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (t0 + t < x.hi) {
        if (!kStates) fq[j] = *reinterpret_cast<const float4*>(q + (t0 + t) * p.qs + c);
        fk[j] = *reinterpret_cast<const float4*>(k + (t0 + t) * p.ks + c);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * kSimtThreads, t = i / (kCols / 4), c = (i % (kCols / 4)) * 4;
      fv[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (t0 + t < x.hi) fv[j] = *reinterpret_cast<const float4*>(v + (t0 + t) * p.vs + c);
    }
  };
  if (x.lo < x.hi) ask(x.lo);
  for (int64_t t0 = x.lo; t0 < x.hi; t0 += kC) {
    const int n = (int)(x.hi - t0 < kC ? x.hi - t0 : kC);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      const int i = tid + j * kSimtThreads, t = i / (D / 4), c = (i % (D / 4)) * 4;
      if (!kStates) *reinterpret_cast<float4*>(&sq[t * S::DP + c]) = fq[j];
      *reinterpret_cast<float4*>(&sk[t * S::DP + c]) = fk[j];
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * kSimtThreads, t = i / (kCols / 4), c = (i % (kCols / 4)) * 4;
      *reinterpret_cast<float4*>(&sv[t * S::VP + c]) = fv[j];
    }
    if (t0 + kC < x.hi) ask(t0 + kC);
    if (!kStates) {
#pragma unroll
      for (int i = 0; i < RPT; ++i)
        *reinterpret_cast<float4*>(&ss[(r0 + i) * S::VP + tx * 4]) =
            make_float4(st[i][0], st[i][1], st[i][2], st[i][3]);
    }
    if (tid < 32) {
      const float g = tid < n ? p.g[(t0 + tid) * p.gs + h] : 0.0f;
      const bool nan = __any_sync(0xffffffffu, g != g);
      float2 u = log_scan(log_pair(g), tid);
      const float2 all = make_float2(__shfl_sync(0xffffffffu, u.x, 31),
                                     __shfl_sync(0xffffffffu, u.y, 31));
      if (nan) u.x = __int_as_float(0x7fffffff);  // a NaN decay spoils its chunk
      gam[tid] = u;
      s_in[tid] = exp2f(u.x + u.y);
      s_out[tid] = decay_between(all, u);
      if (tid == 0) {
        s_total = decay_between(all, make_float2(nan ? u.x : 0.0f, 0.0f));
        log_sum = log_add(log_sum, all);
      }
    }
    __syncthreads();
    if (!kStates) {
      const int i = tid >> 3;
      float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int c = 0; c < D; c += 4) {
        const float4 a = *reinterpret_cast<const float4*>(&sq[i * S::DP + c]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float4 b = *reinterpret_cast<const float4*>(&sk[((tid & 7) + 8 * m) * S::DP + c]);
          acc[m] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, acc[m]))));
        }
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int j = (tid & 7) + 8 * m;
        sp[i * S::PP + j] = j <= i ? acc[m] * decay_between(gam[i], gam[j]) : 0.0f;
      }
      __syncthreads();
      const int i0 = ty * 2;
      float out[2][4] = {};
      for (int r = 0; r < D; r += 4) {
        const float4 qa = *reinterpret_cast<const float4*>(&sq[i0 * S::DP + r]);
        const float4 qb = *reinterpret_cast<const float4*>(&sq[(i0 + 1) * S::DP + r]);
        const float a[4] = {qa.x, qa.y, qa.z, qa.w}, b[4] = {qb.x, qb.y, qb.z, qb.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 f = *reinterpret_cast<const float4*>(&ss[(r + e) * S::VP + tx * 4]);
          out[0][0] = fmaf(a[e], f.x, out[0][0]); out[0][1] = fmaf(a[e], f.y, out[0][1]);
          out[0][2] = fmaf(a[e], f.z, out[0][2]); out[0][3] = fmaf(a[e], f.w, out[0][3]);
          out[1][0] = fmaf(b[e], f.x, out[1][0]); out[1][1] = fmaf(b[e], f.y, out[1][1]);
          out[1][2] = fmaf(b[e], f.z, out[1][2]); out[1][3] = fmaf(b[e], f.w, out[1][3]);
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) out[m][c] *= s_in[i0 + m];
      auto add = [&](float (&x)[4], float w, const float4& f) {
        x[0] = fmaf(w, f.x, x[0]); x[1] = fmaf(w, f.y, x[1]);
        x[2] = fmaf(w, f.z, x[2]); x[3] = fmaf(w, f.w, x[3]);
      };
      // later rows do not reach a row, NaN included
      for (int j = 0; j <= i0; ++j) {
        const float4 f = *reinterpret_cast<const float4*>(&sv[j * S::VP + tx * 4]);
        add(out[0], sp[i0 * S::PP + j], f);
        add(out[1], sp[(i0 + 1) * S::PP + j], f);
      }
      add(out[1], sp[(i0 + 1) * S::PP + i0 + 1],
          *reinterpret_cast<const float4*>(&sv[(i0 + 1) * S::VP + tx * 4]));
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (i0 + m < n)
          *reinterpret_cast<float4*>((T*)p.o + ((t0 + i0 + m) * p.H + h) * D + c0) =
              make_float4(p.scale * out[m][0], p.scale * out[m][1], p.scale * out[m][2],
                          p.scale * out[m][3]);
    }
    const float a = s_total;
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) st[i][c] *= a;
    for (int j = 0; j < n; ++j) {
      const float w = s_out[j];
      const float4 f = *reinterpret_cast<const float4*>(&sv[j * S::VP + tx * 4]);
      const float vv[4] = {f.x * w, f.y * w, f.z * w, f.w * w};
      float kk[RPT];
#pragma unroll
      for (int i = 0; i < RPT; i += 4) {
        const float4 r = *reinterpret_cast<const float4*>(&sk[j * S::DP + r0 + i]);
        kk[i] = r.x; kk[i + 1] = r.y; kk[i + 2] = r.z; kk[i + 3] = r.w;
      }
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) st[i][c] = fmaf(kk[i], vv[c], st[i][c]);
    }
  }
  float* exit_state = nullptr;
  if (kStates) {
    exit_state = added + ((int64_t)x.place * p.H + h) * (D * D);
    if (tid == 0 && blockIdx.z == 0) added_log[x.place * p.H + h] = log_sum.x;
  } else if (x.last && p.final_state) {
    exit_state = p.final_state + ((int64_t)x.seq * p.H + h) * (D * D);
  }
  if (exit_state) {
#pragma unroll
    for (int i = 0; i < RPT; ++i)
      *reinterpret_cast<float4*>(exit_state + (int64_t)(r0 + i) * D + c0) =
          make_float4(st[i][0], st[i][1], st[i][2], st[i][3]);
  }
}

// The scan: place j of a sequence goes from the state that segment j adds to the state after it,
// which is the entry state of segment j + 1. One thread per four elements of a (sequence, head).
template <int D>
__global__ void __launch_bounds__(256)
decay_scan_kernel(const DecayParams p, int seg, float* added, const float* added_log) {
  constexpr int kParts = D * D / 1024;
  const int h = blockIdx.y;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Segment y;  // a sequence's first segment scans for all
  if (!find_segment<true>(p, seg, blockIdx.x / kParts, threadIdx.x & 31, false, y) || !y.first) return;
  const int64_t c0 = y.lo, c1 = p.cu ? p.cu[y.seq + 1] : p.total;
  const int e = (blockIdx.x % kParts * 256 + threadIdx.x) * 4;
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (p.init)
    x = *reinterpret_cast<const float4*>(p.init + ((int64_t)y.seq * p.H + h) * (D * D) + e);
  const int64_t first = c0 / seg, n = (c1 - c0 + seg - 1) / seg - 1;
  // four places at a time: their loads do not wait for one another
  for (int64_t j0 = first; j0 < first + n; j0 += 4) {
    const int m = (int)(first + n - j0 < 4 ? first + n - j0 : 4);
    float4 f[4];
    float a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= m) break;
      a[i] = added_log[(j0 + i) * p.H + h];
      f[i] = *reinterpret_cast<const float4*>(added + ((j0 + i) * p.H + h) * (int64_t)(D * D) + e);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= m) break;
      const float b = exp2f(a[i]);
      x = make_float4(fmaf(b, x.x, f[i].x), fmaf(b, x.y, f[i].y), fmaf(b, x.z, f[i].z),
                      fmaf(b, x.w, f[i].w));
      *reinterpret_cast<float4*>(added + ((j0 + i) * p.H + h) * (int64_t)(D * D) + e) = x;
    }
  }
}

// Tokens of a segment: so that all heads' segments are at most one per SM (bf16) or four (CUDA cores:
// 64 value columns each), but not so few that the state that a segment has to write and read outweighs
// them. bf16, with one per SM and with two: 65536 tokens x 4 heads 99 and 115 us, 40 prompts up to 1000
// x 16 heads 95 and 112; where heads do not divide the SMs, segments are missing: 16384 x 32 180 and 178,
// x 40 230 and 217, x 64 336 and 349, x 80 (one segment, half of the SMs) 456 and 452. At least 256
// tokens: 2048 x 8 29 us, with 512 37; 8192 x 2 31 us, with 128 36, with 512 37. (But 300 x 4 17 us in
// one, 22 in three.)
// fp32, 5 prompts up to 1301 x 6: 50 us, with 256 tokens at least 84; 8192 x 16: 605, with half as
// many segments 650, with twice as many 671.
int segment_tokens(kda_dtype dt, int total, int H, int d) {
  const int64_t units = (int64_t)H * (dt == KDA_BF16 ? 1 : d / kCols);
  const int64_t all = dt == KDA_BF16 ? kSms : 4 * kSms, want = units < all ? all / units : 1;
  const int64_t seg = ((total + want - 1) / want + 63) / 64 * 64;
  const int64_t least = dt != KDA_BF16 ? 64 : total > 512 ? 256 : 512;
  return (int)(seg < least ? least : seg);
}

template <int D>
kda_status launch_simt(const DecayParams& p, int seg, float* added, float* added_log,
                       cudaStream_t s) {
  const size_t smem = SimtShape<D>::floats * sizeof(float);
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    cudaFuncSetAttribute(decay_chunk_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         (int)smem);
    cudaFuncSetAttribute(decay_chunk_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         (int)smem);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  const dim3 grid((unsigned)(p.total / seg + p.n_seqs), (unsigned)p.H, D / kCols);
  if (p.total > seg) {
    const dim3 places((unsigned)(p.total / seg), (unsigned)p.H, D / kCols);
    decay_chunk_kernel<D, true><<<places, kSimtThreads, smem, s>>>(p, seg, added, added_log);
    launch_decay_scan(p, D, seg, added, added_log, s);
    count_launches(1);
  }
  decay_chunk_kernel<D, false><<<grid, kSimtThreads, smem, s>>>(p, seg, added, added_log);
  count_launches(1);
  return check_launch("kda_decay_prefill");
}

}  // namespace

namespace decay {

void launch_decay_scan(const DecayParams& p, int d, int seg, float* added, const float* added_log,
                       cudaStream_t s) {
  const dim3 grid((unsigned)(p.total / seg * (d * d / 1024)), (unsigned)p.H);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (d == 128) cudaLaunchKernelEx(&cfg, decay_scan_kernel<128>, p, seg, added, added_log);
  else cudaLaunchKernelEx(&cfg, decay_scan_kernel<64>, p, seg, added, added_log);
  count_launches(1);
}

}  // namespace decay

size_t decay_prefill_workspace_bytes(kda_dtype dt, int total, int H, int d) {
  const int seg = segment_tokens(dt, total, H, d);
  if (total <= seg) return 0;
  return (size_t)(total / seg) * H * ((size_t)d * d + 1) * sizeof(float);
}

kda_status launch_decay_prefill(const DecayParams& p, kda_dtype dt, int d, cudaStream_t s) {
  const int seg = segment_tokens(dt, p.total, p.H, d);
  float* added = (float*)p.ws;
  float* added_log = added ? added + (int64_t)(p.total / seg) * p.H * (d * d) : nullptr;
  if (dt == KDA_BF16) return launch_tc(p, d, seg, added, added_log, s);
  return d == 128 ? launch_simt<128>(p, seg, added, added_log, s)
                  : launch_simt<64>(p, seg, added, added_log, s);
}

kda_status launch_decay_window(const DecayParams& p, kda_dtype dt, int d, cudaStream_t s) {
  if (dt == KDA_BF16)
    return d == 128 ? launch_window_t<128, __nv_bfloat16>(p, s)
                    : launch_window_t<64, __nv_bfloat16>(p, s);
  return d == 128 ? launch_window_t<128, float>(p, s) : launch_window_t<64, float>(p, s);
}

}  // namespace kda
