// The paged 8-bit K/V cache: quantising new tokens as they are written (kda_cache_write) and
// reading them back (kda_cache_read).
//
// A page holds 64 tokens; each (page, head) has one power-of-two scale s, with m <= 448 s for
// the largest value m that was written. Division by s is then exact, the codes do not depend on
// the precision of the arithmetic, and since e4m3 is a floating format the relative precision
// does not depend on s as long as values stay above its subnormals. When a later token needs a
// larger scale, the codes that the page already holds are multiplied by the (power of two) ratio:
// exact again but for codes that fall into the subnormals.
//
// Both passes are HBM streams (write: an element in, a byte out; read: the reverse). The work
// items are (page of a sequence, head, k or v): one CTA owns the page's slice, so that scale and
// codes change without atomics, and holds all its new values in registers between the maximum
// and the rounding (8 chunks of 16 bytes a thread), so that they are read once. 16384 tokens x 32
// heads at d = 128 in bf16, one GB300: written in 69 us (5.8 TB/s, 86% of the copy rate; 73 with
// 16 rows a pass in 256 threads; with a streaming hint on the codes 66, but then what reads them
// next finds fewer in L2 and the pair is 2 us slower), read back in 63 us (6.4 TB/s, 95%; 65
// with 128 threads).
#include "kda_internal.cuh"
#include "kda_fp8.cuh"

namespace kda {
namespace {

// Items: sequence s owns the numbers cu[s] / 64 + 2 s .. cu[s+1] / 64 + 2 (s+1) - 1, which are at
// least as many as the pages that any start makes it touch (a run of n tokens touches at most
// n / 64 + 2 pages).
int cache_items(const CacheParams& p) { return p.total / kPage + 2 * p.n_seqs; }

struct PageRun {
  int seq;
  int64_t page;   // page id
  int64_t first;  // position of the page's first token
  int64_t lo, hi; // positions covered, absolute
  int64_t tok0;   // packed row of position lo
  bool present;   // page is in the pool
};

// The item's page and the positions in it that the sequence covers. false: nothing to do.
__device__ __forceinline__ bool find_run(const CacheParams& p, int item, bool flag, PageRun& r) {
  int a = 0, b = p.n_seqs - 1;  // the last sequence whose first item is <= item
  if (p.cu) {
    while (a < b) {
      const int m = (a + b + 1) >> 1;
      if (p.cu[m] / kPage + 2 * m <= item) a = m;
      else b = m - 1;
    }
  }
  const int64_t c0 = p.cu ? p.cu[a] : 0;
  int64_t c1 = p.cu ? p.cu[a + 1] : p.total;
  if (c0 < 0 || c1 > p.total || c1 < c0) {
    if (flag && p.status) atomicOr(p.status, KDA_STATUS_BAD_OFFSETS);
    return false;
  }
  if (p.lens) {
    const int64_t len = p.lens[a] > 0 ? p.lens[a] : 0;
    if (c0 + len < c1) c1 = c0 + len;
  }
  const int64_t local = item - (c0 / kPage + 2 * (int64_t)a);
  const int64_t st = p.start[a];
  r.seq = a;
  r.present = st >= 0;
  const int64_t s0 = st >= 0 ? st : 0;  // a skipped sequence is still walked (reads give zeros)
  const int64_t blk = s0 / kPage + local;
  r.first = blk * kPage;
  r.lo = r.first > s0 ? r.first : s0;
  const int64_t end = s0 + (c1 - c0);
  r.hi = r.first + kPage < end ? r.first + kPage : end;
  if (local < 0 || r.lo >= r.hi) return false;
  r.tok0 = c0 + (r.lo - s0);
  r.page = -1;
  if (r.present) {
    if (blk >= p.max_pages) {
      if (flag && p.status) atomicOr(p.status, KDA_STATUS_BAD_PAGE);
    } else {
      r.page = p.table[(int64_t)a * p.max_pages + blk];
      if (r.page >= p.n_pages) {
        if (flag && p.status) atomicOr(p.status, KDA_STATUS_BAD_PAGE);
        r.page = -1;
      }
    }
  }
  r.present = r.page >= 0;
  return true;
}

template <class T, int D>
struct WriteShape {
  static constexpr int N = Vec16<T>::N;
  static constexpr int LPR = D / N;          // threads per token row
  static constexpr int ROWS = 8;             // rows per pass
  static constexpr int THREADS = LPR * ROWS;
  static constexpr int PASSES = kPage / ROWS;
};

template <class T, int D>
__global__ void __launch_bounds__(WriteShape<T, D>::THREADS)
cache_write_kernel(const CacheParams p) {
  using S = WriteShape<T, D>;
  constexpr int N = S::N;
  __shared__ uint32_t wmax[S::THREADS / 32];
  const int h = blockIdx.y, side = blockIdx.z;
  PageRun r;
  if (!find_run(p, blockIdx.x, threadIdx.x == 0 && h == 0 && side == 0, r) || !r.present) return;
  const int row = threadIdx.x / S::LPR, e0 = (threadIdx.x % S::LPR) * N;
  const int lo = (int)(r.lo - r.first), hi = (int)(r.hi - r.first);

  const T* x = (const T*)p.x[side] + (int64_t)h * D + e0;
  uint4 raw[S::PASSES];
#pragma unroll
  for (int i = 0; i < S::PASSES; ++i) {
    const int t = i * S::ROWS + row;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (t >= lo && t < hi)
      raw[i] = __ldcs(reinterpret_cast<const uint4*>(x + (r.tok0 + (t - lo)) * p.stride[side]));
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < S::PASSES; ++i) {
    float f[N];
    Vec16<T>::unpack(raw[i], f);
#pragma unroll
    for (int j = 0; j < N; ++j) m = max(m, finite_abs_bits(f[j]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  float* sp = p.scale[side] + r.page * p.H + h;
  const float s_old = lo > 0 ? *sp : 0.0f;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < S::THREADS / 32; ++i) m = max(m, wmax[i]);
  float s = pow2f(scale_exponent(m));
  uint8_t* code = p.code[side] + (r.page * p.H + h) * (int64_t)(kPage * D);
  if (s_old >= s) {
    s = s_old;
  } else if (lo > 0) {  // the kept tokens' codes move to the larger scale
    const float ratio = s_old / s;
    uint4* c4 = reinterpret_cast<uint4*>(code);
    for (int i = threadIdx.x; i < lo * D / 16; i += S::THREADS) {
      uint4 c = c4[i];
      uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = f32x2_from_f16x2(f16x2_from_e4m3(w[j] & 0xffffu));
        const float2 b = f32x2_from_f16x2(f16x2_from_e4m3(w[j] >> 16));
        w[j] = e4m3x2_from_f32(a.x * ratio, a.y * ratio) |
               e4m3x2_from_f32(b.x * ratio, b.y * ratio) << 16;
      }
      c4[i] = c;
    }
  }
  // 1 / s: exact, s is a power of two
  const float inv = 1.0f / s;
#pragma unroll
  for (int i = 0; i < S::PASSES; ++i) {
    const int t = i * S::ROWS + row;
    if (t < lo || t >= hi) continue;
    float f[N];
    Vec16<T>::unpack(raw[i], f);
    uint32_t w[N / 4];
#pragma unroll
    for (int j = 0; j < N / 4; ++j)
      w[j] = e4m3x2_from_f32(f[4 * j] * inv, f[4 * j + 1] * inv) |
             e4m3x2_from_f32(f[4 * j + 2] * inv, f[4 * j + 3] * inv) << 16;
    if constexpr (N == 8)
      *reinterpret_cast<uint2*>(code + t * D + e0) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(code + t * D + e0) = w[0];
  }
  if (threadIdx.x == 0) *sp = s;
}

constexpr int kReadThreads = 256;

template <class T, int D>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const CacheParams p) {
  constexpr int N = Vec16<T>::N;
  constexpr int LPR = D / 16;                   // threads per token row (16 codes each)
  constexpr int ROWS = kReadThreads / LPR;
  constexpr int PASSES = kPage / ROWS;
  const int h = blockIdx.y, side = blockIdx.z;
  if (!p.x[side]) return;
  PageRun r;
  if (!find_run(p, blockIdx.x, threadIdx.x == 0 && h == 0 && (side == 0 || !p.x[0]), r)) return;
  const int row = threadIdx.x / LPR, e0 = (threadIdx.x % LPR) * 16;
  const int lo = (int)(r.lo - r.first), hi = (int)(r.hi - r.first);
  uint4 raw[PASSES];
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
  if (r.present) {
    s = p.scale[side][r.page * p.H + h];
    const uint8_t* code = p.code[side] + (r.page * p.H + h) * (int64_t)(kPage * D);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int t = i * ROWS + row;
      if (t >= lo && t < hi) raw[i] = __ldcs(reinterpret_cast<const uint4*>(code + t * D + e0));
    }
  }
  T* out = (T*)p.x[side] + (int64_t)h * D + e0;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int t = i * ROWS + row;
    if (t < lo || t >= hi) continue;
    float f[16];
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = f32x2_from_f16x2(f16x2_from_e4m3(w[j] & 0xffffu));
      const float2 b = f32x2_from_f16x2(f16x2_from_e4m3(w[j] >> 16));
      f[4 * j] = a.x * s; f[4 * j + 1] = a.y * s;
      f[4 * j + 2] = b.x * s; f[4 * j + 3] = b.y * s;
    }
    if (!r.present) {
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = 0.0f;
    }
    uint4* o = reinterpret_cast<uint4*>(out + (r.tok0 + (t - lo)) * p.stride[side]);
#pragma unroll
    for (int j = 0; j < 16 / N; ++j) __stcs(o + j, Vec16<T>::pack(f + j * N));
  }
}

template <class T, int D>
kda_status launch_write_t(const CacheParams& p, cudaStream_t s) {
  dim3 grid((unsigned)cache_items(p), (unsigned)p.H, 2);
  cache_write_kernel<T, D><<<grid, WriteShape<T, D>::THREADS, 0, s>>>(p);
  count_launches(1);
  return check_launch("kda_cache_write");
}
template <class T, int D>
kda_status launch_read_t(const CacheParams& p, cudaStream_t s) {
  dim3 grid((unsigned)cache_items(p), (unsigned)p.H, 2);
  cache_read_kernel<T, D><<<grid, kReadThreads, 0, s>>>(p);
  count_launches(1);
  return check_launch("kda_cache_read");
}

}  // namespace

kda_status launch_cache_write(const CacheParams& p, kda_dtype dt, int d, cudaStream_t s) {
  if (dt == KDA_BF16)
    return d == 128 ? launch_write_t<__nv_bfloat16, 128>(p, s)
                    : launch_write_t<__nv_bfloat16, 64>(p, s);
  return d == 128 ? launch_write_t<float, 128>(p, s) : launch_write_t<float, 64>(p, s);
}

kda_status launch_cache_read(const CacheParams& p, kda_dtype dt, int d, cudaStream_t s) {
  if (dt == KDA_BF16)
    return d == 128 ? launch_read_t<__nv_bfloat16, 128>(p, s)
                    : launch_read_t<__nv_bfloat16, 64>(p, s);
  return d == 128 ? launch_read_t<float, 128>(p, s) : launch_read_t<float, 64>(p, s);
}

}  // namespace kda
