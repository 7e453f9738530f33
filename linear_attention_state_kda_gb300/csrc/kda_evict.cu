// Eviction from the paged 8-bit cache by accumulated attention weight: adding a window's softmax
// weights to a weight per cached token and head (kda_cache_weigh), and keeping a budget of tokens
// by these weights, moved into new pages (kda_cache_evict).
#include <cuda_fp16.h>

#include "kda_internal.cuh"
#include "kda_fp8.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

// ---------------------------------------------------------------- weighing
//
//     weight[t] = keep * weight[t] + sum_i exp(s_it - lse_i),   s_it = scale q_i . k_t
//
// over the query rows i (tokens of the window x query heads of the group) that see position t, for
// up to 64 rows (or fp32, or d = 64; else kda_weigh_tc.cu).
//
// Bound by the K codes, d bytes a key. A cluster owns one (row, key/value head) and its CTAs
// contiguous ranges of its pages, so that the codes are read once: the scores stay in shared
// memory while the row statistics (running maximum and sum) are joined over the cluster, and become
// weights there. Keys beyond the room for scores are scored again. (Clusters do not fill the GPU
// where there are few of them: 8 clusters of 16 CTAs land on 64 SMs. There the statistics are taken
// by one launch and the weights by a second that scores again, mostly from L2: one row of 131072
// tokens and 8 heads took 286 us as clusters of 8, 66 us so.)
//
// A warp takes a page, 32 keys in flight at once (with 64, 341 us where 32 take 280: fewer CTAs per
// SM); its id and scale are fetched with those of the warp's next pages. Scores are warp-level f16
// MMAs with the keys as the rows: 16 keys x 16 channels times 16 channels x 8 query rows. The sum
// over the channels is in any order, so lane (g, t) takes channels 16 t .. and 64 + 16 t .. of keys
// g and g + 8 from global memory in 16-byte loads (four lanes read 64 bytes on end: whole sectors),
// which are the A fragments after widening (e4m3 to f16 is exact). Query rows are scaled by a power
// of two into f16's upper range: bf16 entries down to 2^-30 of the row's largest are exact, fp32
// entries are two f16 parts.
//
// Measured, Hq 32, Hkv 8, d 128: 128 rows of 16384 tokens, one query token each, 280 us (4.6 TB/s
// of codes); 16 rows of 8192 with 4 query tokens 48 us; the same with 2 in fp32 35 us; 2 rows of 100
// 8.9 us, which is latency: ids, codes, the cluster's two barriers.
constexpr int kWThreads = 128, kWMaxWarps = kWThreads / 32;
// Query rows whose statistics the two launches keep at a time (a window of more takes further pairs):
// the workspace does not grow with the window past 8 KB for each range of keys. A multiple of 32.
constexpr int kStatRows = 1024;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 64-bit word at `p` of the cluster's CTA `rank` holds two floats.
__device__ __forceinline__ float2 ld_cluster_f2(const float2* p, uint32_t rank) {
  const uint64_t v = ptx::ld_cluster_u64(reinterpret_cast<const uint64_t*>(p), rank);
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}

// (m, l) of two parts of a row's keys.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x), at = m == -INFINITY ? 0.0f : m;
  return make_float2(m, a.y * ptx::ex2_approx(a.x - at) + b.y * ptx::ex2_approx(b.x - at));
}

// NT: tiles of 8 query rows scored at once. P: f16 parts of a query. How a unit's keys are shared:
// by a cluster of `cs` CTAs, or by `cs` CTAs of a launch that takes the statistics and of one that sums
// the weights, each for query rows row0 .. row0 + stat_rows - 1 (a cluster takes all).
enum Share { kCluster, kStats, kWeights };
template <int D, int NT, int P, class T, Share kShare>
__global__ void __launch_bounds__(kWThreads, NT == 1 ? 6 : 4)
weigh_kernel(const WeighParams p, int cs, int cap_keys, int row0, int stat_rows) {
  constexpr int KC = D / 16;      // 16-channel steps
  constexpr int LB = D / 4;       // bytes of a key per lane
  constexpr int ROWS = NT * 8;
  constexpr int BT = 2;           // tiles of 16 keys in flight: half a page
  extern __shared__ __align__(16) unsigned char wsm[];
  // query fragments [P][NT][KC][32 lanes] x 8 bytes, then the scores [rows][cap_keys + 4] (a row
  // begins 4 banks on: the 8 keys x 4 rows of an accumulator register fall into distinct banks)
  uint2* frag = reinterpret_cast<uint2*>(wsm);
  float* score = reinterpret_cast<float*>(wsm + (size_t)P * NT * KC * 256);
  const int stride = cap_keys + 4;
  __shared__ float row_mul[ROWS];          // 2^e of a query row
  __shared__ float2 part[kWMaxWarps][ROWS];
  __shared__ float2 cta_ml[ROWS];
  __shared__ float row_lse[ROWS];

  const int rank = blockIdx.x % cs, bh = blockIdx.x / cs;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  constexpr int warps = kWMaxWarps;
  const int start = p.start[b];
  int n = start < 0 ? 0 : p.lens ? p.lens[b] : p.window;
  n = n < 0 ? 0 : n > p.window ? p.window : n;
  if (n == 0) return;  // the whole cluster
  const int G = p.Hq / p.Hkv, R = kShare == kCluster ? n * G : min(n * G, row0 + stat_rows);
  const int64_t most = (int64_t)p.max_pages * kPage;  // at most 2^30
  const int keys = (int)((int64_t)start + n < most ? (int64_t)start + n : most);
  if (kShare != kWeights && rank == 0 && tid == 0 && h == 0 && p.status && (int64_t)start + n > most)
    atomicOr(p.status, KDA_STATUS_BAD_PAGE);
  const int pages = (keys + kPage - 1) / kPage;
  const int per = (pages + cs - 1) / cs;
  const int pg0 = min(pages, rank * per), pg1 = min(pages, pg0 + per);
  const int32_t* table = p.table + (int64_t)b * p.max_pages;

  // Ids and scales (times scale log2 e) of the warp's pages pg0 + warp + warps * k: lane l has those
  // of k = base + l.
  int id_l = -1, have = -1;
  float ks_l = 0.0f;
  auto fetch = [&](int k) {  // (k the same in all lanes)
    if (have >= 0 && k >= have && k < have + 32) return;
    have = k & ~31;
    const int pg = pg0 + warp + warps * (have + lane);
    id_l = pg < pg1 ? table[pg] : -1;
    if (id_l >= p.n_pages) {
      if (p.status) atomicOr(p.status, KDA_STATUS_BAD_PAGE);
      id_l = -1;
    }
    ks_l = id_l < 0 ? 0.0f : p.ks[(int64_t)id_l * p.Hkv + h] * (p.scale * kLog2e);
  };
  {  // (the first pages' ids on their way before the queries)
    const int pg = pg0 + warp + warps * lane;
    if (pg < pg1) asm volatile("prefetch.global.L1 [%0];" ::"l"(table + pg));
  }

  for (int r0 = kShare == kCluster ? 0 : row0; r0 < R; r0 += ROWS) {
    const int rows = min(ROWS, R - r0);
    __syncthreads();
    // the group's query rows: scale, then fragments. A warp takes a row.
    for (int r = warp; r < ROWS; r += warps) {
      float f[D / 32];
      float m = 0.0f;
      const int row = r0 + r;
      const int j = row / G, gh = row - j * G;
      const T* q = (const T*)p.q + (((int64_t)b * p.window + j) * p.Hq + h * G + gh) * D;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        f[i] = r < rows ? ld_elem(q, lane * (D / 32) + i) : 0.0f;
        m = fmaxf(m, __uint_as_float(finite_abs_bits(f[i])));
      }
      m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
      // 2^e with m 2^-e in [2^14, 2^15); e from the bits, m = 0 counts as 2^-126
      const int ex = (int)(__float_as_uint(m) >> 23);
      const int e = (ex ? ex : 1) - 127 - 14;  // -140 .. 113
      const float down = e > 0 ? pow2f(-e) : 1.0f;
      const float up1 = e < 0 ? pow2f(-e < 126 ? -e : 126) : 1.0f;
      const float up2 = e < -126 ? pow2f(-e - 126) : 1.0f;
      // channel c of the row: in 16-byte piece c / 16, of lane c / 16 % 4 and its load c / 64
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const float x = f[i] * down * up1 * up2;
        const int c = lane * (D / 32) + i;
        const int tq = c / 16 % 4, kc = c / 64 * 4 + c % 16 / 4, el = c % 4;
        __half hi = __float2half_rn(x);
        __half* dst = reinterpret_cast<__half*>(
            &frag[(((r >> 3) * KC) + kc) * 32 + (r & 7) * 4 + tq]);
        dst[el] = hi;
        if (P == 2) {
          float lo = x - __half2float(hi);
          if (!(fabsf(lo) <= 64.0f)) lo = 0.0f;  // of an infinity or NaN
          dst[(size_t)NT * KC * 128 + el] = __float2half_rn(lo);
        }
      }
      // (2^e may be below the normal numbers, and nothing but a power of two is exact there)
      if (lane == 0) row_mul[r] = pow2f(e < -126 ? -126 : e) * (e < -126 ? pow2f(e + 126) : 1.0f);
    }
    __syncthreads();

    // Codes that the second launch reads again stay in L2 where they fit: 2 rows of 65536 tokens 48 us,
    // marked to be evicted first 54; 64 fp32 tokens over one row of 32768 673 and 706. (The same for a
    // cluster's further query rows, asked at run time: 64 tokens over 16 rows of 2048 at d = 64 169 us for
    // 187, but 8 tokens over 16 rows of 8192, which have none, 99 for 93.)
    constexpr bool read_again = kShare == kStats;
    // the last token of the group sees the most, its first token the least
    const int seen = (int)min((int64_t)keys, (int64_t)start + (r0 + rows - 1) / G + 1);
    const int64_t seen_by_all = (int64_t)start + r0 / G + 1;
    // the lane's rows 2 t4, 2 t4 + 1 of each tile: how far they see, their factors and statistics
    int vis[NT][2];
    float mul[NT][2];
    float2 ml[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = i * 8 + t4 * 2 + e;
        vis[i][e] = r < rows ? (int)min((int64_t)keys, (int64_t)start + (r0 + r) / G + 1) : 0;
        mul[i][e] = row_mul[r];
        ml[i][e] = make_float2(-INFINITY, 0.0f);
      }

    // Scores of tiles t0 .. t0 + BT - 1 (16 keys each) of a page in base-2 exponents, masked.
    auto score_tiles = [&](int id, float ks, int page, int t0, float (&acc)[BT][NT][4]) {
      const uint8_t* base =
          p.kc + ((int64_t)id * p.Hkv + h) * (int64_t)(kPage * D) + (t0 * 16 + g) * D + t4 * 16;
      uint32_t w[BT][2][LB / 4];
#pragma unroll
      for (int t = 0; t < BT; ++t)
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < LB / 16; ++i) {
            const uint4* src = reinterpret_cast<const uint4*>(base + (t * 16 + 8 * half) * D + 64 * i);
            *reinterpret_cast<uint4*>(&w[t][half][4 * i]) = read_again ? *src : __ldcs(src);
          }
#pragma unroll
      for (int t = 0; t < BT; ++t) {
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.0f;
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) {
          uint32_t a[4];
          f16x4_from_e4m3(w[t][0][kc], a[0], a[2]);
          f16x4_from_e4m3(w[t][1][kc], a[1], a[3]);
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int part_i = 0; part_i < P; ++part_i) {
              const uint2 q2 = frag[((part_i * NT + i) * KC + kc) * 32 + lane];
              mma16816(acc[t][i], a, q2.x, q2.y);
            }
        }
      }
      const bool whole = (int64_t)(page + 1) * kPage <= seen_by_all;
#pragma unroll
      for (int t = 0; t < BT; ++t)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][i][e] *= ks * mul[i][e & 1];
      if (!whole) {
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int pos = page * kPage + (t0 + t) * 16 + g + 8 * (e >> 1);
              acc[t][i][e] = pos < vis[i][e & 1] ? acc[t][i][e] : -INFINITY;
            }
      }
    };

    for (int k = 0, pg = pg0 + warp; kShare != kWeights && pg < pg1; ++k, pg += warps) {
      if ((int64_t)pg * kPage >= seen) break;
      fetch(k);
      const int id = __shfl_sync(0xffffffffu, id_l, k & 31);
      if (id < 0) continue;
      const float ks = __shfl_sync(0xffffffffu, ks_l, k & 31);
      const int local = (pg - pg0) * kPage;
      if (kShare == kCluster && lane < 2)  // the page's weights, for later
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.weights + ((int64_t)id * p.Hkv + h) * kPage +
                                                      32 * lane));
#pragma unroll 1
      for (int t0 = 0; t0 < kPage / 16; t0 += BT) {
        float acc[BT][NT][4];
        score_tiles(id, ks, pg, t0, acc);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float2& s = ml[i][e];
            float m = s.x;
#pragma unroll
            for (int t = 0; t < BT; ++t) m = fmaxf(m, fmaxf(acc[t][i][e], acc[t][i][e + 2]));
            const float at = m == -INFINITY ? 0.0f : m;
            float l = s.y * ptx::ex2_approx(s.x - at);
#pragma unroll
            for (int t = 0; t < BT; ++t)
              l += ptx::ex2_approx(acc[t][i][e] - at) + ptx::ex2_approx(acc[t][i][e + 2] - at);
            s = make_float2(m, l);
          }
        if (local < cap_keys) {
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = i * 8 + t4 * 2 + e;
              if (r < rows) {
                float* dst = score + r * stride + local + t0 * 16 + g;
#pragma unroll
                for (int t = 0; t < BT; ++t) {
                  dst[t * 16] = acc[t][i][e];
                  dst[t * 16 + 8] = acc[t][i][e + 2];
                }
              }
            }
        }
      }
    }
    // row statistics: lanes of a row, warps, CTAs (16 lanes to a row)
    auto of_row = [&](float2 s) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
        s = join(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o),
                                __shfl_xor_sync(0xffffffffu, s.y, o)));
      return s;
    };
    // a row that sees nothing adds nothing, nor does one past the last
    auto set_lse = [&](int r, float2 s) {
      const bool none = r >= rows || (s.x == -INFINITY && !(s.y != s.y));
      row_lse[r] = none ? INFINITY : (s.x == -INFINITY ? 0.0f : s.x) + log2f(s.y);
    };
    float2* stats = kShare == kCluster ? nullptr : p.stats + (int64_t)bh * cs * stat_rows + (r0 - row0);
    if (kShare != kWeights) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float2 s = ml[i][e];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            s = join(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o),
                                    __shfl_xor_sync(0xffffffffu, s.y, o)));
          if (g == 0) part[warp][i * 8 + t4 * 2 + e] = s;
        }
      __syncthreads();
      for (int i = tid; i < ROWS * 16; i += kWThreads) {
        const int r = i >> 4, w = i & 15;
        const float2 s = of_row(w < kWMaxWarps ? part[w][r] : make_float2(-INFINITY, 0.0f));
        if (w == 0) {
          if (kShare == kCluster) cta_ml[r] = s;
          else if (r < rows) stats[(int64_t)rank * stat_rows + r] = s;
        }
      }
    }
    if (kShare == kStats) continue;
    if (kShare == kCluster) {
      ptx::cluster_sync();
      for (int i = tid; i < ROWS * 16; i += kWThreads) {
        const int r = i >> 4, c = i & 15;
        const float2 s = of_row(c < cs ? ld_cluster_f2(&cta_ml[r], c) : make_float2(-INFINITY, 0.0f));
        if (c == 0) set_lse(r, s);
      }
      __syncthreads();
      ptx::cluster_arrive();  // this CTA has read the others' statistics; waited for below
    } else {
      for (int i = tid; i < ROWS * 16; i += kWThreads) {
        const int r = i >> 4;
        float2 s = make_float2(-INFINITY, 0.0f);
        for (int c = i & 15; c < cs && r < rows; c += 16)
          s = join(s, stats[(int64_t)c * stat_rows + r]);
        s = of_row(s);
        if ((i & 15) == 0) set_lse(r, s);
      }
      __syncthreads();
    }

    // weights: from the scores in shared memory, else scored again
    const bool fresh = r0 == 0;
    for (int k = 0, pg = pg0 + warp; pg < pg1; ++k, pg += warps) {
      fetch(k);
      const int id = __shfl_sync(0xffffffffu, id_l, k & 31);
      if (id < 0) continue;
      const int local = (pg - pg0) * kPage;
      const bool reached = (int64_t)pg * kPage < seen;
      if (!reached && !fresh) continue;
      float* wp = p.weights + ((int64_t)id * p.Hkv + h) * kPage;
      if (local < cap_keys || !reached) {
        // lane l: keys 2 l and 2 l + 1 of the page
        const int at = 2 * lane, pos = pg * kPage + at;
        float2 sum = make_float2(0.0f, 0.0f), old = sum;
        if (pos < keys && (!fresh || (pos < start && p.keep != 0.0f)))
          old = *reinterpret_cast<const float2*>(wp + at);
        if (reached)
          for (int r = 0; r < rows; ++r) {
            const float2 x = *reinterpret_cast<const float2*>(&score[r * stride + local + at]);
            sum.x += ptx::ex2_approx(x.x - row_lse[r]);
            sum.y += ptx::ex2_approx(x.y - row_lse[r]);
          }
        if (fresh) {
          old.x = pos < start && p.keep != 0.0f ? p.keep * old.x : 0.0f;
          old.y = pos + 1 < start && p.keep != 0.0f ? p.keep * old.y : 0.0f;
        }
        if (pos + 1 < keys)
          *reinterpret_cast<float2*>(wp + at) = make_float2(old.x + sum.x, old.y + sum.y);
        else if (pos < keys)
          wp[at] = old.x + sum.x;
      } else {
        const float ks = __shfl_sync(0xffffffffu, ks_l, k & 31);
#pragma unroll 1
        for (int t0 = 0; t0 < kPage / 16; t0 += BT) {
          float acc[BT][NT][4];
          score_tiles(id, ks, pg, t0, acc);
#pragma unroll
          for (int t = 0; t < BT; ++t) {
            float sum[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                sum[e >> 1] += ptx::ex2_approx(acc[t][i][e] - row_lse[i * 8 + t4 * 2 + (e & 1)]);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              sum[half] += __shfl_xor_sync(0xffffffffu, sum[half], 1);
              sum[half] += __shfl_xor_sync(0xffffffffu, sum[half], 2);
              const int at = (t0 + t) * 16 + g + 8 * half, pos = pg * kPage + at;
              if (t4 == 0 && pos < keys) {
                const float old =
                    !fresh ? wp[at] : pos < start && p.keep != 0.0f ? p.keep * wp[at] : 0.0f;
                wp[at] = old + sum[half];
              }
            }
          }
        }
      }
    }
    if (kShare == kCluster) {
      // the others have read this CTA's statistics: they may be written again, or the CTA leave
      __syncwarp();
      ptx::cluster_wait();
    }
  }
}

// CTAs that share a unit's keys. Few units with long contexts take two launches: 16 units of 65536
// tokens 106 us as clusters, 49 so; 16 units of 32768 with 16 query rows 90 and 40; but 32 units of
// 32768 47 and 54, 32 of 8192 19 and 25, 8 of 8192 17 and 21. One CTA of a wave to a range: 6 per SM, 4 with more rows.
struct Sharing {
  bool cluster;
  int cs;
};
Sharing sharing_of(int batch, int Hkv, int rows, int max_pages) {
  const int64_t units = (int64_t)batch * Hkv;
  if (units < 32 && max_pages >= 512) {
    const int64_t most = kSms * (rows <= 8 ? 6 : 4) / units, cs = max_pages / 4;
    return {false, (int)(cs < most ? cs : most)};
  }
  // a cluster: up to 2048 keys to a CTA (128 rows of 16384 tokens, 8 heads: 280 us; with 8192, 314;
  // with 1024 the same as with 2048), fewer where the units are few
  int cs = 1;
  const int64_t keys = (int64_t)max_pages * kPage;
  while (cs < 8 && max_pages > cs && (keys > (int64_t)cs * 2048 || units * cs < 128))
    cs *= 2;
  return {true, cs};
}

template <int D, int NT, int P, class T>
kda_status launch_weigh_nt(const WeighParams& p, cudaStream_t s) {
  const int64_t units = (int64_t)p.batch * p.Hkv;
  const Sharing sh = sharing_of(p.batch, p.Hkv, p.max_rows, p.max_pages);
  constexpr size_t frag = (size_t)P * NT * (D / 16) * 256;
  static_assert(frag <= 32 * 1024, "shared memory");
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    const auto kernel = weigh_kernel<D, NT, P, T, kCluster>;
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
    cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  const unsigned grid = (unsigned)(units * sh.cs);
  if (!sh.cluster) {
    const int at_once = p.max_rows < kStatRows ? p.max_rows : kStatRows;
    for (int r = 0; r < p.max_rows; r += at_once) {
      weigh_kernel<D, NT, P, T, kStats><<<grid, kWThreads, frag, s>>>(p, sh.cs, 0, r, at_once);
      weigh_kernel<D, NT, P, T, kWeights><<<grid, kWThreads, frag, s>>>(p, sh.cs, 0, r, at_once);
      count_launches(2);
    }
    return check_launch("kda_cache_weigh");
  }
  const int64_t rows64 = (int64_t)(p.Hq / p.Hkv) * p.window;
  const int rows = rows64 < NT * 8 ? (int)rows64 : NT * 8;
  const int64_t per = (p.max_pages + sh.cs - 1) / sh.cs;
  int64_t cap = (int64_t)((100 * 1024 - frag) / ((size_t)rows * 4) - 4) / kPage;
  if (cap > per) cap = per;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kWThreads);
  cfg.dynamicSmemBytes = frag + (size_t)(cap * kPage + 4) * rows * 4;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)sh.cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, weigh_kernel<D, NT, P, T, kCluster>, p, sh.cs, (int)(cap * kPage), 0, 0);
  count_launches(1);
  return check_launch("kda_cache_weigh");
}
template <int D, int P, class T>
kda_status launch_weigh_t(const WeighParams& p, cudaStream_t s) {
  const int64_t rows = (int64_t)(p.Hq / p.Hkv) * p.window;
  if (rows <= 8) return launch_weigh_nt<D, 1, P, T>(p, s);
  if (rows <= 16) return launch_weigh_nt<D, 2, P, T>(p, s);
  return launch_weigh_nt<D, 4, P, T>(p, s);
}

// ---------------------------------------------------------------- eviction
//
// Two kernels. The first keeps, for each (row, head), the budget's positions: a cluster holds the
// candidates' weights as order-preserving integers in shared memory and finds the smallest one that
// is kept by three rounds of counts (digits of 11, 11 and 10 bits, the first counted as the weights
// arrive), then writes the kept positions in order, each warp those of its own range. Latency: five
// cluster barriers around passes over shared memory. (Four rounds of 8 bits, warps agreeing on
// their distinct digits before they count, took 69 us for 32 rows of 16384 tokens and 8 heads; this
// takes 31. 3 rows of 500: 9 us, nearly all latency.)
// The second moves the kept tokens, one CTA per (new page, head). It is bound by the codes, read
// and written once: all of a thread's loads are in flight before the page's scale is known. 32 rows
// of 4096 kept tokens: 88 us, 6.1 TB/s (102 us with the loads after the scale).
constexpr int kEThreads = 512;
constexpr int kEWarps = kEThreads / 32;
constexpr int kEBins = 2048;
static_assert(kEThreads * 4 >= kEBins, "a thread adds up four bins");
constexpr int kEMaxKeys = 49152;  // of a CTA in shared memory, tiles of 128; later ones are read again
static_assert(kEMaxKeys % 128 == 0, "whole tiles");

// Orders like the weights; NaN lowest, zeros of both signs equal. 0 is no candidate.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 1u;
  const uint32_t b = w == 0.0f ? 0u : __float_as_uint(w);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint4 ld_cluster_u32x4(const uint32_t* p, uint32_t rank) {
  uint32_t a;
  uint4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t scan_lanes(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

__global__ void __launch_bounds__(kEThreads) evict_select_kernel(const EvictParams p, int cs, int cap) {
  extern __shared__ __align__(16) uint32_t s_key[];
  __shared__ __align__(16) uint32_t hist[3][kEBins];
  __shared__ uint32_t warp_sum[kEWarps], s_pick[2];
  __shared__ __align__(8) uint32_t s_count[2];
  __shared__ uint2 warp_count[kEWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int rank = blockIdx.x % cs, bh = blockIdx.x / cs;
  const int b = bh / p.Hkv, h = bh % p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int raw = p.length[b];
  int32_t* kept = p.kept + ((int64_t)b * p.Hkv + h) * p.budget;
  if (raw < 0) {  // a padding row: the whole cluster
    for (int i = rank * kEThreads + tid; i < p.budget; i += cs * kEThreads) kept[i] = -1;
    if (rank == 0 && tid == 0 && h == 0) p.new_length[b] = raw;
    return;
  }
  for (int i = tid; i < 3 * kEBins / 4; i += kEThreads)
    reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
  const int64_t most = (int64_t)p.max_pages * kPage;  // at most 2^30
  if (raw > most && rank == 0 && tid == 0 && h == 0 && p.status)
    atomicOr(p.status, KDA_STATUS_BAD_PAGE);
  const int len = (int)(raw < most ? raw : most);
  const int pages = (len + kPage - 1) / kPage, per = (pages + cs - 1) / cs;
  const int pg0 = min(pages, rank * per), pg1 = min(pages, pg0 + per);
  const int first = pg0 * kPage;
  const int n = max(0, min(pg1 * kPage, len) - first);
  const int32_t* table = p.table + (int64_t)b * p.max_pages;
  // the warp's positions: w0 .. w1 - 1 of the CTA's, four on end to a lane, 128 at a time
  const int span = (n + kEWarps * 128 - 1) / (kEWarps * 128) * 128;
  const int w0 = min(n, warp * span), w1 = min(n, w0 + span);

  // the keys of four positions i + .., from the weights
  constexpr int kBatch = 4;
  auto load = [&](int i0, int batch, uint4 (&k)[kBatch]) {
    int id[kBatch];
    float4 w[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * 128 + lane * 4;
      id[u] = u < batch && i < w1 ? table[(first + i) / kPage] : -1;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int pos = first + i0 + u * 128 + lane * 4;
      w[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (id[u] >= 0 && id[u] < p.n_pages)
        w[u] = *reinterpret_cast<const float4*>(
            p.weights + ((int64_t)id[u] * p.Hkv + h) * kPage + (pos & (kPage - 1)));
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int pos = first + i0 + u * 128 + lane * 4;
      auto key = [&](int at, float x) -> uint32_t {
        if (id[u] < 0 || id[u] >= p.n_pages || at >= len) return 0u;
        return at < p.sinks || at >= len - p.recent ? 0xffffffffu : weight_key(x);
      };
      k[u] = make_uint4(key(pos, w[u].x), key(pos + 1, w[u].y), key(pos + 2, w[u].z),
                        key(pos + 3, w[u].w));
      if (id[u] >= p.n_pages && h == 0 && p.status) atomicOr(p.status, KDA_STATUS_BAD_PAGE);
    }
  };
  auto get = [&](int i0) -> uint4 {
    const int i = i0 + lane * 4;
    if (i0 + 128 <= cap) return i < w1 ? *reinterpret_cast<const uint4*>(s_key + i)
                                       : make_uint4(0, 0, 0, 0);
    uint4 k[kBatch];
    load(i0, 1, k);
    return k[0];
  };
  // counts digits (k - prefix) >> shift of the keys in prefix .. prefix + 2^bits - 1
  auto count = [&](uint32_t* bins, const uint4& k4, bool (&in)[4], uint32_t prefix, int shift) {
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    if (!__any_sync(0xffffffffu, in[0] | in[1] | in[2] | in[3])) return;
    const uint32_t lead = __shfl_sync(0xffffffffu, k4.x, 0);
    bool same = in[0] & in[1] & in[2] & in[3];
#pragma unroll
    for (int j = 0; j < 4; ++j) same &= (k[j] ^ lead) >> shift == 0u;
    if (__all_sync(0xffffffffu, same)) {  // equal weights, kept ends: one addition
      if (lane == 0) atomicAdd(&bins[(lead - prefix) >> shift], 128u);
      return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (in[j]) atomicAdd(&bins[(k[j] - prefix) >> shift], 1u);
  };

  __syncthreads();
#pragma unroll 1
  for (int i0 = w0; i0 < w1; i0 += kBatch * 128) {
    uint4 k[kBatch];
    load(i0, kBatch, k);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * 128;
      if (i >= w1) break;
      if (i + 128 <= cap && i + lane * 4 < w1) *reinterpret_cast<uint4*>(s_key + i + lane * 4) = k[u];
      bool in[4] = {k[u].x != 0u, k[u].y != 0u, k[u].z != 0u, k[u].w != 0u};
      count(hist[0], k[u], in, 0u, 21);
    }
  }

  // the smallest kept key, and how many of that value are kept: digits from the top
  uint32_t prefix = 0, left = 0, want = 0;
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
    if (round > 0) {
      // (keys 0 may be counted: they are below any that is kept)
      const uint32_t range = round == 1 ? 1u << 21 : 1u << 10;
#pragma unroll 1
      for (int i0 = w0; i0 < w1; i0 += 128) {
        const uint4 k = get(i0);
        bool in[4] = {k.x - prefix < range, k.y - prefix < range, k.z - prefix < range,
                      k.w - prefix < range};
        count(hist[round], k, in, prefix, shift);
      }
    }
    ptx::cluster_sync();
    // this thread's four bins, the highest digits to the first threads
    const int bin = kEBins - 4 - 4 * tid;
    uint32_t t[4] = {0, 0, 0, 0};
    for (int c = 0; c < cs && bin >= 0; ++c) {
      const uint4 v = ld_cluster_u32x4(&hist[round][bin], c);
      t[0] += v.w; t[1] += v.z; t[2] += v.y; t[3] += v.x;
    }
    const uint32_t sum = t[0] + t[1] + t[2] + t[3];
    uint32_t upto = scan_lanes(sum, lane);
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    const uint32_t of_warps = scan_lanes(lane < kEWarps ? warp_sum[lane] : 0u, lane);
    if (warp > 0) upto += __shfl_sync(0xffffffffu, of_warps, warp - 1);
    if (round == 0) {
      want = min(__shfl_sync(0xffffffffu, of_warps, 31), (uint32_t)p.budget);
      left = want;
      if (want == 0) break;  // (in the whole cluster)
    }
    uint32_t before = upto - sum;
    if (before < left && left <= upto) {
      int j = 0;
      while (before + t[j] < left) before += t[j++];
      s_pick[0] = (uint32_t)(bin + 3 - j);
      s_pick[1] = left - before;
    }
    __syncthreads();
    prefix |= s_pick[0] << shift;
    left = s_pick[1];
  }

  // `prefix` is the smallest kept key; `left` of its positions are kept, the earliest ones.
  // Where this warp's positions begin among the kept: counts of the warps and CTAs before it.
  auto counts = [&](const uint4& k, uint32_t& gt, uint32_t& eq) {
    gt = (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
    eq = (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
  };
  uint32_t gt = 0, eq = 0;
  if (want > 0) {
#pragma unroll 1
    for (int i0 = w0; i0 < w1; i0 += 128) {
      uint32_t g1, e1;
      counts(get(i0), g1, e1);
      gt += g1;
      eq += e1;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) warp_count[warp] = make_uint2(gt, eq);
    __syncthreads();
    const uint2 wc = lane < kEWarps ? warp_count[lane] : make_uint2(0, 0);
    gt = __reduce_add_sync(0xffffffffu, lane < warp ? wc.x : 0u);
    eq = __reduce_add_sync(0xffffffffu, lane < warp ? wc.y : 0u);
    if (warp == kEWarps - 1 && lane == 0) {
      s_count[0] = gt + warp_count[warp].x;
      s_count[1] = eq + warp_count[warp].y;
    }
    ptx::cluster_sync();
    uint64_t of_cta = 0;
    if (lane < rank) of_cta = ptx::ld_cluster_u64(reinterpret_cast<const uint64_t*>(s_count), lane);
    gt += __reduce_add_sync(0xffffffffu, (uint32_t)of_cta);
    eq += __reduce_add_sync(0xffffffffu, (uint32_t)(of_cta >> 32));
  }
  __syncwarp();
  ptx::cluster_arrive();  // this thread has read the others' counts; waited for below
  if (want > 0) {
#pragma unroll 1
    for (int i0 = w0; i0 < w1; i0 += 128) {
      const uint4 k4 = get(i0);
      const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
      uint32_t g1, e1;
      counts(k4, g1, e1);
      const uint32_t own = g1 | e1 << 16, upto = scan_lanes(own, lane);
      uint32_t g = gt + ((upto - own) & 0xffffu), e = eq + ((upto - own) >> 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool is_eq = k[j] == prefix;
        if (k[j] > prefix || (is_eq && e < left)) kept[g + min(e, left)] = first + i0 + lane * 4 + j;
        g += k[j] > prefix;
        e += is_eq;
      }
      const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
      gt += all & 0xffffu;
      eq += all >> 16;
    }
  }
  for (int i = (int)want + rank * kEThreads + tid; i < p.budget; i += cs * kEThreads) kept[i] = -1;
  if (rank == 0 && tid == 0 && h == 0) p.new_length[b] = (int32_t)want;
  __syncwarp();
  ptx::cluster_wait();  // no CTA leaves while its counts are read
}

// Moves 64 kept tokens of a head into a new page. The page's scale is the largest of the tokens'
// pages', so a code moves as it is where its page had that scale, else by an exact power of two
// (rounded again only among the format's subnormals).
constexpr int kMThreads = 256;
template <int D>
__global__ void __launch_bounds__(kMThreads) evict_move_kernel(const EvictParams p) {
  __shared__ int64_t src[kPage];      // row of the caches, -1: none
  __shared__ float scale[2][kPage];
  const int width = (p.budget + kPage - 1) / kPage;
  const int pg = blockIdx.x % width, h = blockIdx.y, b = blockIdx.x / width;
  const int tid = threadIdx.x, lane = tid & 31;
  int dst = -1;
  if (pg < p.new_max_pages) dst = p.new_table[(int64_t)b * p.new_max_pages + pg];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what is kept, of the kernel before
  const int i = pg * kPage + tid;
  int pos = 0;
  if (tid < kPage && i < p.budget) pos = p.kept[((int64_t)b * p.Hkv + h) * p.budget + i];
  const int count = p.new_length[b];
  if (count < 0 || (int64_t)pg * kPage >= count) return;
  if (pg >= p.new_max_pages || dst >= p.n_pages) {
    if (tid == 0 && h == 0 && p.status) atomicOr(p.status, KDA_STATUS_BAD_PAGE);
    return;
  }
  if (dst < 0) return;
  int64_t slice = 0, row = -1;
  if (tid < kPage) {
    if (i < count) {
      slice = (int64_t)p.table[(int64_t)b * p.max_pages + pos / kPage] * p.Hkv + h;
      row = slice * kPage + (pos & (kPage - 1));
    }
    src[tid] = row;
  }
  __syncthreads();
  constexpr int LPR = D / 16, ROWS = kMThreads / LPR, N = kPage / ROWS;
  const int part = tid % LPR * 16, r0 = tid / LPR;
  uint4 c[2][N];
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t at = src[r0 + k * ROWS];
      if (at >= 0) c[side][k] = __ldcs(reinterpret_cast<const uint4*>(p.code[side] + at * D + part));
    }
  if (tid < kPage) {
    scale[0][tid] = row < 0 ? 0.0f : p.scale[0][slice];
    scale[1][tid] = row < 0 ? 0.0f : p.scale[1][slice];
    p.weights[((int64_t)dst * p.Hkv + h) * kPage + tid] = row < 0 ? 0.0f : p.weights[row];
  }
  __syncthreads();
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    float top = fmaxf(scale[side][lane], scale[side][lane + 32]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    uint8_t* out = p.code[side] + ((int64_t)dst * p.Hkv + h) * (int64_t)(kPage * D) + part;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int r = r0 + k * ROWS;
      if (src[r] < 0) continue;
      uint4 v = c[side][k];
      const float old = scale[side][r];
      if (old != top) {
        const float f = old / top;
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = f32x2_from_f16x2(f16x2_from_e4m3(w[j] & 0xffffu));
          const float2 y = f32x2_from_f16x2(f16x2_from_e4m3(w[j] >> 16));
          w[j] = e4m3x2_from_f32(x.x * f, x.y * f) | e4m3x2_from_f32(y.x * f, y.y * f) << 16;
        }
      }
      *reinterpret_cast<uint4*>(out + r * D) = v;
    }
    if (tid == 0) p.scale[side][(int64_t)dst * p.Hkv + h] = top;
  }
}

}  // namespace

size_t cache_weigh_workspace_bytes(kda_dtype dt, int batch, int window, int Hq, int Hkv, int d,
                                   int max_pages) {
  if (weigh_tc_applies(dt, window, Hq, Hkv, d)) return cache_weigh_tc_workspace(batch, window, Hq, Hkv);
  const int rows = Hq / Hkv * window;
  const Sharing sh = sharing_of(batch, Hkv, rows, max_pages);
  return sh.cluster ? 0 : (size_t)batch * Hkv * sh.cs * (rows < kStatRows ? rows : kStatRows) * sizeof(float2);
}

kda_status launch_cache_weigh(const WeighParams& p, kda_dtype dt, int d, cudaStream_t s) {
  if (weigh_tc_applies(dt, p.window, p.Hq, p.Hkv, d)) return launch_cache_weigh_tc(p, s);
  if (dt == KDA_BF16)
    return d == 128 ? launch_weigh_t<128, 1, __nv_bfloat16>(p, s)
                    : launch_weigh_t<64, 1, __nv_bfloat16>(p, s);
  return d == 128 ? launch_weigh_t<128, 2, float>(p, s) : launch_weigh_t<64, 2, float>(p, s);
}

kda_status launch_cache_evict(const EvictParams& p, int d, cudaStream_t s) {
  const int64_t units = (int64_t)p.batch * p.Hkv;
  // up to 8192 keys to a CTA. 32 rows of 16384, moves and read-back included: 243 us, as with 16384,
  // and 263 with 4096; 8 rows of 32768: 133, 135 and 162 us.
  int cs = 1;
  while (cs < 8 && (int64_t)p.max_pages * kPage > (int64_t)cs * 8192) cs *= 2;
  // room for whole tiles of 128 keys (64 rows of one page: 34 us, with the keys read again 40)
  const int64_t per = (((int64_t)p.max_pages + cs - 1) / cs * kPage + 127) / 128 * 128;
  const int cap = (int)(per < kEMaxKeys ? per : kEMaxKeys);
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         kEMaxKeys * 4);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cs));
  cfg.blockDim = dim3(kEThreads);
  cfg.dynamicSmemBytes = (size_t)cap * 4;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, evict_select_kernel, p, cs, cap);
  count_launches(1);
  if (p.budget > 0) {  // its CTAs start while the last of the selection run
    cfg.gridDim = dim3((unsigned)p.batch * ((p.budget + kPage - 1) / kPage), (unsigned)p.Hkv);
    cfg.blockDim = dim3(kMThreads);
    cfg.dynamicSmemBytes = 0;
    at[0] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    if (d == 128) cudaLaunchKernelEx(&cfg, evict_move_kernel<128>, p);
    else cudaLaunchKernelEx(&cfg, evict_move_kernel<64>, p);
    count_launches(1);
  }
  return check_launch("kda_cache_evict");
}

}  // namespace kda
