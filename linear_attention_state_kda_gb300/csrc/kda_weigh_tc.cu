// Weights of cached tokens for windows of many queries (bf16, d = 128, more than 64 query rows per
// key/value head): the end of a prompt weighing the whole of it.
//
//     weight[t] = keep * weight[t] + sum_i 2^(x_it - lse_i),   x_it = scale log2(e) q_i . k_t
//
// Two kernels over the keys, 256 query rows at a time: the first takes the rows' statistics (running
// maximum and sum) of ranges of keys into the workspace, the second joins them and sums the weights
// over the rows. In both the products are tcgen05 kind::f8f6f4 on the codes as they lie (TMA), with
// the operands swapped: the first has a query row per accumulator lane, so that maximum and sum stay
// in one thread; the second a key per lane, so that the sum over the rows does. (One kernel with the
// statistics joined over a cluster per key/value head measured 117 us on one row of 32k keys and 8
// heads: clusters of 8 use 64 SMs, and of clusters of 16 only 7 run at once.)
//
// A query row enters as three 8-bit parts: x = q / 2^e in [-448, 448], e4m3(x), e4m3 of the rest, and
// e5m2 of the rest of that. bf16 has 8 significant bits, two e4m3 parts hold 8 where their exponents
// reach, from |x| = 1/4 up. Below, what they leave is under 2^-10, and its e5m2 is off by at most 2^-14,
// with the row's largest above 224 less than 2^-21 of it.
//
// Bound by the exponentials (two for each query row and key, 16 a cycle and SM), then by the products
// (three parts). One row of 32768 tokens, 64 query tokens x 32 heads, 8 key/value heads: 62 us, of
// which either kernel's exponentials are 15 and its products 11. A step of 128 keys x 256 rows takes
// 2240 cycles of the first kernel (1750 of products, and two looks at barriers) and 3600 of the second
// (2050 of exponentials; the rows' constants come from shared memory beside the products' operands).
// Splitting the queries once per CTA and joining the statistics are 5 us together.
#include "kda_internal.cuh"
#include "kda_fp8.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

constexpr int D = 128;
constexpr int kRows = 256;          // query rows at a time
constexpr int kTile = 128;          // keys of a step: two pages
constexpr int kStages = 4;
constexpr int kParts = 3;
constexpr int kThreads = 640;       // loads, products, two idle; 16 warps of exponentials
constexpr uint32_t kTries = 1u << 19;
constexpr float kLog2e = 1.4426950408889634f;

struct Smem {
  static constexpr int Q = 0;                               // [part][row tile][128 rows][128 B]
  static constexpr int K = Q + kParts * kRows * D;          // [stage][128 keys][128 B]
  static constexpr int SMALL = K + kStages * kTile * D;
};
struct Small {
  uint64_t full[kStages], empty[kStages], d_full[2], d_empty[2], drain;
  float ks[kStages][2];             // scale log2(e) times a step's pages' scales; 0 where there is none
  int page[kStages][2];             // -1: none
  alignas(16) float2 row[kRows];    // 2^e, and minus lse
  float2 late[kRows];               // statistics of the second half of the ranges
  float part[2][3][kTile];          // sums over the last three quarters of the rows
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, int* abort) {
  const bool done = __all_sync(0xffffffffu, ptx::mbar_wait_short(bar, parity, kTries, abort));
  if (!done) *(volatile int*)abort = 1;
  return done;
}
__device__ __forceinline__ uint32_t e5m2x2_from_f32(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// How the work is cut: statistics by (unit, 256 rows, range of keys), weights by (unit, range of keys),
// a unit being a row's key/value head.
struct Cut {
  int groups, stat_ranges, ranges;
};

template <bool kStats>
__global__ void __launch_bounds__(kThreads, 1)
weigh_tc_kernel(const __grid_constant__ CUtensorMap map, const WeighParams p, const Cut cut) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Small& sm = *reinterpret_cast<Small*>(smem + Smem::SMALL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (kStats) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int ranges = kStats ? cut.stat_ranges : cut.ranges;
  const int range = blockIdx.x % ranges;
  const int first_group = kStats ? blockIdx.x / ranges % cut.groups : 0;
  const int bh = kStats ? blockIdx.x / ranges / cut.groups : blockIdx.x / ranges;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int start = p.start[b];
  int n = start < 0 ? 0 : p.lens ? p.lens[b] : p.window;
  n = n < 0 ? 0 : n > p.window ? p.window : n;
  const int G = p.Hq / p.Hkv, R = n * G;
  if (first_group * kRows >= R) return;
  const int64_t most = (int64_t)p.max_pages * kPage;
  const int64_t keys = (int64_t)start + n < most ? (int64_t)start + n : most;
  if (kStats && range == 0 && first_group == 0 && threadIdx.x == 0 && h == 0 && p.status &&
      (int64_t)start + n > most)
    atomicOr(p.status, KDA_STATUS_BAD_PAGE);
  const int32_t* table = p.table + (int64_t)b * p.max_pages;
  // weights: a contiguous range of steps (two pages each)
  const int steps = (int)((keys + kTile - 1) / kTile);
  const int per = (steps + ranges - 1) / ranges;
  const int w0 = min(steps, range * per), w1 = min(steps, w0 + per);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&sm.full[i], 1);
      ptx::mbar_init(&sm.empty[i], 1 + 16);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sm.d_full[i], 1);
      ptx::mbar_init(&sm.d_empty[i], 16);
    }
    ptx::mbar_init(&sm.drain, 1);
    ptx::fence_mbar_init();
    sm.abort = 0;
  }
  if (warp == 1) {
    ptx::tmem_alloc(&sm.tmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
  const uint32_t base = ptx::smem_u32(smem);
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_all(bar, parity, &sm.abort); };

  int step = 0;  // steps of all groups so far: stages and accumulators take turns
  const int last_group = kStats ? first_group + 1 : (R + kRows - 1) / kRows;
#pragma unroll 1
  for (int group = first_group; group < last_group; ++group) {
    const int r0 = group * kRows, rows = min(kRows, R - r0);
    const int tiles = rows > 128 ? 2 : 1;
    // positions that some row of the group sees, and the steps that this CTA takes of them
    const int64_t seen = min(keys, (int64_t)start + (r0 + rows - 1) / G + 1);
    const int all_steps = (int)((seen + kTile - 1) / kTile);
    const int stat_per = (all_steps + ranges - 1) / ranges;
    const int s0 = kStats ? min(all_steps, range * stat_per) : w0;
    const int s1 = kStats ? min(all_steps, s0 + stat_per) : max(w0, min(w1, all_steps));
    const int count = s1 - s0;
    // the group's query rows: a warp takes four at a time, a lane 16 channels of one
    const int piece = lane & 7;
#pragma unroll 1
    for (int r = (int)threadIdx.x >> 3; r < tiles * 128; r += kThreads / 8) {
      const int at = r0 + r, j = at / G;
      uint4 v[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      if (r < rows) {
        const uint4* src = reinterpret_cast<const uint4*>(
            (const __nv_bfloat16*)p.q +
            (((int64_t)b * p.window + j) * p.Hq + h * G + (at - j * G)) * D + piece * 16);
        v[0] = src[0];
        v[1] = src[1];
      }
      const uint32_t u[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
      float f[16];
      uint32_t m = 0;
      bool bad = false;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        f[c] = __uint_as_float(c & 1 ? u[c / 2] & 0xffff0000u : u[c / 2] << 16);
        m = max(m, finite_abs_bits(f[c]));
        bad |= !(fabsf(f[c]) < INFINITY);
      }
      // (a row is within a warp's eight lanes, all of them here)
      const uint32_t row_lanes = 0xffu << (lane & 24);
      m = __reduce_max_sync(row_lanes, m);
      bad = __any_sync(row_lanes, bad);
      // 2^e, the smallest power of two with m <= 448 2^e, at least 2^-126: bf16 ends at 2^-133, so that
      // smaller rows are multiples of 2^-7 after it, which two parts hold
      const int e = max(exponent_of(m), -126);
#pragma unroll
      for (int c = 0; c < 16; ++c) f[c] *= pow2f(-e);
      const uint32_t off = base + Smem::Q + (r >> 7) * (128 * D) + (r & 127) * D +
                           ((piece ^ (r & 7)) << 4);
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        uint32_t code[4];
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
          if (part < 2) {
            const uint32_t lo = e4m3x2_from_f32(f[c], f[c + 1]);
            const uint32_t hi = e4m3x2_from_f32(f[c + 2], f[c + 3]);
            const float2 x = f32x2_from_f16x2(f16x2_from_e4m3(lo));
            const float2 y = f32x2_from_f16x2(f16x2_from_e4m3(hi));
            f[c] -= x.x; f[c + 1] -= x.y; f[c + 2] -= y.x; f[c + 3] -= y.y;
            code[c / 4] = lo | hi << 16;
          } else {
            code[c / 4] = e5m2x2_from_f32(f[c], f[c + 1]) | e5m2x2_from_f32(f[c + 2], f[c + 3]) << 16;
          }
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(off + part * (kRows * D)),
                     "r"(code[0]), "r"(code[1]), "r"(code[2]), "r"(code[3])
                     : "memory");
      }
      // a row with an infinity or NaN has no weights but NaN
      if (piece == 0)
        sm.row[r].x = bad ? __int_as_float(0x7fffffff) : pow2f(e);
    }
    // the rows' statistics, by two threads a row
    const int mine = (int)threadIdx.x - 128, row = mine & (kRows - 1);
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (!kStats && group == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!kStats && mine >= 0 && row < tiles * 128) {
      const float2* src =
          p.stats + ((int64_t)bh * cut.groups + group) * (2 * cut.stat_ranges) * kRows + row;
      const int i0 = mine < kRows ? 0 : cut.stat_ranges, i1 = i0 + cut.stat_ranges;
      constexpr int kBatch = 10;  // side by side
#pragma unroll 1
      for (int i = i0; i < i1; i += kBatch) {
        float2 x[kBatch];
        float top = ml.x;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          x[k] = i + k < i1 ? src[(int64_t)(i + k) * kRows] : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) top = fmaxf(top, x[k].x);
        const float at = top == -INFINITY ? 0.0f : top;
        ml.y *= ptx::ex2_approx(ml.x - at);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) ml.y += x[k].y * ptx::ex2_approx(x[k].x - at);
        ml.x = top;
      }
      if (mine >= kRows) sm.late[row] = ml;
    }
    __syncthreads();
    if (!kStats && mine >= 0 && mine < tiles * 128) {
      const float2 x = sm.late[row];
      const float m = fmaxf(ml.x, x.x), at = m == -INFINITY ? 0.0f : m;
      const float l = ml.y * ptx::ex2_approx(ml.x - at) + x.y * ptx::ex2_approx(x.x - at);
      // a row past the last, or that sees nothing, adds nothing
      const bool none = row >= rows || (m == -INFINITY && !(l != l));
      sm.row[row].y = none ? -INFINITY : -(at + log2f(l));
      if (none) sm.row[row].x = 0.0f;
    }
    ptx::fence_proxy_async_smem();
    __syncthreads();

    {
      if (warp == 0) {
        // ---------------------------------------------------------------- loads
        int id = -1;  // of page 2 i + lane, and its scale, 16 steps ahead
        float ks = 0.0f;
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
          const int at = step + i, s = at % kStages, from = (i & 15) * 2;
          if (from == 0) {
            const int pg = (s0 + i) * 2 + lane;
            // (a step's second page also where no row of this group sees it: its weights begin here)
            id = (int64_t)pg * kPage < keys && pg < 2 * s1 ? table[pg] : -1;
            if (id >= p.n_pages) {
              if (p.status) atomicOr(p.status, KDA_STATUS_BAD_PAGE);
              id = -1;
            }
            // (with the page's scale, not with 2^e, which it could bring below the normal numbers)
            ks = id < 0 ? 0.0f : p.ks[(int64_t)id * p.Hkv + h] * (p.scale * kLog2e);
          }
          const int a = __shfl_sync(0xffffffffu, id, from);
          const int c = __shfl_sync(0xffffffffu, id, from + 1);
          const float ka = __shfl_sync(0xffffffffu, ks, from);
          const float kc = __shfl_sync(0xffffffffu, ks, from + 1);
          if (at >= kStages && !wait(&sm.empty[s], ((at / kStages) - 1) & 1)) break;
          if (lane == 0) {
            sm.page[s][0] = a < 0 ? -1 : a;
            sm.page[s][1] = c < 0 ? -1 : c;
            sm.ks[s][0] = ka;
            sm.ks[s][1] = kc;
            uint8_t* dst = smem + Smem::K + s * (kTile * D);
            ptx::mbar_arrive_expect_tx(&sm.full[s], (uint32_t)(((a >= 0) + (c >= 0)) * kPage * D));
            if (a >= 0) ptx::tma_load_3d(dst, &map, &sm.full[s], 0, 0, a * p.Hkv + h);
            if (c >= 0) ptx::tma_load_3d(dst + kPage * D, &map, &sm.full[s], 0, 0, c * p.Hkv + h);
          }
          __syncwarp();
        }
      } else if (warp == 1) {
        // ---------------------------------------------------------------- products
        for (int i = 0; i < count; ++i) {
          const int at = step + i, s = at % kStages, buf = at & 1;
          if (!wait(&sm.full[s], (at / kStages) & 1) ||
              (at >= 2 && !wait(&sm.d_empty[buf], ((at >> 1) - 1) & 1)))
            break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            const uint64_t k = ptx::sdesc_sw128(base + Smem::K + s * (kTile * D), 16, 1024);
            const uint64_t q = ptx::sdesc_sw128(base + Smem::Q, 16, 1024);
            const uint32_t d = tmem + buf * kRows;
#pragma unroll 1
            for (int part = 0; part < kParts; ++part) {
              const uint32_t fmt = part < 2 ? ptx::kFmtE4M3 : ptx::kFmtE5M2;
              if (kStats) {
                const uint32_t id = ptx::idesc_make2(fmt, ptx::kFmtE4M3, 128, kTile);
                for (int t = 0; t < tiles; ++t)
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    ptx::mma_f8(d + t * kTile,
                                ptx::desc_add(q, part * (kRows * D) + t * 128 * D + j * 32),
                                ptx::desc_add(k, j * 32), id, part + j > 0);
              } else {
                const uint32_t id = ptx::idesc_make2(ptx::kFmtE4M3, fmt, 128, (uint32_t)tiles * 128);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  ptx::mma_f8(d, ptx::desc_add(k, j * 32),
                              ptx::desc_add(q, part * (kRows * D) + j * 32), id, part + j > 0);
              }
            }
            ptx::mma_commit(&sm.empty[s]);
            ptx::mma_commit(&sm.d_full[buf]);
          }
          __syncwarp();
        }
      } else if (warp >= 4) {
        // ---------------------------------------------------------------- exponentials
        const int w = warp & 3, g = ((warp - 4) >> 2) & 1, half = (warp - 4) >> 3;
        const uint32_t lanes = (uint32_t)(w * 32) << 16;
        if (kStats) {
          // a query row: row tile g, lane; half of a step's keys
          const int r = g * 128 + w * 32 + lane;
          const float c = g < tiles ? sm.row[r].x : 0.0f;
          const int64_t vis = r < rows ? min(keys, (int64_t)start + (r0 + r) / G + 1) : 0;
          float m = -INFINITY, l = 0.0f;
          for (int i = 0; i < count; ++i) {
            const int at = step + i, s = at % kStages, buf = at & 1;
            if (!wait(&sm.d_full[buf], (at >> 1) & 1)) break;
            ptx::tc_fence_after();
            if (g < tiles) {
              const int64_t pos0 = (int64_t)(s0 + i) * kTile;
#pragma unroll 1
              for (int q4 = 2 * half; q4 < 2 * half + 2; ++q4) {  // 32 keys
                float x[32];
                ptx::tmem_ld32(tmem + lanes + buf * kRows + g * kTile + q4 * 32, x);
                const float f = c * sm.ks[s][q4 >> 1];
                const int64_t left = sm.page[s][q4 >> 1] < 0 ? 0 : vis - (pos0 + q4 * 32);
                const ptx::f32x2 ff = ptx::pack2(f, f);
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                  ptx::unpack2(ptx::mul2(ptx::pack2(x[j], x[j + 1]), ff), x[j], x[j + 1]);
                if (__any_sync(0xffffffffu, left < 32)) {
#pragma unroll
                  for (int j = 0; j < 32; ++j) x[j] = j < left ? x[j] : -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < 32; j += 2) top = fmaxf(top, fmaxf(x[j], x[j + 1]));
                if (top > m) {
                  l *= ptx::ex2_approx(m - top);
                  m = top;
                }
                const float mm = m == -INFINITY ? 0.0f : m;
                const ptx::f32x2 nm = ptx::pack2(-mm, -mm);
                ptx::f32x2 sum = ptx::pack2(0.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                  float a, e;
                  ptx::unpack2(ptx::add2(ptx::pack2(x[j], x[j + 1]), nm), a, e);
                  sum = ptx::add2(sum, ptx::pack2(ptx::ex2_approx(a), ptx::ex2_approx(e)));
                }
                float a, e;
                ptx::unpack2(sum, a, e);
                l += a + e;
              }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              ptx::mbar_arrive(&sm.d_empty[buf]);
              ptx::mbar_arrive(&sm.empty[s]);
            }
          }
          if (g < tiles)
            p.stats[((((int64_t)bh * cut.groups + group) * ranges + range) * 2 + half) * kRows + r] =
                make_float2(m, l);
        } else {
          // a key: a quarter of the query rows, half of row tile g
          const int quarter = g * 2 + half;
          for (int i = 0; i < count; ++i) {
            const int at = step + i, s = at % kStages, buf = at & 1;
            const bool ok = wait(&sm.d_full[buf], (at >> 1) & 1);
            ptx::tc_fence_after();
            const int64_t pos0 = (int64_t)(s0 + i) * kTile, pos = pos0 + w * 32 + lane;
            const int id = sm.page[s][w >> 1];
            const float ks = sm.ks[s][w >> 1];
            const ptx::f32x2 kk = ptx::pack2(ks, ks);
            // rows from `from` on see this key
            const int64_t hidden = (pos - start) * G - r0;
            const int from = pos >= keys ? kRows : hidden > 0 ? (int)min(hidden, (int64_t)kRows) : 0;
            const bool all = __all_sync(0xffffffffu, from == 0);
            ptx::f32x2 sum = ptx::pack2(0.0f, 0.0f);
            if (ok && g < tiles) {
#pragma unroll 1
              for (int q4 = 2 * half; q4 < 2 * half + 2; ++q4) {  // 32 rows
                float x[32];
                ptx::tmem_ld32(tmem + lanes + buf * kRows + g * 128 + q4 * 32, x);
                const int rr = g * 128 + q4 * 32;
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                  // (c, -lse) of two rows
                  const float4 t = *reinterpret_cast<const float4*>(&sm.row[rr + j]);
                  float a, e;
                  ptx::unpack2(ptx::fma2(ptx::pack2(x[j], x[j + 1]),
                                         ptx::mul2(ptx::pack2(t.x, t.z), kk), ptx::pack2(t.y, t.w)),
                               a, e);
                  a = ptx::ex2_approx(a);
                  e = ptx::ex2_approx(e);
                  if (!all) {
                    a = rr + j >= from ? a : 0.0f;
                    e = rr + j + 1 >= from ? e : 0.0f;
                  }
                  sum = ptx::add2(sum, ptx::pack2(a, e));
                }
              }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              ptx::mbar_arrive(&sm.d_empty[buf]);
              ptx::mbar_arrive(&sm.empty[s]);
            }
            float a, e;
            ptx::unpack2(sum, a, e);
            a += e;
            if (quarter > 0) sm.part[at & 1][quarter - 1][w * 32 + lane] = a;
            // the four warps of these keys
            asm volatile("bar.sync %0, 128;" ::"r"(2 + w) : "memory");
            if (quarter == 0 && ok && id >= 0 && pos < keys) {
#pragma unroll
              for (int j = 0; j < 3; ++j) a += sm.part[at & 1][j][w * 32 + lane];
              float* wp = p.weights + ((int64_t)id * p.Hkv + h) * kPage + (pos & (kPage - 1));
              const float old = r0 > 0 ? *wp : pos < start && p.keep != 0.0f ? p.keep * *wp : 0.0f;
              *wp = old + a;
            }
          }
          // (a part is written again two steps on, behind the next step's barrier)
          if (r0 == 0 && quarter == 0) {
            // positions that the window holds, but no row of this group sees, begin at zero
            for (int i = s1; i < w1; ++i) {
              const int64_t pos = (int64_t)i * kTile + w * 32 + lane;
              const int pg = (int)(pos / kPage);
              const int id = pos < keys ? table[pg] : -1;
              if (id >= 0 && id < p.n_pages) {
                float* wp = p.weights + ((int64_t)id * p.Hkv + h) * kPage + (pos & (kPage - 1));
                *wp = pos < start && p.keep != 0.0f ? p.keep * *wp : 0.0f;
              }
            }
          }
        }
      }
      step += count;
    }
    __syncthreads();
  }
  if (warp == 1 && __any_sync(0xffffffffu, *(volatile int*)&sm.abort)) {
    if (ptx::elect_one()) ptx::mma_commit(&sm.drain);
    __syncwarp();
    ptx::mbar_wait_tries(&sm.drain, 0, kTries);
    __syncwarp();
  }
  if (warp == 0 && *(volatile int*)&sm.abort) __nanosleep(1000000);  // loads in flight land
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && sm.abort && p.status) atomicOr(p.status, KDA_STATUS_TIMEOUT);
  if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

}  // namespace

static Cut cut_of(int batch, int window, int Hq, int Hkv) {
  const int64_t units = (int64_t)batch * Hkv, rows = (int64_t)(Hq / Hkv) * window;
  Cut c;
  c.groups = (int)((rows + kRows - 1) / kRows);
  // about one range per SM
  const int64_t stats = units * c.groups;
  c.stat_ranges = (int)(stats < kSms ? kSms / stats : 1);
  c.ranges = (int)(units < kSms ? kSms / units : 1);
  return c;
}

bool weigh_tc_applies(kda_dtype dt, int window, int Hq, int Hkv, int d) {
  return dt == KDA_BF16 && d == 128 && (int64_t)window * (Hq / Hkv) > 64;
}

size_t cache_weigh_tc_workspace(int batch, int window, int Hq, int Hkv) {
  const Cut c = cut_of(batch, window, Hq, Hkv);
  return (size_t)batch * Hkv * c.groups * c.stat_ranges * 2 * kRows * sizeof(float2);
}

kda_status launch_cache_weigh_tc(const WeighParams& p, cudaStream_t s) {
  CUtensorMap map;
  if (!chunk_tc_available())
    return set_error(KDA_ERR_UNSUPPORTED,
                     "kda_cache_weigh: the CUDA driver does not provide cuTensorMapEncodeTiled, which "
                     "windows of many queries need");
  if (!make_map_pages(&map, p.kc, D, (uint64_t)p.n_pages * p.Hkv))
    return set_error(KDA_ERR_CUDA, "kda_cache_weigh: cuTensorMapEncodeTiled failed");
  constexpr int bytes = Smem::SMALL + (int)sizeof(Small);
  static_assert(bytes <= 232448, "shared memory");
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    cudaFuncSetAttribute(weigh_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    cudaFuncSetAttribute(weigh_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  const Cut c = cut_of(p.batch, p.window, p.Hq, p.Hkv);
  const int64_t units = (int64_t)p.batch * p.Hkv;
  const unsigned stats = (unsigned)(units * c.groups * c.stat_ranges);
  weigh_tc_kernel<true><<<stats, kThreads, bytes, s>>>(map, p, c);
  // its CTAs split their queries while the last statistics are taken
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * c.ranges));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, weigh_tc_kernel<false>, map, p, c);
  count_launches(2);
  return check_launch("kda_cache_weigh");
}

}  // namespace kda
