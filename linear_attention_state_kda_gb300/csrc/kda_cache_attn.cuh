// Shared by the attention kernels over the 8-bit cache: the split of the work over workers, and
// what both keep per query row.
//
// The key slices that the row groups see are laid end to end (row, head, row group, slice) and cut
// into equal ranges, one per worker. A "unit" is one (row, head, row group); a worker's "piece" is
// the part of a unit in its range. Beginning and ending a unit counts as unit_cost slices more.
//
// The loops here run a few times per CTA and are kept rolled: unrolled, they were 30 KB of each
// kernel's code, more than the loops over the keys, and pushed those out of the instruction cache.
#pragma once

#include "kda_internal.cuh"

namespace kda {
namespace attn {

constexpr int kMaxSms = 160;       // SMs used at most (sizes the workspace)
constexpr int kWindows = 512;      // windows of rows in the search for a worker's first row
// P is 2^kPBase for a term equal to the row's M, and M is raised only when a term exceeds it by
// more than 2^kSlack: P <= 2^15 fits f16, and the accumulators are rescaled once or twice per
// unit instead of in most steps.
constexpr float kPBase = 7.0f, kSlack = 8.0f;
constexpr int kNoEnd = 1 << 30;    // beyond the positions of the largest page table
// Value scales below 2^kMinScaleExp count as this one in M. l is then at most 2^(15 + 80) a key, in range
// for 2^30 keys; P of a smaller scale 2^e starts at 2^(e + 87) instead of 2^7, 2^-13 for the smallest.
constexpr int kMinScaleExp = -80;

// Two fp32 values in one register pair, and the packed operations on them.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

struct UnitDesc {  // of a unit that is cut: the worker that began it, and how many share it (else 0)
  int32_t worker, pieces;
};

// Query tokens of row b.
__device__ __forceinline__ int row_tokens(const CacheAttnParams& p, int b) {
  if (p.start[b] < 0) return 0;
  const int n = p.lens ? p.lens[b] : p.window;
  return n < 0 ? 0 : (n > p.window ? p.window : n);
}
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Piece {
  int b, h, rg, unit;  // unit: within the row
  int first, last;     // slices
  bool whole;
  UnitDesc desc;       // to be written by the piece with first == 0
};

// A worker's walk over its range. Every lane of a warp calls; all lanes get the same answers.
template <int kSlice>
struct Ranges {
  int G, unit_rows, nrg, U, unit_cost, worker;
  int64_t total, workers, pos, end, at;
  int base, row;
  int64_t cost, cost_l;  // of a head of the current row; of the lane's row of the 32 from `base` on
  bool few;

  // Key slices that some query of the row's group rg sees, within the page table: a long window's
  // first groups see fewer, and groups past the row's last token none.
  __device__ __forceinline__ int group_slices(const CacheAttnParams& p, int start, int n,
                                              int rg) const {
    if (rg >= nrg || rg * unit_rows >= n * G) return 0;
    int j = nrg == 1 ? n : (rg * unit_rows + unit_rows - 1) / G + 1;
    j = j < n ? j : n;
    const int64_t keys = (int64_t)start + j, most = (int64_t)p.max_pages * kPage;
    return (int)(((keys < most ? keys : most) + kSlice - 1) / kSlice);
  }
  struct Sums {
    int64_t slices;
    int units;
  };
  // Slices and units with slices of a head of row b.
  __device__ __forceinline__ Sums row_sums(const CacheAttnParams& p, int b, bool flag) const {
    Sums s = {0, 0};
    if (b >= p.batch) return s;
    const int n = row_tokens(p, b);
    if (n == 0) return s;
    const int start = p.start[b];
    if (flag && p.status && (int64_t)start + n > (int64_t)p.max_pages * kPage)
      atomicOr(p.status, KDA_STATUS_BAD_PAGE);
#pragma unroll 1
    for (int rg = 0; rg < nrg; ++rg) {
      const int c = group_slices(p, start, n, rg);
      s.slices += c;
      s.units += c > 0;
    }
    return s;
  }
  __device__ __forceinline__ int64_t cost_of(const Sums& s) const {
    return s.slices + (int64_t)s.units * unit_cost;
  }

  // Counts all slices and finds this worker's range. Every thread of the CTA calls (it has a
  // barrier for more than 32 rows or several groups); s_win and s_rows hold kWindows entries.
  // `flag`: report rows past the page table. With no more slices than workers, one each: there is
  // no one to balance with.
  __device__ __forceinline__ void plan(const CacheAttnParams& p, int rows_of_unit, int n_warps,
                                       int my_worker, int64_t max_workers, int cost_of_unit,
                                       int64_t* s_win, int* s_rows, bool flag) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    G = p.Hq / p.Hkv;
    unit_rows = rows_of_unit;
    nrg = (G * p.window + unit_rows - 1) / unit_rows;
    U = p.Hkv * nrg;
    const int per_win = (p.batch + 32 * kWindows - 1) / (32 * kWindows) * 32;
    const int n_win = (p.batch + per_win - 1) / per_win;
    int64_t slices = 0, units = 0;
    Sums sums_l = {0, 0};
    if (p.batch <= 32) {
      if (nrg == 1) {
        sums_l = row_sums(p, lane, flag);
      } else {
        // a warp sums a row, its lanes the groups
#pragma unroll 1
        for (int b = warp; b < p.batch; b += n_warps) {
          const int n = row_tokens(p, b), start = p.start[b];
          int64_t c = 0, u = 0;
#pragma unroll 1
          for (int rg = lane; rg < nrg; rg += 32) {
            const int x = group_slices(p, start, n, rg);
            c += x;
            u += x > 0;
          }
          c = warp_sum(c);
          u = warp_sum(u);
          if (lane == 0) {
            s_win[b] = c;
            s_rows[b] = (int)u;
            if (flag && p.status && n > 0 && (int64_t)start + n > (int64_t)p.max_pages * kPage)
              atomicOr(p.status, KDA_STATUS_BAD_PAGE);
          }
        }
        __syncthreads();
        if (lane < p.batch) sums_l = {s_win[lane], s_rows[lane]};
      }
      slices = warp_sum(sums_l.slices);
      units = warp_sum(sums_l.units);
    } else {
#pragma unroll 1
      for (int w = warp; w < n_win; w += n_warps) {
        int64_t c = 0, u = 0;
#pragma unroll 1
        for (int i = lane; i < per_win; i += 32) {
          const Sums x = row_sums(p, w * per_win + i, flag);
          c += x.slices;
          u += x.units;
        }
        c = warp_sum(c);
        u = warp_sum(u);
        if (lane == 0) {
          s_win[w] = c;
          s_rows[w] = (int)u;
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int w = lane; w < n_win; w += 32) {
        slices += s_win[w];
        units += s_rows[w];
      }
      slices = warp_sum(slices);
      units = warp_sum(units);
    }
    worker = my_worker;
    workers = max_workers;
    few = slices * p.Hkv <= workers;
    unit_cost = few ? 0 : cost_of_unit;
    total = (slices + units * unit_cost) * p.Hkv;
    if (few) workers = total;
    cost_l = cost_of(sums_l);
    pos = end = at = 0;
    base = row = 0;
    cost = 0;
    if (worker < workers) {
      pos = few ? worker : total * worker / workers;
      end = few ? worker + 1 : total * (worker + 1) / workers;
    }
    if (pos >= end) return;
    // the row that holds pos: its window, then the 32 rows
    if (p.batch > 32) {
#pragma unroll 1
      for (int w = 0;; w += 32) {
        int64_t c = w + lane < n_win
                        ? (s_win[w + lane] + (int64_t)s_rows[w + lane] * unit_cost) * p.Hkv
                        : 0;
        const int64_t mine = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t u = __shfl_up_sync(0xffffffffu, c, o);
          if (lane >= o) c += u;
        }
        const unsigned past = __ballot_sync(0xffffffffu, at + c <= pos);
        const int k = __popc(past);  // windows that end at or before pos
        if (k < 32) {
          at += __shfl_sync(0xffffffffu, c - mine, k);
          base = (w + k) * per_win;
          break;
        }
        at += __shfl_sync(0xffffffffu, c, 31);
      }
#pragma unroll 1
      for (;;) {
        cost_l = cost_of(row_sums(p, base + lane, false));
        const int64_t c = warp_sum(cost_l) * p.Hkv;
        if (at + c > pos) break;
        at += c;
        base += 32;
      }
    }
    cost = __shfl_sync(0xffffffffu, cost_l, 0);
  }

  __device__ __forceinline__ bool next(const CacheAttnParams& p, Piece& x) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    while (pos < end) {
#pragma unroll 1
      while (at + cost * p.Hkv <= pos) {
        at += cost * p.Hkv;
        if (++row == 32) {
          row = 0;
          base += 32;
          cost_l = cost_of(row_sums(p, base + lane, false));
        }
        cost = __shfl_sync(0xffffffffu, cost_l, row);
      }
      x.b = base + row;
      x.h = (int)((pos - at) / cost);
      int64_t in_head = (pos - at) - x.h * cost;  // position within the head, then within the unit
      x.rg = 0;
      int c = (int)cost;  // of the unit
      if (nrg > 1) {
        const int n = row_tokens(p, x.b), start = p.start[x.b];
#pragma unroll 1
        for (; x.rg < nrg; x.rg += 32) {
          const int s = group_slices(p, start, n, x.rg + lane);
          const int mine = s > 0 ? s + unit_cost : 0;
          int64_t upto = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += u;
          }
          const int k = __popc(__ballot_sync(0xffffffffu, upto <= in_head));
          if (k < 32) {
            in_head -= __shfl_sync(0xffffffffu, upto - mine, k);
            c = __shfl_sync(0xffffffffu, mine, k);
            x.rg += k;
            break;
          }
          in_head -= __shfl_sync(0xffffffffu, upto, 31);
        }
        if (x.rg >= nrg) return false;
      }
      x.unit = x.h * nrg + x.rg;
      const int n_slices = c - unit_cost;
      const int x0 = (int)in_head;
      const int x1 = end - pos < c - x0 ? x0 + (int)(end - pos) : c;
      const int64_t pos0 = pos, stop = pos + (c - x0);  // end of the unit
      pos += x1 - x0;
      x.first = x0 > unit_cost ? x0 - unit_cost : 0;
      x.last = x1 > unit_cost ? x1 - unit_cost : 0;
      if (x.first == x.last) continue;  // the range ends before the unit's first slice
      x.whole = x.first == 0 && x.last == n_slices;
      x.desc = {worker, 0};
      // the last piece is in the first range that ends at or after the unit's end
      if (x.first == 0 && !x.whole)
        x.desc.pieces = (int)(few ? stop - pos0 : (stop * workers + total - 1) / total - worker);
      return true;
    }
    return false;
  }

  // Units without keys: their output is zeros and they are not cut. `step` warps share them.
  template <class T>
  __device__ __forceinline__ void zero_units(const CacheAttnParams& p, int d, int first, int step,
                                             UnitDesc* desc) const {
    const int lane = threadIdx.x & 31;
    const int64_t units = (int64_t)p.batch * U;
    const int chunks = d * (int)sizeof(T) / 16;
#pragma unroll 1
    for (int64_t i0 = (int64_t)first * 32; i0 < units; i0 += (int64_t)step * 32) {
      const int64_t i = i0 + lane;
      const int b = i < units ? (int)(i / U) : 0, unit = (int)(i - (int64_t)b * U);
      const bool dead = i < units && group_slices(p, p.start[b], row_tokens(p, b), unit % nrg) == 0;
      if (dead) desc[i] = {0, 0};
#pragma unroll 1
      for (unsigned left = __ballot_sync(0xffffffffu, dead); left; left &= left - 1) {
        const int from = __ffs(left) - 1;
        const int zb = __shfl_sync(0xffffffffu, b, from), zu = __shfl_sync(0xffffffffu, unit, from);
        const int h = zu / nrg, r0 = (zu - h * nrg) * unit_rows;
        const int rows = min(unit_rows, G * p.window - r0);
#pragma unroll 1
        for (int k = lane; k < rows * chunks; k += 32) {
          const int gr = r0 + k / chunks, j = gr / G;
          uint4* o = reinterpret_cast<uint4*>(
              (T*)p.o + ((int64_t)(zb * (int64_t)p.window + j) * p.Hq + h * G + (gr - j * G)) * d);
          o[k % chunks] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
  }
};

// Workspace: the pieces' sums, their (M, l), then a descriptor per unit (of 16 rows at least) and, for
// units of 256 rows, the unit that each worker began and did not end (-1: none). An SM has up to 8
// workers with units of up to 32 rows, or 4 with 64, or one with 256.
inline size_t piece_rows_of(int R) { return (size_t)2 * kMaxSms * 8 * (R < 32 ? R : 32); }

// The tcgen05 kernel for bf16 queries: rows of its units, and its launch over the parts of the
// workspace.
constexpr int kTcRows = 256;
kda_status launch_attn_tc(const CacheAttnParams& p, int d, int ctas, int piece_rows, float* ws_o,
                          float2* ws_ml, UnitDesc* desc, int32_t* cut, cudaStream_t s);

}  // namespace attn
}  // namespace kda
