// Attention of one decoded token, or of a verify window, over the paged 8-bit cache
// (kda_cache_attention): o = sum_t softmax_t(scale q . k_t) v_t in one pass over the cache with
// the running maximum and sum of the softmax.
//
// What bounds it: the cache is read once, 2 d bytes per token and key/value head, so a single
// decoded token per row is HBM-bound; the 4 d operations per (query row, key) are tensor-core
// work. A "unit" is one (batch row, key/value head) with up to 16 MT query rows (the window's tokens
// times the query heads of the group), so that the cache is read once for all of them.
//
// Arithmetic. e4m3 codes are exact in f16, so both products run as f16 x f16 -> fp32 warp MMAs
// on codes; the page's power-of-two scales are applied around them. A query row is multiplied by
// a power of two that puts its largest entry in [2^13, 2^14) and rounded to f16: exact for bf16
// entries down to 2^-28 of the largest; fp32 queries are carried as the sum of two f16 parts (22
// bits). With x_t the score in units of log2 and e_t the exponent of t's value scale, the row
// keeps M = max_t (x_t + e_t) and accumulates
//     P_t = 2^(x_t + e_t - M + 14) (f16; two parts for fp32),  O = sum_t P_t code_t,
//     l = sum_t 2^(x_t - M + 14) = sum_t P_t 2^-e_t (fp32),    o = O / l.
// P is at most 2^14 whatever the scales of the pages, and what f16 drops is below 2^-38 of the
// row's largest term.
//
// Layout. Lane (g, t) = (lane / 4, lane % 4) of an m16n8k16 MMA. The order of the channels in the
// first product and of the columns in the second is free as long as both operands agree, and is
// chosen so that a lane reads 16-byte pieces of a cached row as they lie: channels 32 t .. 32 t +
// 31 of key g for the scores, and channels 16 g .. 16 g + 15 of keys 2t, 2t+1, 2t+8, 2t+9 for the
// values, whose bytes are interleaved pairwise to give two keys of one channel (d = 128; half of
// that for d = 64). A lane's outputs are then 32 consecutive channels of its row.
//
// Every warp walks 16-key slices of its own through a private ring of kStages shared-memory
// buffers filled with 16-byte asynchronous copies; nothing in the loop waits for another warp.
// The warps' results are joined at the end of the unit.
//
// Work split. The rows' 64-key blocks are laid end to end (row, head, row group, block) and cut
// into as many equal ranges as CTAs fit on the GPU, so that ragged lengths and few rows load
// every SM alike. A unit that lies in one range is finished there; the pieces of a unit that is
// cut go to the workspace (each CTA has at most two) and a second kernel, launched ahead of time
// and released when the first ends, joins them in order: no atomics, the same bits every time.
#include "kda_internal.cuh"
#include "kda_fp8.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

constexpr int kSlice = 32;     // keys per warp step
constexpr int kMaxCtas = 320;  // bound of the grid (sizes the workspace)
// P is 2^kPBase for a term equal to the row's M, and M is raised only when a term exceeds it by
// more than 2^kSlack: P <= 2^15 fits f16, and the accumulators are rescaled once or twice per
// unit instead of in most steps.
constexpr float kPBase = 7.0f, kSlack = 8.0f;
constexpr int kUnitCost = 3;   // what beginning and joining a unit takes, in blocks
constexpr int kMinCost = kUnitCost + 2;  // least work of a CTA: a unit of two blocks
constexpr int kNoEnd = 1 << 30;    // beyond the positions of the largest page table
constexpr int kMinScaleExp = -60;  // clamp of e_t in M, so that l stays in range

struct UnitDesc {  // a unit whose first piece is CTA c's last one
  int32_t b, h, rg, pieces;
};

template <class T, int D, int MT>
struct Shape {
  static constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
  static constexpr int ROWS = 16 * MT;
  static constexpr int WARPS = MT == 1 ? 6 : 8;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int CTAS = MT == 1 ? 2 : 1;     // resident per SM
  static constexpr int STAGES = D == 128 ? 2 : 3;  // slices in a warp's ring
  static constexpr int KSTEPS = D / 16;
  static constexpr int NT = D / 8;                 // n-tiles of the second product
  static constexpr int SLICE_BYTES = kSlice * D;   // one of K, V
  static constexpr int STAGE = 2 * SLICE_BYTES;
  static constexpr int RING = WARPS * STAGES * STAGE;
  // A warp's results in shared memory: each lane's D / 4 channels of a row 4 floats further than
  // the last lane's, so that 16-byte accesses of 8 lanes touch every bank once.
  static constexpr int LANE_F = D / 4 + 4, ROW_F = 4 * LANE_F;
  static constexpr int MERGE = WARPS * ROWS * ROW_F * 4;
  static constexpr int BUF = RING > MERGE ? RING : MERGE;
  static constexpr int QFRAG = MT * PARTS * KSTEPS * 512;
  static constexpr int SMEM = BUF + QFRAG;
};

// Byte of 16-byte chunk c of row r of a slice: chunks are permuted within the row so that both
// access patterns above touch every bank once (d = 128).
template <int D>
__device__ __forceinline__ int chunk_at(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  else return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma_f16(float* d, const uint4& a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The part of (lo, hi) that f16x2(lo, hi) = h dropped, rounded to f16.
__device__ __forceinline__ uint32_t f16x2_rest(float lo, float hi, uint32_t h) {
  const float2 f = f32x2_from_f16x2(h);
  return f16x2(lo - f.x, hi - f.y);
}

// Query tokens of row b, and 64-key blocks that any of them sees.
__device__ __forceinline__ int row_tokens(const CacheAttnParams& p, int b) {
  if (p.start[b] < 0) return 0;
  const int n = p.lens ? p.lens[b] : p.window;
  return n < 0 ? 0 : (n > p.window ? p.window : n);
}
__device__ __forceinline__ int64_t row_blocks(const CacheAttnParams& p, int b, bool flag) {
  const int n = row_tokens(p, b);
  if (n == 0) return 0;
  const int64_t blocks = ((int64_t)p.start[b] + n + kPage - 1) / kPage;
  if (blocks <= p.max_pages) return blocks;
  if (flag && p.status) atomicOr(p.status, KDA_STATUS_BAD_PAGE);
  return p.max_pages;
}

template <int kThreads>
struct Work {                 // what a CTA knows of the list of blocks
  int64_t pre[kThreads + 1];  // cost of one unit of rows base .. base + i - 1, summed
  int64_t part[kThreads / 32];
};

// pre[] of rows base .. base + kThreads - 1. Every thread calls.
template <int kThreads>
__device__ __forceinline__ void scan_rows(const CacheAttnParams& p, Work<kThreads>& w, int base,
                                          bool flag) {
  const int b = base + threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t v = b < p.batch ? row_blocks(p, b, flag) : 0;
  if (v > 0) v += kUnitCost;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) w.part[warp] = v;
  __syncthreads();
  for (int i = 0; i < warp; ++i) v += w.part[i];
  w.pre[threadIdx.x + 1] = v;
  if (threadIdx.x == 0) w.pre[0] = 0;
  __syncthreads();
}

template <class T, int D, int MT>
struct WarpState {
  float o[MT][D / 8][4];
  float m[MT][2], l[MT][2];
};

// One slice: scores, softmax update, weighted values. kTail: some key of the slice is hidden from
// some row; `left` of its keys are seen by each of the lane's rows.
template <class T, int D, int MT, bool kTail>
__device__ __forceinline__ void slice_step(WarpState<T, D, MT>& st, const uint8_t* kb,
                                           const uint8_t* vb, const uint4* qfrag, float ks, float vs,
                                           const float (&rowf)[MT][2], const int (&left)[MT][2],
                                           int lane) {
  using S = Shape<T, D, MT>;
  constexpr int NK = kSlice / 8;  // key tiles of the first product
  const int g = lane >> 2, t = lane & 3;
  float s[MT][NK][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NK; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[mt][nt][i] = 0.0f;
  // half of the lane's channels at a time
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    uint4 kw[NK];
#pragma unroll
    for (int nt = 0; nt < NK; ++nt)
      kw[nt] = *reinterpret_cast<const uint4*>(kb + chunk_at<D>(nt * 8 + g, (D / 64) * t + j));
#pragma unroll
    for (int k4 = 0; k4 < 4; ++k4) {
      uint32_t b[NK][2];
#pragma unroll
      for (int nt = 0; nt < NK; ++nt) f16x4_from_e4m3((&kw[nt].x)[k4], b[nt][0], b[nt][1]);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int part = 0; part < S::PARTS; ++part) {
          const uint4 a = qfrag[((mt * S::PARTS + part) * S::KSTEPS + 4 * j + k4) * 32 + lane];
#pragma unroll
          for (int nt = 0; nt < NK; ++nt) mma_f16(s[mt][nt], a, b[nt][0], b[nt][1]);
        }
    }
  }
  const int ve = (int)((__float_as_uint(vs) >> 23) & 255u) - 127;
  const float vexp = (float)ve, vref = (float)(ve < kMinScaleExp ? kMinScaleExp : ve);
  const float vinv = __uint_as_float((uint32_t)(127 - ve) << 23);  // 2^-e
  bool over = false;
  float top[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float f = rowf[mt][half] * ks;
      top[mt][half] = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NK; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float& x = s[mt][nt][half * 2 + i];
          x *= f;
          if constexpr (kTail) {
            if (nt * 8 + 2 * t + i >= left[mt][half]) x = -INFINITY;
          }
          top[mt][half] = fmaxf(top[mt][half], x);
        }
      over |= top[mt][half] + vref > st.m[mt][half] + kSlack;
    }
  if (__any_sync(0xffffffffu, over)) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float corr[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x = top[mt][half];
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        const float mo = st.m[mt][half], mn = fmaxf(mo, x + vref);
        st.m[mt][half] = mn;
        corr[half] = ptx::ex2_approx(mo - (mn == -INFINITY ? 0.0f : mn));
        st.l[mt][half] *= corr[half];
      }
#pragma unroll
      for (int n = 0; n < S::NT; ++n) {
        st.o[mt][n][0] *= corr[0]; st.o[mt][n][1] *= corr[0];
        st.o[mt][n][2] *= corr[1]; st.o[mt][n][3] *= corr[1];
      }
    }
  }
  uint4 pa[MT][S::PARTS][kSlice / 16];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float m = st.m[mt][half];
      const float c = vexp - (m == -INFINITY ? 0.0f : m) + kPBase;
      float sum = 0.0f;
#pragma unroll
      for (int nt = 0; nt < NK; ++nt) {
        const float x0 = ptx::ex2_approx(s[mt][nt][half * 2] + c);
        const float x1 = ptx::ex2_approx(s[mt][nt][half * 2 + 1] + c);
        sum += x0 + x1;
        const uint32_t hi = f16x2(x0, x1);
        (&pa[mt][0][nt >> 1].x)[half + 2 * (nt & 1)] = hi;
        if constexpr (S::PARTS == 2)
          (&pa[mt][1][nt >> 1].x)[half + 2 * (nt & 1)] = f16x2_rest(x0, x1, hi);
      }
      st.l[mt][half] = fmaf(sum, vinv, st.l[mt][half]);
    }
#pragma unroll
  for (int kh = 0; kh < kSlice / 16; ++kh) {
    uint32_t vw[4][D / 32];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int key = kh * 16 + 2 * t + (r & 1) + (r >> 1) * 8;
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(vb + chunk_at<D>(key, g));
        vw[r][0] = x.x; vw[r][1] = x.y; vw[r][2] = x.z; vw[r][3] = x.w;
      } else {
        const uint2 x =
            *reinterpret_cast<const uint2*>(vb + chunk_at<D>(key, g >> 1) + (g & 1) * 8);
        vw[r][0] = x.x; vw[r][1] = x.y;
      }
    }
    if constexpr (kTail) {
      // A zero weight does not hide a NaN code of a key that the row does not see (or of what
      // lies after the last token): NaN codes are taken out here and put back into the rows
      // that see them.
      uint32_t nan = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
          nan |= __vcmpeq4(vw[r][w] & 0x7f7f7f7fu, 0x7f7f7f7fu);
      if (__any_sync(0xffffffffu, nan != 0)) {
        uint4 va[MT];  // 1 where the row sees the key
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const int key = kh * 16 + nt * 8 + 2 * t;
              (&va[mt].x)[half + 2 * nt] = (key < left[mt][half] ? 0x3c00u : 0u) |
                                           (key + 1 < left[mt][half] ? 0x3c000000u : 0u);
            }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t ind[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t bad = __vcmpeq4(vw[r][w] & 0x7f7f7f7fu, 0x7f7f7f7fu);
            vw[r][w] &= ~bad;
            ind[r] = bad & 0x38383838u;  // the code of 1.0
          }
#pragma unroll
          for (int q = 0; q < 4; q += 2) {
            const uint32_t sel = q < 2 ? 0x5140u : 0x7362u;
            uint32_t b0[2], b1[2];
            f16x4_from_e4m3(__byte_perm(ind[0], ind[1], sel), b0[0], b0[1]);
            f16x4_from_e4m3(__byte_perm(ind[2], ind[3], sel), b1[0], b1[1]);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                float hit[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_f16(hit, va[mt], b0[u], b1[u]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (hit[i] > 0.0f) st.o[mt][4 * w + q + u][i] = __uint_as_float(0x7fffffffu);
              }
          }
        }
      }
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        const uint32_t sel = q < 2 ? 0x5140u : 0x7362u;
        uint32_t b0[2], b1[2];
        f16x4_from_e4m3(__byte_perm(vw[0][w], vw[1][w], sel), b0[0], b0[1]);
        f16x4_from_e4m3(__byte_perm(vw[2][w], vw[3][w], sel), b1[0], b1[1]);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int part = 0; part < S::PARTS; ++part)
              mma_f16(st.o[mt][4 * w + q + u], pa[mt][part][kh], b0[u], b1[u]);
      }
    }
  }
}

template <class T, int D, int MT>
__global__ void __launch_bounds__(Shape<T, D, MT>::THREADS, Shape<T, D, MT>::CTAS)
attn_kernel(const CacheAttnParams p, float* ws_o, float2* ws_ml, UnitDesc* desc) {
  using S = Shape<T, D, MT>;
  constexpr int kWarps = S::WARPS, kThreads = S::THREADS, kStages = S::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Work<kThreads> work;
  __shared__ float s_rowf[S::ROWS];
  __shared__ int s_seen[S::ROWS];
  __shared__ float s_m[kWarps][S::ROWS], s_l[kWarps][S::ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int G = p.Hq / p.Hkv, R = G * p.window;
  const int nrg = (R + S::ROWS - 1) / S::ROWS;
  const int U = p.Hkv * nrg;
  const bool flag = blockIdx.x == 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // rows without keys get their zeros here
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    if (row_blocks(p, b, false) > 0) continue;
    T* o = (T*)p.o + (int64_t)b * p.window * p.Hq * D;
    for (int i = threadIdx.x; i < p.window * p.Hq * D; i += kThreads) st_elem(o, i, 0.0f);
  }
  if (threadIdx.x == 0) desc[blockIdx.x].pieces = 0;

  // this CTA's range of the list of blocks
  int64_t total = 0;
  int base = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    scan_rows(p, work, b0, flag);
    total += work.pre[kThreads];
    base = b0;
  }
  total *= U;
  int64_t ctas = (total + kMinCost - 1) / kMinCost;
  if (ctas > gridDim.x) ctas = gridDim.x;
  if (blockIdx.x >= ctas) return;
  const int64_t cta = blockIdx.x;
  int64_t pos = total * cta / ctas;
  const int64_t end = total * (cta + 1) / ctas;
  int64_t before = 0;  // blocks (times U) before row `base`
  if (p.batch > kThreads) {
    base = 0;
    for (;;) {
      scan_rows(p, work, base, false);
      if (before + work.pre[kThreads] * U > pos) break;
      before += work.pre[kThreads] * U;
      base += kThreads;
    }
  }
  int row;  // within the scanned rows: the last one that starts at or before pos
  {
    int a = 0, z = kThreads - 1;
    while (a < z) {
      const int mid = (a + z + 1) >> 1;
      if (before + work.pre[mid] * U <= pos) a = mid;
      else z = mid - 1;
    }
    row = a;
  }

  while (pos < end) {
    // the piece [blk0, blk1) of a unit
    while (work.pre[row + 1] == work.pre[row] || before + work.pre[row + 1] * U <= pos) {
      if (++row == kThreads) {
        before += work.pre[kThreads] * U;
        base += kThreads;
        row = 0;
        scan_rows(p, work, base, false);
      }
    }
    const int b = base + row;
    const int64_t cost = work.pre[row + 1] - work.pre[row], nb = cost - kUnitCost;
    const int64_t off = pos - before - work.pre[row] * U;
    const int unit = (int)(off / cost);
    const int64_t x0 = off - unit * cost;
    const int64_t x1 = x0 + (end - pos) < cost ? x0 + (end - pos) : cost;
    const int64_t stop = pos + (cost - x0);  // end of the unit
    pos += x1 - x0;
    const int64_t blk0 = x0 > kUnitCost ? x0 - kUnitCost : 0;
    const int64_t blk1 = x1 > kUnitCost ? x1 - kUnitCost : 0;
    if (blk0 == blk1) continue;  // the range ends before the unit's first block
    const int h = unit / nrg, rg = unit - h * nrg;
    const int rows = R - rg * S::ROWS < S::ROWS ? R - rg * S::ROWS : S::ROWS;
    const int n_tok = row_tokens(p, b);
    const int64_t start = p.start[b];

    // queries: scaled by a power of two, rounded to f16 parts, in the order of the MMA's operand
    for (int r = warp; r < S::ROWS; r += kWarps) {
      constexpr int N = D / 32;
      float q[N];
      uint32_t top = 0;
      const int gr = rg * S::ROWS + r, j = gr / G;
      const bool live = r < rows && j < n_tok;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        q[i] = 0.0f;
        if (live)
          q[i] = ld_elem((const T*)p.q, ((int64_t)(b * p.window + j) * p.Hq + h * G + (gr - j * G)) * D +
                                            lane * N + i);
        top = max(top, finite_abs_bits(q[i]));
      }
      top = __reduce_max_sync(0xffffffffu, top);
      int e = top ? 13 + 127 - (int)(top >> 23) : 0;
      e = e > 100 ? 100 : (e < -100 ? -100 : e);
      if (lane == 0) {
        s_rowf[r] = p.scale * 1.44269504f * pow2f(-e);
        // rows that are not live see everything: they force no mask, and are not stored
        const int64_t n = start + j + 1;
        s_seen[r] = live && n < kNoEnd ? (int)n : kNoEnd;
      }
      const float up = pow2f(e);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        // channels c, c + 1: lane quarter t', k-step k, register pair (c & 2)
        const int c = lane * N + i, tt = c / (D / 4), k = (c % (D / 4)) / 4;
        const int reg = (r & 15) / 8 + (c & 2);
        const uint32_t hi = f16x2(q[i] * up, q[i + 1] * up);
        uint32_t* f = reinterpret_cast<uint32_t*>(smem + S::BUF);
        const int at = (((r / 16) * S::PARTS * S::KSTEPS + k) * 32 + (r & 7) * 4 + tt) * 4 + reg;
        f[at] = hi;
        if constexpr (S::PARTS == 2)
          f[at + S::KSTEPS * 128] = f16x2_rest(q[i] * up, q[i + 1] * up, hi);
      }
    }
    __syncthreads();

    float rowf[MT][2];
    int seen[MT][2], least = kNoEnd;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        rowf[mt][half] = s_rowf[mt * 16 + half * 8 + g];
        seen[mt][half] = s_seen[mt * 16 + half * 8 + g];
      }
    for (int r = lane; r < S::ROWS; r += 32) least = min(least, s_seen[r]);
    least = __reduce_min_sync(0xffffffffu, least);

    WarpState<T, D, MT> st;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int n = 0; n < S::NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.o[mt][n][i] = 0.0f;
      st.m[mt][0] = st.m[mt][1] = -INFINITY;
      st.l[mt][0] = st.l[mt][1] = 0.0f;
    }

    // slices of this warp: warp, warp + kWarps, ... of the piece
    const int first = (int)blk0 * (kPage / kSlice) + warp, last = (int)blk1 * (kPage / kSlice);
    uint8_t* ring = smem + warp * kStages * S::STAGE;
    const uint32_t ring_u = ptx::smem_u32(ring);
    const int32_t* table = p.table + (int64_t)b * p.max_pages;
    const uint4* qf = reinterpret_cast<const uint4*>(smem + S::BUF);
    // 16-byte copies of a lane: chunk lane + 32 c, at rotated places of their rows
    const int put0 = D == 128 ? (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4)
                              : (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
    struct Pending {
      float ks, vs;
      bool present;
    };
    auto page_of = [&](int sl) { return sl < last ? table[sl / (kPage / kSlice)] : -1; };
    auto issue = [&](int sl, int page, int stage) {
      Pending n = {0.0f, 0.0f, page >= 0 && page < p.n_pages};
      if (n.present) {
        const int64_t slice = (int64_t)page * p.Hkv + h;
        const int64_t at =
            slice * (kPage * D) + (sl % (kPage / kSlice)) * S::SLICE_BYTES + lane * 16;
        const uint8_t* kp = p.kc + at;
        const uint8_t* vp = p.vc + at;
        const uint32_t dst = ring_u + stage * S::STAGE;
#pragma unroll
        for (int c = 0; c < S::SLICE_BYTES / 512; ++c)
          cp16(dst + c * 512 + (D == 128 ? put0 ^ ((c & 1) * 64) : put0), kp + c * 512);
#pragma unroll
        for (int c = 0; c < S::SLICE_BYTES / 512; ++c)
          cp16(dst + S::SLICE_BYTES + c * 512 + (D == 128 ? put0 ^ ((c & 1) * 64) : put0),
               vp + c * 512);
        n.ks = p.ks[slice];
        n.vs = p.vs[slice];
      } else if (page >= 0 && lane == 0 && p.status) {
        atomicOr(p.status, KDA_STATUS_BAD_PAGE);
      }
      cp_commit();
      return n;
    };
    Pending pend[kStages - 1];
    int next_page;
    {
      int pg[kStages];
#pragma unroll
      for (int i = 0; i < kStages; ++i) pg[i] = page_of(first + i * kWarps);
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) pend[i] = issue(first + i * kWarps, pg[i], i);
      next_page = pg[kStages - 1];
    }
    int stage = 0;
#pragma unroll 1
    for (int sl = first; sl < last; sl += kWarps) {
      cp_wait<kStages - 2>();
      __syncwarp();
      const Pending cur = pend[0];
#pragma unroll
      for (int i = 0; i < kStages - 2; ++i) pend[i] = pend[i + 1];
      const int ahead = sl + (kStages - 1) * kWarps;
      pend[kStages - 2] = issue(ahead, next_page, stage == 0 ? kStages - 1 : stage - 1);
      next_page = page_of(ahead + kWarps);
      const uint8_t* kb = ring + stage * S::STAGE;
      const uint8_t* vb = kb + S::SLICE_BYTES;
      stage = stage == kStages - 1 ? 0 : stage + 1;
      if (!cur.present) continue;
      int left[MT][2];
      if (sl * kSlice + kSlice <= least) {
        slice_step<T, D, MT, false>(st, kb, vb, qf, cur.ks, cur.vs, rowf, left, lane);
      } else {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) left[mt][half] = seen[mt][half] - sl * kSlice;
        slice_step<T, D, MT, true>(st, kb, vb, qf, cur.ks, cur.vs, rowf, left, lane);
      }
    }
    cp_wait<0>();

    // join the warps
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float l = st.l[mt][half];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (t == 0) {
          s_m[warp][mt * 16 + half * 8 + g] = st.m[mt][half];
          s_l[warp][mt * 16 + half * 8 + g] = l;
        }
      }
    __syncthreads();
    float* acc = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float* o = acc + (warp * S::ROWS + mt * 16 + half * 8 + g) * S::ROW_F + t * S::LANE_F;
#pragma unroll
        for (int n = 0; n < S::NT; n += 4)  // channels t D/4 + n and t D/4 + D/8 + n
#pragma unroll
          for (int u = 0; u < 2; ++u)
            *reinterpret_cast<float4*>(o + u * (D / 8) + n) =
                make_float4(st.o[mt][n][half * 2 + u], st.o[mt][n + 1][half * 2 + u],
                            st.o[mt][n + 2][half * 2 + u], st.o[mt][n + 3][half * 2 + u]);
      }
    __syncthreads();
    const bool whole = blk0 == 0 && blk1 == nb;
    const int slot = 2 * blockIdx.x + (blk0 == 0 ? 1 : 0);
    for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = (i % (D / 4)) * 4;
      float top = -INFINITY, l = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (s_m[w][r] == -INFINITY && s_l[w][r] == 0.0f) continue;  // saw no key
        const float f = ptx::ex2_approx(s_m[w][r] - (top == -INFINITY ? 0.0f : top));
        const float4 x = *reinterpret_cast<const float4*>(
            acc + (w * S::ROWS + r) * S::ROW_F + (c / (D / 4)) * S::LANE_F + c % (D / 4));
        l += f * s_l[w][r];
        o.x += f * x.x; o.y += f * x.y; o.z += f * x.z; o.w += f * x.w;
      }
      if (whole) {
        const int gr = rg * S::ROWS + r, j = gr / G;
        const bool live = j < n_tok;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        T* dst = (T*)p.o + ((int64_t)(b * p.window + j) * p.Hq + h * G + (gr - j * G)) * D + c;
        st_elem(dst, 0, live ? o.x * inv : 0.0f);
        st_elem(dst, 1, live ? o.y * inv : 0.0f);
        st_elem(dst, 2, live ? o.z * inv : 0.0f);
        st_elem(dst, 3, live ? o.w * inv : 0.0f);
      } else {
        *reinterpret_cast<float4*>(ws_o + ((int64_t)slot * S::ROWS + r) * D + c) = o;
        if (c == 0) ws_ml[(int64_t)slot * S::ROWS + r] = make_float2(top, l);
      }
    }
    if (!whole && blk0 == 0 && threadIdx.x == 0) {
      // the pieces of this unit end in the CTA whose range holds its last block
      int pieces = 1;
      while (total * (cta + pieces) / ctas < stop) ++pieces;
      UnitDesc d;
      d.b = b; d.h = h; d.rg = rg; d.pieces = pieces;
      desc[blockIdx.x] = d;
    }
    __syncthreads();
  }
}

constexpr int kJoinWarps = 8;

// Joins the pieces of the unit that CTA c began and others went on with: c's second slot, then
// the first slots of c + 1, c + 2, ... One CTA per (c, row): its warps sum every eighth piece, and
// their sums are added in order.
template <class T, int D, int MT>
__global__ void __launch_bounds__(kJoinWarps * 32)
join_kernel(const CacheAttnParams p, const float* ws_o, const float2* ws_ml, const UnitDesc* desc) {
  using S = Shape<T, D, MT>;
  constexpr int N = D / 32;
  __shared__ float s_o[kJoinWarps][D], s_l[kJoinWarps], s_top[kJoinWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const UnitDesc d = desc[blockIdx.x];
  const int G = p.Hq / p.Hkv, R = G * p.window;
  const int r = blockIdx.y, gr = d.rg * S::ROWS + r;
  if (d.pieces == 0 || gr >= R) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto slot_row = [&](int i) {
    return (int64_t)(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * S::ROWS + r;
  };
  float top = -INFINITY;
  for (int i = threadIdx.x; i < d.pieces; i += kJoinWarps * 32) top = fmaxf(top, ws_ml[slot_row(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_top[w]);
  const float mu = top == -INFINITY ? 0.0f : top;
  float o[N], l = 0.0f;
#pragma unroll
  for (int c = 0; c < N; ++c) o[c] = 0.0f;
#pragma unroll 4
  for (int i = warp; i < d.pieces; i += kJoinWarps) {
    const int64_t at = slot_row(i);
    const float2 ml = ws_ml[at];
    float x[N];
    if constexpr (N == 4) {
      const float4 v = *reinterpret_cast<const float4*>(ws_o + at * D + lane * N);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(ws_o + at * D + lane * N);
      x[0] = v.x; x[1] = v.y;
    }
    // a piece in which the row saw no key has m = -inf and only zeros
    const float f = ptx::ex2_approx(ml.x - mu);
    l = fmaf(f, ml.y, l);
#pragma unroll
    for (int c = 0; c < N; ++c) o[c] = fmaf(f, x[c], o[c]);
  }
#pragma unroll
  for (int c = 0; c < N; ++c) s_o[warp][lane * N + c] = o[c];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  if (threadIdx.x >= D) return;
  float sum = 0.0f;
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    sum += s_o[w][threadIdx.x];
    l += s_l[w];
  }
  const int j = gr / G;
  const bool live = j < row_tokens(p, d.b);
  T* dst = (T*)p.o + ((int64_t)(d.b * p.window + j) * p.Hq + d.h * G + (gr - j * G)) * D;
  st_elem(dst, threadIdx.x, live && l != 0.0f ? sum / l : 0.0f);
}

size_t piece_bytes(int rows, int d) { return (size_t)2 * kMaxCtas * rows * d * sizeof(float); }
size_t ml_bytes(int rows) { return (size_t)2 * kMaxCtas * rows * sizeof(float2); }

template <class T, int D, int MT>
kda_status launch_t(const CacheAttnParams& p, cudaStream_t s) {
  using S = Shape<T, D, MT>;
  static int ctas_of[64] = {};  // resident CTAs of each device, found once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64)
    return set_error(KDA_ERR_CUDA, "kda_cache_attention: no current device");
  if (ctas_of[dev] == 0) {
    int sms = 0, per = 0;
    e = cudaFuncSetAttribute(attn_kernel<T, D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::SMEM);
    if (e == cudaSuccess)
      e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, attn_kernel<T, D, MT>, S::THREADS,
                                                        S::SMEM);
    if (e != cudaSuccess || per < 1)
      return set_error(KDA_ERR_CUDA, std::string("kda_cache_attention: ") + cudaGetErrorString(e));
    ctas_of[dev] = sms * per < kMaxCtas ? sms * per : kMaxCtas;
  }
  const int G = p.Hq / p.Hkv, nrg = (G * p.window + S::ROWS - 1) / S::ROWS;
  // no more CTAs than the page table allows ranges of kMinCost
  const int64_t most =
      ((int64_t)p.batch * p.Hkv * nrg * (p.max_pages + kUnitCost) + kMinCost - 1) / kMinCost;
  const int ctas = most < ctas_of[dev] ? (int)most : ctas_of[dev];
  uint8_t* ws = (uint8_t*)p.ws;
  float* ws_o = (float*)ws;
  float2* ws_ml = (float2*)(ws + piece_bytes(S::ROWS, D));
  UnitDesc* desc = (UnitDesc*)(ws + piece_bytes(S::ROWS, D) + ml_bytes(S::ROWS));
  attn_kernel<T, D, MT><<<ctas, S::THREADS, S::SMEM, s>>>(p, ws_o, ws_ml, desc);
  kda_status st = check_launch("kda_cache_attention");
  if (st != KDA_OK) return st;
  cudaLaunchConfig_t cfg = {};
  const int rows = G * p.window < S::ROWS ? G * p.window : S::ROWS;
  cfg.gridDim = dim3(ctas, rows);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, join_kernel<T, D, MT>, p, (const float*)ws_o, (const float2*)ws_ml,
                     (const UnitDesc*)desc);
  count_launches(2);
  return check_launch("kda_cache_attention");
}

// Rows of a unit: two MMA row tiles when the group and window fill them (bf16), else one.
int row_tiles(kda_dtype dt, int rows) { return dt == KDA_BF16 && rows > 16 ? 2 : 1; }

}  // namespace

size_t cache_attn_workspace_bytes(int, int window, int Hq, int Hkv, int d) {
  const int rows = Hq / Hkv * window > 16 ? 32 : 16;
  return piece_bytes(rows, d) + ml_bytes(rows) + (sizeof(UnitDesc) * kMaxCtas + 255) / 256 * 256;
}

kda_status launch_cache_attn(const CacheAttnParams& p, kda_dtype dt, int d, cudaStream_t s) {
  if (dt == KDA_BF16) {
    if (row_tiles(dt, p.Hq / p.Hkv * p.window) == 2)
      return d == 128 ? launch_t<__nv_bfloat16, 128, 2>(p, s) : launch_t<__nv_bfloat16, 64, 2>(p, s);
    return d == 128 ? launch_t<__nv_bfloat16, 128, 1>(p, s) : launch_t<__nv_bfloat16, 64, 1>(p, s);
  }
  return d == 128 ? launch_t<float, 128, 1>(p, s) : launch_t<float, 64, 1>(p, s);
}

}  // namespace kda
