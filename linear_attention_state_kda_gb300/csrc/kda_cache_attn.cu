// Attention of one decoded token, of a verify window or of a chunk of a prompt over the paged 8-bit
// cache (kda_cache_attention): o = sum_t softmax_t(scale q . k_t) v_t in one pass over the cache
// with the running maximum and sum of the softmax. More than 64 bf16 query rows per key/value head
// run on the kernel of kda_cache_attn_tc.cu.
//
// What bounds it: the cache is read once, 2 d bytes per token and key/value head, so a single
// decoded token per row is HBM-bound; the 4 d operations per (query row, key) are tensor-core
// work. A "unit" is one (batch row, key/value head) with up to 64 query rows (the window's tokens
// times the query heads of the group), so that the cache is read once for all of them.
//
// Arithmetic. e4m3 codes are exact in f16, so both products run as f16 x f16 -> fp32 warp MMAs
// on codes; the page's power-of-two scales are applied around them. A query row is multiplied by
// a power of two that puts its largest entry in [2^13, 2^14) and rounded to f16: exact for bf16
// entries down to 2^-28 of the largest; fp32 queries are carried as the sum of two f16 parts (22
// bits). With x_t the score in units of log2 and e_t the exponent of t's value scale, the row
// keeps M, at most 8 below max_t (x_t + e_t), and accumulates
//     P_t = 2^(x_t + e_t - M + 7) (f16; two parts for fp32),  O = sum_t P_t code_t,
//     l = sum_t 2^(x_t - M + 7) = sum_t P_t 2^-e_t (fp32),    o = O / l.
// P is at most 2^15 whatever the scales of the pages, and what f16 drops is below 2^-32 of the row's
// largest term, as long as the row sees a value scale of 2^-80 or more. In M a smaller e_t counts as
// -80, so that l stays in range; where all are smaller, 2^e at the most, what f16 drops is below
// 2^-(112 + e) of the largest term: 2^-12 for the smallest scale, 2^-100. (l loses what is below 2^-126
// as P: terms below 2^-24 of the largest where a row's value scales are 2^109 apart, larger ones beyond.)
//
// Layout. Lane (g, t) = (lane / 4, lane % 4) of an m16n8k16 MMA. The order of the channels in the
// first product and of the columns in the second is free as long as both operands agree, and is
// chosen so that a lane reads 16-byte pieces of a cached row as they lie: channels 32 t .. 32 t +
// 31 of key g for the scores, and channels 16 g .. 16 g + 15 of keys 2t, 2t+1, 2t+8, 2t+9 for the
// values, whose bytes are interleaved pairwise to give two keys of one channel (d = 128; half of
// that for d = 64). A lane's outputs are then 32 consecutive channels of its row.
//
// Work split. The rows' key slices (32 keys) are laid end to end (row, head, row group, slice) and
// cut into as many equal ranges as workers fit on the GPU, so that ragged lengths and few rows load
// every SM alike. A worker is one warp (8 per SM), or a team of 2 or 4 warps with 16 query rows
// each (12 warps per SM); it walks its range through its own ring of shared-memory buffers filled
// with 16-byte asynchronous copies, and while one begins or ends a unit the others keep the memory
// busy. (A CTA per unit, its warps joined at the unit's end, left 4-8 us of latency per unit
// uncovered: 398 us against 352 on 128 rows of up to 16k tokens. Two row tiles in one warp instead
// of a team: 8 warps of 255 registers, 98 us against 74 on 32 windows of 32 rows. Teams in 16 warps
// of 128 registers spill: 292 us against 149 on 64 windows.) A unit that lies in one range is
// finished there; the pieces of a unit that is cut go to the workspace (each worker has at most
// two) and a second kernel, placed ahead of time and released when the first ends, joins them in
// order: no atomics, the same bits every time. (Only the second kernel is launched that way: the
// launch costs some 2 us more on the host, which the first would not win back.)
#include "kda_cache_attn.cuh"
#include "kda_fp8.cuh"
#include "ptx.cuh"

namespace kda {

using namespace attn;

namespace {

constexpr int kSlice = 32;    // keys per warp step
constexpr int kUnitCost = 4;  // what beginning and ending a unit takes, in slices

// TEAM warps walk a unit's slices together, 16 query rows each: the slice is copied once for all
// of them.
template <class T, int D, int TEAM>
struct Shape {
  static constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
  static constexpr int WARPS = TEAM == 1 ? 8 : 12;  // one CTA per SM: 255 or 168 registers a thread
  static constexpr int THREADS = WARPS * 32;
  static constexpr int TEAMS = WARPS / TEAM;        // workers of a CTA
  static constexpr int ROWS = 16 * TEAM;
  static constexpr int KSTEPS = D / 16;
  static constexpr int NT = D / 8;                // n-tiles of the second product
  static constexpr int SLICE_BYTES = kSlice * D;  // one of K, V
  static constexpr int STAGE = 2 * SLICE_BYTES;
  static constexpr int STAGES = D == 128 ? 2 : 3;
  // Query operands: in registers where there are enough, else in shared memory.
  static constexpr bool QREG = TEAM == 1;
  static constexpr int QFRAGS = PARTS * KSTEPS;
  static constexpr int QBYTES = QREG ? 0 : QFRAGS * 512;  // of a warp
  static constexpr int SMEM = TEAMS * STAGES * STAGE + WARPS * QBYTES;
};

// Barrier of a team's warps.
template <int TEAM>
__device__ __forceinline__ void team_sync(int team) {
  if constexpr (TEAM == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(TEAM * 32) : "memory");
}

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

template <int D>
struct WarpState {
  float o[D / 8][4];
  float m[2], l[2];
};

// One slice: scores, softmax update, weighted values. kTail: some key of the slice is hidden from
// some row; `left` of its keys are seen by each of the lane's rows.
template <class T, int D, int TEAM, bool kTail>
__device__ __forceinline__ void slice_step(
    WarpState<D>& st, const uint8_t* kb, const uint8_t* vb,
    const uint4 (&qreg)[Shape<T, D, TEAM>::QREG ? Shape<T, D, TEAM>::QFRAGS : 1],
    const uint4* qfrag, float ks, float vs, const float (&rowf)[2], const int (&left)[2], int lane) {
  using S = Shape<T, D, TEAM>;
  constexpr int NK = kSlice / 8;  // key tiles of the first product
  const int g = lane >> 2, t = lane & 3;
  float s[NK][4];
#pragma unroll
  for (int nt = 0; nt < NK; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[nt][i] = 0.0f;
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
      for (int part = 0; part < S::PARTS; ++part) {
        const int at = part * S::KSTEPS + 4 * j + k4;
        const uint4 a = S::QREG ? qreg[S::QREG ? at : 0] : qfrag[at * 32 + lane];
#pragma unroll
        for (int nt = 0; nt < NK; ++nt) mma_f16(s[nt], a, b[nt][0], b[nt][1]);
      }
    }
  }
  const int ve = (int)((__float_as_uint(vs) >> 23) & 255u) - 127;
  const float vexp = (float)ve, vref = (float)(ve < kMinScaleExp ? kMinScaleExp : ve);
  const float vinv = __uint_as_float((uint32_t)(127 - ve) << 23);  // 2^-e
  // s becomes log2 P relative to the row's M (0 for one without keys so far)
  bool over = false;
  float top[2], c[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const float f = rowf[half] * ks;
    c[half] = vexp - (st.m[half] == -INFINITY ? 0.0f : st.m[half]) + kPBase;
    const f32x2 f2 = pair(f, f), c2 = pair(c[half], c[half]);
    top[half] = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NK; ++nt) {
      float &y0 = s[nt][half * 2], &y1 = s[nt][half * 2 + 1];
      split(fma2(pair(y0, y1), f2, c2), y0, y1);
      if constexpr (kTail) {
        if (nt * 8 + 2 * t >= left[half]) y0 = -INFINITY;
        if (nt * 8 + 2 * t + 1 >= left[half]) y1 = -INFINITY;
      }
      top[half] = fmaxf(top[half], fmaxf(y0, y1));
    }
    top[half] += vref - c[half];
    over |= top[half] > st.m[half] + kSlack;
  }
  if (__any_sync(0xffffffffu, over)) {
    float corr[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float x = top[half];
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
      const float mo = st.m[half], mn = fmaxf(mo, x), ref = mn == -INFINITY ? 0.0f : mn;
      st.m[half] = mn;
      corr[half] = ptx::ex2_approx(mo - ref);
      st.l[half] *= corr[half];
      const float down = (mo == -INFINITY ? 0.0f : mo) - ref;
#pragma unroll
      for (int nt = 0; nt < NK; ++nt) {
        s[nt][half * 2] += down;
        s[nt][half * 2 + 1] += down;
      }
    }
#pragma unroll
    for (int n = 0; n < S::NT; ++n) {
      st.o[n][0] *= corr[0]; st.o[n][1] *= corr[0];
      st.o[n][2] *= corr[1]; st.o[n][3] *= corr[1];
    }
  }
  uint4 pa[S::PARTS][kSlice / 16];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    f32x2 sums = 0ull;
#pragma unroll
    for (int nt = 0; nt < NK; ++nt) {
      const float x0 = ptx::ex2_approx(s[nt][half * 2]);
      const float x1 = ptx::ex2_approx(s[nt][half * 2 + 1]);
      sums = add2(sums, pair(x0, x1));
      const uint32_t hi = f16x2(x0, x1);
      (&pa[0][nt >> 1].x)[half + 2 * (nt & 1)] = hi;
      if constexpr (S::PARTS == 2)
        (&pa[1][nt >> 1].x)[half + 2 * (nt & 1)] = f16x2_rest(x0, x1, hi);
    }
    float sum0, sum1;
    split(sums, sum0, sum1);
    st.l[half] = fmaf(sum0 + sum1, vinv, st.l[half]);
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
        uint4 va;  // 1 where the row sees the key
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const int key = kh * 16 + nt * 8 + 2 * t;
            (&va.x)[half + 2 * nt] = (key < left[half] ? 0x3c00u : 0u) |
                                     (key + 1 < left[half] ? 0x3c000000u : 0u);
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
            for (int u = 0; u < 2; ++u) {
              float hit[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              mma_f16(hit, va, b0[u], b1[u]);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (hit[i] > 0.0f) st.o[4 * w + q + u][i] = __uint_as_float(0x7fffffffu);
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
          for (int part = 0; part < S::PARTS; ++part)
            mma_f16(st.o[4 * w + q + u], pa[part][kh], b0[u], b1[u]);
      }
    }
  }
}

template <class T, int D, int TEAM>
__global__ void __launch_bounds__(Shape<T, D, TEAM>::THREADS, 1)
attn_kernel(const CacheAttnParams p, int piece_rows, float* ws_o, float2* ws_ml, UnitDesc* desc) {
  using S = Shape<T, D, TEAM>;
  constexpr int kStages = S::STAGES, kWarps = S::WARPS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_win[kWindows];
  __shared__ int s_rows[kWindows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int team = warp / TEAM, member = warp % TEAM;
  const int G = p.Hq / p.Hkv, R = G * p.window;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // consecutive ranges are on different SMs
  const int worker = team * gridDim.x + blockIdx.x;
  Ranges<kSlice> ranges;
  ranges.plan(p, S::ROWS, kWarps, worker, (int64_t)gridDim.x * S::TEAMS, kUnitCost, s_win, s_rows,
              blockIdx.x == 0);

  uint8_t* ring = smem + team * (kStages * S::STAGE);
  const uint32_t ring_u = ptx::smem_u32(ring);
  uint4* qf = reinterpret_cast<uint4*>(smem + S::TEAMS * kStages * S::STAGE + warp * S::QBYTES);
  // 16-byte copies of a lane: chunk lane + 32 c, at rotated places of their rows; the team's
  // members take every TEAM-th c
  const int put0 = D == 128 ? (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4)
                            : (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);

  Piece piece;
  while (ranges.next(p, piece)) {
    const int b = piece.b, h = piece.h, rg = piece.rg, first = piece.first, last = piece.last;
    const int n_tok = row_tokens(p, b);
    const int start = p.start[b];
    const int32_t* table = p.table + (int64_t)b * p.max_pages;
    struct Pending {
      float ks, vs;
      bool present;
    };
    auto page_of = [&](int sl) {
      return sl < last ? table[sl / (kPage / kSlice)] : -1;
    };
    auto issue = [&](int sl, int page, int stage) {
      Pending n = {0.0f, 0.0f, page >= 0 && page < p.n_pages};
      if (n.present) {
        const int64_t slice = (int64_t)page * p.Hkv + h;
        const int64_t off =
            slice * (kPage * D) + (sl % (kPage / kSlice)) * S::SLICE_BYTES + lane * 16;
        const uint8_t* kp = p.kc + off;
        const uint8_t* vp = p.vc + off;
        const uint32_t dst = ring_u + stage * S::STAGE;
#pragma unroll
        for (int i = 0; i < S::SLICE_BYTES / 512 / TEAM; ++i) {
          const int c = i * TEAM + member;
          cp16(dst + c * 512 + (D == 128 ? put0 ^ ((c & 1) * 64) : put0), kp + c * 512);
        }
#pragma unroll
        for (int i = 0; i < S::SLICE_BYTES / 512 / TEAM; ++i) {
          const int c = i * TEAM + member;
          cp16(dst + S::SLICE_BYTES + c * 512 + (D == 128 ? put0 ^ ((c & 1) * 64) : put0),
               vp + c * 512);
        }
        n.ks = p.ks[slice];
        n.vs = p.vs[slice];
      } else if (page >= 0 && lane == 0 && member == 0 && p.status) {
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
      for (int i = 0; i < kStages; ++i) pg[i] = page_of(first + i);
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) pend[i] = issue(first + i, pg[i], i);
      next_page = pg[kStages - 1];
    }

    // Queries: a lane loads its D / 4 channels of rows g and g + 8 of each row tile, scales them
    // by a power of two and rounds them to the f16 parts of its MMA operands.
    const int row0 = rg * S::ROWS + member * 16;  // of this warp's rows
    float rowf[2];
    int seen[2], least = kNoEnd;
    uint4 qreg[S::QREG ? S::QFRAGS : 1];
    {
      uint32_t frag[S::PARTS][S::KSTEPS][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int gr = row0 + half * 8 + g, j = gr / G;
        const bool live = gr < R && j < n_tok;
        float q[D / 4];
#pragma unroll
        for (int i = 0; i < D / 4; ++i) q[i] = 0.0f;
        if (live) {
          const uint4* src = reinterpret_cast<const uint4*>(
              (const T*)p.q + ((int64_t)(b * p.window + j) * p.Hq + h * G + (gr - j * G)) * D +
              t * (D / 4));
          constexpr int N = Vec16<T>::N;
#pragma unroll
          for (int i = 0; i < D / 4 / N; ++i) Vec16<T>::unpack(src[i], q + i * N);
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) top = max(top, finite_abs_bits(q[i]));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e = top ? 13 + 127 - (int)(top >> 23) : 0;
        e = e > 100 ? 100 : e;  // (-114 at the least)
        const float up = pow2f(e);
        rowf[half] = p.scale * 1.44269504f * pow2f(-e);
        // rows that are not live see everything: they force no mask, and are not stored
        const int64_t n = (int64_t)start + j + 1;
        seen[half] = live && n < kNoEnd ? (int)n : kNoEnd;
        least = min(least, seen[half]);
#pragma unroll
        for (int k = 0; k < S::KSTEPS; ++k)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float a0 = q[4 * k + 2 * c] * up, a1 = q[4 * k + 2 * c + 1] * up;
            frag[0][k][half + 2 * c] = f16x2(a0, a1);
            if constexpr (S::PARTS == 2)
              frag[1][k][half + 2 * c] = f16x2_rest(a0, a1, frag[0][k][half + 2 * c]);
          }
      }
#pragma unroll
      for (int part = 0; part < S::PARTS; ++part)
#pragma unroll
        for (int k = 0; k < S::KSTEPS; ++k) {
          const uint4 a = make_uint4(frag[part][k][0], frag[part][k][1], frag[part][k][2],
                                     frag[part][k][3]);
          const int i = part * S::KSTEPS + k;
          if constexpr (S::QREG) qreg[i] = a;
          else qf[i * 32 + lane] = a;
        }
    }
    least = __reduce_min_sync(0xffffffffu, least);

    WarpState<D> st;
#pragma unroll
    for (int n = 0; n < S::NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[n][i] = 0.0f;
    st.m[0] = st.m[1] = -INFINITY;
    st.l[0] = st.l[1] = 0.0f;
    int stage = 0;
#pragma unroll 1
    for (int sl = first; sl < last; ++sl) {
      // the copies of every member, and the end of every member's last step
      cp_wait<kStages - 2>();
      team_sync<TEAM>(team);
      const Pending cur = pend[0];
#pragma unroll
      for (int i = 0; i < kStages - 2; ++i) pend[i] = pend[i + 1];
      pend[kStages - 2] =
          issue(sl + kStages - 1, next_page, stage == 0 ? kStages - 1 : stage - 1);
      next_page = page_of(sl + kStages);
      const uint8_t* kb = ring + stage * S::STAGE;
      const uint8_t* vb = kb + S::SLICE_BYTES;
      stage = stage == kStages - 1 ? 0 : stage + 1;
      if (!cur.present) continue;
      if (row0 >= R) continue;  // a member without rows only copies
      int left[2];
      if (sl * kSlice + kSlice <= least) {
        slice_step<T, D, TEAM, false>(st, kb, vb, qreg, qf, cur.ks, cur.vs, rowf, left, lane);
      } else {
        left[0] = seen[0] - sl * kSlice;
        left[1] = seen[1] - sl * kSlice;
        slice_step<T, D, TEAM, true>(st, kb, vb, qreg, qf, cur.ks, cur.vs, rowf, left, lane);
      }
    }
    cp_wait<0>();
    team_sync<TEAM>(team);  // the ring is free for the next unit

    const int slot = 2 * worker + (first == 0 ? 1 : 0);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float l = st.l[half];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const int gr = row0 + half * 8 + g, j = gr / G;
      if (gr >= R) continue;
      float o[D / 4];  // channels t D/4 + n and t D/4 + D/8 + n
#pragma unroll
      for (int n = 0; n < S::NT; ++n) {
        o[n] = st.o[n][half * 2];
        o[D / 8 + n] = st.o[n][half * 2 + 1];
      }
      if (piece.whole) {
        const bool live = j < n_tok;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint4* dst = reinterpret_cast<uint4*>(
            (T*)p.o + ((int64_t)(b * p.window + j) * p.Hq + h * G + (gr - j * G)) * D +
            t * (D / 4));
        constexpr int N = Vec16<T>::N;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) o[i] = live ? o[i] * inv : 0.0f;
#pragma unroll
        for (int i = 0; i < D / 4 / N; ++i) dst[i] = Vec16<T>::pack(o + i * N);
      } else {
        const int64_t to = (int64_t)slot * piece_rows + (gr - rg * S::ROWS);
        float4* dst = reinterpret_cast<float4*>(ws_o + to * D + t * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        if (t == 0) ws_ml[to] = make_float2(st.m[half], l);
      }
    }
    if (first == 0 && member == 0 && lane == 0)
      desc[(int64_t)b * ranges.U + piece.unit] = piece.desc;
  }
  ranges.zero_units<T>(p, D, warp * gridDim.x + blockIdx.x, gridDim.x * kWarps, desc);
}

// Joins the pieces of a unit that was cut: the second slot of the warp that began it, then the
// first slots of the next ones. kPerRow warps of the CTA sum every kPerRow-th piece of a row relative
// to their own largest M, and their sums are added in order; one warp writes its row by itself.
// blockIdx.x is the unit, or, with `cut`, the worker that began it: of many units of a prompt's chunk
// at most one per worker is cut (4 chunks of 1024 tokens after 16384 have 512 units on 152 workers:
// 616 us a call against 633; without a barrier for rows of one warp 604).
template <class T, int D, int kJoinWarps, int kPerRow, int kBatch>
__global__ void __launch_bounds__(kJoinWarps * 32)
join_kernel(const CacheAttnParams p, int unit_rows, int piece_rows, const float* ws_o,
            const float2* ws_ml, const UnitDesc* desc, const int32_t* cut) {
  constexpr int N = D / 32;
  const int G = p.Hq / p.Hkv, R = G * p.window;
  const int nrg = (R + unit_rows - 1) / unit_rows, U = p.Hkv * nrg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % kPerRow;
  constexpr int kRows = kJoinWarps / kPerRow;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int at_unit = cut ? cut[blockIdx.x] : (int)blockIdx.x;
  if (at_unit < 0) return;
  const UnitDesc d = desc[at_unit];
  const int b = at_unit / U, unit = at_unit - b * U, h = unit / nrg, rg = unit - h * nrg;
  const int n_tok = row_tokens(p, b);
  if (d.pieces == 0) return;
  const int r = blockIdx.y * kRows + warp / kPerRow, gr = rg * unit_rows + r;
  const bool mine = r < unit_rows && gr < R;
  float o[N], l = 0.0f, m = -INFINITY;
#pragma unroll
  for (int c = 0; c < N; ++c) o[c] = 0.0f;
  for (int i0 = sub; mine && i0 < d.pieces; i0 += kPerRow * kBatch) {
    float2 ml[kBatch];
    float x[kBatch][N];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kPerRow;
      ml[k] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int c = 0; c < N; ++c) x[k][c] = 0.0f;
      if (i >= d.pieces) continue;
      const int64_t at =
          (int64_t)(i == 0 ? 2 * d.worker + 1 : 2 * (d.worker + i)) * piece_rows + r;
      ml[k] = ws_ml[at];
      if constexpr (N == 4) {
        const float4 v = *reinterpret_cast<const float4*>(ws_o + at * D + lane * N);
        x[k][0] = v.x; x[k][1] = v.y; x[k][2] = v.z; x[k][3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(ws_o + at * D + lane * N);
        x[k][0] = v.x; x[k][1] = v.y;
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) top = fmaxf(top, ml[k].x);
    const float mu = top == -INFINITY ? 0.0f : top;
    const float keep = ptx::ex2_approx(m - mu);
    m = top;
    l *= keep;
#pragma unroll
    for (int c = 0; c < N; ++c) o[c] *= keep;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      // a piece in which the row saw no key has M = -inf and only zeros
      const float f = ptx::ex2_approx(ml[k].x - mu);
      l = fmaf(f, ml[k].y, l);
#pragma unroll
      for (int c = 0; c < N; ++c) o[c] = fmaf(f, x[k][c], o[c]);
    }
  }
  if constexpr (kPerRow == 1) {
    const int j = gr / G;
    if (!mine) return;
    const bool live = j < n_tok && l != 0.0f;
    T* dst = (T*)p.o + ((int64_t)(b * p.window + j) * p.Hq + h * G + (gr - j * G)) * D;
#pragma unroll
    for (int c = 0; c < N; ++c) st_elem(dst, lane * N + c, live ? o[c] / l : 0.0f);
  } else {
    __shared__ float s_o[kJoinWarps][D], s_l[kJoinWarps], s_m[kJoinWarps];
#pragma unroll
    for (int c = 0; c < N; ++c) s_o[warp][lane * N + c] = o[c];
    if (lane == 0) {
      s_l[warp] = l;
      s_m[warp] = m;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * D; i += kJoinWarps * 32) {
      const int rr = i / D, c = i - rr * D;
      const int gq = rg * unit_rows + blockIdx.y * kRows + rr, j = gq / G;
      if (blockIdx.y * kRows + rr >= unit_rows || gq >= R) continue;
      float top = -INFINITY;
      for (int w = 0; w < kPerRow; ++w) top = fmaxf(top, s_m[rr * kPerRow + w]);
      const float mu = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f, ls = 0.0f;
      for (int w = 0; w < kPerRow; ++w) {
        const float f = ptx::ex2_approx(s_m[rr * kPerRow + w] - mu);
        sum = fmaf(f, s_o[rr * kPerRow + w][c], sum);
        ls = fmaf(f, s_l[rr * kPerRow + w], ls);
      }
      const bool live = j < n_tok && ls != 0.0f;
      T* dst = (T*)p.o + ((int64_t)(b * p.window + j) * p.Hq + h * G + (gq - j * G)) * D;
      st_elem(dst, c, live ? sum / ls : 0.0f);
    }
  }
}

// Warps of a team: as many as the unit's query rows fill, up to four (bf16); more rows are cut into
// groups that read the cache again. fp32 has too many operands for 168 registers.
int team_of(kda_dtype dt, int rows) { return dt == KDA_F32 || rows <= 16 ? 1 : (rows <= 32 ? 2 : 4); }

// bf16 calls with at least this many query rows per key/value head go to the tcgen05 kernel: beyond
// 64 rows the warps' units read and convert the codes again. 64 windows over contexts to 8k, 8
// key/value heads, d = 128: 80 rows 262 us against 469, 128 rows 277 against 489, 256 rows 314
// against 938 (d = 64, 80 rows: 185 against 306); one chunk of 512 tokens after 8192: 83 against 245.
// Only the shortest contexts lose, to the longer start: 64 tokens after 100, 21 us against 17.
constexpr int kTcMinRows = 65;

// SMs used on the current device (0: error, set).
int sms_here() {
  static int sms_of[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    set_error(KDA_ERR_CUDA, "kda_cache_attention: no current device");
    return 0;
  }
  if (sms_of[dev] == 0) {
    int sms = 0;
    const cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess || sms < 1) {
      set_error(KDA_ERR_CUDA, std::string("kda_cache_attention: ") + cudaGetErrorString(e));
      return 0;
    }
    sms_of[dev] = sms < kMaxSms ? sms : kMaxSms;
  }
  return sms_of[dev];
}

// Few units have many pieces each: 16 warps for a row of one. Many units have a few: a warp for a
// row, in small CTAs.
template <class T, int D>
kda_status launch_join(const CacheAttnParams& p, int unit_rows, int rows, int64_t units, int workers,
                       int sms, const float* ws_o, const float2* ws_ml, const UnitDesc* desc,
                       const int32_t* cut, cudaStream_t s) {
  if (cut && units > workers) units = workers;
  else cut = nullptr;
  const bool few = units * rows <= 4 * sms;
  auto kernel = few ? join_kernel<T, D, 16, 16, 8> : join_kernel<T, D, 4, 1, 4>;
  static bool set[2][64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !set[few][dev]) {
    // the same split of L1 and shared memory for both kernels: no SM is drained to change it
    cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                         cudaSharedmemCarveoutMaxShared);
    set[few][dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)units, (unsigned)(few ? rows : (rows + 3) / 4));
  cfg.blockDim = dim3(few ? 512 : 128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, p, unit_rows, rows, ws_o, ws_ml, desc, cut);
  count_launches(2);
  return check_launch("kda_cache_attention");
}

template <class T, int D, int TEAM>
kda_status launch_main(const CacheAttnParams& p, int ctas, int rows, float* ws_o, float2* ws_ml,
                       UnitDesc* desc, cudaStream_t s) {
  using S = Shape<T, D, TEAM>;
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !set[dev]) {
    cudaFuncSetAttribute(attn_kernel<T, D, TEAM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         S::SMEM);
    set[dev] = true;
  }
  attn_kernel<T, D, TEAM><<<ctas, S::THREADS, S::SMEM, s>>>(p, rows, ws_o, ws_ml, desc);
  return check_launch("kda_cache_attention");
}

template <class T, int D>
kda_status launch_t(const CacheAttnParams& p, kda_dtype dt, cudaStream_t s) {
  const int sms = sms_here();
  if (sms == 0) return KDA_ERR_CUDA;
  const int R = p.Hq / p.Hkv * p.window, team = team_of(dt, R);
  const bool tc = dt == KDA_BF16 && R >= kTcMinRows;
  const int unit_rows = tc ? kTcRows : 16 * team;
  const int nrg = (R + unit_rows - 1) / unit_rows, rows = R < unit_rows ? R : unit_rows;
  // no more CTAs than the page table allows slices
  const int64_t units = (int64_t)p.batch * p.Hkv * nrg;
  const int64_t most = units * p.max_pages * (kPage / kSlice);
  const int ctas = most < sms ? (int)most : sms;
  float* ws_o = (float*)p.ws;
  float2* ws_ml = (float2*)(ws_o + piece_rows_of(R) * D);
  UnitDesc* desc = (UnitDesc*)(ws_ml + piece_rows_of(R));
  int32_t* cut = nullptr;
  kda_status st;
  if (tc) {
    cut = (int32_t*)(desc + units);
    st = launch_attn_tc(p, D, ctas, rows, ws_o, ws_ml, desc, cut, s);
  } else if constexpr (sizeof(T) == 4) {
    st = launch_main<T, D, 1>(p, ctas, rows, ws_o, ws_ml, desc, s);
  } else {
    st = team == 1   ? launch_main<T, D, 1>(p, ctas, rows, ws_o, ws_ml, desc, s)
         : team == 2 ? launch_main<T, D, 2>(p, ctas, rows, ws_o, ws_ml, desc, s)
                     : launch_main<T, D, 4>(p, ctas, rows, ws_o, ws_ml, desc, s);
  }
  if (st != KDA_OK) return st;
  return launch_join<T, D>(p, unit_rows, rows, units, ctas, sms, ws_o, ws_ml, desc, cut, s);
}

}  // namespace

size_t cache_attn_workspace_bytes(int batch, int window, int Hq, int Hkv, int d) {
  const int R = Hq / Hkv * window;
  const size_t units = (size_t)batch * Hkv * ((R + 15) / 16);
  return piece_rows_of(R) * (d * sizeof(float) + sizeof(float2)) +
         (sizeof(UnitDesc) * units + sizeof(int32_t) * kMaxSms + 255) / 256 * 256;
}

kda_status launch_cache_attn(const CacheAttnParams& p, kda_dtype dt, int d, cudaStream_t s) {
  if (dt == KDA_F32) return d == 128 ? launch_t<float, 128>(p, dt, s) : launch_t<float, 64>(p, dt, s);
  return d == 128 ? launch_t<__nv_bfloat16, 128>(p, dt, s) : launch_t<__nv_bfloat16, 64>(p, dt, s);
}

}  // namespace kda
