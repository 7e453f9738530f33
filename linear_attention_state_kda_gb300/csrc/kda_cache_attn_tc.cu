// Attention over the paged 8-bit cache on the fifth-generation tensor cores, for chunks of a prompt:
// bf16 queries, units of up to 256 query rows (the chunk's tokens times the query heads of a group).
//
// The mathematics is kda_cache_attn.cu's: e4m3 codes widened to f16 (exact), queries scaled by a
// power of two per row and rounded to f16, the pages' scales applied around both products, P in
// f16 relative to a running maximum that is raised rarely, sums in fp32. There, warp MMAs run at a
// quarter of the tensor cores' rate and each warp widens the codes for its own 16 rows; here the
// codes are widened once for 256 rows.
//
// One CTA per SM, persistent over its range of 128-key tiles. A unit's rows are two tiles of 128,
// which take turns: while one is in the softmax, the tensor cores work for the other.
//     S [128 rows x 128 keys]  = Q . K^T        operands in shared memory
//     O [128 rows x d]        += P . V          P in tensor memory, over the first half of its S
// Roles, each on its own warps and over all of the CTA's pieces without a common barrier:
//   warp 0        issues the MMAs of the row tiles in turn
//   warp 2        zeros of the units without keys
//   warp 3        walks the CTA's range and hands its pieces to the other roles (each doing so for
//                 itself would hold 25 registers more); descriptors of the units that begin here
//   warps 4-11    softmax, a warpgroup per row tile and a lane per row: scores from tensor memory,
//                 maximum, sum, P; its queries before a piece and its output after it. A row lies in
//                 one thread, so these warps need no barrier among themselves
//   warps 12-15   load the codes of a tile into registers while the tile before is in work, and
//                 widen them into two stages of K and of V (128-byte swizzle)
//
// What bounds it: the products take 2048 cycles per 256 x 128 scores, the exponentials as long at
// their full rate, and waits of some 150 cycles lie between a row tile's scores, softmax and values;
// measured 3.9 thousand. 4 chunks of 1024 tokens after 16384, 32/8 heads: 602 us, 1203 TFLOP/s (62%
// of the measured bf16 rate, 70% of the sustained one); 321 TFLOP/s with warp MMAs. Taking out the
// widening gains 2%, the loads of the codes 5%, the exponentials nothing. What it took, in TFLOP/s
// there:
//   530 -> 885   the issuing warp stays converged and its operands are known to be the same in all
//                lanes, with one lane elected at the instruction: from a branch of lane 0 each MMA
//                took four times as long to issue
//   885 -> 994   one rolled loop of steps for the issuing warp
//   994 -> 1068  less code: the waits count tries, loops that run once a piece are rolled (the
//                instruction cache missed on a third of its requests)
//  1068 -> 1146  barriers that are due together are looked at together
//  1146 -> 1200  the join of the units that were cut (join_kernel)
//  1212 -> 1203  waits for a whole piece, which look whether another role gave up
// Handing P over a page at a time gave 509 against 477 TFLOP/s where only one row tile has rows, and
// 1090 against 1146 there; taking the exponentials while the largest score is looked for, and
// beginning the tile again where it turns out too large, 1068 against 1213. Neither was kept.
// Tensor memory: 128 columns of S and d of O per row tile.
#include "kda_cache_attn.cuh"
#include "kda_fp8.cuh"
#include "ptx.cuh"

namespace kda {

using namespace attn;

namespace {

constexpr int kTile = 128;  // keys per step: two pages
constexpr int kThreads = 512;
// What beginning and ending a unit takes, in tiles (2 measured 17% slower on 64 windows of 256 rows,
// 6 and 10 within 3% either way).
constexpr int kUnitCost = 4;
constexpr uint32_t kTmemCols = 512;
constexpr int kScales = 4;  // ring of the tiles' scales
constexpr int kPieces = 4;  // ring of pieces
// Tries of a wait for a tile (2 s) and for a whole piece (63 s: the longest is 2^23 tiles, the keys of
// the largest page table, some 17 s).
constexpr uint32_t kTileTries = 1u << 19, kPieceTries = 1u << 24;

template <int D>
struct Smem {  // offsets; every operand tile starts on 1024 bytes
  static constexpr int QTILE = 128 * D * 2, KV = kTile * D * 2;
  static constexpr int Q = 0;
  static constexpr int K = Q + 2 * QTILE;
  static constexpr int V = K + 2 * KV;
  static constexpr int BYTES = V + 2 * KV;
};

// Every wait is by parity, which tells a phase only from the one before it. So a role may wait for a
// phase only where the phase before is known to be complete and the one after it cannot be:
//   k_full, v_full, by the MMAs: tiles in order; a stage's next tile waits for k_empty / v_empty of
//     this one. v_full, by the softmax: once the scores of tile n are there, a converter warp has put
//     V of n - 1 before K of n, and V of n + 2 waits for this row tile's P of n
//   k_empty, v_empty: tiles in order, two behind
//   q_full, s_full, p_full, o_full: of one row tile, each waited for by the other side in every tile
//     (piece) that the row tile has rows in; S, P and O take turns
//   scales: in order, by a row tile with rows in every piece; see there for one that skips some
//   piece_full, piece_empty: every role takes every piece
struct Bars {
  // codes widened (4 converter warps) and read by both row tiles' MMAs
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t scales[kScales];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2];  // by row tile
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint64_t drain;  // the MMAs in flight when a role gave up
};

struct Scales {  // of a tile's two pages
  float k[2], v[2];
  int there[2];
};

struct Work {  // a piece; without tiles: there are no more
  int b, h, rg, first, last, whole;
  int start, tokens;  // of its row
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 16 bytes to a shared-memory address.
__device__ __forceinline__ void st_shared(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
template <int N>
__device__ __forceinline__ void regs_give() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
// Empty statements that keep every use of loaded columns behind the wait.
__device__ __forceinline__ void tmem_loaded(uint32_t* r, int n) {
#pragma unroll
  for (int i = 0; i < n; ++i) asm volatile("" : "+r"(r[i]));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const CacheAttnParams p, int piece_rows, float* ws_o, float2* ws_ml, UnitDesc* desc,
               int32_t* cut) {
  using M = Smem<D>;
  constexpr int CPK = D / 16;            // 16-code chunks of a key
  constexpr int NL = kTile * CPK / 128;  // chunks of a tile that a converter thread takes
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ Bars bars;
  __shared__ Scales s_scales[kScales];
  __shared__ Work s_work[kPieces];
  // NaN codes of keys that some row does not see: a bit per channel, and whether a warp wrote any
  __shared__ __align__(16) uint16_t s_nan[2][kTile][CPK];
  __shared__ int s_nan_any[2][4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv, R = G * p.window;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars.k_full[i], 4);
      ptx::mbar_init(&bars.k_empty[i], 1);
      ptx::mbar_init(&bars.v_full[i], 4);
      ptx::mbar_init(&bars.v_empty[i], 1);
      ptx::mbar_init(&bars.q_full[i], 4);
      ptx::mbar_init(&bars.s_full[i], 1);
      ptx::mbar_init(&bars.p_full[i], 4);
      ptx::mbar_init(&bars.o_full[i], 1);
    }
    for (int i = 0; i < kScales; ++i) ptx::mbar_init(&bars.scales[i], 1);
    for (int i = 0; i < kPieces; ++i) {
      ptx::mbar_init(&bars.piece_full[i], 1);
      ptx::mbar_init(&bars.piece_empty[i], 13);
    }
    ptx::mbar_init(&bars.drain, 1);
    ptx::fence_mbar_init();
    s_abort = 0;
  }
  if (warp == 1) {
    ptx::tmem_alloc(&s_tmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  // the operand tiles are not in use yet
  int64_t* s_win = reinterpret_cast<int64_t*>(smem);
  int* s_rows = reinterpret_cast<int*>(s_win + kWindows);
  Ranges<kTile> ranges;
  ranges.plan(p, kTcRows, kThreads / 32, blockIdx.x, gridDim.x, kUnitCost, s_win, s_rows,
              blockIdx.x == 0);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);  // (known to be the same in all lanes)
  const uint32_t tmem_o = tmem + 2 * kTile;

  // A wait of a whole warp (all lanes get the same answer) for what another role does with a tile.
  // One that gives up records it, and the warp leaves; so do those that wait for it.
  auto outcome = [&](bool done) {
    if (__all_sync(0xffffffffu, done)) return true;
    if (p.status) atomicOr(p.status, KDA_STATUS_TIMEOUT);
    *(volatile int*)&s_abort = 1;
    return false;
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return outcome(ptx::mbar_wait_tries(bar, parity, kTileTries));
  };
  // For what takes another role a whole piece, or the search for the next one: as long as that takes,
  // and no longer than until a role gives up.
  auto wait_long = [&](uint64_t* bar, uint32_t parity) {
    return outcome(ptx::mbar_wait_tries_or(bar, parity, kPieceTries, &s_abort));
  };
  // Of two barriers, which are looked at together.
  auto wait2 = [&](uint64_t* a, uint32_t parity_a, uint64_t* b, uint32_t parity_b) {
    const bool ra = ptx::mbar_try_wait(a, parity_a), rb = ptx::mbar_try_wait(b, parity_b);
    return __all_sync(0xffffffffu, ra && rb) || (wait(a, parity_a) && wait(b, parity_b));
  };
  // Positions that the first row of a piece's unit sees.
  auto unit_first_sees = [&](const Work& x) {
    return (int64_t)x.start + x.rg * kTcRows / G + 1;
  };

  int n = 0;           // tiles of the pieces so far
  uint32_t taken = 0;  // pieces so far
  // The next piece, if there is one: for the 13 warps of the MMAs, the softmax and the converters.
  Work piece;
  auto take = [&]() {
    const uint32_t slot = taken % kPieces;
    if (!wait_long(&bars.piece_full[slot], (taken / kPieces) & 1)) return false;
    piece = s_work[slot];
    piece.first = __shfl_sync(0xffffffffu, piece.first, 0);
    piece.last = __shfl_sync(0xffffffffu, piece.last, 0);
    __syncwarp();  // every lane has read it (a shuffle orders no memory)
    if (lane == 0) ptx::mbar_arrive(&bars.piece_empty[slot]);
    ++taken;
    return piece.last > piece.first;
  };
  // registers of the four warpgroups: 72 + 176 + 176 + 88 = 4 x 128
  if (warp < 4) {
    regs_give<72>();
    if (warp == 0) {
      // ------------------------------------------------------------------ MMAs
      const uint32_t id_s = ptx::idesc_make(ptx::kFmtF16, 128, kTile, false, false);
      const uint32_t id_o = ptx::idesc_make(ptx::kFmtF16, 128, D, false, true);
      const uint32_t base = ptx::smem_u32(smem);
      uint32_t nq[2] = {0, 0};  // pieces of each row tile so far
      uint32_t parity = 0;      // bit g: of row tile g's next O product
      bool ok = true;
      while (ok && take()) {
        const int tiles = piece.last - piece.first;
        const int halves = R - piece.rg * kTcRows > 128 ? 2 : 1;
        for (int g = 0; ok && g < halves; ++g) ok = wait(&bars.q_full[g], nq[g]++ & 1);
        // Steps (tile, row tile): the values' product of the tile, then the scores of the next
        // tile, which overwrite the P that the product reads. Tile -1 has only scores.
#pragma unroll 1
        for (int i = -1, g = 0; ok && i < tiles;) {
          const int m = n + i, buf = m & 1;
          const bool final = g == halves - 1;  // frees the stages
          if (i >= 0) {
            ok = wait2(&bars.v_full[buf], (m >> 1) & 1, &bars.p_full[g], parity >> g & 1);
            if (!ok) break;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
              const uint64_t b = ptx::sdesc_sw128(base + M::V + buf * M::KV, kTile * 128, 1024);
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k)
                ptx::mma_f16_ts(tmem_o + g * D, tmem + g * kTile + k * 8, ptx::desc_add(b, k * 2048),
                                id_o, i > 0 || k > 0);
              ptx::mma_commit(&bars.o_full[g]);
              if (final) ptx::mma_commit(&bars.v_empty[buf]);
            }
            __syncwarp();
          }
          if (i + 1 < tiles) {
            // (before the first tile the last product of the piece before is looked at: complete)
            ok = wait2(&bars.k_full[buf ^ 1], ((m + 1) >> 1) & 1, &bars.o_full[g],
                       (parity >> g & 1) ^ (i < 0));
            if (!ok) break;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
              const uint64_t a = ptx::sdesc_sw128(base + M::Q + g * M::QTILE, 16, 1024);
              const uint64_t b = ptx::sdesc_sw128(base + M::K + (buf ^ 1) * M::KV, 16, 1024);
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (k >> 2) * (128 * 128) + (k & 3) * 32;
                ptx::mma_f16(tmem + g * kTile, ptx::desc_add(a, off), ptx::desc_add(b, off), id_s,
                             k > 0);
              }
              ptx::mma_commit(&bars.s_full[g]);
              if (final) ptx::mma_commit(&bars.k_empty[buf ^ 1]);
            }
            __syncwarp();
          }
          if (i >= 0) parity ^= 1u << g;
          if (final) ++i;
          g = final ? 0 : 1;
        }
        n += tiles;
      }
      if (__any_sync(0xffffffffu, *(volatile int*)&s_abort)) {
        // a role gave up: the MMAs in flight end first
        if (ptx::elect_one()) ptx::mma_commit(&bars.drain);
        __syncwarp();
        ptx::mbar_wait_tries(&bars.drain, 0, kTileTries);
        __syncwarp();
      }
    } else if (warp == 2) {
      ranges.zero_units<__nv_bfloat16>(p, D, blockIdx.x, gridDim.x, desc);
    } else if (warp == 3) {
      Piece x = {};
      bool ok = true;
      int begun = -1;
      for (bool more = true; more; ++taken) {
        more = ranges.next(p, x);
        if (!more) x.first = x.last = 0;
        else if (x.first == 0) {
          const int at = x.b * ranges.U + x.unit;
          if (lane == 0) desc[at] = x.desc;
          if (!x.whole) begun = at;
        }
        const int start = more ? p.start[x.b] : 0, tokens = more ? row_tokens(p, x.b) : 0;
        // (descriptors are written to the end also when the other roles have left)
        const uint32_t slot = taken % kPieces;
        ok = ok && wait_long(&bars.piece_empty[slot], ((taken / kPieces) & 1) ^ 1);
        if (ok && lane == 0) {
          s_work[slot] = {x.b, x.h, x.rg, x.first, x.last, x.whole, start, tokens};
          ptx::mbar_arrive(&bars.piece_full[slot]);
        }
      }
      if (lane == 0) cut[blockIdx.x] = begun;
    }
  } else if (warp < 12) {
    // -------------------------------------------------------------------- softmax
    regs_take<176>();
    const int g = (warp - 4) >> 2, w = warp & 3, r = w * 32 + lane;
    const uint32_t lanes = (uint32_t)(w * 32) << 16;
    const uint32_t t_s = tmem + lanes + g * kTile, t_o = tmem_o + lanes + g * D;
    uint32_t use = 0;  // tiles of this row tile so far
    bool ok = true, skipped = false;
    while (ok && take()) {
      const int tiles = piece.last - piece.first;
      const int gr = piece.rg * kTcRows + g * 128 + r;
      if (R - piece.rg * kTcRows <= g * 128) {  // no rows
        n += tiles;
        skipped = true;
        continue;
      }
      const int j = gr / G, n_tok = piece.tokens;
      const bool live = gr < R && j < n_tok;
      const int64_t at_row =
          ((int64_t)piece.b * p.window + j) * p.Hq + piece.h * G + (gr - j * G);  // of q and o
      float rowf;
      {
        const uint4* src = reinterpret_cast<const uint4*>((const __nv_bfloat16*)p.q + at_row * D);
        // (rolled: this is run once a piece, and what it takes of the instruction cache is fetched
        // each time)
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        uint32_t top = 0;
#pragma unroll 8
        for (int i = 0; i < D / 8; ++i) {
          float q[8];
          Vec16<__nv_bfloat16>::unpack(live ? src[i] : zero, q);
#pragma unroll
          for (int u = 0; u < 8; ++u) top = max(top, finite_abs_bits(q[u]));
        }
        int e = top ? 13 + 127 - (int)(top >> 23) : 0;
        e = e > 100 ? 100 : e;  // (-114 at the least)
        const float up = pow2f(e);
        rowf = p.scale * 1.44269504f * pow2f(-e);
        const uint32_t dst =
            ptx::smem_u32(smem) + M::Q + g * M::QTILE + (r >> 3) * 1024 + (r & 7) * 128;
#pragma unroll 8
        for (int i = 0; i < D / 8; ++i) {
          float q[8];
          Vec16<__nv_bfloat16>::unpack(live ? src[i] : zero, q);
          st_shared(dst + (i >> 3) * (128 * 128) + (((i & 7) ^ (r & 7)) << 4),
                    make_uint4(pack_f16(q[0] * up, q[1] * up), pack_f16(q[2] * up, q[3] * up),
                               pack_f16(q[4] * up, q[5] * up), pack_f16(q[6] * up, q[7] * up)));
        }
      }
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();  // O of the piece before has been read
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars.q_full[g]);

      // rows that are not live see everything: they force no mask, and are not stored
      const int64_t sees = (int64_t)piece.start + j + 1;
      const int seen = live && sees < kNoEnd ? (int)sees : kNoEnd;
      const int64_t first_sees = unit_first_sees(piece);
      float m = -INFINITY, l = 0.0f;
      uint4 nan = make_uint4(0u, 0u, 0u, 0u);  // channels in which the row saw a NaN
      // After a skipped piece, the first scores before the first scales. A wait by parity tells a
      // phase only from the one before it, and the converters may still be many tiles behind: the
      // ring's word is another tile's then, and its parity may let the wait pass. s_full counts this
      // row tile's own tiles. With the scores of tile n there, tile n - 4's scales have been published,
      // and tile n + 4's cannot be: they wait until the keys of n + 2 have been read, and so for this
      // row tile's P of tile n. Without a skip the scores of the tile before say the same.
      if (skipped) ok = wait_long(&bars.s_full[g], use & 1);
      skipped = false;
#pragma unroll 1
      for (int i = piece.first; i < piece.last; ++i, ++n, ++use) {
        ok = ok && wait(&bars.scales[n % kScales], (n / kScales) & 1);
        const Scales sc = s_scales[n % kScales];
        const int left = seen - i * kTile;
        const bool masked =
            __any_sync(0xffffffffu, left < kTile || !sc.there[0] || !sc.there[1]);
        float f[2], vexp[2], vref[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          f[hf] = rowf * sc.k[hf];
          const int ve = (int)((__float_as_uint(sc.v[hf]) >> 23) & 255u) - 127;
          vexp[hf] = (float)ve;
          vref[hf] = (float)(ve < kMinScaleExp ? kMinScaleExp : ve);
        }
        ok = ok && wait(&bars.s_full[g], use & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        uint32_t s[kTile];  // scores, then log2 P
#pragma unroll 1
        for (bool again = false;; again = true) {
#pragma unroll
          for (int c = 0; c < 4; ++c) ptx::tmem_ld32_nowait(t_s + c * 32, s + c * 32);
          ptx::tmem_ld_wait();
          tmem_loaded(s, kTile);
          const float m0 = m == -INFINITY ? 0.0f : m;
          float top[2];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float c = vexp[hf] - m0 + kPBase;
            const f32x2 f2 = pair(f[hf], f[hf]), c2 = pair(c, c);
#pragma unroll
            for (int k = hf * 32; k < hf * 32 + 32; ++k) {
              float y0, y1;
              split(fma2(pair(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), f2, c2), y0,
                    y1);
              s[2 * k] = __float_as_uint(y0);
              s[2 * k + 1] = __float_as_uint(y1);
            }
          }
          if (masked) {
            // keys of each page that the row sees (opaque, or the comparisons are made ahead of the
            // branch for every tile)
            int see[2];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              see[hf] = sc.there[hf] ? left - hf * kPage : 0;
              asm volatile("" : "+r"(see[hf]));
            }
#pragma unroll
            for (int k = 0; k < kTile; ++k)
              if (k % kPage >= see[k / kPage]) s[k] = 0xff800000u;
          }
          bool over = false;
          float most = m;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float t[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              t[u] = __uint_as_float(s[hf * 64 + u]);
#pragma unroll
              for (int k = 4 + u; k < 64; k += 4) t[u] = fmaxf(t[u], __uint_as_float(s[hf * 64 + k]));
            }
            // y = x + vexp - m0 + kPBase; M must stay within kSlack of x + vref
            top[hf] = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) - (vexp[hf] - vref[hf] + kPBase) +
                      m0;
            over |= top[hf] > m + kSlack;
            most = fmaxf(most, top[hf]);
          }
          if (again || !__any_sync(0xffffffffu, over)) break;
          const float corr = ptx::ex2_approx(m - (most == -INFINITY ? 0.0f : most));
          m = most;
          l *= corr;
          if (i > piece.first) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              ptx::tmem_ld32(t_o + c * 32, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] *= corr;
              ptx::tmem_st32(t_o + c * 32, o);
            }
          }
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          f32x2 sum[2] = {0ull, 0ull};
#pragma unroll
          for (int k = hf * 32; k < hf * 32 + 32; ++k) {
            const float e0 = ptx::ex2_approx(__uint_as_float(s[2 * k]));
            const float e1 = ptx::ex2_approx(__uint_as_float(s[2 * k + 1]));
            sum[k & 1] = add2(sum[k & 1], pair(e0, e1));
            s[k] = pack_f16(e0, e1);
          }
          float a, b;
          split(add2(sum[0], sum[1]), a, b);
          const float vinv = __uint_as_float((uint32_t)(127 - (int)vexp[hf]) << 23);  // 2^-e
          l = fmaf(a + b, vinv, l);
          ptx::tmem_st32_nowait(t_s + hf * 32, reinterpret_cast<const float*>(s + hf * 32));
        }
        if ((int64_t)i * kTile + kTile > first_sees) {
          // what the converters took out is put back into the rows that see it
          ok = wait(&bars.v_full[n & 1], (n >> 1) & 1);
          if (!ok) break;
          const int* any = s_nan_any[n & 1];
          if (any[0] | any[1] | any[2] | any[3]) {
#pragma unroll 1
            for (int k = 0; k < kTile && k < left; ++k) {
              if (!any[k * CPK % 128 / 32]) continue;
              const uint32_t* x = reinterpret_cast<const uint32_t*>(s_nan[n & 1][k]);
              nan.x |= x[0];
              nan.y |= x[1];
              if constexpr (D == 128) {
                nan.z |= x[2];
                nan.w |= x[3];
              }
            }
            __syncwarp();
          }
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars.p_full[g]);
      }
      ok = ok && wait(&bars.o_full[g], (use - 1) & 1);
      if (!ok) break;
      ptx::tc_fence_after();
      const int slot = 2 * (int)blockIdx.x + (piece.first == 0 ? 1 : 0);
      const int64_t to = (int64_t)slot * piece_rows + g * 128 + r;
      const float inv = live && l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        __syncwarp();
        ptx::tmem_ld32(t_o + c * 32, o);
        const uint32_t bad = c < 2 ? (c == 0 ? nan.x : nan.y) : (c == 2 ? nan.z : nan.w);
        if (bad) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (bad >> k & 1u) o[k] = __uint_as_float(0x7fffffffu);
        }
        if (gr < R && piece.whole) {
          uint4* dst = reinterpret_cast<uint4*>((__nv_bfloat16*)p.o + at_row * D + c * 32);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = inv != 0.0f ? o[k] * inv : 0.0f;
#pragma unroll
          for (int k = 0; k < 4; ++k) dst[k] = Vec16<__nv_bfloat16>::pack(o + k * 8);
        } else if (gr < R) {
          float4* dst = reinterpret_cast<float4*>(ws_o + to * D + c * 32);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
      if (gr < R && !piece.whole) ws_ml[to] = make_float2(m, l);
    }
  } else {
    // -------------------------------------------------------------------- K and V to f16
    regs_give<88>();
    const int tid = threadIdx.x - 384, w = warp - 12;
    // Channels 16 c .. 16 c + 15 of keys key0 + i (128 / CPK). Eight lanes take four chunks of two
    // keys, so that the two 16-byte pieces of their f16 go to eight different places of a row.
    const int c = D == 128 ? (tid & 3) + (tid >> 1 & 4) : tid & 3;
    const int key0 = D == 128 ? (tid >> 2 & 1) + (tid >> 4) * 2 : tid >> 2;
    // (128 / CPK is a multiple of 8: every i has the same rotation of the row's pieces)
    const uint32_t row0 = (c >> 2) * (kTile * 128) + (key0 >> 3) * 1024 + (key0 & 7) * 128;
    const uint32_t put0 = row0 + (((2 * (c & 3)) ^ (key0 & 7)) << 4);
    const uint32_t put1 = row0 + (((2 * (c & 3) + 1) ^ (key0 & 7)) << 4);
    const uint32_t tiles_at = ptx::smem_u32(smem);
    bool ok = true;
    while (ok && take()) {
      const int32_t* table = p.table + (int64_t)piece.b * p.max_pages;
      const int n_tok = piece.tokens, start = piece.start;
      const int j1 = (piece.rg * kTcRows + kTcRows - 1) / G;
      const int64_t first_sees = unit_first_sees(piece);
      // positions that some row of the unit sees
      const int64_t reach = (int64_t)start + (j1 < n_tok ? j1 + 1 : n_tok);
      int page[2];  // of the tile whose codes are loaded next
      auto look = [&](int i) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int at = 2 * i + hf;
          page[hf] = i < piece.last && at < p.max_pages && (int64_t)at * kPage < reach ? table[at] : -1;
        }
      };
      uint4 kraw[NL], vraw[NL];
      auto load = [&](uint4 (&raw)[NL], const uint8_t* codes) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const int pg = page[i / (NL / 2)];
          raw[i] = make_uint4(0u, 0u, 0u, 0u);
          if (pg >= 0 && pg < p.n_pages)
            raw[i] = *reinterpret_cast<const uint4*>(
                codes + ((int64_t)pg * p.Hkv + piece.h) * (kPage * D) +
                (key0 * CPK + c + 128 * (i % (NL / 2))) * 16);
        }
      };
      Scales next;
      auto load_scales = [&]() {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int pg = page[hf];
          next.there[hf] = pg >= 0 && pg < p.n_pages;
          next.k[hf] = next.v[hf] = 1.0f;
          if (next.there[hf]) {
            next.k[hf] = p.ks[(int64_t)pg * p.Hkv + piece.h];
            next.v[hf] = p.vs[(int64_t)pg * p.Hkv + piece.h];
          } else if (pg >= 0 && p.status) {
            atomicOr(p.status, KDA_STATUS_BAD_PAGE);
          }
        }
      };
      // f16 of chunk i into a tile
      auto put = [&](uint32_t tile, int i, const uint4& x) {
        uint4 a, b;
        f16x4_from_e4m3(x.x, a.x, a.y);
        f16x4_from_e4m3(x.y, a.z, a.w);
        f16x4_from_e4m3(x.z, b.x, b.y);
        f16x4_from_e4m3(x.w, b.z, b.w);
        st_shared(tile + put0 + i * (128 / CPK) * 128, a);
        st_shared(tile + put1 + i * (128 / CPK) * 128, b);
      };
      look(piece.first);
      load(kraw, p.kc);
      load(vraw, p.vc);
      if (tid == 0) load_scales();
      look(piece.first + 1);
#pragma unroll 1
      for (int i = piece.first; ok && i < piece.last; ++i, ++n) {
        const int buf = n & 1;
        if (n >= 2) ok = wait(&bars.k_empty[buf], ((n - 2) >> 1) & 1);
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < NL; ++x) put(tiles_at + M::K + buf * M::KV, x, kraw[x]);
        if (tid == 0) s_scales[n % kScales] = next;
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars.k_full[buf]);
        if (tid == 0) {
          ptx::mbar_arrive(&bars.scales[n % kScales]);
          load_scales();
        }
        load(kraw, p.kc);
        if (n >= 2) ok = wait(&bars.v_empty[buf], ((n - 2) >> 1) & 1);
        if (!ok) break;
        if ((int64_t)i * kTile + kTile > first_sees) {
          // some rows do not see all of these keys, and a zero weight does not hide a NaN: NaN
          // codes are taken out and noted for the rows that see them
          uint32_t any = 0;
          uint16_t marks[NL];
#pragma unroll
          for (int x = 0; x < NL; ++x) {
            uint32_t* q = &vraw[x].x;
            marks[x] = 0;
            if ((int64_t)i * kTile + key0 + x * (128 / CPK) < first_sees) continue;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint32_t bad = __vcmpeq4(q[u] & 0x7f7f7f7fu, 0x7f7f7f7fu);
              q[u] &= ~bad;
              marks[x] |= (uint16_t)(((bad & 1u) | (bad >> 7 & 2u) | (bad >> 14 & 4u) | (bad >> 21 & 8u))
                                     << (4 * u));
            }
            any |= marks[x];
          }
          any = __any_sync(0xffffffffu, any != 0);
          if (any) {
#pragma unroll
            for (int x = 0; x < NL; ++x) s_nan[buf][key0 + x * (128 / CPK)][c] = marks[x];
          }
          if (lane == 0) s_nan_any[buf][w] = any;
        } else if (lane == 0) {
          s_nan_any[buf][w] = 0;
        }
#pragma unroll
        for (int x = 0; x < NL; ++x) put(tiles_at + M::V + buf * M::KV, x, vraw[x]);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars.v_full[buf]);
        load(vraw, p.vc);
        look(i + 2);
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) ptx::tmem_dealloc(tmem, kTmemCols);
}

template <int D>
kda_status launch_d(const CacheAttnParams& p, int ctas, int piece_rows, float* ws_o, float2* ws_ml,
                    UnitDesc* desc, int32_t* cut, cudaStream_t s) {
  constexpr int bytes = Smem<D>::BYTES + 1024;
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !set[dev]) {
    cudaFuncSetAttribute(attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    set[dev] = true;
  }
  attn_tc_kernel<D><<<ctas, kThreads, bytes, s>>>(p, piece_rows, ws_o, ws_ml, desc, cut);
  return check_launch("kda_cache_attention");
}

}  // namespace

namespace attn {

kda_status launch_attn_tc(const CacheAttnParams& p, int d, int ctas, int piece_rows, float* ws_o,
                          float2* ws_ml, UnitDesc* desc, int32_t* cut, cudaStream_t s) {
  return d == 128 ? launch_d<128>(p, ctas, piece_rows, ws_o, ws_ml, desc, cut, s)
                  : launch_d<64>(p, ctas, piece_rows, ws_o, ws_ml, desc, cut, s);
}

}  // namespace attn
}  // namespace kda
