// Linear attention with one decay per head on the tensor cores: prompts in bf16.
//
// Chunks of 64 tokens. With gamma the running sum of the log-decays in a chunk, Gamma its total and S
// the state before it (fp32, transposed: a thread has a value channel and half of the key channels),
//     O^T = e^gamma_t * (S^T Q^T) + V^T P^T,   P_ts = [s <= t] e^(gamma_t - gamma_s) q_t . k_s
//     S'^T = e^Gamma S^T + V'^T K,             V'_s = e^(Gamma - gamma_s) v_s
// Every product is a tcgen05 bf16 product with fp32 sums. Operands that are not inputs are carried in
// several bf16 parts, so that an output is as exact as its own rounding lets it be: S and P in two
// (2^-15 of a term; rounded to one, outputs whose terms cancel were off by up to 16 times their own
// rounding), V' in three (24 bits: states are fp32, and what a token adds stays for the rest of the
// sequence). Each chunk's V'^T K is a sum of its own, added to the state in registers. The two sums of
// O have accumulators of their own and meet in fp32, so that Q needs no decayed copy.
//
// Roles of a CTA (28 warps): one takes the units of work (segments of a head), one loads (TMA), one
// sums the decays, one issues the products; 8 put V and V' into TMEM, transposed on the way; 4 turn
// q.k into P; 8 keep the state; 4 write outputs. The chunks of all units run through them as one
// stream, so that a unit's ends are covered by its neighbours. Order of the products per chunk: q.k,
// V'^T K, which the state waits for, S^T Q^T and V^T P^T. The state's high part lies in TMEM, which is
// full then, the low part in shared memory: three chunks of q, k and v fit beside it.
//
// 16384 tokens x 32 heads (d = 128): 180 us, of which what the segments add takes 55, the scan 7
// and the outputs 120 (with S and P in one part each 163 and 105). The outputs move 537 MB in that, 4.5
// TB/s; a chunk takes some 3500 cycles: 2300 in which the warp that issues has products to issue (44;
// the three parts of V' are 12 of them and nearly half of the tensor time), the rest its looks at
// barriers and its waits for the last chunk's outputs and the state's parts, whose warps share the issue
// slots. Measured and left: both parts of the state in TMEM, the scores in the second sum's columns
// (205 us: P and the outputs then wait for one another); the two parts of S^T Q^T behind barriers of
// their own (188-208: more looks); V'^T K before q.k (189); all looks in one before the last products
// (204: they wait for the slowest). What a segment adds takes 1350 cycles a chunk: three of four
// segments a head, 201 MB, on 96 of the SMs.
#include "kda_decay.cuh"
#include "kda_fp8.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

using namespace decay;

constexpr int kC = 64;
constexpr int kStages = 4;  // chunks that the roles work on
constexpr int kData = 3;    // of these, with their q, k and v in shared memory (released earlier)
constexpr int kThreads = 896;
constexpr int kAhead = 2, kAddAhead = 8;  // chunks whose decays are asked for ahead (room; latency)
constexpr uint32_t kTries = 1u << 19;  // of a wait inside a CTA: 2 s

struct Maps {
  CUtensorMap q, k, v, o;
};

// What the roles know of a stage's chunk.
struct Chunk {
  const float* entry;  // of the unit's first chunk: the state before it, or nullptr (zeros)
  float* exit;         // of a unit's last chunk: where the state after it goes, or nullptr
  int t0;              // first token
  int head;
  short tokens;        // how many of the 64 belong to the segment
  short kind;
};
constexpr int kFirst = 1, kStop = 2, kLast = 4;  // kinds: begins or ends a unit; none, the roles leave

// A unit of the work: a segment of one head. The scheduling warp takes the units that this CTA runs
// (its own block's, then those of blocks that were not launched yet: a long unit holds no one up) and
// finds their segments; the warps that load and that sum decays follow it through a ring.
constexpr int kUnits = 2;
struct Unit {
  const float* entry;
  float* exit;
  int lo, hi, head;
  int place;  // -1: there are no more units
};
struct UnitRing {
  uint64_t full[kUnits], empty[kUnits], clc, ask;
  alignas(16) uint32_t response[4];
  Unit unit[kUnits];
};

// Offsets in shared memory. Operand tiles are [64 tokens][64 channels] blocks of 8 KB (128-byte
// swizzle), D / 64 of them side by side.
template <int D>
struct Out {
  static constexpr int TILE = kC * D * 2, STAGE = 3 * TILE;
  static constexpr int Q = 0, K = TILE, V = 2 * TILE;
  static constexpr int P = kData * STAGE;  // two parts of 8 KB
  static constexpr int O = P + 2 * 8192;   // outputs, as Q
  static constexpr int LO = O + TILE;      // low part of the state: [128 value channels][64 key channels]
  static constexpr int SMALL = LO + 128 * D * 2;
};
// Every wait is by parity, which tells a phase only from the one before it, so none may be two phases
// behind. Each barrier's next phase needs, at some remove, what its waiters do after this one: a
// stage's chunk is replaced once every role has left it, its data once the products and V' have; the
// next scores wait for p_full, the next P for sc_full (which comes behind V^T P^T of the last), the
// next sum and V' for kv_done and u_empty, the next parts of the state for sq_done, the next V for
// o_full, the next outputs for o_empty.
struct OutSmall {
  UnitRing units;
  uint64_t full[kStages], empty[kStages], data_full[kData], data_empty[kData];
  uint64_t sc_full, p_full, v_full, vt_full, u_empty, hi_full;
  uint64_t kv_done, sq_done, o_full, o_empty, drain;
  float ghi[kStages][kC], glo[kStages][kC];  // running sums of log2 decays, high and low parts
  float in[kStages][kC], out[kStages][kC];   // decays from the chunk's start, and to its end
  float g[kAhead][kC];                       // log-decays of the next chunks
  float total[kStages];                      // decay of a whole chunk
  Chunk chunk[kStages];
  uint32_t tmem;
  int abort;
};
// TMEM columns: what a chunk adds to the state (fp32), the state's high part, V' in three parts and
// V (transposed, two tokens a column), the scores, and the two sums of O, all 512 at D = 128.
template <int D>
struct Tm {
  static constexpr int U = 0, HI = D, VP = HI + D / 2, VT = VP + 96, SC = VT + 32, OI = SC + 64,
                       OA = OI + 64;
  static_assert(OA + 64 <= 512, "TMEM");
};

__device__ __forceinline__ void st_shared(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
// Upper halves of two words (a's in the low half): bf16 by truncation.
__device__ __forceinline__ uint32_t tops(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The bf16 of a pair by truncation, and the exact rest.
__device__ __forceinline__ uint32_t take_top(ptx::f32x2& x) {
  float a, b;
  ptx::unpack2(x, a, b);
  const uint32_t t = tops(a, b);
  float ra, rb;
  asm("{\n\t.reg .b16 lo, hi, m;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "mov.b16 m, 0xbf80;\n\t"
      "fma.rn.f32.bf16 %0, lo, m, %3;\n\t"
      "fma.rn.f32.bf16 %1, hi, m, %4;\n\t}"
      : "=f"(ra), "=f"(rb)
      : "r"(t), "f"(a), "f"(b));
  x = ptx::pack2(ra, rb);
  return t;
}
// A pair in two bf16 parts: the first cut (it never overflows), the rest rounded, 2^-15 in all. An
// infinity or NaN stays one: its rest is NaN.
__device__ __forceinline__ void split2(ptx::f32x2 x, uint32_t& hi, uint32_t& lo) {
  hi = take_top(x);
  float a, b;
  ptx::unpack2(x, a, b);
  lo = pack_bf16(a, b);
}
// Two bf16 values times two weights in three parts of 8 bits: the fp32 products exactly.
__device__ __forceinline__ void weigh3(uint32_t v, ptx::f32x2 w, uint32_t part[3]) {
  ptx::f32x2 f =
      ptx::mul2(ptx::pack2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)), w);
  part[0] = take_top(f);
  part[1] = take_top(f);
  float a, b;
  ptx::unpack2(f, a, b);
  part[2] = tops(a, b);
}

// D x 64 tile of a head's rows from token t0.
template <int D>
__device__ __forceinline__ void load_tile(void* dst, const CUtensorMap* m, uint64_t* bar, int head,
                                          int t0) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    ptx::tma_load_2d((uint8_t*)dst + i * 8192, m, bar, head * D + i * 64, t0);
}

// V'^T K of a chunk: three parts of V' (TMEM), K (MN-major). Products round their sums toward zero,
// so the parts go from the smallest to the largest and each chunk into a sum of its own, which is
// then added in registers: summed up over chunks in place, a slowly decaying state was off by 2e-6
// after 500 tokens (and 4e-6 after 4000), now by 2e-7.
template <int D>
__device__ __forceinline__ void issue_kv(uint32_t tmem_u, uint32_t vp, uint32_t k) {
  const uint32_t id = ptx::idesc_make(ptx::kFmtBF16, 128, D, false, true);
  const uint64_t b = ptx::sdesc_sw128(k, 8192, 1024);
#pragma unroll 1
  for (int part = 2; part >= 0; --part)
#pragma unroll
    for (uint32_t i = 0; i < kC / 16; ++i)
      ptx::mma_f16_ts(tmem_u, vp + (uint32_t)part * 32 + i * 8, ptx::desc_add(b, i * 2048), id,
                      part < 2 || i > 0);
}

// 16 bytes (8 channels) number i of a tile: row i / (D / 8), swizzled place.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int i) {
  const int t = i / (D / 8), c = i % (D / 8);
  return (uint32_t)((c >> 3) * 8192 + t * 128 + (((c & 7) ^ (t & 7)) << 4));
}
// A ring of the next chunks' log-decays: lane l has tokens 2 l and 2 l + 1. Loaded kAhead chunks
// before their use: the latency of one load is as long as a chunk.
template <int kAhead>
struct DecayRing {
  float (*ring)[kC];
  const float* g;
  int64_t stride;
  int lane;
  // Asks for the tokens from t0 on (those at or after t_end count as 0); every call is a group.
  __device__ __forceinline__ void ask(int n, int t0, int t_end) const {
    float* dst = &ring[n % kAhead][2 * lane];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + 2 * lane + i;
      if (t < t_end) ptx::cp_async4(dst + i, g + t * stride);
      else dst[i] = 0.0f;
    }
    ptx::cp_async_commit();
  }
  // The next `chunks` of those asked for have arrived.
  template <int chunks>
  __device__ __forceinline__ void wait() const {
    ptx::cp_async_wait<kAhead - chunks>();
  }
  __device__ __forceinline__ float2 get(int n) const {
    return *reinterpret_cast<const float2*>(&ring[n % kAhead][2 * lane]);
  }
};

// 16 channels x 32 tokens of V, transposed: words 2 i + c hold tokens 8 i + 2 t, + 1 (t = lane % 4) of
// channel 8 c + lane / 4.
__device__ __forceinline__ void load_vt(uint32_t v, int ch, int tok, int lane, uint32_t* r) {
  // lane's row: token tok + (lane >> 4) * 8 + (lane & 7), channels ch + ((lane >> 3) & 1) * 8 ..
  const int t = tok + (lane >> 4) * 8 + (lane & 7), c = (ch + ((lane >> 3) & 1) * 8) >> 3;
  const uint32_t at = v + (c >> 3) * 8192 + t * 128 + (((c & 7) ^ (t & 7)) << 4);
  ptx::ld_matrix4_trans(at, r);
  ptx::ld_matrix4_trans(at + 16 * 128, r + 4);  // (16 tokens on: the same swizzle)
}
__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fffffff); }

// What every role needs to wait: gives up after kTries or when another role did. (The roles' code has
// to stay within the instruction cache: the caller's status is set once, at the kernel's end.)
struct Waiter {
  int* abort;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    const bool done =
        __all_sync(0xffffffffu, ptx::mbar_wait_short(bar, parity, kTries, abort));
    if (!done) *(volatile int*)abort = 1;
    return done;
  }
  // Of two barriers, which are looked at together: a look takes some 200 cycles beside the traffic of
  // the products.
  __device__ __forceinline__ bool both(uint64_t* a, uint32_t parity_a, uint64_t* b,
                                       uint32_t parity_b) const {
    const bool ra = ptx::mbar_test(a, parity_a), rb = ptx::mbar_test(b, parity_b);
    return __all_sync(0xffffffffu, ra && rb) || ((*this)(a, parity_a) && (*this)(b, parity_b));
  }
};
// The scheduling warp. find(block, unit): the unit of a block; false where it has none.
template <class Find>
__device__ __forceinline__ void schedule(UnitRing& ring, const Waiter& wait, int lane,
                                         const Find& find) {
  int block = blockIdx.x;
  uint32_t asked = 0, n = 0;
  bool ok = true;
#pragma unroll 1
  while (ok) {
    const bool more = block >= 0;
    Unit u;
    u.place = -1;
    if (!more || find(block, u)) {
      const uint32_t at = n % kUnits;
      ok = n < kUnits || wait(&ring.empty[at], ((n / kUnits) - 1) & 1);
      if (ok && lane == 0) {
        ring.unit[at] = u;
        ptx::mbar_arrive(&ring.full[at]);
      }
      // the next is taken late, so that no CTA sits on units that another could begin
      if (more && ok) ok = wait(&ring.ask, n & 1);
      ++n;
    }
    if (!more || !ok) break;
    if (lane == 0) {
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive_expect_tx(&ring.clc, 16);
      ptx::clc_try_cancel(ring.response, &ring.clc);
    }
    if (!wait(&ring.clc, asked++ & 1)) {
      ok = false;
      break;
    }
    block = ptx::clc_block(ring.response);
    __syncwarp();
  }
}
// The next unit, for the warps that follow; false: none, or a wait gave up.
__device__ __forceinline__ bool next_unit(UnitRing& ring, const Waiter& wait, int lane, uint32_t& n,
                                          Unit& u) {
  const uint32_t at = n % kUnits;
  if (!wait(&ring.full[at], (n / kUnits) & 1)) return false;
  u = ring.unit[at];
  __syncwarp();  // every lane has read it
  if (lane == 0) ptx::mbar_arrive(&ring.empty[at]);
  ++n;
  return __shfl_sync(0xffffffffu, u.place, 0) >= 0;
}
// Barrier of `threads` threads with the conjunction of their answers.
__device__ __forceinline__ bool group_and(int id, int threads, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %3, 0;\n\t"
      "barrier.cta.red.and.pred p, %1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
decay_tc_kernel(const __grid_constant__ Maps maps, const DecayParams p, int seg, const float* added) {
  using M = Out<D>;
  using T = Tm<D>;
  constexpr int NQ = D / 32;  // warps that hold the accumulators' rows
  extern __shared__ __align__(1024) uint8_t smem[];
  OutSmall& sm = *reinterpret_cast<OutSmall*>(smem + M::SMALL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&sm.full[i], 2);
      ptx::mbar_init(&sm.empty[i], 4 + 5 * NQ);
    }
    for (int i = 0; i < kData; ++i) {
      ptx::mbar_init(&sm.data_full[i], 1);
      ptx::mbar_init(&sm.data_empty[i], 1 + 2 * NQ);
    }
    for (int i = 0; i < kUnits; ++i) {
      ptx::mbar_init(&sm.units.full[i], 1);
      ptx::mbar_init(&sm.units.empty[i], 2);
    }
    ptx::mbar_init(&sm.units.clc, 1);
    ptx::mbar_init(&sm.units.ask, 1);
    ptx::mbar_init(&sm.sc_full, 1);
    ptx::mbar_init(&sm.p_full, 4);
    ptx::mbar_init(&sm.v_full, 2 * NQ);
    ptx::mbar_init(&sm.vt_full, 2 * NQ);
    ptx::mbar_init(&sm.u_empty, 2 * NQ);
    ptx::mbar_init(&sm.hi_full, 2 * NQ);
    ptx::mbar_init(&sm.kv_done, 1);
    ptx::mbar_init(&sm.sq_done, 1);
    ptx::mbar_init(&sm.o_full, 1);
    ptx::mbar_init(&sm.o_empty, NQ);
    ptx::mbar_init(&sm.drain, 1);
    ptx::fence_mbar_init();
    sm.abort = 0;
  }
  if (warp == 25) {
    ptx::tmem_alloc(&sm.tmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
  const uint32_t base = ptx::smem_u32(smem);
  const Waiter wait{&sm.abort};
  auto arrive = [&](uint64_t* bar) {  // of a warp, after all its lanes
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
  };
  // The next chunk n, for P's warps; false: none, or a wait gave up.
  auto take = [&](int n, Chunk& c) {
    if (!wait(&sm.full[n % kStages], (n / kStages) & 1)) return false;
    c = sm.chunk[n % kStages];
    return __shfl_sync(0xffffffffu, c.kind, 0) != kStop;
  };

  // registers of the seven warpgroups: 64 + 96 + 96 + 64 + 64 + 64 + 56 = 7 x 72
  if (warp >= 4 && warp < 12) {
    ptx::regs_take<96>();
    // ------------------------------------------------------------------ the state
    const int w = warp & 3, half = (warp - 4) >> 2;  // 32 value channels, half of the key channels
    if (w < NQ) {
      const uint32_t lanes = (uint32_t)(w * 32) << 16;
      const uint32_t t_u = tmem + lanes + T::U + half * (D / 2);
      const uint32_t t_hi = tmem + lanes + T::HI + half * (D / 4);
      // the row of the low part: blocks of 64 key channels, 128-byte swizzle
      const uint32_t row = w * 32 + lane, lo = base + M::LO + row * 128 + (D == 128 ? half * 16384 : 0);
      const uint32_t lo0 = D == 128 ? 0 : half * 4;
      const int at = half * (D / 2) * D + w * 32 + lane;  // of the state's matrix
      float* exit_state = nullptr;
      Chunk c;
      ptx::f32x2 st[D / 4];
      asm volatile("griddepcontrol.wait;" ::: "memory");  // the scan before this kernel, if any
#pragma unroll 1
      for (int n = 0;; ++n) {
        const int s = n % kStages;
        if (!wait(&sm.full[s], (n / kStages) & 1)) break;
        c = sm.chunk[s];
        const int kind = __shfl_sync(0xffffffffu, c.kind, 0);
        if (kind & (kFirst | kStop)) {  // the unit before has ended
          if (exit_state) {
#pragma unroll
            for (int i = 0; i < D / 4; ++i) {
              float x, y;
              ptx::unpack2(st[i], x, y);
              exit_state[at + (2 * i) * D] = x;
              exit_state[at + (2 * i + 1) * D] = y;
            }
          }
          if (kind == kStop) break;
#pragma unroll
          for (int i = 0; i < D / 4; ++i) {
            float x = 0.0f, y = 0.0f;
            if (c.entry) {  // (the scan may write it while this kernel runs: no read-only loads)
              x = __ldcg(c.entry + at + (2 * i) * D);
              y = __ldcg(c.entry + at + (2 * i + 1) * D);
            }
            st[i] = ptx::pack2(x, y);
          }
        }
        exit_state = c.exit;
        if (n > 0 && !wait(&sm.sq_done, (n - 1) & 1)) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int b = 0; b < D / 4; b += 8) {
          uint32_t hi[8], l[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) split2(st[b + i], hi[i], l[i]);
          ptx::tmem_st8(t_hi + b, hi);
#pragma unroll
          for (int i = 0; i < 8; i += 4)
            st_shared(lo + ((((b + i) / 4 + lo0) ^ (row & 7)) << 4),
                      make_uint4(l[i], l[i + 1], l[i + 2], l[i + 3]));
        }
        ptx::fence_proxy_async_smem();
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        arrive(&sm.hi_full);
        const float a = sm.total[s];
        const ptx::f32x2 aa = ptx::pack2(a, a);
        if (!wait(&sm.kv_done, n & 1)) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int b = 0; b < D / 4; b += 8) {
          uint32_t f[16];
          ptx::tmem_ld16_nowait(t_u + 2 * b, f);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(f[i]));
#pragma unroll
          for (int i = 0; i < 8; ++i)
            st[b + i] = ptx::fma2(st[b + i], aa, ptx::pack2(__uint_as_float(f[2 * i]),
                                                            __uint_as_float(f[2 * i + 1])));
        }
        ptx::tc_fence_before();
        arrive(&sm.u_empty);
        if (lane == 0) ptx::mbar_arrive(&sm.empty[s]);
      }
    }
  } else if (warp >= 24) {
    ptx::regs_give<56>();
    if (warp == 24) {
      // ------------------------------------------------------------------ loads
      int n = 0;
      uint32_t unit = 0;
      Unit u;
      bool ok = true;
      auto room = [&](int n) {
        return (n < kStages || wait(&sm.empty[n % kStages], ((n / kStages) - 1) & 1)) &&
               (n < kData || wait(&sm.data_empty[n % kData], ((n / kData) - 1) & 1));
      };
#pragma unroll 1
      while (ok && next_unit(sm.units, wait, lane, unit, u)) {
        const int hk = u.head / (p.H / p.Hk);
        if (lane == 0 && u.entry) ptx::bulk_prefetch_l2(u.entry, D * D * 4);
        Chunk c;
        c.entry = u.entry;
        c.head = u.head;
        int t = u.lo;
#pragma unroll 1
        do {
          const int s = n % kStages;
          c.t0 = t;
          c.tokens = (short)(u.hi - t < kC ? u.hi - t : kC);
          c.kind = (short)((t == u.lo ? kFirst : 0) | (u.hi - t <= kC ? kLast : 0));
          c.exit = c.kind & kLast ? u.exit : nullptr;
          if ((c.kind & kLast) && lane == 0) ptx::mbar_arrive(&sm.units.ask);
          if (!(ok = room(n))) break;
          if (lane == 0) {
            sm.chunk[s] = c;
            ptx::mbar_arrive(&sm.full[s]);
            uint64_t* bar = &sm.data_full[n % kData];
            uint8_t* st = smem + n % kData * M::STAGE;
            if (c.tokens > 0) {
              ptx::mbar_arrive_expect_tx(bar, M::STAGE);
              load_tile<D>(st + M::K, &maps.k, bar, hk, t);
              load_tile<D>(st + M::Q, &maps.q, bar, hk, t);
              load_tile<D>(st + M::V, &maps.v, bar, u.head, t);
            } else {  // an empty sequence: all rows are cleared, the state passes through
              ptx::mbar_arrive(bar);
            }
          }
          ++n;
          t += kC;
        } while (t < u.hi);
      }
      if (ok && room(n) && lane == 0) {
        sm.chunk[n % kStages].kind = kStop;
        ptx::mbar_arrive(&sm.full[n % kStages]);
        ptx::mbar_arrive(&sm.data_full[n % kData]);
      }
      if (*(volatile int*)&sm.abort) {  // the loads in flight land before the CTA leaves
        __nanosleep(1000000);
        __syncwarp();
      }
    } else if (warp == 26) {
      // ------------------------------------------------------------------ sums of the decays
      int n = 0;
      uint32_t unit = 0;
      Unit u;
      bool ok = true;
#pragma unroll 1
      while (ok && next_unit(sm.units, wait, lane, unit, u)) {
        const DecayRing<kAhead> ring{sm.g, p.g + u.head, p.gs, lane};
#pragma unroll 1
        for (int i = 0; i < kAhead; ++i) ring.ask(i, u.lo + i * kC, u.hi);
        int i = 0;
#pragma unroll 1
        do {
          const int s = n % kStages;
          ring.wait<1>();
          const float2 g = ring.get(i);
          const bool nan = __any_sync(0xffffffffu, g.x != g.x || g.y != g.y);
          const float2 second = log_pair(g.y);
          float2 b = log_scan(log_add(log_pair(g.x), second), lane), a = log_sub(b, second);
          ring.ask(i + kAhead, u.lo + (i + kAhead) * kC, u.hi);
          if (nan) a.x = b.x = nan_f();  // a NaN decay spoils its chunk
          if (n >= kStages && !(ok = wait(&sm.empty[s], ((n / kStages) - 1) & 1))) break;
          *reinterpret_cast<float2*>(&sm.ghi[s][2 * lane]) = make_float2(a.x, b.x);
          *reinterpret_cast<float2*>(&sm.glo[s][2 * lane]) = make_float2(a.y, b.y);
          const float ea = ptx::ex2_approx(a.x + a.y), eb = ptx::ex2_approx(b.x + b.y);
          const float2 all = make_float2(__shfl_sync(0xffffffffu, b.x, 31),
                                         __shfl_sync(0xffffffffu, b.y, 31));
          *reinterpret_cast<float2*>(&sm.in[s][2 * lane]) = make_float2(ea, eb);
          *reinterpret_cast<float2*>(&sm.out[s][2 * lane]) =
              make_float2(ptx::ex2_approx((all.x - a.x) + (all.y - a.y)),
                          ptx::ex2_approx((all.x - b.x) + (all.y - b.y)));
          if (lane == 31) sm.total[s] = eb;
          arrive(&sm.full[s]);
          ++n;
          ++i;
        } while (u.lo + i * kC < u.hi);
      }
      const int s = n % kStages;
      if (ok && n >= kStages) ok = wait(&sm.empty[s], ((n / kStages) - 1) & 1);
      if (ok) arrive(&sm.full[s]);
      ptx::cp_async_wait<0>();
    } else if (warp == 27) {
      // ------------------------------------------------------------------ the units
      schedule(sm.units, wait, lane, [&](int block, Unit& u) {
        const int h = block % p.H;
        Segment x;
        if (!find_segment<false>(p, seg, block / p.H, lane, lane == 0 && h == 0, x)) return false;
        u.lo = (int)x.lo;
        u.hi = (int)x.hi;
        u.head = h;
        u.place = 0;
        u.entry = !x.first ? added + ((int64_t)(x.place - 1) * p.H + h) * (D * D)
                  : p.init ? p.init + ((int64_t)x.seq * p.H + h) * (D * D) : nullptr;
        u.exit = x.last && p.final_state ? p.final_state + ((int64_t)x.seq * p.H + h) * (D * D)
                                         : nullptr;
        return x.hi > x.lo || u.exit != nullptr;
      });
    } else {
      // ------------------------------------------------------------------ products
      // (loops rolled: unrolled, this role's code alone did not fit the instruction cache)
      const uint32_t id_o = ptx::idesc_make(ptx::kFmtBF16, 128, kC, false, false);
      const uint32_t id_sc = ptx::idesc_make(ptx::kFmtBF16, kC, kC, false, false);
#pragma unroll 1
      for (int n = 0;; ++n) {
        const uint32_t st = base + n % kData * M::STAGE, ph = n & 1;
        // (V' says that the chunk itself is there, or that there is none)
        if (n == 0 ? !wait(&sm.v_full, 0) : !wait.both(&sm.u_empty, ph ^ 1, &sm.v_full, ph)) break;
        if (__shfl_sync(0xffffffffu, (int)sm.chunk[n % kStages].kind, 0) == kStop) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint64_t a = ptx::sdesc_sw128(st + M::Q, 16, 1024);
          const uint64_t b = ptx::sdesc_sw128(st + M::K, 16, 1024);
#pragma unroll 1
          for (uint32_t i = 0; i < D / 64; ++i)
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
              ptx::mma_f16(tmem + T::SC, ptx::desc_add(a, i * 8192 + j * 32),
                           ptx::desc_add(b, i * 8192 + j * 32), id_sc, i + j > 0);
          ptx::mma_commit(&sm.sc_full);
          issue_kv<D>(tmem + T::U, tmem + T::VP, st + M::K);
          ptx::mma_commit(&sm.kv_done);
        }
        __syncwarp();
        if (n == 0 ? !wait(&sm.hi_full, 0) : !wait.both(&sm.hi_full, ph, &sm.o_empty, ph ^ 1)) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint64_t b = ptx::sdesc_sw128(st + M::Q, 16, 1024);
          const uint64_t lo = ptx::sdesc_sw128(base + M::LO, 16, 1024);
#pragma unroll 1
          for (uint32_t i = 0; i < D / 64; ++i)
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
              ptx::mma_f16_ts(tmem + T::OI, tmem + T::HI + i * 32 + j * 8,
                              ptx::desc_add(b, i * 8192 + j * 32), id_o, i + j > 0);
#pragma unroll 1
          for (uint32_t i = 0; i < D / 64; ++i)
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
              ptx::mma_f16(tmem + T::OI, ptx::desc_add(lo, i * 16384 + j * 32),
                           ptx::desc_add(b, i * 8192 + j * 32), id_o, 1);
          ptx::mma_commit(&sm.sq_done);
          ptx::mma_commit(&sm.data_empty[n % kData]);
        }
        __syncwarp();
        if (!wait.both(&sm.p_full, ph, &sm.vt_full, ph)) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint64_t b = ptx::sdesc_sw128(base + M::P, 16, 1024);
#pragma unroll 1
          for (uint32_t part = 0; part < 2; ++part)
#pragma unroll
            for (uint32_t i = 0; i < kC / 16; ++i)
              ptx::mma_f16_ts(tmem + T::OA, tmem + T::VT + i * 8,
                              ptx::desc_add(b, part * 8192 + i * 32), id_o, part + i > 0);
          ptx::mma_commit(&sm.o_full);
        }
        __syncwarp();
      }
      if (__any_sync(0xffffffffu, *(volatile int*)&sm.abort)) {  // the products in flight end first
        if (ptx::elect_one()) ptx::mma_commit(&sm.drain);
        __syncwarp();
        ptx::mbar_wait_tries(&sm.drain, 0, kTries);
        __syncwarp();
      }
    }
  } else if (warp >= 16) {
    ptx::regs_give<64>();
    // ------------------------------------------------------------------ V and V', transposed
    const int w = warp & 3, tok = ((warp - 16) >> 2) * 32;  // 32 channels, half of the tokens
    if (w < NQ) {
      const uint32_t lanes = (uint32_t)(w * 32) << 16;
#pragma unroll 1
      for (int n = 0;; ++n) {
        const int s = n % kStages;
        if (!wait.both(&sm.full[s], (n / kStages) & 1, &sm.data_full[n % kData], (n / kData) & 1)) break;
        if (__shfl_sync(0xffffffffu, (int)sm.chunk[s].kind, 0) == kStop) {
          // which the products learn from this barrier, once they have left its last phase
          if (n == 0 || wait(&sm.kv_done, (n - 1) & 1)) arrive(&sm.v_full);
          break;
        }
        const int m = sm.chunk[s].tokens;
        const uint32_t st = base + n % kData * M::STAGE;
        ptx::f32x2 weight[4];
        uint32_t raw[2][8];
        load_vt(st + M::V, w * 32, tok, lane, raw[0]);
        load_vt(st + M::V, w * 32 + 16, tok, lane, raw[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = *reinterpret_cast<const float2*>(&sm.out[s][tok + i * 8 + 2 * (lane & 3)]);
          weight[i] = ptx::pack2(f.x, f.y);
        }
        if (m < kC) {  // rows of the next sequence, whatever they hold: zeros, in K too
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = tok + i * 8 + 2 * (lane & 3);
            const uint32_t keep = (t < m ? 0xffffu : 0u) | (t + 1 < m ? 0xffff0000u : 0u);
            raw[0][2 * i] &= keep;
            raw[0][2 * i + 1] &= keep;
            raw[1][2 * i] &= keep;
            raw[1][2 * i + 1] &= keep;
          }
          for (int i = (warp - 16) / 4 * (NQ * 32) + w * 32 + lane; i < kC * D / 8;
               i += 2 * NQ * 32)
            if (i / (D / 8) >= m) st_shared(st + M::K + tile_at<D>(i), make_uint4(0u, 0u, 0u, 0u));
          ptx::fence_proxy_async_smem();
        }
        arrive(&sm.empty[s]);
        if (lane == 0) ptx::mbar_arrive(&sm.data_empty[n % kData]);
        if (n > 0 && !wait(&sm.kv_done, (n - 1) & 1)) break;
        ptx::tc_fence_after();
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
          uint32_t part[3][8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t x[3];
            weigh3(b ? raw[1][i] : raw[0][i], weight[i >> 1], x);
            part[0][i] = x[0];
            part[1][i] = x[1];
            part[2][i] = x[2];
          }
#pragma unroll
          for (int j = 0; j < 3; ++j)
            ptx::tmem_st_rows16_nowait(
                tmem + lanes + ((uint32_t)(b * 16) << 16) + T::VP + j * 32 + tok / 2, part[j]);
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        arrive(&sm.v_full);
        if (n > 0 && !wait(&sm.o_full, (n - 1) & 1)) break;
        ptx::tc_fence_after();
        ptx::tmem_st_rows16_nowait(tmem + lanes + T::VT + tok / 2, raw[0]);
        ptx::tmem_st_rows16_nowait(tmem + lanes + (16u << 16) + T::VT + tok / 2, raw[1]);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        arrive(&sm.vt_full);
      }
    }
  } else if (warp >= 12) {
    ptx::regs_give<64>();
    // ------------------------------------------------------------------ outputs
    const int w = warp - 12;
    if (w < NQ) {
      const int tid = w * 32 + lane;
      const uint32_t stage = base + M::O + (w >> 1) * 8192;  // its block of 64 channels
      const uint32_t t_o = tmem + ((uint32_t)(w * 32) << 16);
      const ptx::f32x2 scale = ptx::pack2(p.scale, p.scale);
      Chunk c;
#pragma unroll 1
      for (int n = 0;; ++n) {
        const int s = n % kStages;
        bool ok = wait(&sm.full[s], (n / kStages) & 1);
        if (ok) {
          c = sm.chunk[s];
          ok = __shfl_sync(0xffffffffu, c.kind, 0) != kStop && wait(&sm.o_full, n & 1);
        }
        if (tid == 0) ptx::bulk_wait_read0();  // the last chunk's rows have left
        ok = group_and(1, NQ * 32, ok);
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll 1
        for (int tok = 0; tok < kC; tok += 32) {
          ptx::f32x2 ee[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = *reinterpret_cast<const float2*>(&sm.in[s][tok + i * 8 + 2 * (lane & 3)]);
            ee[i] = ptx::pack2(f.x, f.y);
          }
#pragma unroll 1
          for (uint32_t ch0 = 0; ch0 < 32; ch0 += 16) {  // 16 channels x 32 tokens
            uint32_t x[16], y[16];
            ptx::tmem_ld_frag32_nowait(t_o + (ch0 << 16) + T::OI + tok, x);
            ptx::tmem_ld_frag32_nowait(t_o + (ch0 << 16) + T::OA + tok, y);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(x[i]), "+r"(y[i]));
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const ptx::f32x2 inter =
                  ptx::pack2(__uint_as_float(x[j]), __uint_as_float(x[j + 1]));
              const ptx::f32x2 intra =
                  ptx::pack2(__uint_as_float(y[j]), __uint_as_float(y[j + 1]));
              float y0, y1;
              ptx::unpack2(ptx::mul2(ptx::fma2(ee[j >> 2], inter, intra), scale), y0, y1);
              o[j >> 1] = pack_bf16(y0, y1);
            }
            // matrices (channels 0-7, 8-15) x (two groups of 8 tokens): row = token
            const int ch = ((w & 1) * 32 + (int)ch0) / 8 + ((lane >> 3) & 1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int t = tok + i * 16 + (lane >> 4) * 8 + (lane & 7);
              ptx::st_matrix4_trans(stage + t * 128 + ((ch ^ (t & 7)) << 4), o[4 * i], o[4 * i + 1],
                                    o[4 * i + 2], o[4 * i + 3]);
            }
          }
        }
        ptx::tc_fence_before();
        arrive(&sm.o_empty);
        if (lane == 0) ptx::mbar_arrive(&sm.empty[s]);
        ptx::fence_proxy_async_smem();
        group_and(1, NQ * 32, true);
        if (c.tokens >= kC) {
          if (tid == 0) {
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
              ptx::tma_store_2d(&maps.o, smem + M::O + i * 8192, c.head * D + i * 64, c.t0);
            ptx::bulk_commit();
          }
        } else {  // the rows after the segment belong to another one
          for (int i = tid; i < c.tokens * (D / 8); i += NQ * 32) {
            const int t = c.t0 + i / (D / 8);
            *reinterpret_cast<uint4*>((__nv_bfloat16*)p.o + ((int64_t)t * p.H + c.head) * D +
                                      i % (D / 8) * 8) = ld_shared(base + M::O + tile_at<D>(i));
          }
        }
      }
      if (tid == 0) ptx::bulk_wait0();
    }
  } else {
    ptx::regs_give<64>();
    // ------------------------------------------------------------------ P (warps 0 .. 3)
    // The scores are a product with M = 64: rows 16 w .. 16 w + 15 are in the first lanes of
    // quarter w. A lane has two columns of every eight of rows g and g + 8.
    const int w = warp, g = lane >> 2, t4 = lane & 3;
    const uint32_t t_sc = tmem + ((uint32_t)(w * 32) << 16) + T::SC;
    // columns that the rows never reach stay zeros
    for (int i = lane; i < 2 * 16 * 4; i += 32) {
      const int row = w * 16 + (i >> 2 & 15);
      st_shared(base + M::P + (i >> 6) * 8192 + row * 128 + (((4 + (i & 3)) ^ (row & 7)) << 4),
                make_uint4(0u, 0u, 0u, 0u));
    }
    __syncwarp();
    const ptx::f32x2 minus = ptx::pack2(-1.0f, -1.0f);
    Chunk c;
#pragma unroll 1
    for (int n = 0; take(n, c); ++n) {
      const int s = n % kStages;
      if (!wait(&sm.sc_full, n & 1)) break;  // (the last P has been read)
      ptx::tc_fence_after();
      const int row = w * 16 + g;
      const ptx::f32x2 gh[2] = {ptx::pack2(sm.ghi[s][row], sm.ghi[s][row]),
                                ptx::pack2(sm.ghi[s][row + 8], sm.ghi[s][row + 8])};
      const ptx::f32x2 gl[2] = {ptx::pack2(sm.glo[s][row], sm.glo[s][row]),
                                ptx::pack2(sm.glo[s][row + 8], sm.glo[s][row + 8])};
#pragma unroll 1
      for (int c0 = 0; c0 <= w * 16; c0 += 32) {
        uint32_t r[16];
        ptx::tmem_ld_frag32_nowait(t_sc + c0, r);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(r[j]));
        uint32_t o[2][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = c0 + 8 * i + 2 * t4;
          const float2 h2 = *reinterpret_cast<const float2*>(&sm.ghi[s][col]);
          const float2 l2 = *reinterpret_cast<const float2*>(&sm.glo[s][col]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float d0, d1, y0, y1;
            ptx::unpack2(ptx::add2(ptx::fma2(ptx::pack2(h2.x, h2.y), minus, gh[e]),
                                   ptx::fma2(ptx::pack2(l2.x, l2.y), minus, gl[e])),
                         d0, d1);
            ptx::unpack2(ptx::mul2(ptx::pack2(ptx::ex2_approx(d0), ptx::ex2_approx(d1)),
                                   ptx::pack2(__uint_as_float(r[4 * i + 2 * e]),
                                              __uint_as_float(r[4 * i + 2 * e + 1]))),
                         y0, y1);
            y0 = col <= row + 8 * e ? y0 : 0.0f;
            y1 = col < row + 8 * e ? y1 : 0.0f;
            split2(ptx::pack2(y0, y1), o[0][2 * i + e], o[1][2 * i + e]);
          }
        }
        // matrices (rows 0-7, 8-15) x (two groups of 8 columns)
        const int at = w * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int blk = c0 / 8 + 2 * i + (lane >> 4);
            const uint32_t* x = &o[part][4 * i];
            ptx::st_matrix4(base + M::P + part * 8192 + at * 128 + ((blk ^ (at & 7)) << 4), x[0], x[1],
                            x[2], x[3]);
          }
      }
      ptx::tc_fence_before();  // the scores are read, too
      ptx::fence_proxy_async_smem();
      arrive(&sm.p_full);
      if (lane == 0) ptx::mbar_arrive(&sm.empty[s]);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && sm.abort && p.status) atomicOr(p.status, KDA_STATUS_TIMEOUT);
  if (warp == 25) ptx::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- what a segment adds
//
// sum_s e^(sum of g after s) k_s v_s^T over a whole segment, from its last chunk to its first: the
// decays behind a chunk are known when it is reached, so the accumulator is never rescaled. And the
// rows that the outputs' kernel reads first are the ones that this one read last.
template <int D>
struct Add {
  static constexpr int TILE = kC * D * 2, STAGE = 2 * TILE, STAGES = D == 128 ? 6 : 8;
  static constexpr int V = 0, K = TILE;
  static constexpr int SMALL = STAGES * STAGE;
};
struct AddSmall {
  UnitRing units;
  uint64_t full[8], empty[8];
  uint64_t v_full[2], v_empty[2], acc_full[2], acc_empty[2], drain;
  float w[8][kC];
  float g[kAddAhead][kC];
  float* out[8];  // of a chunk's unit
  int kind[8];
  uint32_t tmem;
  int abort;
};
constexpr int kAddThreads = 896;  // 16 + 8 + 4 warps

template <int D>
__global__ void __launch_bounds__(kAddThreads, 1)
decay_add_kernel(const __grid_constant__ Maps maps, const DecayParams p, int seg, float* added,
                 float* added_log) {
  using M = Add<D>;
  constexpr int NQ = D / 32, kStages = M::STAGES;
  constexpr int VP = 256;  // TMEM: two chunks' sums, then two sets of three parts of V'
  extern __shared__ __align__(1024) uint8_t smem[];
  AddSmall& sm = *reinterpret_cast<AddSmall*>(smem + M::SMALL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int N = seg / kC;  // segments that are not their sequence's last are whole

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&sm.full[i], 2);
      ptx::mbar_init(&sm.empty[i], 1 + 4 * NQ + 2 * NQ);
    }
    for (int i = 0; i < kUnits; ++i) {
      ptx::mbar_init(&sm.units.full[i], 1);
      ptx::mbar_init(&sm.units.empty[i], 2);
    }
    ptx::mbar_init(&sm.units.clc, 1);
    ptx::mbar_init(&sm.units.ask, 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sm.v_full[i], 2 * NQ);
      ptx::mbar_init(&sm.v_empty[i], 1);
      ptx::mbar_init(&sm.acc_full[i], 1);
      ptx::mbar_init(&sm.acc_empty[i], 2 * NQ);
    }
    ptx::mbar_init(&sm.drain, 1);
    ptx::fence_mbar_init();
    sm.abort = 0;
  }
  if (warp == 25) {
    ptx::tmem_alloc(&sm.tmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
  const uint32_t base = ptx::smem_u32(smem);
  const Waiter wait{&sm.abort};
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
  };
  auto take = [&](int n, int& kind) {
    if (!wait(&sm.full[n % kStages], (n / kStages) & 1)) return false;
    kind = __shfl_sync(0xffffffffu, sm.kind[n % kStages], 0);
    return kind != kStop;
  };

  // registers of the seven warpgroups: 4 x 72 (as launched) + 2 x 88 + 40 = 7 x 72
  if (warp < 16) {
    // ------------------------------------------------------------------ V'
    // two sets of 8 warps take chunks in turn: 32 channels, half of the tokens each
    const int w = warp & 3, tok = ((warp >> 2) & 1) * 32, b = warp >> 3;
    if (w < NQ) {
      const uint32_t lanes = (uint32_t)(w * 32) << 16;
#pragma unroll 1
      for (int n = 0;; ++n) {
        const int s = n % kStages;
        if (!wait(&sm.full[s], (n / kStages) & 1)) break;
        const bool stop = __shfl_sync(0xffffffffu, sm.kind[s], 0) == kStop;
        if ((n & 1) != b) {  // (every warp sees every phase of a stage: parities do not run ahead)
          if (stop) break;
          arrive(&sm.empty[s]);
          continue;
        }
        if (stop) {  // which the products learn from this barrier, once they have left its last phase
          if (n < 2 || wait(&sm.v_empty[b], ((n >> 1) - 1) & 1)) arrive(&sm.v_full[b]);
          break;
        }
        const uint32_t st = base + s * M::STAGE;
        uint32_t raw[2][8];
        load_vt(st + M::V, w * 32, tok, lane, raw[0]);
        load_vt(st + M::V, w * 32 + 16, tok, lane, raw[1]);
        ptx::f32x2 weight[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = *reinterpret_cast<const float2*>(&sm.w[s][tok + i * 8 + 2 * (lane & 3)]);
          weight[i] = ptx::pack2(f.x, f.y);
        }
        arrive(&sm.empty[s]);
        // all of V' before its room is free
        uint32_t part[2][3][8];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t x[3];
            weigh3(raw[c][i], weight[i >> 1], x);
            part[c][0][i] = x[0];
            part[c][1][i] = x[1];
            part[c][2][i] = x[2];
          }
        if (n >= 2 && !wait(&sm.v_empty[b], ((n >> 1) - 1) & 1)) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 3; ++j)
            ptx::tmem_st_rows16_nowait(
                tmem + lanes + ((uint32_t)(c * 16) << 16) + VP + b * 96 + j * 32 + tok / 2, part[c][j]);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        arrive(&sm.v_full[b]);
      }
    }
  } else if (warp < 24) {
    ptx::regs_take<88>();
    // ------------------------------------------------------------------ sums over the chunks
    const int w = warp & 3, half = (warp - 16) >> 2;  // 32 value channels, half of the key channels
    if (w < NQ) {
      const int at = half * (D / 2) * D + w * 32 + lane;
      const uint32_t t_u = tmem + ((uint32_t)(w * 32) << 16) + half * (D / 2);
      ptx::f32x2 sum[D / 4];
      int kind;
#pragma unroll 1
      for (int n = 0; take(n, kind); ++n) {
        const int s = n % kStages, b = n & 1;
        float* out = sm.out[s] + at;
        arrive(&sm.empty[s]);
        if (kind & kFirst) {
#pragma unroll
          for (int i = 0; i < D / 4; ++i) sum[i] = ptx::pack2(0.0f, 0.0f);
        }
        if (!wait(&sm.acc_full[b], (n >> 1) & 1)) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int c = 0; c < D / 4; c += 8) {
          uint32_t f[16];
          ptx::tmem_ld16_nowait(t_u + b * 128 + 2 * c, f);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(f[i]));
#pragma unroll
          for (int i = 0; i < 8; ++i)
            sum[c + i] = ptx::add2(sum[c + i], ptx::pack2(__uint_as_float(f[2 * i]),
                                                          __uint_as_float(f[2 * i + 1])));
        }
        ptx::tc_fence_before();
        arrive(&sm.acc_empty[b]);
        if (kind & kLast) {
#pragma unroll
          for (int i = 0; i < D / 4; ++i) {
            float x, y;
            ptx::unpack2(sum[i], x, y);
            out[(2 * i) * D] = x;
            out[(2 * i + 1) * D] = y;
          }
        }
      }
    }
  } else {
    ptx::regs_give<40>();
    if (warp == 24) {
    // ------------------------------------------------------------------ loads
    int n = 0;
    uint32_t unit = 0;
    Unit u;
    bool ok = true;
#pragma unroll 1
    while (ok && next_unit(sm.units, wait, lane, unit, u)) {
      const int hk = u.head / (p.H / p.Hk);
#pragma unroll 1
      for (int i = 0; i < N; ++i, ++n) {
        const int s = n % kStages, t = u.lo + (N - 1 - i) * kC;
        if (i == N - 1 && lane == 0) ptx::mbar_arrive(&sm.units.ask);
        if (n >= kStages && !(ok = wait(&sm.empty[s], ((n / kStages) - 1) & 1))) break;
        if (lane == 0) {
          uint8_t* st = smem + s * M::STAGE;
          sm.kind[s] = (i == 0 ? kFirst : 0) | (i == N - 1 ? kLast : 0);
          sm.out[s] = u.exit;
          ptx::mbar_arrive_expect_tx(&sm.full[s], M::STAGE);
          load_tile<D>(st + M::V, &maps.v, &sm.full[s], u.head, t);
          load_tile<D>(st + M::K, &maps.k, &sm.full[s], hk, t);
        }
      }
    }
    const int s = n % kStages;
    if (ok && n >= kStages) ok = wait(&sm.empty[s], ((n / kStages) - 1) & 1);
    if (ok && lane == 0) {
      sm.kind[s] = kStop;
      ptx::mbar_arrive(&sm.full[s]);
    }
    if (*(volatile int*)&sm.abort) {  // the loads in flight land before the CTA leaves
      __nanosleep(1000000);
      __syncwarp();
    }
    } else if (warp == 26) {
    // ------------------------------------------------------------------ sums of the decays
    int n = 0;
    uint32_t unit = 0;
    Unit u;
    bool ok = true;
#pragma unroll 1
    while (ok && next_unit(sm.units, wait, lane, unit, u)) {
      const DecayRing<kAddAhead> ring{sm.g, p.g + u.head, p.gs, lane};
      auto ask = [&](int i) {
        const int t = i < N ? u.lo + (N - 1 - i) * kC : 0;
        ring.ask(i, t, i < N ? t + kC : 0);
      };
#pragma unroll 1
      for (int i = 0; i < kAddAhead; ++i) ask(i);
      float2 later = make_float2(0.0f, 0.0f);
      // two chunks side by side: one's sums alone took as long as everything else of a chunk
#pragma unroll 1
      for (int i = 0; i < N; i += 2) {
        float2 second[2], sum[2], all[2];
        bool nan[2];
        ring.wait<2>();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float2 g = ring.get(i + c);
          nan[c] = __any_sync(0xffffffffu, g.x != g.x || g.y != g.y);
          second[c] = log_pair(g.y);
          sum[c] = log_add(log_pair(g.x), second[c]);
        }
        log_scan(sum, lane);
        ask(i + kAddAhead);
        ask(i + 1 + kAddAhead);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          all[c] = make_float2(__shfl_sync(0xffffffffu, sum[c].x, 31),
                               __shfl_sync(0xffffffffu, sum[c].y, 31));
#pragma unroll
        for (int c = 0; c < 2 && i + c < N && ok; ++c, ++n) {
          const int s = n % kStages;
          const float2 upto = log_add(later, all[c]), b = log_sub(upto, sum[c]),
                       a = log_add(b, second[c]);
          float wa = ptx::ex2_approx(a.x + a.y), wb = ptx::ex2_approx(b.x + b.y);
          if (nan[c]) wa = wb = nan_f();
          later = upto;
          if (n >= kStages && !(ok = wait(&sm.empty[s], ((n / kStages) - 1) & 1))) break;
          *reinterpret_cast<float2*>(&sm.w[s][2 * lane]) = make_float2(wa, wb);
          arrive(&sm.full[s]);
        }
        if (!ok) break;
      }
      if (lane == 0) added_log[u.place] = later.x;
    }
    const int s = n % kStages;
    if (ok && n >= kStages) ok = wait(&sm.empty[s], ((n / kStages) - 1) & 1);
    if (ok) arrive(&sm.full[s]);
    ptx::cp_async_wait<0>();
    } else if (warp == 27) {
    // ------------------------------------------------------------------ the units
    schedule(sm.units, wait, lane, [&](int block, Unit& u) {
      Segment x;
      if (!find_segment<true>(p, seg, block / p.H, lane, false, x)) return false;
      u.lo = (int)x.lo;
      u.hi = (int)x.hi;
      u.head = block % p.H;
      u.place = x.place * p.H + u.head;
      u.entry = nullptr;
      u.exit = added + (int64_t)u.place * (D * D);
      return true;
    });
    } else {
    // ------------------------------------------------------------------ products
    // (a look at a barrier takes some 300 cycles: V' says that the chunk itself is there too)
#pragma unroll 1
    for (int n = 0;; ++n) {
      const int s = n % kStages, b = n & 1;
      if (n < 2 ? !wait(&sm.v_full[b], 0)
                : !wait.both(&sm.v_full[b], (n >> 1) & 1, &sm.acc_empty[b], ((n >> 1) - 1) & 1))
        break;
      if (__shfl_sync(0xffffffffu, sm.kind[s], 0) == kStop) break;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        issue_kv<D>(tmem + b * 128, tmem + VP + b * 96, base + s * M::STAGE + M::K);
        ptx::mma_commit(&sm.v_empty[b]);
        ptx::mma_commit(&sm.empty[s]);
        ptx::mma_commit(&sm.acc_full[b]);
      }
      __syncwarp();
    }
    if (__any_sync(0xffffffffu, *(volatile int*)&sm.abort)) {
      if (ptx::elect_one()) ptx::mma_commit(&sm.drain);
      __syncwarp();
      ptx::mbar_wait_tries(&sm.drain, 0, kTries);
      __syncwarp();
    }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && sm.abort && p.status) atomicOr(p.status, KDA_STATUS_TIMEOUT);
  if (warp == 25) ptx::tmem_dealloc(tmem, 512);
}

template <int D>
kda_status launch_d(const DecayParams& p, int seg, float* added, float* added_log, cudaStream_t s) {
  Maps m;
  const uint64_t rows = p.total > 0 ? (uint64_t)p.total : 1;
  // (without tokens nothing is loaded: the maps are not used)
  if (p.total > 0 &&
      !(make_map_tokens(&m.q, p.q, (uint64_t)p.Hk * D, rows, (uint64_t)p.qs * 2, 64, kC) &&
        make_map_tokens(&m.k, p.k, (uint64_t)p.Hk * D, rows, (uint64_t)p.ks * 2, 64, kC) &&
        make_map_tokens(&m.v, p.v, (uint64_t)p.H * D, rows, (uint64_t)p.vs * 2, 64, kC) &&
        make_map_tokens(&m.o, p.o, (uint64_t)p.H * D, rows, (uint64_t)p.H * D * 2, 64, kC)))
    return set_error(KDA_ERR_CUDA, "kda_decay_prefill: cuTensorMapEncodeTiled failed");
  constexpr int out_bytes = Out<D>::SMALL + (int)sizeof(OutSmall);
  constexpr int add_bytes = Add<D>::SMALL + (int)sizeof(AddSmall);
  static_assert(out_bytes <= 232448 && add_bytes <= 232448, "shared memory");
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    cudaFuncSetAttribute(decay_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, out_bytes);
    cudaFuncSetAttribute(decay_add_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, add_bytes);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  const int slots = p.total / seg + p.n_seqs;
  if (p.total > seg) {
    const unsigned places = (unsigned)(p.total / seg * p.H);
    decay_add_kernel<D><<<places, kAddThreads, add_bytes, s>>>(m, p, seg, added, added_log);
    launch_decay_scan(p, D, seg, added, added_log, s);
    count_launches(1);
  }
  // behind a scan, its CTAs start while the scan's last ones run
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(slots * p.H));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = out_bytes;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.total > seg ? 1 : 0;
  cudaLaunchKernelEx(&cfg, decay_tc_kernel<D>, m, p, seg, (const float*)added);
  count_launches(1);
  return check_launch("kda_decay_prefill");
}

}  // namespace

namespace decay {

kda_status launch_tc(const DecayParams& p, int d, int seg, float* added, float* added_log,
                     cudaStream_t s) {
  if (!chunk_tc_available())
    return set_error(KDA_ERR_UNSUPPORTED,
                     "kda_decay_prefill: the CUDA driver does not provide cuTensorMapEncodeTiled, "
                     "which the tensor-core path needs");
  return d == 128 ? launch_d<128>(p, seg, added, added_log, s)
                  : launch_d<64>(p, seg, added, added_log, s);
}

}  // namespace decay
}  // namespace kda
