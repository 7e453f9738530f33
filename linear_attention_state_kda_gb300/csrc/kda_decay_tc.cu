// Linear attention with one decay per head on the tensor cores: prompts in bf16.
//
// Chunks of 64 tokens. With gamma the running sum of the log-decays in a chunk, Gamma its total and S
// the state before it (fp32, kept transposed in TMEM: lanes are value channels),
//     O^T = e^gamma_t * (S^T Q^T) + V^T P^T,   P_ts = [s <= t] e^(gamma_t - gamma_s) q_t . k_s
//     S'^T = e^Gamma S^T + V'^T K,             V'_s = e^(Gamma - gamma_s) v_s
// Every product is a tcgen05 bf16 product with fp32 sums. Operands that are not inputs are carried in
// several bf16 parts, so that a product is as exact as its user needs: S and P in two (16 bits, under
// the rounding of the bf16 outputs), V' in three (24 bits: states are fp32, and what a token adds to
// them stays for the rest of the sequence). The two sums of O have accumulators of their own and
// meet in fp32, so that Q needs no decayed copy.
//
// Roles of a CTA (one segment of one head, 16 warps): one warp loads (TMA) and sums the decays; one
// issues the products; 4 build V'; 2 turn q.k into P; 4 split and decay the state; 4 write outputs.
// Order of the products per chunk: q.k of the next chunk; V'^T K, whose result the next chunk's
// state waits for; then S^T Q^T and V^T P^T, which run while the state is split again.
#include "kda_decay.cuh"
#include "kda_fp8.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

using namespace decay;

constexpr int kC = 64;
constexpr int kStages = 3;
constexpr int kThreads = 512;
constexpr uint32_t kTries = 1u << 19;  // of a wait inside a CTA: 2 s

struct Maps {
  CUtensorMap q, k, v, o;
};

// Offsets in shared memory. Operand tiles are [64 tokens][64 channels] blocks of 8 KB (128-byte
// swizzle), D / 64 of them side by side. Products with M = 128 read the 64 rows or channels after
// a tile's own, into accumulator lanes that no one reads: the order Q, V, K keeps those reads inside
// the stage, and V' before P inside the operands.
template <int D>
struct Out {
  static constexpr int TILE = kC * D * 2, STAGE = 3 * TILE;
  static constexpr int Q = 0, V = TILE, K = 2 * TILE;
  static constexpr int VP = kStages * STAGE;      // three parts
  static constexpr int P = VP + 3 * TILE;         // two parts of 8 KB
  static constexpr int O = P + 2 * 8192;          // [64][D] bf16
  static constexpr int SMALL = O + TILE;
};
struct OutSmall {
  uint64_t full[kStages], empty[kStages];
  uint64_t sc_full[2], sc_empty[2];
  uint64_t p_full, v_full, st_full, kv_done, o_full, o_empty, drain;
  alignas(16) float2 gam[kStages][kC];  // running sums of log2 decays, as pairs
  float ein[kStages][kC];   // 2^gamma
  float2 total[kStages];
  uint32_t tmem;
  int abort;
};
// TMEM columns
template <int D>
struct Tm {
  static constexpr int S = 0, HI = D, LO = HI + D / 2, SC = LO + D / 2, OI = SC + 128, OA = OI + 64;
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
__device__ __forceinline__ float top(float x) {
  return __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two values in two bf16 parts: the first truncated, the rest rounded (2^-16 in all). An infinity or
// NaN stays one: its rest is NaN.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = tops(a, b);
  lo = pack_bf16(a - top(a), b - top(b));
}
// Eight values in three parts: 8 bits each, exact.
__device__ __forceinline__ void split3(const float* x, uint4& hi, uint4& mid, uint4& lo) {
  uint32_t h[4], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x[2 * i], b = x[2 * i + 1];
    h[i] = tops(a, b);
    const float ra = a - top(a), rb = b - top(b);
    m[i] = tops(ra, rb);
    l[i] = tops(ra - top(ra), rb - top(rb));
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  mid = make_uint4(m[0], m[1], m[2], m[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// D x 64 tile of a head's rows from token t0.
template <int D>
__device__ __forceinline__ void load_tile(void* dst, const CUtensorMap* m, uint64_t* bar, int head,
                                          int t0) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    ptx::tma_load_2d((uint8_t*)dst + i * 8192, m, bar, head * D + i * 64, t0);
}

// V'^T K of a chunk into the state: three parts of V' (MN-major), K (MN-major).
template <int D>
__device__ __forceinline__ void issue_kv(uint32_t tmem_s, uint32_t vp, uint32_t k, bool fresh) {
  const uint32_t id = ptx::idesc_make(ptx::kFmtBF16, 128, D, true, true);
  const uint64_t b = ptx::sdesc_sw128(k, 8192, 1024);
#pragma unroll
  for (int part = 0; part < 3; ++part) {
    const uint64_t a = ptx::sdesc_sw128(vp + part * (kC * D * 2), 8192, 1024);
#pragma unroll
    for (int i = 0; i < kC / 16; ++i)
      ptx::mma_f16(tmem_s, ptx::desc_add(a, i * 2048), ptx::desc_add(b, i * 2048), id,
                   !fresh || part > 0 || i > 0);
  }
}

// 16 bytes (8 channels) number i of a tile: row i / (D / 8), swizzled place.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int i) {
  const int t = i / (D / 8), c = i % (D / 8);
  return (uint32_t)((c >> 3) * 8192 + t * 128 + (((c & 7) ^ (t & 7)) << 4));
}
__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fffffff); }

// What every role needs to wait: gives up after kTries or when another role did.
struct Waiter {
  int* abort;
  uint32_t* status;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    const bool done = ptx::mbar_wait_tries_or(bar, parity, kTries, abort);
    if (__all_sync(0xffffffffu, done)) return true;
    if (status) atomicOr(status, KDA_STATUS_TIMEOUT);
    *(volatile int*)abort = 1;
    return false;
  }
};
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
  const int h = blockIdx.x % p.H;
  Segment x;
  if (!find_segment(p, seg, blockIdx.x / p.H, threadIdx.x == 0 && h == 0, x)) return;
  const int hk = h / (p.H / p.Hk);
  const int N = (int)((x.hi - x.lo + kC - 1) / kC);
  const int t_first = (int)x.lo, t_end = (int)x.hi;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&sm.full[i], 2);
      ptx::mbar_init(&sm.empty[i], 1 + 4 + 2 + 2 * NQ);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sm.sc_full[i], 1);
      ptx::mbar_init(&sm.sc_empty[i], 2);
    }
    ptx::mbar_init(&sm.p_full, 2);
    ptx::mbar_init(&sm.v_full, 4);
    ptx::mbar_init(&sm.st_full, NQ);
    ptx::mbar_init(&sm.kv_done, 1);
    ptx::mbar_init(&sm.o_full, 1);
    ptx::mbar_init(&sm.o_empty, NQ);
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
  const Waiter wait{&sm.abort, p.status};
  auto arrive = [&](uint64_t* bar) {  // of a warp, after all its lanes
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ loads and decays
    float g0 = 0.0f, g1 = 0.0f;
    auto load_g = [&](int n) {
      const int t = t_first + n * kC + 2 * lane;
      g0 = t < t_end ? __ldg(p.g + t * p.gs + h) : 0.0f;
      g1 = t + 1 < t_end ? __ldg(p.g + (t + 1) * p.gs + h) : 0.0f;
    };
    load_g(0);
    int n = 0;
#pragma unroll 1
    for (; n < N; ++n) {
      const int s = n % kStages;
      if (n >= kStages && !wait(&sm.empty[s], ((n / kStages) - 1) & 1)) break;
      if (lane == 0) {
        uint8_t* st = smem + s * M::STAGE;
        const int t = t_first + n * kC;
        ptx::mbar_arrive_expect_tx(&sm.full[s], M::STAGE);
        load_tile<D>(st + M::K, &maps.k, &sm.full[s], hk, t);
        load_tile<D>(st + M::Q, &maps.q, &sm.full[s], hk, t);
        load_tile<D>(st + M::V, &maps.v, &sm.full[s], h, t);
      }
      const bool nan = __any_sync(0xffffffffu, g0 != g0 || g1 != g1);
      const int64_t u0 = log_units(g0), u1 = log_units(g1);
      if (n + 1 < N) load_g(n + 1);
      int64_t sum = u0 + u1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t w = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += w;
      }
      float2 a = log_pair(sum - u1), b = log_pair(sum);
      if (nan) a.x = b.x = nan_f();  // a NaN decay spoils its chunk
      *reinterpret_cast<float4*>(&sm.gam[s][2 * lane]) = make_float4(a.x, a.y, b.x, b.y);
      *reinterpret_cast<float2*>(&sm.ein[s][2 * lane]) =
          make_float2(ptx::ex2_approx(a.x + a.y), ptx::ex2_approx(b.x + b.y));
      if (lane == 31) sm.total[s] = b;
      arrive(&sm.full[s]);
    }
    if (*(volatile int*)&sm.abort) {  // the loads in flight land before the CTA leaves
      for (int i = n > kStages ? n - kStages : 0; i < n; ++i)
        ptx::mbar_wait_tries(&sm.full[i % kStages], (i / kStages) & 1, kTries);
      __syncwarp();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ products
    const uint32_t id_qk = ptx::idesc_make(ptx::kFmtBF16, 128, kC, false, false);
    const uint32_t id_pv = ptx::idesc_make(ptx::kFmtBF16, 128, kC, true, false);
    auto issue_qk = [&](int n) {
      const uint32_t st = base + (n % kStages) * M::STAGE;
      if (ptx::elect_one()) {
        const uint64_t a = ptx::sdesc_sw128(st + M::Q, 16, 1024);
        const uint64_t b = ptx::sdesc_sw128(st + M::K, 16, 1024);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t off = (i >> 2) * 8192 + (i & 3) * 32;
          ptx::mma_f16(tmem + T::SC + (n & 1) * 64, ptx::desc_add(a, off), ptx::desc_add(b, off),
                       id_qk, i > 0);
        }
        ptx::mma_commit(&sm.sc_full[n & 1]);
      }
      __syncwarp();
    };
    bool ok = N == 0 || wait(&sm.full[0], 0);
    if (ok && N > 0) issue_qk(0);
#pragma unroll 1
    for (int n = 0; ok && n < N; ++n) {
      const int s = n % kStages;
      const uint32_t st = base + s * M::STAGE;
      if (n + 1 < N) {
        ok = wait(&sm.full[(n + 1) % kStages], ((n + 1) / kStages) & 1) &&
             (n < 1 || wait(&sm.sc_empty[(n + 1) & 1], (((n + 1) >> 1) - 1) & 1));
        if (!ok) break;
        ptx::tc_fence_after();
        issue_qk(n + 1);
      }
      ok = wait(&sm.v_full, n & 1) && wait(&sm.st_full, n & 1);
      if (!ok) break;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        issue_kv<D>(tmem + T::S, base + M::VP, st + M::K, false);
        ptx::mma_commit(&sm.kv_done);
      }
      __syncwarp();
      if (n > 0 && !(ok = wait(&sm.o_empty, (n - 1) & 1))) break;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        const uint64_t b = ptx::sdesc_sw128(st + M::Q, 16, 1024);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            ptx::mma_f16_ts(tmem + T::OI, tmem + (part ? T::LO : T::HI) + i * 8,
                            ptx::desc_add(b, (i >> 2) * 8192 + (i & 3) * 32),
                            ptx::idesc_make(ptx::kFmtBF16, 128, kC, false, false), part > 0 || i > 0);
      }
      __syncwarp();
      if (!(ok = wait(&sm.p_full, n & 1))) break;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        const uint64_t a = ptx::sdesc_sw128(st + M::V, 8192, 1024);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint64_t b = ptx::sdesc_sw128(base + M::P + part * 8192, 16, 1024);
#pragma unroll
          for (int i = 0; i < kC / 16; ++i)
            ptx::mma_f16(tmem + T::OA, ptx::desc_add(a, i * 2048), ptx::desc_add(b, i * 32), id_pv,
                         part > 0 || i > 0);
        }
        ptx::mma_commit(&sm.o_full);
        ptx::mma_commit(&sm.empty[s]);
      }
      __syncwarp();
    }
    if (__any_sync(0xffffffffu, *(volatile int*)&sm.abort)) {  // the products in flight end first
      if (ptx::elect_one()) ptx::mma_commit(&sm.drain);
      __syncwarp();
      ptx::mbar_wait_tries(&sm.drain, 0, kTries);
      __syncwarp();
    }
  } else if (warp < 4 || warp >= 14) {
    // ------------------------------------------------------------------ V'
    const int tid = (warp < 4 ? warp - 2 : warp - 12) * 32 + lane;
#pragma unroll 1
    for (int n = 0; n < N; ++n) {
      const int s = n % kStages;
      const uint32_t st = base + s * M::STAGE;
      const int m = t_end - (t_first + n * kC);  // tokens left
      if (!wait(&sm.full[s], (n / kStages) & 1)) break;
      if (n > 0 && !wait(&sm.kv_done, (n - 1) & 1)) break;
      const float2 total = sm.total[s];
#pragma unroll
      for (int i = 0; i < kC * D / 8 / 128; ++i) {
        const int at = i * 128 + tid, t = at / (D / 8);
        const uint32_t off = tile_at<D>(at);
        const float2 gt = sm.gam[s][t];
        const float w = ptx::ex2_approx((total.x - gt.x) + (total.y - gt.y));
        float f[8];
        Vec16<__nv_bfloat16>::unpack(ld_shared(st + M::V + off), f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= w;
        uint4 part[3];
        split3(f, part[0], part[1], part[2]);
        if (t >= m) {  // rows of the next sequence, whatever they hold
          const uint4 z = make_uint4(0u, 0u, 0u, 0u);
          part[0] = part[1] = part[2] = z;
          st_shared(st + M::V + off, z);
          st_shared(st + M::K + off, z);
        }
#pragma unroll
        for (int j = 0; j < 3; ++j) st_shared(base + M::VP + j * M::TILE + off, part[j]);
      }
      ptx::fence_proxy_async_smem();
      arrive(&sm.v_full);
      if (lane == 0) ptx::mbar_arrive(&sm.empty[s]);
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------ the state
    const int w = warp - 4;
    if (w < NQ) {
      const uint32_t lanes = (uint32_t)(w * 32) << 16;
      const int dv = w * 32 + lane;
      const float* entry = !x.first ? added + ((x.place - 1) * p.H + h) * (int64_t)(D * D)
                           : p.init ? p.init + ((int64_t)x.seq * p.H + h) * (D * D) : nullptr;
      float* exit_state =
          x.last && p.final_state ? p.final_state + ((int64_t)x.seq * p.H + h) * (D * D) : nullptr;
      bool ok = true;
#pragma unroll 1
      for (int n = 0; n < N; ++n) {
        const int s = n % kStages;
        ok = wait(&sm.full[s], (n / kStages) & 1) &&
             (n == 0 || (wait(&sm.kv_done, (n - 1) & 1) && wait(&sm.o_full, (n - 1) & 1)));
        if (!ok) break;
        ptx::tc_fence_after();
        const float a = ptx::ex2_approx(sm.total[s].x + sm.total[s].y);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float f[32];
          if (n > 0) {
            ptx::tmem_ld32(tmem + lanes + T::S + c * 32, f);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = entry ? entry[(c * 32 + i) * D + dv] : 0.0f;
          }
          float hi[16], lo[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint32_t u, v;
            split2(f[2 * i], f[2 * i + 1], u, v);
            hi[i] = __uint_as_float(u);
            lo[i] = __uint_as_float(v);
            f[2 * i] *= a;
            f[2 * i + 1] *= a;
          }
          ptx::tmem_st16(tmem + lanes + T::HI + c * 16, hi);
          ptx::tmem_st16(tmem + lanes + T::LO + c * 16, lo);
          ptx::tmem_st32_nowait(tmem + lanes + T::S + c * 32, f);
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        arrive(&sm.st_full);
        if (lane == 0) ptx::mbar_arrive(&sm.empty[s]);
      }
      if (ok && exit_state) {
        if (N > 0) ok = wait(&sm.kv_done, (N - 1) & 1);
        ptx::tc_fence_after();
        if (ok) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float f[32];
            if (N > 0) {
              ptx::tmem_ld32(tmem + lanes + T::S + c * 32, f);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) f[i] = entry ? entry[(c * 32 + i) * D + dv] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) exit_state[(c * 32 + i) * D + dv] = f[i];
          }
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ outputs
    const int w = warp - 8;
    if (w < NQ) {
      const uint32_t lanes = (uint32_t)(w * 32) << 16;
      const int dv = w * 32 + lane, tid = dv;
      __nv_bfloat16* stage = reinterpret_cast<__nv_bfloat16*>(smem + M::O);
      bool ok = true;
#pragma unroll 1
      for (int n = 0; n < N; ++n) {
        const int s = n % kStages;
        const int t0 = t_first + n * kC;
        ok = wait(&sm.o_full, n & 1) && wait(&sm.full[s], (n / kStages) & 1);
        if (tid == 0) ptx::bulk_wait_read0();  // the last chunk's rows have left
        ok = group_and(1, NQ * 32, ok);
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t a[32], b[32];
          ptx::tmem_ld32_nowait(tmem + lanes + T::OI + c * 32, a);
          ptx::tmem_ld32_nowait(tmem + lanes + T::OA + c * 32, b);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(a[i]), "+r"(b[i]));
          if (c == 1) {
            ptx::tc_fence_before();
            arrive(&sm.o_empty);
          }
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 e = *reinterpret_cast<const float2*>(&sm.ein[s][c * 32 + i]);
            const uint32_t r = pack_bf16(
                p.scale * fmaf(e.x, __uint_as_float(a[i]), __uint_as_float(b[i])),
                p.scale * fmaf(e.y, __uint_as_float(a[i + 1]), __uint_as_float(b[i + 1])));
            stage[(c * 32 + i) * D + dv] = __ushort_as_bfloat16((unsigned short)r);
            stage[(c * 32 + i + 1) * D + dv] = __ushort_as_bfloat16((unsigned short)(r >> 16));
          }
        }
        arrive(&sm.empty[s]);
        ptx::fence_proxy_async_smem();
        ok = group_and(1, NQ * 32, true);
        const int m = t_end - t0;
        if (m >= kC) {
          if (tid == 0) {
            ptx::tma_store_2d(&maps.o, stage, h * D, t0);
            ptx::bulk_commit();
          }
        } else {  // the rows after the segment belong to another one
          for (int i = tid; i < m * (D / 8); i += NQ * 32) {
            const int t = i / (D / 8), c = i % (D / 8);
            *reinterpret_cast<uint4*>((__nv_bfloat16*)p.o + ((int64_t)(t0 + t) * p.H + h) * D + c * 8) =
                *reinterpret_cast<const uint4*>(stage + t * D + c * 8);
          }
        }
      }
      if (tid == 0) ptx::bulk_wait0();
    }
  } else {
    // ------------------------------------------------------------------ P (warps 12, 13)
    const int w = warp - 12, i = w * 32 + lane;  // the row
    const uint32_t lanes = (uint32_t)(w * 32) << 16;
#pragma unroll 1
    for (int n = 0; n < N; ++n) {
      const int s = n % kStages;
      if (!(wait(&sm.full[s], (n / kStages) & 1) && wait(&sm.sc_full[n & 1], (n >> 1) & 1) &&
            (n == 0 || wait(&sm.o_full, (n - 1) & 1))))
        break;
      ptx::tc_fence_after();
      const float2 gi = sm.gam[s][i];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float f[32];
        if (c <= w) ptx::tmem_ld32(tmem + lanes + T::SC + (n & 1) * 64 + c * 32, f);
        if (c == w) {
          ptx::tc_fence_before();
          arrive(&sm.sc_empty[n & 1]);
        }
        if (c <= w) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float2 gj = sm.gam[s][c * 32 + j];
            const float d = ptx::ex2_approx((gi.x - gj.x) + (gi.y - gj.y));
            f[j] = c * 32 + j <= i ? f[j] * d : 0.0f;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] = 0.0f;
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(f[b * 8 + 2 * e], f[b * 8 + 2 * e + 1], hi[e], lo[e]);
          const uint32_t off = base + M::P + i * 128 + (((c * 4 + b) ^ (i & 7)) << 4);
          st_shared(off, make_uint4(hi[0], hi[1], hi[2], hi[3]));
          st_shared(off + 8192, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
      }
      ptx::fence_proxy_async_smem();
      arrive(&sm.p_full);
      if (lane == 0) ptx::mbar_arrive(&sm.empty[s]);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- what a segment adds
//
// sum_s e^(sum of g after s) k_s v_s^T over a whole segment, from its last chunk to its first: the
// decays behind a chunk are known when it is reached, so the accumulator is never rescaled. And the
// rows that the outputs' kernel reads first are the ones that this one read last.
template <int D>
struct Add {
  static constexpr int TILE = kC * D * 2, STAGE = 2 * TILE;
  static constexpr int V = 0, K = TILE;
  static constexpr int VP = kStages * STAGE;  // two sets of three parts, then one tile of slack for D = 64
  static constexpr int SMALL = VP + 6 * TILE + (D == 64 ? TILE : 0);
};
struct AddSmall {
  uint64_t full[kStages], empty[kStages];
  uint64_t v_full[2], v_empty[2], done, drain;
  float w[kStages][kC];
  uint32_t tmem;
  int abort;
};
constexpr int kAddThreads = 320;  // 2 + 8 warps

template <int D>
__global__ void __launch_bounds__(kAddThreads, 1)
decay_add_kernel(const __grid_constant__ Maps maps, const DecayParams p, int seg, float* added,
                 float* added_log) {
  using M = Add<D>;
  constexpr int NQ = D / 32;
  constexpr uint32_t kCols = D;
  extern __shared__ __align__(1024) uint8_t smem[];
  AddSmall& sm = *reinterpret_cast<AddSmall*>(smem + M::SMALL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x % p.H;
  Segment x;
  if (!find_segment(p, seg, blockIdx.x / p.H, false, x) || x.last) return;
  const int hk = h / (p.H / p.Hk);
  const int N = seg / kC;  // segments that are not their sequence's last are whole
  const int t_first = (int)x.lo;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&sm.full[i], 2);
      ptx::mbar_init(&sm.empty[i], 1 + 8);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sm.v_full[i], 8);
      ptx::mbar_init(&sm.v_empty[i], 1);
    }
    ptx::mbar_init(&sm.done, 1);
    ptx::mbar_init(&sm.drain, 1);
    ptx::fence_mbar_init();
    sm.abort = 0;
  }
  if (warp == 1) {
    ptx::tmem_alloc(&sm.tmem, kCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
  const uint32_t base = ptx::smem_u32(smem);
  const Waiter wait{&sm.abort, p.status};
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
  };

  if (warp == 0) {
    float g0 = 0.0f, g1 = 0.0f;
    auto load_g = [&](int n) {
      const int t = t_first + (N - 1 - n) * kC + 2 * lane;
      g0 = __ldg(p.g + t * p.gs + h);
      g1 = __ldg(p.g + (t + 1) * p.gs + h);
    };
    load_g(0);
    int64_t later = 0;
    int n = 0;
#pragma unroll 1
    for (; n < N; ++n) {
      const int s = n % kStages;
      if (n >= kStages && !wait(&sm.empty[s], ((n / kStages) - 1) & 1)) break;
      if (lane == 0) {
        uint8_t* st = smem + s * M::STAGE;
        const int t = t_first + (N - 1 - n) * kC;
        ptx::mbar_arrive_expect_tx(&sm.full[s], M::STAGE);
        load_tile<D>(st + M::V, &maps.v, &sm.full[s], h, t);
        load_tile<D>(st + M::K, &maps.k, &sm.full[s], hk, t);
      }
      const bool nan = __any_sync(0xffffffffu, g0 != g0 || g1 != g1);
      const int64_t u0 = log_units(g0), u1 = log_units(g1);
      if (n + 1 < N) load_g(n + 1);
      int64_t sum = u0 + u1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t w = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += w;
      }
      const int64_t all = __shfl_sync(0xffffffffu, sum, 31);
      const float2 a = log_pair(later + all - (sum - u1)), b = log_pair(later + all - sum);
      float wa = ptx::ex2_approx(a.x + a.y), wb = ptx::ex2_approx(b.x + b.y);
      if (nan) wa = wb = nan_f();
      *reinterpret_cast<float2*>(&sm.w[s][2 * lane]) = make_float2(wa, wb);
      later += all;
      arrive(&sm.full[s]);
    }
    if (lane == 0) added_log[x.place * p.H + h] = log_pair(later).x;
    if (*(volatile int*)&sm.abort) {
      for (int i = n > kStages ? n - kStages : 0; i < n; ++i)
        ptx::mbar_wait_tries(&sm.full[i % kStages], (i / kStages) & 1, kTries);
      __syncwarp();
    }
  } else if (warp == 1) {
    bool ok = true;
#pragma unroll 1
    for (int n = 0; ok && n < N; ++n) {
      const int s = n % kStages, b = n & 1;
      ok = wait(&sm.full[s], (n / kStages) & 1) && wait(&sm.v_full[b], (n >> 1) & 1);
      if (!ok) break;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        issue_kv<D>(tmem, base + M::VP + b * 3 * M::TILE, base + s * M::STAGE + M::K, n == 0);
        ptx::mma_commit(&sm.v_empty[b]);
        ptx::mma_commit(&sm.empty[s]);
        if (n == N - 1) ptx::mma_commit(&sm.done);
      }
      __syncwarp();
    }
    if (__any_sync(0xffffffffu, *(volatile int*)&sm.abort)) {
      if (ptx::elect_one()) ptx::mma_commit(&sm.drain);
      __syncwarp();
      ptx::mbar_wait_tries(&sm.drain, 0, kTries);
      __syncwarp();
    }
  } else {
    const int tid = (warp - 2) * 32 + lane;
    bool ok = true;
#pragma unroll 1
    for (int n = 0; n < N; ++n) {
      const int s = n % kStages, b = n & 1;
      const uint32_t st = base + s * M::STAGE, vp = base + M::VP + b * 3 * M::TILE;
      ok = wait(&sm.full[s], (n / kStages) & 1) &&
           (n < 2 || wait(&sm.v_empty[b], ((n >> 1) - 1) & 1));
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < kC * D / 8 / 256; ++i) {
        const int at = i * 256 + tid;
        const uint32_t off = tile_at<D>(at);
        const float w = sm.w[s][at / (D / 8)];
        float f[8];
        Vec16<__nv_bfloat16>::unpack(ld_shared(st + M::V + off), f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= w;
        uint4 part[3];
        split3(f, part[0], part[1], part[2]);
#pragma unroll
        for (int j = 0; j < 3; ++j) st_shared(vp + j * M::TILE + off, part[j]);
      }
      ptx::fence_proxy_async_smem();
      arrive(&sm.v_full[b]);
      if (lane == 0) ptx::mbar_arrive(&sm.empty[s]);
    }
    // warps 4 .. 7 hold the accumulator's rows
    const int w = warp & 3;
    if (ok && warp >= 4 && warp < 8 && w < NQ && wait(&sm.done, 0)) {
      ptx::tc_fence_after();
      float* out = added + (x.place * p.H + h) * (int64_t)(D * D) + w * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float f[32];
        ptx::tmem_ld32(tmem + ((uint32_t)(w * 32) << 16) + c * 32, f);
#pragma unroll
        for (int i = 0; i < 32; ++i) out[(c * 32 + i) * D] = f[i];
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) ptx::tmem_dealloc(tmem, kCols);
}

template <int D>
kda_status launch_d(const DecayParams& p, int seg, float* added, float* added_log, cudaStream_t s) {
  Maps m;
  const uint64_t rows = p.total > 0 ? (uint64_t)p.total : 1;
  // (without tokens nothing is loaded: the maps are not used)
  if (p.total > 0 &&
      !(make_map_tokens(&m.q, p.q, (uint64_t)p.Hk * D, rows, (uint64_t)p.qs * 2, 64, kC, true) &&
        make_map_tokens(&m.k, p.k, (uint64_t)p.Hk * D, rows, (uint64_t)p.ks * 2, 64, kC, true) &&
        make_map_tokens(&m.v, p.v, (uint64_t)p.H * D, rows, (uint64_t)p.vs * 2, 64, kC, true) &&
        make_map_tokens(&m.o, p.o, (uint64_t)p.H * D, rows, (uint64_t)p.H * D * 2, D, kC, false)))
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
  const unsigned grid = (unsigned)((p.total / seg + p.n_seqs) * p.H);
  if (p.total > seg) {
    decay_add_kernel<D><<<grid, kAddThreads, add_bytes, s>>>(m, p, seg, added, added_log);
    launch_decay_scan(p, D, seg, added, added_log, s);
    count_launches(1);
  }
  decay_tc_kernel<D><<<grid, kThreads, out_bytes, s>>>(m, p, seg, added);
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
