// Shared by the kernels of linear attention with one decay per head: how packed sequences are cut
// into segments, and the decays inside a chunk.
//
// A prompt is cut into segments of `seg` tokens (a multiple of the chunk) that are walked side by
// side: the state that a segment adds is summed first (from zero), a scan over a sequence's
// segments gives each its entry state (elementwise, since a segment's decay is one number), and
// the segments then run with their outputs. Lengths live on the device, so segments are numbered
// from the packed offsets: segment j of sequence s is in slot floor(cu[s] / seg) + s + j. All but
// a sequence's last are full, and their added states are in place floor(cu[s] / seg) + j of a
// workspace of floor(total / seg) places: sequence s + 1 begins at least that many places on.
#pragma once

#include "kda_internal.cuh"

namespace kda {
namespace decay {

struct Segment {
  int seq;
  int lo, hi;          // tokens
  int place;           // of the state that it adds; the entry state is in place - 1
  bool first, last;    // of its sequence
};

// The segment in a slot, or (kPlaces) the one with a place, i.e. not its sequence's last; false: none.
// `flag`: report malformed offsets. (Offsets are at most 2^30, so that 32 bits do; a negative one is
// malformed.) By a whole warp, whose lanes probe 32 sequences at once.
template <bool kPlaces>
__device__ __forceinline__ bool find_segment(const DecayParams& p, int seg, int slot, int lane,
                                             bool flag, Segment& x) {
  int a = 0;  // the last sequence whose first slot (or place) is <= slot: among n from a on
  if (p.cu) {
    for (int n = p.n_seqs; n > 1;) {
      const int step = (n + 31) / 32, off = lane * step, m = a + off;
      bool upto = lane == 0;
      if (lane > 0 && off < n) upto = p.cu[m] / seg + (kPlaces ? 0 : m) <= slot;
      const int last = (31 - __clz(__ballot_sync(0xffffffffu, upto))) * step;
      a += last;
      n = min(step, n - last);
    }
  }
  int c0 = p.cu ? p.cu[a] : 0, c1 = p.cu ? p.cu[a + 1] : p.total;
  const int j = slot - (c0 / seg + (kPlaces ? 0 : a));
  if (j < 0) return false;
  if (c0 < 0 || c1 > p.total || c1 < c0) {
    if (flag && p.status) atomicOr(p.status, KDA_STATUS_BAD_OFFSETS);
    if (j > 0) return false;
    c0 = c1 = 0;  // an empty sequence
  }
  if (j > (c1 - c0) / seg) return false;
  x.seq = a;
  x.lo = c0 + j * seg;
  x.hi = c1 - x.lo > seg ? x.lo + seg : c1;
  x.first = j == 0;
  x.last = x.hi == c1;
  x.place = c0 / seg + j;
  return kPlaces ? !x.last : x.first || x.lo < c1;
}

// Sums of log-decays, in base-2 exponents, as pairs of floats (high + low part): their error stays
// below 2^-30 however strong the decays, so the decay between two tokens does not lose bits to a
// strong decay before both. A token's decay below e^-277 (2^-400) counts as that: no fp32 state
// survives it either way. (As 64-bit integers or in double precision the conversions alone took
// 2000 cycles a chunk.)
__device__ __forceinline__ float2 log_pair(float g) {
  g = g < -277.0f ? -277.0f : g;  // (a NaN stays)
  const float c0 = 1.4426950216293335f, c1 = 1.9259629911266175e-8f;  // 1 / ln 2
  const float a = g * c0;
  return make_float2(a, fmaf(g, c1, fmaf(g, c0, -a)));
}
__device__ __forceinline__ float2 log_add(float2 a, float2 b) {
  const float s = __fadd_rn(a.x, b.x), t = __fsub_rn(s, a.x);
  float e = __fadd_rn(__fsub_rn(a.x, __fsub_rn(s, t)), __fsub_rn(b.x, t));  // s + e = a.x + b.x
  e = __fadd_rn(e, __fadd_rn(a.y, b.y));
  const float hi = __fadd_rn(s, e);
  return make_float2(hi, __fsub_rn(e, __fsub_rn(hi, s)));
}
__device__ __forceinline__ float2 log_sub(float2 a, float2 b) {
  return log_add(a, make_float2(-b.x, -b.y));
}
// Sums over the lanes up to each, of N lists side by side (one alone waits for its own latencies).
template <int N>
__device__ __forceinline__ void log_scan(float2 (&v)[N], int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    float2 w[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      w[i] = make_float2(__shfl_up_sync(0xffffffffu, v[i].x, o),
                         __shfl_up_sync(0xffffffffu, v[i].y, o));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 x = log_add(v[i], w[i]);
      if (lane >= o) v[i] = x;
    }
  }
}
__device__ __forceinline__ float2 log_scan(float2 v, int lane) {
  float2 x[1] = {v};
  log_scan(x, lane);
  return x[0];
}
// 2^(a - b).
__device__ __forceinline__ float decay_between(float2 a, float2 b) {
  return exp2f((a.x - b.x) + (a.y - b.y));
}

// The scan over the segments' added states, and the tensor-core kernels for bf16.
void launch_decay_scan(const DecayParams& p, int d, int seg, float* added, const float* added_log,
                       cudaStream_t s);
kda_status launch_tc(const DecayParams& p, int d, int seg, float* added, float* added_log,
                     cudaStream_t s);

}  // namespace decay
}  // namespace kda
