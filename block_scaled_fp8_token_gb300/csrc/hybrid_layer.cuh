// hybrid_layer.cuh -- what the kernels of a hybrid decoder's operators share: BF16 vectors,
// the functions of their gates, and which request of a ragged step a tile of tokens belongs to.
#pragma once

#include "attention_layer.cuh"
#include "act_math.cuh"
#include "hybrid_layer.h"

namespace bfp8 {
namespace dev {

// Eight BF16 of a 16-byte vector, and back with one rounding each.
BFP8_DEV void widen8(const uint4& r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
BFP8_DEV uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
BFP8_DEV uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// 16 bytes from global to shared memory past the registers. A thread's groups complete in
// order; what a thread copied itself it may read after its own wait.
BFP8_DEV void cp_async16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
BFP8_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
BFP8_DEV void cp_async_wait_group() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// 1 / (1 + e^-x), relative error below (4 + 1.2 max(0, -x)) 2^-23: 2^x's approximation is
// within 2 units, its argument's product with log2 e adds 1.16 |x|, and both count in full
// where e^-x outweighs the 1; the reciprocal adds 1. That is under 2^-16 down to x = -87, below
// which e^-x overflows (or its reciprocal is subnormal) and the result is 0: for results that
// BF16 or E4M3 rounds (2^-8, 2^-4).
BFP8_DEV float sigmoid(float x) { return rcp_approx(1.0f + ex2_approx(x * -1.4426950408889634f)); }

// The same of two BF16 x, within 4 2^-23 and as much again where e^-x outweighs the 1: x times the
// upper 16 bits of log2 e is exact, and the rest of the exponent is put right to first order: 1 + x k,
// as 1.5 - (0.5 - x k) within 2^-25, the latter kept in [0, 1] so that an infinite x meets no 0 of e^-x.
BFP8_DEV float saturated_fma(float a, float b, float c) {
  float r;
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
BFP8_DEV float2 sigmoid_bf16(float2 x) {
  const float2 t = __fmul2_rn(x, make_float2(kNegLog2eHi, kNegLog2eHi));
  const float2 e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
  const float2 rest = make_float2(saturated_fma(x.x, -kNegLog2eLoLn2, 0.5f), saturated_fma(x.y, -kNegLog2eLoLn2, 0.5f));
  const float2 right = __ffma2_rn(rest, make_float2(-1.0f, -1.0f), make_float2(1.5f, 1.5f));
  const float2 d = __ffma2_rn(e, right, make_float2(1.0f, 1.0f));
  return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}

// The requests of a step lie one behind another: request b has the tokens
// [offsets[b], offsets[b + 1]), within [0, T] whatever the array holds.
struct Requests {
  const int32_t* offsets;
  const int32_t* slots_in;
  const int32_t* slots_out;
  int64_t tokens, n_slots;
  int32_t batch;
};
BFP8_DEV int64_t clamp_token(const Requests& q, int32_t t) {
  return t < 0 ? 0 : t > q.tokens ? q.tokens : t;
}
BFP8_DEV int64_t first_token(const Requests& q, int b) { return clamp_token(q, __ldg(q.offsets + b)); }
// The slot that request b reads (out: writes), -1 for none.
BFP8_DEV int64_t slot_of(const Requests& q, const int32_t* slots, int b) {
  if (!slots) return -1;
  const int32_t s = __ldg(slots + b);
  return s < 0 || s >= q.n_slots ? -1 : s;
}

// Tiles of 2^shift tokens that begin with each request's first: request b's are numbered
// from key(b) = (offsets[b] >> shift) + b on. As ceil(n / 2^shift) <= (offsets[b + 1] >>
// shift) - (offsets[b] >> shift) + 1, no two requests share a number, all lie below
// (T >> shift) + batch, and the numbers need no sum over the requests ahead.
BFP8_DEV int64_t tile_key(const Requests& q, int b, int shift) {
  return (first_token(q, b) >> shift) + b;
}
// The request whose tile y would be: the last with key(b) <= y, or -1. The whole warp
// searches, 32 probes at a time.
BFP8_DEV int find_request(const Requests& q, int64_t y, int shift) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = q.batch;
  while (true) {
    const int step = (n + 31) >> 5;
    const int at = lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, at < n && tile_key(q, lo + at, shift) <= y);
    if (m == 0) return -1;
    const int c = 31 - __clz(m);
    lo += c * step;
    if (step == 1) return lo;
    n = min(step, n - c * step);
  }
}

}  // namespace dev
}  // namespace bfp8
