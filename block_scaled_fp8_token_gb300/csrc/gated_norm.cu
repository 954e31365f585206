// gated_norm.cu -- the heads' outputs of a linear-attention layer normed and gated, and
// quantized for the output projection, in one pass:
//
//   y = x * rsqrt(mean(x^2) + eps) * (w + offset) * act(z)     per token and head
//   out = bf16(y);  s = max(max|y|, 1e-10f) / 448 per 128 columns of a token's heads,
//   q = RNE_satfinite_e4m3(y / s)
//
// act is SiLU or the sigmoid; without w there is no norm (the gate of a full-attention
// layer's heads). Bound by HBM: x and z are read once, and the codes (a quarter of the
// bytes) or the BF16 row written once. 8192 rows of 48 heads to codes, 253 MB, take 51 us, 5.0
// TB/s, of which looking for codes that FP32 may miss and settling them is 6.5; with one token's
// loads ahead in registers, 32 warps an SM had too few bytes under way (55 us in place of 44),
// and without any 67.
#include "hybrid_layer.cuh"

namespace bfp8 {
namespace {

using namespace dev;

constexpr int kGatedThreads = 256, kGatedAhead = 4;   // tokens whose loads a warp has under way

struct GatedParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* z;
  const void* w;
  __nv_bfloat16* out;
  uint8_t* q;
  float* s;
  int64_t xt, xh, zt, zh, ot, oh, ldq, ssm, sskb, tokens, warps;
  int32_t cols, segs, w_f32, is_sigmoid;
  float eps, w_offset;
};

// A code may hang on FP32's last bits: y / s within kNear units of its last place of the middle
// between two codes, which lies where the 20 bits below a code's are 0x80000. (Of 78 million codes
// none was off by more than 4 units. Below 2^-6 the middles lie elsewhere, and a step is 2^-9 of
// 448.) Twelve bits up, so that two operations an entry find the nearest.
constexpr int kNotes = 16;                             // of a warp
constexpr uint32_t kNear = 8;
constexpr uint32_t kBothSides = (2 * kNear) << 12;
BFP8_DEV uint32_t from_tie(float f) { return __float_as_uint(f) * 4096u - ((0x80000u - kNear) << 12); }
BFP8_DEV bool is_near(float f) { return from_tie(f) <= kBothSides; }

// For those few, sums of two floats (by Knuth's and Dekker's error-free sums and products): entries
// within 2^-32, so that of codes whose quotient is not the middle itself none but one in some 2^32
// differs from exact arithmetic's.
struct Two {
  float hi, lo;
};
// (Each operation rounded on its own: a product that the compiler took into a sum would count its
// rest twice.)
BFP8_DEV Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), c = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, c)), __fsub_rn(b, c))};
}
BFP8_DEV Two two_parts(float h, float l) {
  const float s = __fadd_rn(h, l);
  return {s, __fadd_rn(__fsub_rn(h, s), l)};
}
BFP8_DEV Two two_times(Two a, Two b) {
  const float h = __fmul_rn(a.hi, b.hi);
  return two_parts(h, __fadd_rn(fmaf(a.hi, b.hi, -h), fmaf(a.hi, b.lo, __fmul_rn(a.lo, b.hi))));
}
BFP8_DEV Two two_over(Two a, Two b) {
  const float r = rcp_approx(b.hi), q = __fmul_rn(a.hi, r);
  return two_parts(q, __fmul_rn(__fadd_rn(fmaf(-q, b.hi, a.hi), fmaf(-q, b.lo, a.lo)), r));
}
// 1 + e^-z for a BF16 z in [-60, 40], within 2^-32: e^r by its series, its terms from r^4 / 24 on in
// one float, with r = -z - k ln 2 (Cody and Waite's reduction: ln 2 in pieces of 12 and 13 bits, exact
// times k, and the rest).
BFP8_DEV Two one_and_exp(float z) {
  const float k = rintf(z * -1.4426950408889634f);
  const Two a = two_sum(fmaf(-k, 0.693115234375f, -z), __fmul_rn(k, -3.1948089599609375e-5f));
  const Two r = two_sum(a.hi, fmaf(k, 1.9046543e-9f, a.lo));
  const float x = r.hi;
  float s = 2.7557319e-7f;                             // 1 / 10!, 1 / 9!, ...
  s = fmaf(s, x, 2.7557319e-6f), s = fmaf(s, x, 2.4801587e-5f), s = fmaf(s, x, 1.9841270e-4f);
  s = fmaf(s, x, 1.3888889e-3f), s = fmaf(s, x, 8.3333333e-3f), s = fmaf(s, x, 4.1666667e-2f);
  const Two r2 = two_times(r, r), r3 = two_times(r2, r);
  const Two third = two_times(r3, {0.16666667f, -4.9670537e-9f});
  const Two u = two_sum(third.hi, __fmul_rn(__fmul_rn(s, r2.hi), r2.hi)), v = two_sum(__fmul_rn(0.5f, r2.hi), u.hi);
  const Two w = two_sum(r.hi, v.hi);
  const Two e = two_sum(1.0f, w.hi);
  const float rest = e.lo + (w.lo + (v.lo + (u.lo + (third.lo + (0.5f * r2.lo + r.lo)))));
  const float up = __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(k)) << 23);
  const Two d = two_sum(__fmul_rn(up, e.hi), 1.0f);
  return two_sum(d.hi, fmaf(up, rest, d.lo));
}
// x * w * act(z) in column c of a row, with the head's factor where a group has two; NaN where it
// leaves the range in which the products' errors are exact.
template <int DIM>
BFP8_DEV Two entry(const GatedParams& p, int64_t row, int c) {
  const int head = c / DIM, d = c % DIM;
  const __nv_bfloat16* const px = p.x + row * p.xt + head * p.xh;
  const float x = __bfloat162float(px[d]), z = __bfloat162float(p.z[row * p.zt + head * p.zh + d]);
  float w = 1.0f;
  if (p.w) w = p.w_f32 ? static_cast<const float*>(p.w)[d] : __bfloat162float(static_cast<const __nv_bfloat16*>(p.w)[d]);
  Two y = {p.is_sigmoid ? x : x * z, 0.0f};            // exact: 16 bits
  if (!(y.hi == 0.0f || (fabsf(y.hi) > 0x1p-60f && fabsf(y.hi) < 0x1p60f)) || !(z > -60.0f)) y.hi = NAN;
  if (p.w) y = two_times(y, two_sum(w, p.w_offset));
  y = two_over(y, one_and_exp(fminf(fmaxf(z, -60.0f), 40.0f)));
  if (DIM < 128 && p.w) {
    double ss = 0.0;
#pragma unroll 1
    for (int k = 0; k < DIM; k += 8) {
      float f[8];
      widen8(*reinterpret_cast<const uint4*>(px + k), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += static_cast<double>(f[e]) * f[e];
    }
    const double r = rsqrt(ss / DIM + p.eps);
    y = two_times(y, {static_cast<float>(r), static_cast<float>(r - static_cast<float>(r))});
  }
  return y;
}
// 8 weights from column d of a head on, with their offset.
BFP8_DEV void load_weights(const GatedParams& p, int d, float2 (&w)[4]) {
  if (p.w_f32) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.w) + d));
    const float4 g = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.w) + d + 4));
    w[0] = make_float2(f.x, f.y), w[1] = make_float2(f.z, f.w), w[2] = make_float2(g.x, g.y), w[3] = make_float2(g.z, g.w);
  } else {
    float f[8];
    widen8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.w) + d)), f);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = make_float2(f[2 * e], f[2 * e + 1]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e].x += p.w_offset, w[e].y += p.w_offset;
}
// y of a lane's 8 columns of a row. The whole warp.
template <int DIM>
BFP8_DEV void row_values(const GatedParams& p, const uint4& xr, const uint4& zr, const float2 (&w)[4], float2 (&y)[4]) {
  float x[8], z[8];
  widen8(xr, x);
  widen8(zr, z);
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = make_float2(x[2 * e], x[2 * e + 1]);
  if (p.w) {
    float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int e = 0; e < 4; ++e) s2 = __ffma2_rn(y[e], y[e], s2);
    float ss = s2.x + s2.y;
#pragma unroll
    for (int o = DIM / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(fmaf(ss, 1.0f / DIM, p.eps));
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = __fmul2_rn(y[e], __fmul2_rn(w[e], make_float2(r, r)));
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 a = make_float2(z[2 * e], z[2 * e + 1]);
    float2 g = sigmoid_bf16(a);
    if (!p.is_sigmoid) g = __fmul2_rn(g, a);
    y[e] = __fmul2_rn(y[e], g);
  }
}
// The largest |y| of a lane's group, its scale, and 1 / scale.
BFP8_DEV float group_scale(const float2 (&y)[4], float& sc, float& inv) {
  float am = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) am = fmaxf(am, fmaxf(fabsf(y[e].x), fabsf(y[e].y)));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  // am / 448 rounded (its remainder is exact), and 1 / s within 2^-23
  am = fmaxf(am, 1e-10f);
  sc = am * (1.0f / 448.0f);
  if (am <= 3.0e38f) sc = fmaf(fmaf(-448.0f, sc, am), 1.0f / 448.0f, sc);
  inv = rcp_approx(sc);
  if (am <= 3.0e38f) inv = fmaf(fmaf(-sc, inv, 1.0f), inv, inv);
  return am;
}
BFP8_DEV void quotients(const float2 (&y)[4], float inv, float2 (&f)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = __fmul2_rn(y[e], make_float2(inv, inv));
}
BFP8_DEV bool may_be_near(float am) { return am > 1e-10f && am <= 3.0e38f; }
// The place of its largest entry in a lane's group, the first of equal ones. The whole warp.
BFP8_DEV uint32_t group_top(const float2 (&y)[4], float am, int lane) {
  uint32_t top = 8;
#pragma unroll
  for (int e = 3; e >= 0; --e) top = fabsf(y[e].x) == am ? 2 * e : fabsf(y[e].y) == am ? 2 * e + 1 : top;
  const uint32_t tops = __ballot_sync(0xffffffffu, top < 8) & (lane < 16 ? 0xFFFFu : 0xFFFF0000u);
  const int src = tops ? __ffs(tops) - 1 : lane;
  return 8 * (src & 15) + (__shfl_sync(0xffffffffu, top, src) & 7);
}
// The code of y. A quotient that is the middle itself goes to the even code: entries with one gate and
// one weight have their bits of x alone, and one in 16 of those can be such a tie. Their divisors by
// the gate are the same, so that a quotient is within 2^-42 (three divisions of 2^-44 and four products
// of 2^-47), and what is within 2^-40 of the middle counts as it: of others that is one in some 2^36.
BFP8_DEV uint8_t settled_code(Two y) {
  const uint32_t middle = (__float_as_uint(y.hi) & 0xFFF00000u) | 0x80000u;
  const float m = __uint_as_float(middle);
  // towards zero, with what is cut off as an odd last bit: rounding that once more is exact
  uint32_t bits = __float_as_uint(y.hi);
  if (y.lo != 0.0f) bits = (bits - (((__float_as_uint(y.lo) ^ bits) >> 31) & 1u)) | 1u;
  if (fabsf((y.hi - m) + y.lo) <= 0x1p-40f * fabsf(m)) bits = middle;
  return static_cast<uint8_t>(f32x2_to_e4m3x2(__uint_as_float(bits), 0.0f));
}
// The warp's doubtful codes settled, two lanes each: one has the code's column, the other that with
// the largest entry of its group. A note is a row (x), a column of the warp's in bits 0 - 7 (y), and
// from bit 8 on that of its group.
template <int DIM>
__device__ __noinline__ void settle(const GatedParams& p, const uint2* notes, int count, int c) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  const bool valid = (lane & 15) < count;
  const uint2 note = valid ? notes[lane & 15] : make_uint2(0u, 0u);
  c += note.y & 0xFF;
  Two y = {1.0f, 0.0f};
  if (valid) y = entry<DIM>(p, note.x, lane < 16 ? c : (c & ~127) + static_cast<int>(note.y >> 8));
  const Two m = {__shfl_down_sync(0xffffffffu, y.hi, 16), __shfl_down_sync(0xffffffffu, y.lo, 16)};
  y = two_times(two_over(y, m), {m.hi < 0.0f ? -448.0f : 448.0f, 0.0f});
  if (valid && lane < 16 && fabsf(y.hi) < 449.0f)      // not NaN
    p.q[note.x * p.ldq + c] = settled_code(y);
  __syncwarp();
}
// The same of rows `step` apart, each formed once more with the loop's own operations, for any number
// of doubtful codes; c is the lane's column.
template <int DIM>
__device__ __noinline__ void settle_rows(const GatedParams& p, uint2* notes, int64_t row, int64_t end, int64_t step, int c) {
  const int lane = threadIdx.x & 31, head = c / DIM, d = c % DIM;
  const bool in = c < p.cols;
  float2 w[4], y[4], f[4];
  if (p.w) load_weights(p, d, w);
  for (; row < end; row += step) {
    uint4 x = make_uint4(0u, 0u, 0u, 0u), z = x;
    if (in) {
      x = *reinterpret_cast<const uint4*>(p.x + row * p.xt + head * p.xh + d);
      z = *reinterpret_cast<const uint4*>(p.z + row * p.zt + head * p.zh + d);
    }
    row_values<DIM>(p, x, z, w, y);
    float sc, inv;
    const float am = group_scale(y, sc, inv);
    quotients(y, inv, f);
    uint32_t near = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (in && may_be_near(am) && is_near(e & 1 ? f[e >> 1].y : f[e >> 1].x)) near |= 1u << e;
    const uint32_t top = group_top(y, am, lane);
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      const uint32_t ones = __ballot_sync(0xffffffffu, near >> e & 1u);
      for (int done = 0; done < __popc(ones); done += kNotes) {
        const int at = __popc(ones & ((1u << lane) - 1)) - done;
        if ((near >> e & 1u) && at >= 0 && at < kNotes) notes[at] = make_uint2(static_cast<uint32_t>(row), top << 8 | (8 * lane + e));
        settle<DIM>(p, notes, __popc(ones) - done, c - 8 * lane);
      }
    }
  }
}

// A warp takes 256 columns, 8 a lane, of one token after the other: a head of DIM columns is
// DIM / 8 consecutive lanes, a group of 128 columns 16, so both reductions stay in the warp,
// and the weights stay in registers. A lane copies its 16 bytes of the next tokens to places of
// its own in shared memory, four ahead, and waits for nobody else.
//
// Codes that FP32 may have missed are noted in shared memory and settled behind the warp's last row,
// two lanes each (one in 60,000 is noted; where a warp has a 17th, all of its rows are looked through
// again, so that a row's codes are its own, whatever is beside it): a call inside the loop, though
// never taken, cost the loop 14 of 62 us. A row that its own output overwrites (IN_PLACE) cannot wait,
// and has room for as many notes as codes; with that call in the loop, three blocks an SM of 80 registers
// each take 58 us (codes and rows), four of 64, which spill, 64.
template <int DIM, bool IN_PLACE>
__global__ void __launch_bounds__(kGatedThreads, IN_PLACE ? 3 : 4) gated_norm_kernel(const __grid_constant__ GatedParams p) {
  __shared__ alignas(16) uint4 ring[kGatedAhead][2][kGatedThreads];
  constexpr int kRoom = IN_PLACE ? 256 : kNotes;       // a row's codes, or a few of the warp's rows'
  __shared__ uint2 doubtful[kGatedThreads / 32 * kRoom];
  const int lane = threadIdx.x & 31;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * (kGatedThreads / 32) + (threadIdx.x >> 5);
  const int64_t step = p.warps / p.segs;               // tokens between a warp's: p.warps is a multiple of segs
  const int c = (static_cast<int>(at % p.segs) * 32 + lane) * 8;
  const bool in = c < p.cols;
  const int head = c / DIM, d = c % DIM;
  pdl_wait();
  pdl_launch_dependents();
  int64_t row = at / p.segs;
  if (at >= p.warps || row >= p.tokens) return;
  const __nv_bfloat16* px = p.x + row * p.xt + head * p.xh + d;
  const __nv_bfloat16* pz = p.z + row * p.zt + head * p.zh + d;
  __nv_bfloat16* po = p.out + row * p.ot + head * p.oh + d;
  uint8_t* pq = p.q + row * p.ldq + c;
  float* ps = p.s + row * p.ssm + (c >> 7) * p.sskb;
  int64_t asked = row;
  const uint32_t place = smem_u32(&ring[0][0][threadIdx.x]);
  if (!in) {                                           // lanes past the last column take zeros for ever
#pragma unroll
    for (int s = 0; s < kGatedAhead; ++s) ring[s][0][threadIdx.x] = ring[s][1][threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
  }
  auto ask = [&](int s) {
    if (in && asked < p.tokens) {
      cp_async16(place + s * static_cast<uint32_t>(sizeof(ring[0])), px);
      cp_async16(place + s * static_cast<uint32_t>(sizeof(ring[0])) + static_cast<uint32_t>(sizeof(ring[0][0])), pz);
    }
    cp_async_commit();
    asked += step, px += step * p.xt, pz += step * p.zt;
  };
#pragma unroll
  for (int s = 0; s < kGatedAhead; ++s) ask(s);
  float2 w[4];
  if (p.w) load_weights(p, d, w);
  uint2* const notes = doubtful + (threadIdx.x >> 5) * kRoom;
  int count = 0;
  for (int s = 0; row < p.tokens; s = (s + 1) % kGatedAhead, row += step) {
    cp_async_wait_group<kGatedAhead - 1>();
    const uint4 xr = lds128(place + s * static_cast<uint32_t>(sizeof(ring[0])));
    const uint4 zr = lds128(place + s * static_cast<uint32_t>(sizeof(ring[0])) + static_cast<uint32_t>(sizeof(ring[0][0])));
    ask(s);
    float2 y[4];
    row_values<DIM>(p, xr, zr, w, y);
    if (p.q) {
      float sc, inv;
      const float am = group_scale(y, sc, inv);
      float2 f[4];
      quotients(y, inv, f);
      uint2 cw;
      cw.x = static_cast<uint32_t>(f32x2_to_e4m3x2(f[0].x, f[0].y)) | (static_cast<uint32_t>(f32x2_to_e4m3x2(f[1].x, f[1].y)) << 16);
      cw.y = static_cast<uint32_t>(f32x2_to_e4m3x2(f[2].x, f[2].y)) | (static_cast<uint32_t>(f32x2_to_e4m3x2(f[3].x, f[3].y)) << 16);
      const uint32_t near = min(min(min(from_tie(f[0].x), from_tie(f[0].y)), min(from_tie(f[1].x), from_tie(f[1].y))),
                                min(min(from_tie(f[2].x), from_tie(f[2].y)), min(from_tie(f[3].x), from_tie(f[3].y))));
      if (in) {
        if ((lane & 15) == 0) *ps = sc;
        *reinterpret_cast<uint2*>(pq) = cw;
      }
      const bool near_one = near <= kBothSides && in && may_be_near(am);
      if (__any_sync(0xffffffffu, near_one)) {
        const uint32_t top = group_top(y, am, lane);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool one = near_one && is_near(e & 1 ? f[e >> 1].y : f[e >> 1].x);
          const uint32_t ones = __ballot_sync(0xffffffffu, one);
          const int at = count + __popc(ones & ((1u << lane) - 1));
          if (one && at < kRoom) notes[at] = make_uint2(static_cast<uint32_t>(row), top << 8 | (8 * lane + e));
          count += __popc(ones);
        }
        if (IN_PLACE) {
          int done = 0;
#pragma unroll 1
          do {
            settle<DIM>(p, notes + done, count - done, c - 8 * lane);
          } while ((done += kNotes) < count);
          count = 0;
        }
      }
    }
    if (p.out && in)
      *reinterpret_cast<uint4*>(po) =
          make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y), pack_bf16x2(y[2].x, y[2].y),
                     pack_bf16x2(y[3].x, y[3].y));
    po += step * p.ot, pq += step * p.ldq, ps += step * p.ssm;
  }
  if (IN_PLACE || count == 0) return;
  if (count <= kNotes) settle<DIM>(p, notes, count, c - 8 * lane);
  else settle_rows<DIM>(p, notes, at / p.segs, p.tokens, step, c);
}

bool off16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

}  // namespace

int launch_gated_norm(const bfp8_gated_norm_args& a, void* stream) {
  if (a.tokens < 0 || a.heads < 0) return BFP8_ERR_INVALID_ARG;
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return BFP8_ERR_UNSUPPORTED;
  if (a.tokens == 0 || a.heads == 0) return BFP8_OK;
  if (a.heads > (1 << 20)) return BFP8_ERR_UNSUPPORTED;
  const int64_t D = a.head_dim, cols = a.heads * D, groups = (cols + 127) / 128;
  if (!a.x_bf16 || !a.gate_bf16 || (!a.out_bf16 && !a.q_e4m3)) return BFP8_ERR_INVALID_ARG;
  if (a.gate_act != BFP8_ACT_SILU && a.gate_act != BFP8_ACT_SIGMOID) return BFP8_ERR_INVALID_ARG;
  const int64_t strides[6] = {a.x_stride_token,    a.x_stride_head,
                              a.gate_stride_token, a.gate_stride_head,
                              a.out_bf16 ? a.out_stride_token : D, a.out_bf16 ? a.out_stride_head : D};
  for (int64_t s : strides)
    if (s < D) return BFP8_ERR_INVALID_ARG;
  if (a.q_e4m3 && (!a.scales || a.ldq < cols || a.s_stride_m < 0 || a.s_stride_kb < 0 ||
                   (a.tokens > 1 && a.s_stride_m == 0) || (groups > 1 && a.s_stride_kb == 0)))
    return BFP8_ERR_INVALID_ARG;
  if (!(a.eps >= 0.0f)) return BFP8_ERR_INVALID_ARG;
  if (a.weight && a.w_dtype != BFP8_DT_BF16 && a.w_dtype != BFP8_DT_F32) return BFP8_ERR_SCALE_DTYPE;
  for (int64_t s : strides)
    if (s % 8) return BFP8_ERR_UNSUPPORTED;
  if (off16(a.x_bf16) || off16(a.gate_bf16) || off16(a.weight) || off16(a.out_bf16) ||
      (a.q_e4m3 && (a.ldq % 8 || reinterpret_cast<uintptr_t>(a.q_e4m3) % 8)))
    return BFP8_ERR_UNSUPPORTED;
  // over its own input, but laid out otherwise: rows would go before they are read
  for (int i = 0; i < 2; ++i)
    if (a.out_bf16 && a.out_bf16 == (i ? a.gate_bf16 : a.x_bf16) &&
        ((a.tokens > 1 && strides[2 * i] != strides[4]) || (a.heads > 1 && strides[2 * i + 1] != strides[5])))
      return BFP8_ERR_INVALID_ARG;
  int rc = check_device_ptrs({a.x_bf16, a.gate_bf16, a.weight, a.out_bf16, a.q_e4m3,
                              a.q_e4m3 ? a.scales : nullptr});
  if (rc != BFP8_OK) return rc;
  GatedParams p{};
  p.x = static_cast<const __nv_bfloat16*>(a.x_bf16);
  p.z = static_cast<const __nv_bfloat16*>(a.gate_bf16);
  p.w = a.weight;
  p.out = static_cast<__nv_bfloat16*>(a.out_bf16);
  p.q = static_cast<uint8_t*>(a.q_e4m3);
  p.s = a.scales;
  p.xt = a.x_stride_token, p.xh = a.x_stride_head;
  p.zt = a.gate_stride_token, p.zh = a.gate_stride_head;
  p.ot = a.out_stride_token, p.oh = a.out_stride_head;
  p.ldq = a.ldq, p.ssm = a.s_stride_m, p.sskb = a.s_stride_kb;
  p.cols = static_cast<int32_t>(cols);
  p.segs = static_cast<int32_t>((cols + 255) / 256);
  p.w_f32 = a.w_dtype == BFP8_DT_F32;
  p.is_sigmoid = a.gate_act == BFP8_ACT_SIGMOID;
  p.eps = a.eps;
  p.w_offset = a.weight_offset;
  p.tokens = a.tokens;
  int sms = 0;
  rc = sm_count(&sms);
  if (rc != BFP8_OK) return rc;
  // A warp to each 256 columns of a token, up to 96 warps an SM, three times what is resident:
  // later blocks fill in where earlier ones end (8192 x 48 heads, before codes were
  // settled: 51, 45, 44, 49 us with 32, 64, 128 and 256).
  constexpr int kPer = kGatedThreads / 32, kFit = 96;  // warps of a block, and of an SM
  int64_t rows = (int64_t{sms} * kFit + p.segs - 1) / p.segs;
  rows = rows < a.tokens ? rows : a.tokens;
  p.warps = rows * p.segs;
  const int64_t blocks = (p.warps + kPer - 1) / kPer;
  if (blocks > 0x7FFFFFFF) return BFP8_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(blocks));
  const bool in_place = a.out_bf16 && a.q_e4m3 && (a.out_bf16 == a.x_bf16 || a.out_bf16 == a.gate_bf16);
  auto launch = [&](auto kernel, auto kernel_in_place) {
    return launch_dependent(in_place ? kernel_in_place : kernel, grid, kGatedThreads, 0, st, p);
  };
  switch (a.head_dim) {
    case 64: return launch(gated_norm_kernel<64, false>, gated_norm_kernel<64, true>);
    case 128: return launch(gated_norm_kernel<128, false>, gated_norm_kernel<128, true>);
    default: return launch(gated_norm_kernel<256, false>, gated_norm_kernel<256, true>);
  }
}

}  // namespace bfp8
