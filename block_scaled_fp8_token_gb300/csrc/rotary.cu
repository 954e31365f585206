// rotary.cu -- rotary positions of one to four axes on the heads of the step's queries and
// keys, with the heads' norm ahead of them where a model has one:
//
//   x <- x * rsqrt(mean(x^2) + eps) * (w + offset)                         (w absent: x)
//   angle_i = positions[axis(i)][t] * inv_freq[i]       i = 0 .. rotary_dim / 2 - 1
//   (a, b) <- factor * (a cos - b sin, b cos + a sin)   for the pair (a, b) number i
//
// Pair i is (x[i], x[i + rotary_dim / 2]), or (x[2i], x[2i + 1]) where `adjacent`; columns
// from rotary_dim on are not turned. Bound by HBM: a row is read once and written once.
//
// The angle of a position in the millions leaves a float32 no digits, so it is counted in
// turns: inv_freq / (2 pi) as a 64-bit binary fraction, times the position modulo 2^64,
// which drops whole turns without a rounding. What is rounded is the fraction (2^-64 of a
// turn for each position) and its top 32 bits' conversion to float32 (2^-25 of half a turn).
#include "hybrid_layer.cuh"

namespace bfp8 {
namespace {

using namespace dev;

constexpr int kRotaryThreads = 256;

struct RotaryTensor {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  const void* w;
  int64_t xt, xh, ot, oh;
  int32_t heads, groups;   // groups of 256 / DIM heads
};
struct RotaryParams {
  RotaryTensor t[2];       // queries, keys
  const int32_t* positions;
  const float* inv_freq;
  int64_t ldp, tokens;
  int32_t axes, half, split, w_f32, interleaved;
  int32_t end[4];          // sections: of one behind another the ends; in turns, the lengths
  float eps, w_offset, factor;
};

// 1 / (2 pi) as a binary fraction: bits 1-32, 33-64 and 65-96.
constexpr uint64_t kTurn0 = 0x28BE60DBu, kTurn1 = 0x9391054Au, kTurn2 = 0x7F09D5F4u;

// f / (2 pi) modulo 1 in units of 2^-64, for |f| < 2^32: f = m 2^e with a 24-bit m, and m's
// 120-bit product with the 96 bits above is shifted into place.
BFP8_DEV uint64_t turns_of(float f) {
  const uint32_t bits = __float_as_uint(f);
  const int ex = (bits >> 23) & 0xFF;
  const uint64_t m = ex ? (bits & 0x7FFFFFu) | 0x800000u : bits & 0x7FFFFFu;
  const int e = (ex ? ex : 1) - 150;               // f = m 2^e
  const uint64_t p2 = m * kTurn2, p1 = m * kTurn1 + (p2 >> 32), p0 = m * kTurn0 + (p1 >> 32);
  // the product in units of 2^-96: p0 : low word of p1 : low word of p2
  const uint64_t hi = p0 >> 32, lo = (p0 << 32) | (p1 & 0xFFFFFFFFu);   // hi : lo . (p2), units 2^-64
  uint64_t r;
  if (e >= 0) {                                    // 2^23 <= |f| < 2^32, e < 9
    r = (lo << e) | (e ? (p2 & 0xFFFFFFFFu) >> (32 - e) : 0u);
  } else {
    const int s = -e;
    r = s < 64 ? (lo >> s) | (hi << (64 - s)) : s < 128 ? hi >> (s - 64) : 0;
  }
  return bits >> 31 ? 0 - r : r;
}

template <int DIM>
BFP8_DEV void load_norm_weight(const RotaryParams& p, const void* w, int d, float (&v)[8]) {
  if (p.w_f32) {
    const float* f = static_cast<const float*>(w) + d;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __ldg(f + e);
  } else {
    widen8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + d)), v);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] += p.w_offset;
}

// A warp takes 256 / DIM heads of one token at a time, 8 columns a lane, and `split` warps
// share a token's heads. Its angles' sines and cosines are formed once and serve all of the
// warp's heads. The partner of a lane's columns is in the lane half / 8 away.
template <int DIM, bool ADJACENT>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryParams p) {
  __shared__ uint64_t turns[DIM / 2];
  __shared__ uint8_t axis[DIM / 2];
  pdl_wait();
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < p.half; i += kRotaryThreads) {
    turns[i] = turns_of(__ldg(p.inv_freq + i));
    int a = 0;
    if (p.interleaved) {
      a = i % p.axes;
      if (i / p.axes >= p.end[a]) a = 0;
    } else {
      while (a + 1 < p.axes && i >= p.end[a]) ++a;
    }
    axis[i] = static_cast<uint8_t>(a);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kRotaryThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = item / p.split;
  if (t >= p.tokens) return;
  int32_t pos[4] = {};
  for (int a = 0; a < p.axes; ++a) {
    pos[a] = __ldg(p.positions + a * p.ldp + t);
    if (pos[a] < 0) return;                        // a row of no request
  }
  constexpr int kLanes = DIM / 8;                  // of one head
  constexpr int N = ADJACENT ? 4 : 8;              // angles a lane needs
  const int d = (lane % kLanes) * 8, half = p.half;
  const bool turned = d < 2 * half;
  const bool second = !ADJACENT && d >= half;
  const int partner = (lane & ~(kLanes - 1)) + (((second ? d - half : d + half) & (DIM - 1)) >> 3);
  float cs[N], sn[N];
  if (turned) {
    const int first = ADJACENT ? d / 2 : second ? d - half : d;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int a = axis[first + j];
      const uint32_t at = a == 0 ? pos[0] : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3];
      const uint64_t phase = at * turns[first + j];
      const float x = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
      sincospif(x, &sn[j], &cs[j]);
      const float f = __ldg(p.inv_freq + first + j);
      if (!(fabsf(f) < 0x1p32f)) sn[j] = cs[j] = __int_as_float(0x7FFFFFFF);
      cs[j] *= p.factor;
      sn[j] *= second ? p.factor : -p.factor;      // what the partner is multiplied by
    }
  }
  const int all = p.t[0].groups + p.t[1].groups;
  for (int g = static_cast<int>(item - t * p.split); g < all; g += p.split) {
    const bool key = g >= p.t[0].groups;
    const RotaryTensor& q = key ? p.t[1] : p.t[0];
    const int head = (key ? g - p.t[0].groups : g) * (32 / kLanes) + lane / kLanes;
    const bool in = head < q.heads;
    const uint4 raw = in ? *reinterpret_cast<const uint4*>(q.x + t * q.xt + head * q.xh + d)
                         : make_uint4(0u, 0u, 0u, 0u);
    float x[8], other[8];
    widen8(raw, x);
    if (!ADJACENT) {
      const uint4 r = make_uint4(__shfl_sync(0xffffffffu, raw.x, partner), __shfl_sync(0xffffffffu, raw.y, partner),
                                 __shfl_sync(0xffffffffu, raw.z, partner), __shfl_sync(0xffffffffu, raw.w, partner));
      widen8(r, other);
    }
    if (q.w) {
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(fmaf(ss, 1.0f / DIM, p.eps));
      float w[8];
      load_norm_weight<DIM>(p, q.w, d, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= r * w[e];
      if (!ADJACENT) {
        load_norm_weight<DIM>(p, q.w, (partner % kLanes) * 8, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) other[e] *= r * w[e];
      }
    }
    if (turned) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (ADJACENT) {
          const float a = x[2 * j], b = x[2 * j + 1];
          x[2 * j] = fmaf(b, sn[j], a * cs[j]);    // sn holds -sin
          x[2 * j + 1] = fmaf(-a, sn[j], b * cs[j]);
        } else {
          x[j] = fmaf(other[j], sn[j], x[j] * cs[j]);
        }
      }
    }
    if (in) *reinterpret_cast<uint4*>(q.out + t * q.ot + head * q.oh + d) = pack8(x);
  }
}

bool off16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

}  // namespace

int launch_rotary(const bfp8_rotary_args& a, void* stream) {
  if (a.tokens < 0 || a.q_heads < 0 || a.k_heads < 0) return BFP8_ERR_INVALID_ARG;
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return BFP8_ERR_UNSUPPORTED;
  const int64_t D = a.head_dim;
  if (a.rotary_dim < 2 || a.rotary_dim > D || a.axes < 1 || a.axes > 4) return BFP8_ERR_INVALID_ARG;
  if (a.rotary_dim % 16) return BFP8_ERR_UNSUPPORTED;
  const int32_t half = a.rotary_dim / 2;
  int64_t pairs = 0;
  for (int i = 0; i < a.axes; ++i) {
    if (a.sections[i] < 0 || a.sections[i] > half) return BFP8_ERR_INVALID_ARG;
    pairs += a.sections[i];
  }
  if (pairs != half) return BFP8_ERR_INVALID_ARG;
  if (a.tokens == 0 || (a.q_heads == 0 && a.k_heads == 0)) return BFP8_OK;
  if (!a.positions || !a.inv_freq || (a.axes > 1 && a.ld_positions < a.tokens)) return BFP8_ERR_INVALID_ARG;
  if ((a.q_heads > 0 && (!a.q_bf16 || !a.q_out_bf16)) || (a.k_heads > 0 && (!a.k_bf16 || !a.k_out_bf16)))
    return BFP8_ERR_INVALID_ARG;
  if (!(a.eps >= 0.0f) || !(a.factor > -3.0e38f && a.factor < 3.0e38f)) return BFP8_ERR_INVALID_ARG;
  if ((a.q_weight || a.k_weight) && a.w_dtype != BFP8_DT_BF16 && a.w_dtype != BFP8_DT_F32)
    return BFP8_ERR_SCALE_DTYPE;
  const int64_t strides[2][4] = {{a.q_stride_token, a.q_stride_head, a.q_out_stride_token, a.q_out_stride_head},
                                 {a.k_stride_token, a.k_stride_head, a.k_out_stride_token, a.k_out_stride_head}};
  for (int i = 0; i < 2; ++i) {
    if ((i ? a.k_heads : a.q_heads) == 0) continue;
    for (int64_t s : strides[i])
      if (s < D) return BFP8_ERR_INVALID_ARG;
    for (int64_t s : strides[i])
      if (s % 8) return BFP8_ERR_UNSUPPORTED;
  }
  if (off16(a.q_bf16) || off16(a.q_out_bf16) || off16(a.k_bf16) || off16(a.k_out_bf16) ||
      off16(a.q_weight) || off16(a.k_weight) || a.q_heads > (1 << 20) || a.k_heads > (1 << 20))
    return BFP8_ERR_UNSUPPORTED;
  int rc = check_device_ptrs({a.q_heads ? a.q_bf16 : nullptr, a.q_heads ? a.q_out_bf16 : nullptr,
                              a.k_heads ? a.k_bf16 : nullptr, a.k_heads ? a.k_out_bf16 : nullptr,
                              a.positions, a.inv_freq, a.q_weight, a.k_weight});
  if (rc != BFP8_OK) return rc;
  int sms = 0;
  rc = sm_count(&sms);
  if (rc != BFP8_OK) return rc;
  RotaryParams p{};
  const int per = static_cast<int>(256 / D);
  p.t[0] = {static_cast<const __nv_bfloat16*>(a.q_bf16), static_cast<__nv_bfloat16*>(a.q_out_bf16), a.q_weight,
            a.q_stride_token, a.q_stride_head, a.q_out_stride_token, a.q_out_stride_head,
            static_cast<int32_t>(a.q_heads), static_cast<int32_t>((a.q_heads + per - 1) / per)};
  p.t[1] = {static_cast<const __nv_bfloat16*>(a.k_bf16), static_cast<__nv_bfloat16*>(a.k_out_bf16), a.k_weight,
            a.k_stride_token, a.k_stride_head, a.k_out_stride_token, a.k_out_stride_head,
            static_cast<int32_t>(a.k_heads), static_cast<int32_t>((a.k_heads + per - 1) / per)};
  p.positions = a.positions;
  p.inv_freq = a.inv_freq;
  p.ldp = a.axes > 1 ? a.ld_positions : 0;
  p.tokens = a.tokens;
  p.axes = a.axes;
  p.half = half;
  p.interleaved = a.interleaved != 0;
  for (int i = 0, at = 0; i < a.axes; ++i) p.end[i] = p.interleaved ? a.sections[i] : at += a.sections[i];
  p.w_f32 = a.w_dtype == BFP8_DT_F32;
  p.eps = a.eps;
  p.w_offset = a.weight_offset;
  p.factor = a.factor;
  // few tokens: as many warps share one as fill the GPU, down to a warp a group of heads
  const int64_t groups = p.t[0].groups + p.t[1].groups;
  int64_t split = (int64_t{sms} * 32 + a.tokens - 1) / a.tokens;
  p.split = static_cast<int32_t>(split < groups ? split : groups);
  const int64_t warps = a.tokens * p.split, blocks = (warps + kRotaryThreads / 32 - 1) / (kRotaryThreads / 32);
  if (blocks > 0x7FFFFFFF) return BFP8_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto kernel) { return launch_dependent(kernel, grid, kRotaryThreads, 0, st, p); };
  if (a.adjacent)
    return D == 64 ? go(rotary_kernel<64, true>) : D == 128 ? go(rotary_kernel<128, true>) : go(rotary_kernel<256, true>);
  return D == 64 ? go(rotary_kernel<64, false>) : D == 128 ? go(rotary_kernel<128, false>) : go(rotary_kernel<256, false>);
}

}  // namespace bfp8
