// rotary.cu -- rotary positions of one to four axes on the heads of the step's queries and
// keys, with the heads' norm ahead of them where a model has one:
//
//   x <- x * rsqrt(mean(x^2) + eps) * (w + offset)                         (w absent: x)
//   angle_i = positions[axis(i)][t] * inv_freq[i]       i = 0 .. rotary_dim / 2 - 1
//   (a, b) <- factor * (a cos - b sin, b cos + a sin)   for the pair (a, b) number i
//
// Pair i is (x[i], x[i + rotary_dim / 2]), or (x[2i], x[2i + 1]) where `adjacent`; columns
// from rotary_dim on are not turned. Bound by HBM: a row is read once and written once. 8192
// tokens of 18 normed heads of 256, 151 MB, take 30 us, 5.0 TB/s (54 with the angles formed by
// every lane and one head's loads under way; 38 with the angles shared, 30 with four heads'
// loads); 8000 tokens of 72 heads of 128, 295 MB, 50 us. Few tokens: 2.6 us for one, 3.6 for 64.
// At 64 registers each variant spills 8 bytes a thread, those of adjacent pairs 16 to 28.
//
// The angle of a position in the millions leaves a float32 no digits, so it is counted in
// turns: inv_freq / (2 pi) as a 64-bit binary fraction, times the position modulo 2^64,
// which drops whole turns without a rounding. What is rounded is the fraction (2^-64 of a
// turn for each position) and its top 32 bits' conversion to float32 (2^-25 of half a turn).
#include "hybrid_layer.cuh"

namespace bfp8 {
namespace {

using namespace dev;

constexpr int kRotaryThreads = 256, kRotaryAhead = 4;   // groups of heads whose loads a warp has under way

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
  int32_t axes, half, block_tokens, blocks, w_f32, interleaved;
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

BFP8_DEV float norm_weight(const RotaryParams& p, const void* w, int d) {
  const float v = p.w_f32 ? __ldg(static_cast<const float*>(w) + d)
                          : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(w) + d));
  return v + p.w_offset;
}

// A warp takes 256 / DIM heads of one token at a time, 8 columns a lane. A block has one token
// or several; its sines and cosines are formed once, an angle a thread, and with the norm's
// weights they make two factors a column that serve all of a token's heads:
//   out = r (x cw + partner sw),   r the head's norm factor.
// A column's partner is in the lane half / 8 away, or next to it in the same word.
template <int DIM, bool ADJACENT>
__global__ void __launch_bounds__(kRotaryThreads, 4) rotary_kernel(const RotaryParams p) {
  constexpr int kWarps = kRotaryThreads / 32;
  __shared__ float2 turned_by[kWarps][DIM / 2];    // cosine and sine of each token's pairs
  __shared__ alignas(16) float weight[2][DIM];
  __shared__ alignas(16) uint4 ring[kRotaryAhead][kRotaryThreads];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t block = blockIdx.x / p.blocks;     // of tokens; p.blocks > 1 blocks share one token
  const int per = kWarps / p.block_tokens;         // warps of a token in this block
  const int mine = (tid >> 5) / per;               // the warp's token among the block's
  const int64_t t = block * p.block_tokens + mine;
  const int split = per * p.blocks, first = (tid >> 5) % per * p.blocks + static_cast<int>(blockIdx.x % p.blocks);
  constexpr int kLanes = DIM / 8;                  // of one head
  const int d = (lane % kLanes) * 8, half = p.half;
  const int64_t step = static_cast<int64_t>(split) * (32 / kLanes);
  const uint32_t place = smem_u32(&ring[0][tid]);
  // groups are dealt on from the queries' to the keys'
  const int keys = (first + split - p.t[0].groups % split) % split;
  const __nv_bfloat16* x = nullptr;
  int asked = 0;
  auto ask = [&](const RotaryTensor& q, int s) {   // a lane copies its own columns of a head
    if (asked < q.heads) cp_async16(place + s * static_cast<uint32_t>(sizeof(ring[0])), x);
    cp_async_commit();
    asked += static_cast<int>(step), x += step * q.xh;
  };
  auto begin = [&](const RotaryTensor& q, int g) {
    asked = g * (32 / kLanes) + lane / kLanes;
    x = q.x + t * q.xt + asked * q.xh + d;
#pragma unroll
    for (int s = 0; s < kRotaryAhead; ++s) ask(q, s);
  };
  const bool queries = first < p.t[0].groups;
  if (t < p.tokens && queries) begin(p.t[0], first);   // under way while the angles are formed
  for (int i = tid; i < p.block_tokens * p.half; i += kRotaryThreads) {
    const int k = i / p.half, pair = i - k * p.half;
    if (block * p.block_tokens + k >= p.tokens) break;
    int a = 0;
    if (p.interleaved) {
      a = pair % p.axes;
      if (pair / p.axes >= p.end[a]) a = 0;
    } else {
      while (a + 1 < p.axes && pair >= p.end[a]) ++a;
    }
    const float f = __ldg(p.inv_freq + pair);
    const uint64_t phase = static_cast<uint32_t>(__ldg(p.positions + a * p.ldp + block * p.block_tokens + k)) * turns_of(f);
    float2 cs;
    sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &cs.y, &cs.x);
    if (!(fabsf(f) < 0x1p32f)) cs.x = cs.y = __int_as_float(0x7FFFFFFF);
    turned_by[k][pair] = make_float2(cs.x * p.factor, cs.y * p.factor);
  }
  for (int i = tid; i < 2 * DIM; i += kRotaryThreads) {
    const void* w = i < DIM ? p.t[0].w : p.t[1].w;
    if (w) weight[i / DIM][i % DIM] = norm_weight(p, w, i % DIM);
  }
  __syncthreads();
  if (t >= p.tokens) return;
  for (int a = 0; a < p.axes; ++a)
    if (__ldg(p.positions + a * p.ldp + t) < 0) {  // a row of no request
      cp_async_wait_group<0>();
      return;
    }
  const bool turned = d < 2 * half, second = !ADJACENT && d >= half;
  const int partner = turned ? (lane & ~(kLanes - 1)) + ((second ? d - half : d + half) >> 3) : lane;

  auto walk = [&](const RotaryTensor& q, int g, const float2 (&cw)[4], const float2 (&sw)[4]) {
    int head = g * (32 / kLanes) + lane / kLanes;
    __nv_bfloat16* out = q.out + t * q.ot + head * q.oh + d;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (int s = 0; g < q.groups; g += split, out += step * q.oh, head += static_cast<int>(step), s = (s + 1) % kRotaryAhead) {
      const bool in = head < q.heads;
      cp_async_wait_group<kRotaryAhead - 1>();
      const uint4 raw = in ? lds128(place + s * static_cast<uint32_t>(sizeof(ring[0]))) : zero;
      ask(q, s);
      uint4 other;
      if (ADJACENT) {
        other = make_uint4(__byte_perm(raw.x, 0u, 0x1032), __byte_perm(raw.y, 0u, 0x1032), __byte_perm(raw.z, 0u, 0x1032),
                           __byte_perm(raw.w, 0u, 0x1032));
      } else {
        other = make_uint4(__shfl_sync(0xffffffffu, raw.x, partner), __shfl_sync(0xffffffffu, raw.y, partner),
                           __shfl_sync(0xffffffffu, raw.z, partner), __shfl_sync(0xffffffffu, raw.w, partner));
      }
      if (!turned) other = zero;                   // an infinity there stays one
      const uint32_t xw[4] = {raw.x, raw.y, raw.z, raw.w}, ow[4] = {other.x, other.y, other.z, other.w};
      float2 y[4];
      float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = make_float2(__uint_as_float(xw[e] << 16), __uint_as_float(xw[e] & 0xFFFF0000u));
        const float2 b = make_float2(__uint_as_float(ow[e] << 16), __uint_as_float(ow[e] & 0xFFFF0000u));
        if (q.w) s2 = __ffma2_rn(a, a, s2);
        y[e] = __ffma2_rn(a, cw[e], __fmul2_rn(b, sw[e]));
      }
      if (q.w) {
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(fmaf(ss, 1.0f / DIM, p.eps));
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __fmul2_rn(y[e], make_float2(r, r));
      }
      if (in)
        *reinterpret_cast<uint4*>(out) = make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y),
                                                    pack_bf16x2(y[2].x, y[2].y), pack_bf16x2(y[3].x, y[3].y));
    }
  };

#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const RotaryTensor& q = k ? p.t[1] : p.t[0];
    const int g = k ? keys : first;
    if (g >= q.groups) continue;
    if (k) {
      cp_async_wait_group<0>();                    // the places are free: what the queries asked for has come
      begin(q, g);
    }
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = 1.0f, s[e] = 0.0f;
      if (turned) {
        const float2 cs = turned_by[mine][ADJACENT ? (d + e) >> 1 : second ? d + e - half : d + e];
        c[e] = cs.x;
        s[e] = (ADJACENT ? e & 1 : second) ? cs.y : -cs.y;
      }
      if (q.w) {
        c[e] *= weight[k][d + e];
        if (turned) s[e] *= weight[k][ADJACENT ? (d + e) ^ 1 : second ? d + e - half : d + e + half];
      }
    }
    float2 cw[4], sw[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) cw[e] = make_float2(c[2 * e], c[2 * e + 1]), sw[e] = make_float2(s[2 * e], s[2 * e + 1]);
    walk(q, g, cw, sw);
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
  // over its own input, but laid out otherwise: rows would go before they are read
  for (int i = 0; i < 2; ++i) {
    const int64_t heads = i ? a.k_heads : a.q_heads, *s = strides[i];
    if (heads > 0 && (i ? a.k_bf16 == a.k_out_bf16 : a.q_bf16 == a.q_out_bf16) &&
        ((a.tokens > 1 && s[0] != s[2]) || (heads > 1 && s[1] != s[3])))
      return BFP8_ERR_INVALID_ARG;
  }
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
  // A token's angles are formed by each block that has it: eight tokens to a block, fewer where
  // that leaves SMs without a block, and several blocks to a token where one each does. (A block
  // an SM, two, four: 949 tokens of 72 heads 8.5, 9.6, 10.9 us; 64 tokens 3.7, 4.2, 4.2.)
  const int64_t groups = p.t[0].groups + p.t[1].groups, want = sms;
  p.block_tokens = a.tokens >= 8 * want ? 8 : a.tokens >= 4 * want ? 4 : a.tokens >= 2 * want ? 2 : 1;
  int64_t share = (want + a.tokens - 1) / a.tokens;
  const int64_t most = (groups + kRotaryThreads / 32 - 1) / (kRotaryThreads / 32);
  p.blocks = static_cast<int32_t>(p.block_tokens > 1 ? 1 : share < most ? share : most);
  const int64_t blocks = (a.tokens + p.block_tokens - 1) / p.block_tokens * p.blocks;
  if (blocks > 0x7FFFFFFF) return BFP8_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto kernel) { return launch_dependent(kernel, grid, kRotaryThreads, 0, st, p); };
  if (a.adjacent)
    return D == 64 ? go(rotary_kernel<64, true>) : D == 128 ? go(rotary_kernel<128, true>) : go(rotary_kernel<256, true>);
  return D == 64 ? go(rotary_kernel<64, false>) : D == 128 ? go(rotary_kernel<128, false>) : go(rotary_kernel<256, false>);
}

}  // namespace bfp8
