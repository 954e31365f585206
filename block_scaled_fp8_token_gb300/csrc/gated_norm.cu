// gated_norm.cu -- the heads' outputs of a linear-attention layer normed and gated, and
// quantized for the output projection, in one pass:
//
//   y = x * rsqrt(mean(x^2) + eps) * (w + offset) * act(z)     per token and head
//   out = bf16(y);  s = max(max|y|, 1e-10f) / 448 per 128 columns of a token's heads,
//   q = RNE_satfinite_e4m3(y / s)
//
// act is SiLU or the sigmoid; without w there is no norm (the gate of a full-attention
// layer's heads). Bound by HBM: x and z are read once, and the codes (a quarter of the
// bytes) or the BF16 row written once. 8192 rows of 48 heads to codes, 253 MB, take 44 us, 5.8
// TB/s; with one token's loads ahead in registers, 32 warps an SM had too few bytes under way
// (55 us), and without any 67.
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

// A warp takes 256 columns, 8 a lane, of one token after the other: a head of DIM columns is
// DIM / 8 consecutive lanes, a group of 128 columns 16, so both reductions stay in the warp,
// and the weights stay in registers. A lane copies its 16 bytes of the next tokens to places of
// its own in shared memory, four ahead, and waits for nobody else.
template <int DIM>
__global__ void __launch_bounds__(kGatedThreads, 4) gated_norm_kernel(const GatedParams p) {
  __shared__ alignas(16) uint4 ring[kGatedAhead][2][kGatedThreads];
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
  if (p.w) {
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
  for (int s = 0; row < p.tokens; s = (s + 1) % kGatedAhead, row += step) {
    float x[8], z[8];
    cp_async_wait_group<kGatedAhead - 1>();
    widen8(lds128(place + s * static_cast<uint32_t>(sizeof(ring[0]))), x);
    widen8(lds128(place + s * static_cast<uint32_t>(sizeof(ring[0])) + static_cast<uint32_t>(sizeof(ring[0][0]))), z);
    ask(s);
    float2 y[4];
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
    float am = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = z[2 * e], b = z[2 * e + 1];
      float2 g = make_float2(sigmoid_bf16(a), sigmoid_bf16(b));
      if (!p.is_sigmoid) g = __fmul2_rn(g, make_float2(a, b));
      y[e] = __fmul2_rn(y[e], g);
      am = fmaxf(am, fmaxf(fabsf(y[e].x), fabsf(y[e].y)));
    }
    if (p.out && in)
      *reinterpret_cast<uint4*>(po) =
          make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y), pack_bf16x2(y[2].x, y[2].y),
                     pack_bf16x2(y[3].x, y[3].y));
    if (p.q) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
      // am / 448 rounded (its remainder is exact), and 1 / s within 2^-23
      am = fmaxf(am, 1e-10f);
      float sc = am * (1.0f / 448.0f);
      if (am <= 3.0e38f) sc = fmaf(fmaf(-448.0f, sc, am), 1.0f / 448.0f, sc);
      float inv = rcp_approx(sc);
      if (am <= 3.0e38f) inv = fmaf(fmaf(-sc, inv, 1.0f), inv, inv);
      if (in) {
        if ((lane & 15) == 0) *ps = sc;
        uint32_t cw[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f = __fmul2_rn(y[2 * j], make_float2(inv, inv)), g = __fmul2_rn(y[2 * j + 1], make_float2(inv, inv));
          cw[j] = static_cast<uint32_t>(f32x2_to_e4m3x2(f.x, f.y)) | (static_cast<uint32_t>(f32x2_to_e4m3x2(g.x, g.y)) << 16);
        }
        *reinterpret_cast<uint2*>(pq) = make_uint2(cw[0], cw[1]);
      }
    }
    po += step * p.ot, pq += step * p.ldq, ps += step * p.ssm;
  }
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
  // later blocks fill in where earlier ones end (8192 x 48 heads: 51, 45, 44, 49 us with 32, 64,
  // 128 and 256).
  constexpr int kPer = kGatedThreads / 32, kFit = 96;  // warps of a block, and of an SM
  int64_t rows = (int64_t{sms} * kFit + p.segs - 1) / p.segs;
  rows = rows < a.tokens ? rows : a.tokens;
  p.warps = rows * p.segs;
  const int64_t blocks = (p.warps + kPer - 1) / kPer;
  if (blocks > 0x7FFFFFFF) return BFP8_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(blocks));
  switch (a.head_dim) {
    case 64: return launch_dependent(gated_norm_kernel<64>, grid, kGatedThreads, 0, st, p);
    case 128: return launch_dependent(gated_norm_kernel<128>, grid, kGatedThreads, 0, st, p);
    default: return launch_dependent(gated_norm_kernel<256>, grid, kGatedThreads, 0, st, p);
  }
}

}  // namespace bfp8
