// gated_norm.cu -- the heads' outputs of a linear-attention layer normed and gated, and
// quantized for the output projection, in one pass:
//
//   y = x * rsqrt(mean(x^2) + eps) * (w + offset) * act(z)     per token and head
//   out = bf16(y);  s = max(max|y|, 1e-10f) / 448 per 128 columns of a token's heads,
//   q = RNE_satfinite_e4m3(y / s)
//
// act is SiLU or the sigmoid; without w there is no norm (the gate of a full-attention
// layer's heads). Bound by HBM: x and z are read once, and the codes (a quarter of the
// bytes) or the BF16 row written once.
#include "hybrid_layer.cuh"

namespace bfp8 {
namespace {

using namespace dev;

constexpr int kGatedThreads = 256;

struct GatedParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* z;
  const void* w;
  __nv_bfloat16* out;
  uint8_t* q;
  float* s;
  int64_t xt, xh, zt, zh, ot, oh, ldq, ssm, sskb, items;
  int32_t cols, segs, w_f32, is_sigmoid;
  float eps, w_offset;
};

// A warp takes 256 columns of one token, 8 a lane: a head of DIM columns is DIM / 8
// consecutive lanes, a group of 128 columns 16, so both reductions stay in the warp.
template <int DIM>
__global__ void __launch_bounds__(kGatedThreads) gated_norm_kernel(const GatedParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kGatedThreads / 32) + (threadIdx.x >> 5);
  if (item >= p.items) return;
  const int64_t row = item / p.segs;
  const int lane = threadIdx.x & 31;
  const int c = (static_cast<int>(item - row * p.segs) * 32 + lane) * 8;
  const bool in = c < p.cols;
  const int head = c / DIM, d = c % DIM;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint4 xr = in ? *reinterpret_cast<const uint4*>(p.x + row * p.xt + head * p.xh + d) : zero;
  const uint4 zr = in ? *reinterpret_cast<const uint4*>(p.z + row * p.zt + head * p.zh + d) : zero;
  float y[8], z[8];
  widen8(xr, y);
  widen8(zr, z);
  if (p.w) {
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
    for (int o = DIM / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(fmaf(ss, 1.0f / DIM, p.eps));
    float w[8];
    if (p.w_f32) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.w) + d));
      const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.w) + d + 4));
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
      widen8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.w) + d)), w);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= r * (w[e] + p.w_offset);
  }
  float am = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y[e] *= p.is_sigmoid ? sigmoid(z[e]) : silu(z[e]);
    am = fmaxf(am, fabsf(y[e]));
  }
  if (p.out && in) *reinterpret_cast<uint4*>(p.out + row * p.ot + head * p.oh + d) = pack8(y);
  if (!p.q) return;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  const float sc = __fdiv_rn(fmaxf(am, 1e-10f), 448.0f), inv = __frcp_rn(sc);
  if (!in) return;
  if ((lane & 15) == 0) p.s[row * p.ssm + (c >> 7) * p.sskb] = sc;
  uint32_t cw[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    cw[j] = static_cast<uint32_t>(f32x2_to_e4m3x2(y[4 * j] * inv, y[4 * j + 1] * inv)) |
            (static_cast<uint32_t>(f32x2_to_e4m3x2(y[4 * j + 2] * inv, y[4 * j + 3] * inv)) << 16);
  *reinterpret_cast<uint2*>(p.q + row * p.ldq + c) = make_uint2(cw[0], cw[1]);
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
  p.items = a.tokens * p.segs;
  p.w_f32 = a.w_dtype == BFP8_DT_F32;
  p.is_sigmoid = a.gate_act == BFP8_ACT_SIGMOID;
  p.eps = a.eps;
  p.w_offset = a.weight_offset;
  const int64_t blocks = (p.items + kGatedThreads / 32 - 1) / (kGatedThreads / 32);
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
