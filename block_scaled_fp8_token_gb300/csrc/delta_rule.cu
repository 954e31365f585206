// delta_rule.cu -- the gated delta rule of a linear-attention layer over the ragged tokens
// of a step, with each request's state kept between steps. Per value head, with the state S
// of 128 values by 128 keys, and per token
//
//   alpha = exp(-exp(a_log) softplus(a + dt_bias)),  beta = sigmoid(b)
//   k' = k rsqrt(|k|^2 + eps),  q' = scale q rsqrt(|q|^2 + eps)
//   u = beta (v - alpha S k'),  S <- alpha S + u k'^T,  out = S q'
//
// in FP32; only out is rounded, once, to BF16.
#include "hybrid_layer.cuh"

namespace bfp8 {
namespace {

using namespace dev;

constexpr int kD = 128;

struct DeltaParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* a;
  const __nv_bfloat16* b;
  const float* a_log;
  const float* dt_bias;
  float* state;
  __nv_bfloat16* out;
  int64_t qt, qh, kt, kh, vt, vh, at, bt, ot, oh, s_slot, s_head, max_len;
  Requests req;
  int32_t v_heads, group;
  float scale, eps;
};

// The logarithm of a token's decay, -exp(a_log) softplus(a + dt_bias). (A softplus above 20
// is its argument to FP32's last place.)
BFP8_DEV float log_decay(float a, float dt_bias, float rate) {
  const float z = a + dt_bias;
  return -rate * (z > 20.0f ? z : log1pf(expf(z)));
}
BFP8_DEV float beta_of(float b) { return 1.0f / (1.0f + expf(-b)); }

BFP8_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Eight sums over the warp at once: sum r is left in lanes 4r .. 4r + 3.
BFP8_DEV float warp_sum8(float (&v)[8], int lane) {
#pragma unroll
  for (int n = 4, o = 16; n > 0; n >>= 1, o >>= 1) {
#pragma unroll
    for (int r = 0; r < n; ++r) {
      const float give = lane & o ? v[r] : v[r + n], keep = lane & o ? v[r + n] : v[r];
      v[r] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

constexpr int kStepWarps = 4;

// One token after the other: a warp holds 8 of a head's 128 rows of S, four columns a lane,
// and needs no other warp. Both products with the old state are summed at once, as
// S_new q' = alpha S q' + u (k' . q').
__global__ void __launch_bounds__(32 * kStepWarps) delta_step_kernel(const DeltaParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kParts = kD / (8 * kStepWarps);
  const int lane = threadIdx.x & 31;
  const int64_t item = blockIdx.x / kParts;
  const int b = static_cast<int>(item / p.v_heads), h = static_cast<int>(item - int64_t{b} * p.v_heads);
  const int row0 = (static_cast<int>(blockIdx.x % kParts) * kStepWarps + (threadIdx.x >> 5)) * 8;
  const int64_t first = first_token(p.req, b);
  int64_t n = first_token(p.req, b + 1) - first;
  n = n < p.max_len ? n : p.max_len;
  if (n <= 0) return;
  const int64_t from = slot_of(p.req, p.req.slots_in, b), to = slot_of(p.req, p.req.slots_out, b);
  const int64_t in_head = h * p.s_head + row0 * kD + lane * 4;
  float4 S[8];
  if (from >= 0) {
    const float* s = p.state + from * p.s_slot + in_head;
#pragma unroll
    for (int r = 0; r < 8; ++r) S[r] = *reinterpret_cast<const float4*>(s + r * kD);
  } else {
#pragma unroll
    for (int r = 0; r < 8; ++r) S[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  const float rate = expf(__ldg(p.a_log + h)), dt_bias = __ldg(p.dt_bias + h);
  const int hk = h / p.group;
  const __nv_bfloat16* qp = p.q + first * p.qt + hk * p.qh + lane * 4;
  const __nv_bfloat16* kp = p.k + first * p.kt + hk * p.kh + lane * 4;
  const __nv_bfloat16* vp = p.v + first * p.vt + h * p.vh + row0 + (lane >> 2);
  const __nv_bfloat16* ap = p.a + first * p.at + h;
  const __nv_bfloat16* bp = p.b + first * p.bt + h;
  __nv_bfloat16* op = p.out + first * p.ot + h * p.oh + row0 + (lane >> 2);
  uint2 kr = *reinterpret_cast<const uint2*>(kp), qr = *reinterpret_cast<const uint2*>(qp);
  __nv_bfloat16 vr = *vp, ar = *ap, br = *bp;
  for (int64_t t = 0; t < n; ++t) {
    float k[4] = {__uint_as_float(kr.x << 16), __uint_as_float(kr.x & 0xFFFF0000u),
                  __uint_as_float(kr.y << 16), __uint_as_float(kr.y & 0xFFFF0000u)};
    float q[4] = {__uint_as_float(qr.x << 16), __uint_as_float(qr.x & 0xFFFF0000u),
                  __uint_as_float(qr.y << 16), __uint_as_float(qr.y & 0xFFFF0000u)};
    const float v = __bfloat162float(vr);
    const float alpha = expf(log_decay(__bfloat162float(ar), dt_bias, rate)), beta = beta_of(__bfloat162float(br));
    if (t + 1 < n) {   // the next token's inputs, a token ahead of their use
      kp += p.kt, qp += p.qt, vp += p.vt, ap += p.at, bp += p.bt;
      kr = *reinterpret_cast<const uint2*>(kp), qr = *reinterpret_cast<const uint2*>(qp);
      vr = *vp, ar = *ap, br = *bp;
    }
    const float kn = rsqrtf(warp_sum(fmaf(k[0], k[0], fmaf(k[1], k[1], fmaf(k[2], k[2], k[3] * k[3])))) + p.eps);
    const float qn = rsqrtf(warp_sum(fmaf(q[0], q[0], fmaf(q[1], q[1], fmaf(q[2], q[2], q[3] * q[3])))) + p.eps) * p.scale;
#pragma unroll
    for (int e = 0; e < 4; ++e) k[e] *= kn, q[e] *= qn;
    const float kq = warp_sum(fmaf(k[0], q[0], fmaf(k[1], q[1], fmaf(k[2], q[2], k[3] * q[3]))));
    float sk[8], sq[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      sk[r] = fmaf(S[r].x, k[0], fmaf(S[r].y, k[1], fmaf(S[r].z, k[2], S[r].w * k[3])));
      sq[r] = fmaf(S[r].x, q[0], fmaf(S[r].y, q[1], fmaf(S[r].z, q[2], S[r].w * q[3])));
    }
    const float Sk = warp_sum8(sk, lane), Sq = warp_sum8(sq, lane);
    const float u = beta * fmaf(-alpha, Sk, v);
    if ((lane & 3) == 0) *op = __float2bfloat16_rn(fmaf(alpha, Sq, u * kq));
    op += p.ot;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float ur = __shfl_sync(0xffffffffu, u, 4 * r);
      S[r].x = fmaf(alpha, S[r].x, ur * k[0]);
      S[r].y = fmaf(alpha, S[r].y, ur * k[1]);
      S[r].z = fmaf(alpha, S[r].z, ur * k[2]);
      S[r].w = fmaf(alpha, S[r].w, ur * k[3]);
    }
  }
  if (to >= 0) {
    float* s = p.state + to * p.s_slot + in_head;
#pragma unroll
    for (int r = 0; r < 8; ++r) *reinterpret_cast<float4*>(s + r * kD) = S[r];
  }
}

bool off16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

}  // namespace

size_t delta_rule_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

int launch_delta_rule(const bfp8_delta_rule_args& a, void* stream) {
  if (a.tokens < 0 || a.batch < 0 || a.max_q_len < 0 || a.n_slots < 0 || a.qk_heads < 1 || a.v_heads < 1 ||
      a.v_heads % a.qk_heads)
    return BFP8_ERR_INVALID_ARG;
  if (a.head_dim != kD) return BFP8_ERR_UNSUPPORTED;
  if (!(a.eps >= 0.0f) || !(a.scale > -3.0e38f && a.scale < 3.0e38f)) return BFP8_ERR_INVALID_ARG;
  if (a.tokens == 0 || a.batch == 0 || a.max_q_len == 0) return BFP8_OK;
  if (!a.q_bf16 || !a.k_bf16 || !a.v_bf16 || !a.a_bf16 || !a.b_bf16 || !a.a_log || !a.dt_bias || !a.out_bf16 ||
      !a.q_offsets)
    return BFP8_ERR_INVALID_ARG;
  const int64_t heads[8] = {a.q_stride_token, a.q_stride_head, a.k_stride_token, a.k_stride_head,
                            a.v_stride_token, a.v_stride_head, a.out_stride_token, a.out_stride_head};
  for (int64_t s : heads)
    if (s < kD) return BFP8_ERR_INVALID_ARG;
  if (a.a_stride_token < a.v_heads || a.b_stride_token < a.v_heads) return BFP8_ERR_INVALID_ARG;
  if (a.state ? a.state_stride_head < kD * kD || a.state_stride_slot < kD * kD : a.slots_in || a.slots_out)
    return BFP8_ERR_INVALID_ARG;
  for (int64_t s : heads)
    if (s % 8) return BFP8_ERR_UNSUPPORTED;
  if (a.tokens > 0x7FFFFFFF || a.batch > (1 << 20) || a.v_heads > 65535 || a.batch * a.v_heads > (1 << 28) ||
      off16(a.q_bf16) || off16(a.k_bf16) || off16(a.v_bf16) || off16(a.out_bf16) || off16(a.state) ||
      (a.state && (a.state_stride_slot % 4 || a.state_stride_head % 4)))
    return BFP8_ERR_UNSUPPORTED;
  int rc = check_device_ptrs({a.q_bf16, a.k_bf16, a.v_bf16, a.a_bf16, a.b_bf16, a.a_log, a.dt_bias, a.state,
                              a.out_bf16, a.q_offsets, a.slots_in, a.slots_out});
  if (rc != BFP8_OK) return rc;
  DeltaParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q_bf16);
  p.k = static_cast<const __nv_bfloat16*>(a.k_bf16);
  p.v = static_cast<const __nv_bfloat16*>(a.v_bf16);
  p.a = static_cast<const __nv_bfloat16*>(a.a_bf16);
  p.b = static_cast<const __nv_bfloat16*>(a.b_bf16);
  p.a_log = a.a_log;
  p.dt_bias = a.dt_bias;
  p.state = a.state;
  p.out = static_cast<__nv_bfloat16*>(a.out_bf16);
  p.qt = a.q_stride_token, p.qh = a.q_stride_head;
  p.kt = a.k_stride_token, p.kh = a.k_stride_head;
  p.vt = a.v_stride_token, p.vh = a.v_stride_head;
  p.at = a.a_stride_token, p.bt = a.b_stride_token;
  p.ot = a.out_stride_token, p.oh = a.out_stride_head;
  p.s_slot = a.state_stride_slot, p.s_head = a.state_stride_head;
  p.max_len = a.max_q_len;
  p.req = {a.q_offsets, a.slots_in, a.slots_out, a.tokens, a.n_slots, static_cast<int32_t>(a.batch)};
  p.v_heads = static_cast<int32_t>(a.v_heads);
  p.group = static_cast<int32_t>(a.v_heads / a.qk_heads);
  p.scale = a.scale;
  p.eps = a.eps;
  const unsigned blocks = static_cast<unsigned>(a.batch * a.v_heads * (kD / (8 * kStepWarps)));
  return launch_dependent(delta_step_kernel, dim3(blocks), 32 * kStepWarps, 0, static_cast<cudaStream_t>(stream), p);
}

}  // namespace bfp8
