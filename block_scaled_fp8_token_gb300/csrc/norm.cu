// norm.cu -- the step between two blocks of a decoder layer: the block's
// output normed, gated and added to the scaled residual stream, and the sum
// normed again and quantized for the next projection, in one pass.
//
//   u = y * rsqrt(mean(y^2) + eps) * w_post          (w_post absent: u = y)
//   h = residual_scale * residual + gate * u
//   residual_out = bf16(h)
//   n = h * rsqrt(mean(h^2) + eps) * w_pre
//   norm_out = bf16(n);  s = max(max|n|, 1e-10f) / 448 per 128 columns,
//   q = RNE_satfinite_e4m3(n / s)
//
// The row stays in registers as FP32 from its one read to its writes: the
// second norm takes h and the quantizer takes n before either is rounded to
// BF16, so the codes carry one rounding (to E4M3) where the unfused steps
// carry three. Bound by HBM: a row is read twice (y, residual) and written
// once, plus its codes.
#include "bfp8_internal.h"
#include "ptx.cuh"
#include "act_math.cuh"

namespace bfp8 {
namespace {

using namespace dev;

struct NormParams {
  const __nv_bfloat16* y;
  const __nv_bfloat16* res;
  const __nv_bfloat16* gate;
  const void* w_post;
  const void* w_pre;
  __nv_bfloat16* res_out;
  __nv_bfloat16* norm_out;
  uint8_t* q;
  float* s;
  int64_t T, ldy, ldr, ldg, ldro, ldn, ldq, ssm, sskb;
  int32_t H, w_f32;
  float res_scale, eps, w_offset;
};

// p[c .. c+8) of a BF16 row as four bf16x2 words, zero past H.
template <bool VEC>
BFP8_DEV uint4 load8(const __nv_bfloat16* p, int c, int H) {
  if (VEC) return c < H ? *reinterpret_cast<const uint4*>(p + c) : make_uint4(0u, 0u, 0u, 0u);
  const uint16_t* p16 = reinterpret_cast<const uint16_t*>(p);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = c + 2 * j < H ? p16[c + 2 * j] : 0u;
    const uint32_t hi = c + 2 * j + 1 < H ? p16[c + 2 * j + 1] : 0u;
    w[j] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

BFP8_DEV void widen8(const uint4& r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

// Norm weights c .. c+8 (BF16 or FP32, one branch for the whole grid) plus the
// offset that zero-centred weights are stored without.
template <bool VEC>
BFP8_DEV void load_weight8(const void* w, int w_f32, float offset, int c, int H, float (&v)[8]) {
  if (w_f32) {
    const float* wf = static_cast<const float*>(w);
    if (VEC && c < H) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(wf + c));
      const float4 b = __ldg(reinterpret_cast<const float4*>(wf + c + 4));
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = c + e < H ? __ldg(wf + c + e) : 0.0f;
    }
  } else {
    widen8(load8<VEC>(static_cast<const __nv_bfloat16*>(w), c, H), v);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] += offset;
}

template <bool VEC>
BFP8_DEV void store8(__nv_bfloat16* p, int c, int H, const float (&v)[8]) {
  if (VEC) {
    if (c >= H) return;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
    *reinterpret_cast<uint4*>(p + c) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < H) p[c + e] = __float2bfloat16_rn(v[e]);
  }
}

// Sum over the block, in an order fixed by the launch shape: within the warp by
// shuffles, then every warp adds the warps' sums. `red` alternates between two
// buffers, so the barrier of one reduction also separates the reads of the
// one before it from the writes of the one after.
BFP8_DEV float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < nw ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

BFP8_DEV float inv_rms(float sum_sq, int H, float eps) {
  return __frcp_rn(__fsqrt_rn(__fdiv_rn(sum_sq, static_cast<float>(H)) + eps));
}

// One block per row (grid-stride). Thread t holds the 8-column vectors t,
// t + blockDim, ...: 16 consecutive lanes of a warp hold one 128-column group,
// so a group's maximum is four shuffles. VEC: every row, pitch and H is a
// multiple of 8 elements and 16-byte aligned.
template <bool VEC, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) residual_norm_kernel(const NormParams p) {
  __shared__ float red[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int nt = blockDim.x, tid = threadIdx.x, H = p.H;
  int buf = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    uint4 yr[VPT], rr[VPT], gr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = 8 * (tid + i * nt);
      if (p.y) yr[i] = load8<VEC>(p.y + row * p.ldy, c, H);
      rr[i] = load8<VEC>(p.res + row * p.ldr, c, H);
      if (p.y && p.gate) gr[i] = load8<VEC>(p.gate + row * p.ldg, c, H);
    }
    float ry = 1.0f;
    if (p.y && p.w_post) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float y[8];
        widen8(yr[i], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
      }
      ry = inv_rms(block_sum(ss, red[buf]), H, p.eps);
      buf ^= 1;
    }
    float h[VPT][8];
    float sh = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = 8 * (tid + i * nt);
      widen8(rr[i], h[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] *= p.res_scale;
      if (p.y) {
        // y times weight times gate is exact in FP32 when all are BF16 (8
        // significant bits each), so the row's factor and the sum round once
        float y[8], f[8];
        widen8(yr[i], y);
        if (p.w_post) {
          load_weight8<VEC>(p.w_post, p.w_f32, p.w_offset, c, H, f);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = 1.0f;
        }
        if (p.gate) {
          float g[8];
          widen8(gr[i], g);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = fmaf(y[e] * f[e], ry, h[i][e]);
      }
      if (p.res_out) store8<VEC>(p.res_out + row * p.ldro, c, H, h[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) sh = fmaf(h[i][e], h[i][e], sh);   // columns past H hold 0
    }
    if (!p.q && !p.norm_out) continue;
    const float rh = inv_rms(block_sum(sh, red[buf]), H, p.eps);
    buf ^= 1;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = 8 * (tid + i * nt);
      float w[8];
      load_weight8<VEC>(p.w_pre, p.w_f32, p.w_offset, c, H, w);
      float am = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[i][e] *= w[e];   // n = h * rh
        am = fmaxf(am, fabsf(h[i][e]));
      }
      if (p.norm_out) {
        float n[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = h[i][e] * rh;
        store8<VEC>(p.norm_out + row * p.ldn, c, H, n);
      }
      if (!p.q) continue;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
      // n / s with the row's factor cancelled: h / (max|h| / 448), unless the floor holds
      const float an = am * rh;
      const float sc = __fdiv_rn(fmaxf(an, 1e-10f), 448.0f);
      const float dv = an >= 1e-10f ? __fdiv_rn(am, 448.0f) : __fdiv_rn(sc, rh);
      if ((tid & 15) == 0 && c < H) p.s[row * p.ssm + static_cast<int64_t>(c >> 7) * p.sskb] = sc;
      const float rc = __frcp_rn(dv);
      const float2 y2 = make_float2(rc, rc), ns2 = make_float2(-dv, -dv);
      uint32_t cw[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 a = div_by_scale2(make_float2(h[i][4 * j], h[i][4 * j + 1]), ns2, y2);
        const float2 b = div_by_scale2(make_float2(h[i][4 * j + 2], h[i][4 * j + 3]), ns2, y2);
        cw[j] = static_cast<uint32_t>(f32x2_to_e4m3x2(a.x, a.y)) |
                (static_cast<uint32_t>(f32x2_to_e4m3x2(b.x, b.y)) << 16);
      }
      uint8_t* qrow = p.q + row * p.ldq;
      if (VEC) {
        if (c < H) *reinterpret_cast<uint2*>(qrow + c) = make_uint2(cw[0], cw[1]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < H) qrow[c + e] = static_cast<uint8_t>(cw[e >> 2] >> (8 * (e & 3)));
      }
    }
  }
}

template <bool VEC, int VPT>
int launch_norm(const NormParams& p, int sms, cudaStream_t st) {
  const int vecs = (p.H + 7) / 8;
  const int threads = ((vecs + VPT - 1) / VPT + 31) / 32 * 32;
  const int64_t cap = static_cast<int64_t>(sms) * (2048 / threads > 32 ? 32 : 2048 / threads);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.T < cap ? p.T : cap));
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, residual_norm_kernel<VEC, VPT>, p) != cudaSuccess)
    return BFP8_ERR_CUDA;
  return check_launch();
}

bool aligned(const void* p, uintptr_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

}  // namespace

int launch_residual_norm(const bfp8_norm_args& a, int64_t T, int64_t H, void* stream) {
  const bool norm = a.norm_out || a.q_e4m3;
  if (T < 0 || H < 0) return BFP8_ERR_INVALID_ARG;
  if (T == 0 || H == 0) return BFP8_OK;
  const int64_t Kb = (H + 127) / 128;
  if (!a.residual || a.ld_residual < H) return BFP8_ERR_INVALID_ARG;
  if (a.y ? a.ldy < H : (a.w_post || a.gate)) return BFP8_ERR_INVALID_ARG;
  if (a.gate && a.ld_gate != 0 && a.ld_gate < H) return BFP8_ERR_INVALID_ARG;
  if (a.residual_out ? a.ld_residual_out < H : !norm) return BFP8_ERR_INVALID_ARG;
  if (norm && !a.w_pre) return BFP8_ERR_INVALID_ARG;
  if (a.norm_out && a.ld_norm_out < H) return BFP8_ERR_INVALID_ARG;
  if (a.q_e4m3 && (!a.scales || a.ldq < H || a.s_stride_m < 0 || a.s_stride_kb < 0 ||
                   (T > 1 && a.s_stride_m == 0) || (Kb > 1 && a.s_stride_kb == 0)))
    return BFP8_ERR_INVALID_ARG;
  if (!(a.eps >= 0.0f)) return BFP8_ERR_INVALID_ARG;
  if ((a.w_post || a.w_pre) && a.w_dtype != BFP8_DT_BF16 && a.w_dtype != BFP8_DT_F32)
    return BFP8_ERR_SCALE_DTYPE;
  if (H > 16384) return BFP8_ERR_UNSUPPORTED;
  int rc = check_device_ptrs({a.y, a.residual, a.gate, a.w_post, a.w_pre, a.residual_out,
                              a.norm_out, a.q_e4m3, a.q_e4m3 ? a.scales : nullptr});
  if (rc != BFP8_OK) return rc;
  int sms = 0;
  rc = sm_count(&sms);
  if (rc != BFP8_OK) return rc;
  NormParams p{};
  p.y = static_cast<const __nv_bfloat16*>(a.y);
  p.res = static_cast<const __nv_bfloat16*>(a.residual);
  p.gate = static_cast<const __nv_bfloat16*>(a.gate);
  p.w_post = a.w_post;
  p.w_pre = a.w_pre;
  p.res_out = static_cast<__nv_bfloat16*>(a.residual_out);
  p.norm_out = static_cast<__nv_bfloat16*>(a.norm_out);
  p.q = static_cast<uint8_t*>(a.q_e4m3);
  p.s = a.scales;
  p.T = T;
  p.H = static_cast<int32_t>(H);
  p.ldy = a.ldy;
  p.ldr = a.ld_residual;
  p.ldg = a.ld_gate;
  p.ldro = a.ld_residual_out;
  p.ldn = a.ld_norm_out;
  p.ldq = a.ldq;
  p.ssm = a.s_stride_m;
  p.sskb = a.s_stride_kb;
  p.w_f32 = a.w_dtype == BFP8_DT_F32;
  p.res_scale = a.residual_scale;
  p.eps = a.eps;
  p.w_offset = a.weight_offset;
  auto row16 = [](const void* ptr, int64_t ld) { return !ptr || (aligned(ptr, 16) && ld % 8 == 0); };
  const bool vec = H % 8 == 0 && row16(a.y, a.ldy) && row16(a.residual, a.ld_residual) &&
                   row16(a.gate, a.ld_gate) && row16(a.residual_out, a.ld_residual_out) &&
                   row16(a.norm_out, a.ld_norm_out) && (!a.w_post || aligned(a.w_post, 16)) &&
                   (!a.w_pre || aligned(a.w_pre, 16)) &&
                   (!a.q_e4m3 || (aligned(a.q_e4m3, 8) && a.ldq % 8 == 0));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int vecs = (p.H + 7) / 8;
  // few rows: the most threads a row can use; many rows: fewer threads with
  // more loads in flight each, so that several rows share an SM
  const int vpt = vecs > 1024 ? 4 : (T > sms && vecs >= 256) ? 2 : 1;
  if (vpt == 1) return vec ? launch_norm<true, 1>(p, sms, st) : launch_norm<false, 1>(p, sms, st);
  if (vpt == 2) return vec ? launch_norm<true, 2>(p, sms, st) : launch_norm<false, 2>(p, sms, st);
  return vec ? launch_norm<true, 4>(p, sms, st) : launch_norm<false, 4>(p, sms, st);
}

}  // namespace bfp8
