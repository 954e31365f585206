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
#include "attention_layer.cuh"

#include <type_traits>

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
  float res_scale, eps, w_offset, inv_H;
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
// shuffles, then every warp adds the warps' sums. `red` is zero past the warps
// and alternates between two buffers, so the barrier of one reduction also
// separates the reads of the one before it from the writes of the one after.
BFP8_DEV float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (4 * k >= nw) break;
    const float4 r = reinterpret_cast<const float4*>(red)[k];
    v += (r.x + r.y) + (r.z + r.w);
  }
  return v;
}

BFP8_DEV float inv_rms(float sum_sq, float inv_H, float eps) {
  return rsqrtf(fmaf(sum_sq, inv_H, eps));
}

// A block takes rows blockIdx, blockIdx + gridDim, ... Thread t holds the
// 8-column vectors t, t + blockDim, ...: 16 consecutive lanes of a warp hold one
// 128-column group, so a group's maximum is four shuffles. VEC: every row, pitch
// and H is a multiple of 8 elements and 16-byte aligned.
//
// VPT = 1 is for few rows: the most threads a row can use, everything loaded at
// once. VPT = 4 is for many: a thread has the same columns in every row, so the
// weights are read and widened once, into shared memory (the post-norm's
// multiplied by a gate that all rows share), a row's loads are issued before the
// second reduction of the row ahead of it, and a row's reductions cost fewer
// warps. At 8192 rows of 5120, VPT = 2, 3, 4: 88, 65, 62 us; weights kept in
// registers: 98 us (one block an SM); rows copied to shared memory two ahead
// with the weights shared by four rows: 64 us. At 949 rows of 2072: 10.7 us with
// VPT = 1 and 12.6 with 4.
template <bool VEC, bool ROW_GATE, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512)
    residual_norm_kernel(const NormParams p) {
  constexpr bool kMany = VPT > 1;
  extern __shared__ float4 keep[];   // kMany: [VPT][4][blockDim]: 8 post factors, 8 weights of h
  __shared__ __align__(16) float red[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int nt = blockDim.x, tid = threadIdx.x, H = p.H;
  for (int i = tid; i < 64; i += nt) red[i >> 5][i & 31] = 0.0f;
  __syncthreads();
  const bool norm = p.q || p.norm_out;
  int buf = 0;
  int64_t row = blockIdx.x;
  uint4 yr[VPT], rr[VPT], gr[ROW_GATE ? VPT : 1];
  auto load = [&](int64_t at) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = 8 * (tid + i * nt);
      if (p.y) yr[i] = load8<VEC>(p.y + at * p.ldy, c, H);
      rr[i] = load8<VEC>(p.res + at * p.ldr, c, H);
    }
  };
  load(row);
  // factor of y apart from its row's: weight times shared gate (exact in FP32
  // for BF16 weights: 8 significant bits each)
  auto post = [&](int i, float (&f)[8]) {
    const int c = 8 * (tid + i * nt);
    if (p.w_post) {
      load_weight8<VEC>(p.w_post, p.w_f32, p.w_offset, c, H, f);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = 1.0f;
    }
    if (!ROW_GATE && p.gate) {
      float g[8];
      widen8(load8<VEC>(p.gate, c, H), g);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= g[e];
    }
  };
  auto put8 = [&](int i, int k, const float (&v)[8]) {
    keep[(4 * i + k) * nt + tid] = make_float4(v[0], v[1], v[2], v[3]);
    keep[(4 * i + k + 1) * nt + tid] = make_float4(v[4], v[5], v[6], v[7]);
  };
  auto get8 = [&](int i, int k, float (&v)[8]) {
    const float4 a = keep[(4 * i + k) * nt + tid], b = keep[(4 * i + k + 1) * nt + tid];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  };
  if (kMany) {   // each thread reads back only what it wrote: no barrier
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[8];
      if (p.y) {
        post(i, f);
        put8(i, 0, f);
      }
      if (norm) {
        load_weight8<VEC>(p.w_pre, p.w_f32, p.w_offset, 8 * (tid + i * nt), H, f);
        put8(i, 2, f);
      }
    }
  }
  for (; row < p.T; row += gridDim.x) {
    if (ROW_GATE) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        gr[ROW_GATE ? i : 0] = load8<VEC>(p.gate + row * p.ldg, 8 * (tid + i * nt), H);
    }
    float ry = 1.0f;
    if (p.w_post) {
      float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float y[8];
        widen8(yr[i], y);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 y2 = make_float2(y[e], y[e + 1]);
          ss = __ffma2_rn(y2, y2, ss);
        }
      }
      ry = inv_rms(block_sum(ss.x + ss.y, red[buf]), p.inv_H, p.eps);
      buf ^= 1;
    }
    float h[VPT][8];
    float2 sh = make_float2(0.0f, 0.0f);
    const float2 a2 = make_float2(p.res_scale, p.res_scale), ry2 = make_float2(ry, ry);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = 8 * (tid + i * nt);
      widen8(rr[i], h[i]);
      float y[8], f[8], g[8];
      if (p.y) {
        widen8(yr[i], y);
        if (kMany) get8(i, 0, f);
        else post(i, f);
        if (ROW_GATE) widen8(gr[ROW_GATE ? i : 0], g);
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float2 h2 = __fmul2_rn(make_float2(h[i][e], h[i][e + 1]), a2);
        if (p.y) {
          float2 f2 = make_float2(f[e], f[e + 1]);
          if (ROW_GATE) f2 = __fmul2_rn(f2, make_float2(g[e], g[e + 1]));
          h2 = __ffma2_rn(__fmul2_rn(make_float2(y[e], y[e + 1]), f2), ry2, h2);
        }
        h[i][e] = h2.x, h[i][e + 1] = h2.y;
        sh = __ffma2_rn(h2, h2, sh);   // columns past H hold 0
      }
      if (p.res_out) store8<VEC>(p.res_out + row * p.ldro, c, H, h[i]);
    }
    if (row + gridDim.x < p.T) load(row + gridDim.x);
    if (!norm) continue;
    const float rh = inv_rms(block_sum(sh.x + sh.y, red[buf]), p.inv_H, p.eps);
    buf ^= 1;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = 8 * (tid + i * nt);
      float w[8];
      if (kMany) get8(i, 2, w);
      else load_weight8<VEC>(p.w_pre, p.w_f32, p.w_offset, c, H, w);
      float am = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 h2 = __fmul2_rn(make_float2(h[i][e], h[i][e + 1]), make_float2(w[e], w[e + 1]));
        h[i][e] = h2.x, h[i][e + 1] = h2.y;   // n = h * rh
        am = fmaxf(am, fmaxf(fabsf(h2.x), fabsf(h2.y)));
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
      // The codes are (h w) * (448 / max|h w|), which leaves the row's factor out. The
      // reciprocal's error is taken off by one step from its remainder; the two
      // products, the reciprocal and the two roundings of s keep the quotient within
      // 6 * 2^-24 of n / s. (Of 59 M codes of 949 x 2072, 98 differ from the exact
      // ones', and 108 where n / s is formed by dividing; 102 without that step.)
      const float an = am * rh;
      float sc = an * (1.0f / 448.0f), inv;
      sc = fmaf(fmaf(-448.0f, sc, an), 1.0f / 448.0f, sc);   // the rounded quotient
      if (an >= 1e-10f && am >= 1e-30f && am <= 1e30f && an <= 1e30f) {
        inv = __fdividef(448.0f, am);
        inv = fmaf(fmaf(-am, inv, 448.0f), inv * (1.0f / 448.0f), inv);
      } else {
        sc = __fdiv_rn(fmaxf(an, 1e-10f), 448.0f);
        inv = an >= 1e-10f ? __fdiv_rn(448.0f, am) : __fdiv_rn(rh, sc);
      }
      if ((tid & 15) == 0 && c < H) p.s[row * p.ssm + static_cast<int64_t>(c >> 7) * p.sskb] = sc;
      const float2 inv2 = make_float2(inv, inv);
      uint32_t cw[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 a = __fmul2_rn(make_float2(h[i][4 * j], h[i][4 * j + 1]), inv2);
        const float2 b = __fmul2_rn(make_float2(h[i][4 * j + 2], h[i][4 * j + 3]), inv2);
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

template <bool VEC, bool ROW_GATE, int VPT>
int launch_norm(const NormParams& p, int sms, cudaStream_t st) {
  const int vecs = (p.H + 7) / 8;
  const int threads = ((vecs + VPT - 1) / VPT + 31) / 32 * 32;
  const int smem = VPT > 1 ? VPT * 4 * threads * 16 : 0;
  if (smem > 48 * 1024) {
    const int rc = set_max_dynamic_smem(
        reinterpret_cast<const void*>(residual_norm_kernel<VEC, ROW_GATE, VPT>), VPT * 4 * 512 * 16);
    if (rc != BFP8_OK) return rc;
  }
  // as many blocks as stay resident: each keeps its weights for all its rows
  static const int regs = [] {
    cudaFuncAttributes at{};
    const cudaError_t e = cudaFuncGetAttributes(&at, residual_norm_kernel<VEC, ROW_GATE, VPT>);
    return e == cudaSuccess ? at.numRegs : 128;
  }();
  const int by_regs = 65536 / (threads * ((regs + 7) / 8 * 8));
  const int by_smem = 224 * 1024 / (smem + 2048);
  int fit = by_regs < by_smem ? by_regs : by_smem;
  fit = fit < 1 ? 1 : fit > 2048 / threads ? 2048 / threads : fit > 32 ? 32 : fit;
  const int64_t cap = static_cast<int64_t>(sms) * fit;
  return launch_dependent(residual_norm_kernel<VEC, ROW_GATE, VPT>,
                          dim3(static_cast<unsigned>(p.T < cap ? p.T : cap)), threads, smem, st, p);
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
  p.inv_H = 1.0f / static_cast<float>(H);
  auto row16 = [](const void* ptr, int64_t ld) { return !ptr || (aligned(ptr, 16) && ld % 8 == 0); };
  const bool vec = H % 8 == 0 && row16(a.y, a.ldy) && row16(a.residual, a.ld_residual) &&
                   row16(a.gate, a.ld_gate) && row16(a.residual_out, a.ld_residual_out) &&
                   row16(a.norm_out, a.ld_norm_out) && (!a.w_post || aligned(a.w_post, 16)) &&
                   (!a.w_pre || aligned(a.w_pre, 16)) &&
                   (!a.q_e4m3 || (aligned(a.q_e4m3, 8) && a.ldq % 8 == 0));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int vecs = (p.H + 7) / 8;
  // VPT = 4 where a row has no 1024 threads to itself or the rows are more than two
  // waves of one vector a thread
  const int vpt = vecs > 1024 || T * vecs > sms * int64_t{4096} ? 4 : 1;
  auto go = [&](auto v, auto g) {
    constexpr bool V = decltype(v)::value, G = decltype(g)::value;
    return vpt == 1 ? launch_norm<V, G, 1>(p, sms, st) : launch_norm<V, G, 4>(p, sms, st);
  };
  const std::true_type yes;
  const std::false_type no;
  const bool row_gate = p.gate && p.ldg != 0;
  if (vec) return row_gate ? go(yes, yes) : go(yes, no);
  return row_gate ? go(no, yes) : go(no, no);
}

}  // namespace bfp8
