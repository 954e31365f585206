// delta_rule.cu -- the gated delta rule of a linear-attention layer over the ragged tokens
// of a step, with each request's state kept between steps. Per value head, with the state S
// of 128 values by 128 keys, and per token
//
//   alpha = exp(-exp(a_log) softplus(a + dt_bias)),  beta = sigmoid(b)
//   k' = k rsqrt(|k|^2 + eps),  q' = scale q rsqrt(|q|^2 + eps)
//   u = beta (v - alpha S k'),  S <- alpha S + u k'^T,  out = S q'
//
// State, sums and gates are FP32 and out is rounded once to BF16; what the chunks' products round
// beside is said there.
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
  int64_t qt, qh, kt, kh, vt, vh, at, bt, ot, oh, s_slot, s_head, max_len, step_len;
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
BFP8_DEV float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
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

constexpr int kStepWarps = 4, kMostSteps = 32;         // of a block; tokens of a request, of which up to 20 come
template <int WARPS>
struct StepShared {
  alignas(16) uint2 k[kMostSteps][32];                 // raw rows
  uint2 q[kMostSteps][32];
  alignas(16) __nv_bfloat16 v[kMostSteps][8 * WARPS];  // of the block's values
  float alpha[kMostSteps], beta[kMostSteps], kn[kMostSteps], qn[kMostSteps], kq[kMostSteps];
};

// One token after the other: a warp holds 8 of a head's 128 rows of S, four columns a lane,
// and in the loop needs no other warp. Both products with the old state are summed at once, as
// S_new q' = alpha S q' + u (k' . q'), with the raw key and query, whose factors go behind the
// sums. The tokens' rows and what of them needs no state (gates, factors, k' . q') are in shared
// memory before the first token's turn, so that a turn is one reduction, u's way back to the
// lanes and the update. A block of WARPS warps, number `block`.
//
// Bound by HBM, the state's 64 KB read and written a head: 64 single tokens of 48 heads move 405
// MB in 62 us, 6.5 TB/s. 17 requests of 3 tokens, 32 heads, take 17: at 65 registers seven blocks fit
// an SM, and 2,176 are two waves and a tail of 48.
template <int WARPS>
BFP8_DEV void delta_steps(const DeltaParams& p, int64_t block, StepShared<WARPS>& sh) {
  constexpr int kParts = kD / (8 * WARPS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t item = block / kParts;
  const int b = static_cast<int>(item / p.v_heads), h = static_cast<int>(item - int64_t{b} * p.v_heads);
  const int block_row = static_cast<int>(block % kParts) * (8 * WARPS), row0 = block_row + warp * 8;
  const int64_t first = first_token(p.req, b);
  int64_t len = first_token(p.req, b + 1) - first;
  len = len < p.max_len ? len : p.max_len;
  if (len <= 0 || len > p.step_len) return;
  const int n = static_cast<int>(len);
  const int64_t from = slot_of(p.req, p.req.slots_in, b), to = slot_of(p.req, p.req.slots_out, b);
  const int64_t in_head = h * p.s_head + row0 * kD + lane * 4;
  const int hk = h / p.group;
  const __nv_bfloat16* qp = p.q + first * p.qt + hk * p.qh;
  const __nv_bfloat16* kp = p.k + first * p.kt + hk * p.kh;
  const __nv_bfloat16* vp = p.v + first * p.vt + h * p.vh + block_row;
  for (int t = warp; t < n; t += WARPS) {
    const bool key = lane < 16;
    cp_async16(smem_u32(key ? &sh.k[t][2 * lane] : &sh.q[t][2 * (lane - 16)]),
               (key ? kp + t * p.kt : qp + t * p.qt) + 8 * (lane & 15));
  }
  for (int i = threadIdx.x; i < n * WARPS; i += 32 * WARPS)
    cp_async16(smem_u32(&sh.v[i / WARPS][8 * (i % WARPS)]), vp + (i / WARPS) * p.vt + 8 * (i % WARPS));
  cp_async_commit();
  float2 S[8][2];
#pragma unroll
  for (int r = 0; r < 8; ++r) S[r][0] = S[r][1] = make_float2(0.0f, 0.0f);
  if (from >= 0) {
    const float* s = p.state + from * p.s_slot + in_head;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float4 f = *reinterpret_cast<const float4*>(s + r * kD);
      S[r][0] = make_float2(f.x, f.y), S[r][1] = make_float2(f.z, f.w);
    }
  }
  if (warp == WARPS - 1 && lane < n) {
    const float a = __bfloat162float(p.a[(first + lane) * p.at + h]), g = __bfloat162float(p.b[(first + lane) * p.bt + h]);
    sh.alpha[lane] = expf(log_decay(a, __ldg(p.dt_bias + h), expf(__ldg(p.a_log + h))));
    sh.beta[lane] = beta_of(g);
  }
  cp_async_wait_all();
  __syncthreads();
  auto four = [](uint2 w, float2& lo, float2& hi) {
    lo = make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u));
    hi = make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
  };
  for (int t = warp; t < n; t += WARPS) {
    float2 k01, k23, q01, q23;
    four(sh.k[t][lane], k01, k23);
    four(sh.q[t][lane], q01, q23);
    const float2 kk = __ffma2_rn(k01, k01, __fmul2_rn(k23, k23)), qq = __ffma2_rn(q01, q01, __fmul2_rn(q23, q23));
    const float2 kq = __ffma2_rn(k01, q01, __fmul2_rn(k23, q23));
    const float kn = rsqrtf(warp_sum(kk.x + kk.y) + p.eps), qn = rsqrtf(warp_sum(qq.x + qq.y) + p.eps) * p.scale;
    const float both = warp_sum(kq.x + kq.y);
    if (lane == 0) sh.kn[t] = kn, sh.qn[t] = qn, sh.kq[t] = both * kn * qn;
  }
  __syncthreads();
  __nv_bfloat16* op = p.out + first * p.ot + h * p.oh + row0 + (lane >> 2);
  for (int t = 0; t < n; ++t) {
    float2 k01, k23, q01, q23;
    four(sh.k[t][lane], k01, k23);
    four(sh.q[t][lane], q01, q23);
    const float v = __bfloat162float(sh.v[t][8 * warp + (lane >> 2)]);
    const float alpha = sh.alpha[t], kn = sh.kn[t];
    float sk[8], sq[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float2 a = __ffma2_rn(S[r][0], k01, __fmul2_rn(S[r][1], k23));
      const float2 c = __ffma2_rn(S[r][0], q01, __fmul2_rn(S[r][1], q23));
      sk[r] = a.x + a.y;
      sq[r] = c.x + c.y;
    }
    const float Sk = warp_sum8(sk, lane), Sq = warp_sum8(sq, lane);
    const float u = sh.beta[t] * fmaf(-alpha * kn, Sk, v);
    if ((lane & 3) == 0) *op = __float2bfloat16_rn(fmaf(alpha * sh.qn[t], Sq, u * sh.kq[t]));
    op += p.ot;
    const float uk = u * kn;
    const float2 alpha2 = make_float2(alpha, alpha);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float ur = __shfl_sync(0xffffffffu, uk, 4 * r);
      const float2 u2 = make_float2(ur, ur);
      S[r][0] = __ffma2_rn(u2, k01, __fmul2_rn(alpha2, S[r][0]));
      S[r][1] = __ffma2_rn(u2, k23, __fmul2_rn(alpha2, S[r][1]));
    }
  }
  if (to >= 0) {
    float* s = p.state + to * p.s_slot + in_head;
#pragma unroll
    for (int r = 0; r < 8; ++r)
      *reinterpret_cast<float4*>(s + r * kD) = make_float4(S[r][0].x, S[r][0].y, S[r][1].x, S[r][1].y);
  }
}
__global__ void __launch_bounds__(32 * kStepWarps) delta_step_kernel(const DeltaParams p) {
  __shared__ StepShared<kStepWarps> sh;
  pdl_wait();
  pdl_launch_dependents();
  delta_steps<kStepWarps>(p, blockIdx.x, sh);
}

// ------------------------------------------------------------------ chunks of 64 tokens
//
// Within a chunk of C tokens that begins with the state S0, write Gamma_i = alpha_0 .. alpha_i,
// and k, q for the rows with ck, cq their factors. Then
//   A_ij = beta_i ck_i ck_j (Gamma_i / Gamma_j) (k_i . k_j)      j < i
//   u = (1 + A)^-1 r,   r_i = beta_i (v_i - Gamma_i ck_i S0 k_i)
//   out_i = scale (Gamma_i cq_i S0 q_i + sum_j P_ij u_j),   P_ij = cq_i ck_j (Gamma_i / Gamma_j) (q_i . k_j)   j <= i
//   S = Gamma_C S0 + sum_j (Gamma_C / Gamma_j) ck_j u_j k_j^T
// The first kernel forms T = (1 + A)^-1 and P T of every chunk at once, which need no state;
// the second walks down each request's chunks, three products one behind another a chunk:
//   S0 [K^T | Q^T]  ->  r [T^T | (P T)^T] = [u | sum P u]  ->  u K
// Ratios of Gamma are running products of the alphas, so no difference of sums of logarithms
// loses digits and a decay to 0 gives 0.
//
// On the tensor cores an FP32 value is two F16 parts, the rounded value and its rounded rest:
// 22 bits, and no less than 2^-25 of what the operand's row or matrix is scaled to. Products of
// two rests are left out (2^-24). What each operand is scaled by is a power of two:
//   K, Q   each row to a largest entry in [1, 2): BF16's 8 bits are then exact in F16 down to
//          2^-17 of the largest, and enter as one part; the factors ck, cq take the power back
//   T, P T by 2^12. No entry exceeds 1: column j is what the rule answers to a single value at
//          token j, whose state is a key of length 1 at most and never grows
//   S, r, u: all three are linear in a row of S and of the values, so one power of two a row
//          serves them; the walk watches it (below)
constexpr int kChunk = 64, kShift = 6;
constexpr int kHalfTile = kChunk * 128;                // 64 rows of 128 bytes
constexpr int kTile = 2 * kHalfTile;                   // 128 such rows: K over Q of 64 columns, or T over P T
constexpr int kKq = 2 * kTile;                         // both halves of the columns
constexpr int kScalars = 2 * kTile;                    // of a blob: T over P T, the parts, then
// beta, -beta Gamma ck, Gamma cq 2^12, (Gamma_C / Gamma) ck 2^-12 of each token, and Gamma_C
constexpr int kBeta = 0, kKey = 64, kQuery = 128, kUpdate = 192, kGammaC = 256;
constexpr int kBlob = kScalars + 1152;
constexpr float kTScale = 4096.0f;

__device__ int g_delta_err;

// Of each chunk's slot the workspace has the K and Q rows of each key head, then a blob for
// each value head.
struct ChunkParams {
  DeltaParams d;
  uint8_t* ws;
  float* ends;                                         // of each head's segments but the last: the state behind it
  float* maps;                                         // ... and what it makes of the state ahead of it
  int32_t segments, segment_chunks, second_walk;
  int32_t longest_first;                               // the walk's blocks
  int32_t lead;                                        // the first segment is 1 + lead of the others' chunks long
  uint32_t chunk_blocks;                               // of the first kernel
  int32_t qk_heads, subgroups, per_block;              // value heads a block of the first kernel takes
};
BFP8_DEV int64_t slot_bytes(const ChunkParams& p) {
  return static_cast<int64_t>(p.qk_heads) * kKq + static_cast<int64_t>(p.d.v_heads) * kBlob;
}
BFP8_DEV uint8_t* kq_at(const ChunkParams& p, int64_t slot, int hk) {
  return p.ws + slot * slot_bytes(p) + static_cast<int64_t>(hk) * kKq;
}
BFP8_DEV uint8_t* blob_at(const ChunkParams& p, int64_t slot, int h) {
  return p.ws + slot * slot_bytes(p) + static_cast<int64_t>(p.qk_heads) * kKq + static_cast<int64_t>(h) * kBlob;
}

BFP8_DEV uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// x minus an F16, exactly what rounding left.
BFP8_DEV float minus_f16(float x, uint16_t h) {
  float r;
  asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(r) : "h"(h), "h"(static_cast<uint16_t>(0xBC00)), "f"(x));
  return r;
}
// A pair's two F16 parts.
BFP8_DEV void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16x2(x.x, x.y);
  lo = pack_f16x2(minus_f16(x.x, static_cast<uint16_t>(hi)), minus_f16(x.y, static_cast<uint16_t>(hi >> 16)));
}
// The larger size, of each half of a pair.
BFP8_DEV uint32_t max_abs_f16x2(uint32_t m, uint32_t v) {
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&m), __habs2(*reinterpret_cast<const __half2*>(&v)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
BFP8_DEV float max_f16x2(uint32_t m) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
  return fmaxf(f.x, f.y);
}
BFP8_DEV uint32_t max_abs_bf16x2(uint32_t m, uint32_t v) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                   __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
BFP8_DEV float max_bf16x2(uint32_t m) {
  return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}
// The power of two that brings m to [2^to, 2^(to + 1)), within 2^-125 .. 2^125.
BFP8_DEV float power_for(float m, int to) {
  const int e = 127 + to - static_cast<int>((__float_as_uint(m) >> 23) & 0xFF);
  return __uint_as_float(static_cast<uint32_t>(127 + min(max(e, -125), 125)) << 23);
}

BFP8_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
BFP8_DEV void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
}
// 64 tokens of one head, each half of the columns in rows of 128 bytes with the 128-byte
// swizzle, the halves `apart` bytes apart. Rows past the tensor's are zeros.
BFP8_DEV void load_tile(uint32_t dst, uint32_t apart, const CUtensorMap* map, int head, int row, uint32_t bar) {
  tma_load_3d(dst, map, 0, head, row, bar);
  tma_load_3d(dst + apart, map, 64, head, row, bar);
}
// Of a request the chunks' kernels take: its first token and its length, 0 for the others.
BFP8_DEV int64_t chunked_len(const DeltaParams& p, int b, int64_t& first) {
  first = first_token(p.req, b);
  int64_t n = first_token(p.req, b + 1) - first;
  n = n < p.max_len ? n : p.max_len;
  return n > p.step_len ? n : 0;
}
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_f16_mn(int m, int n) { return idesc_f16(m, n) | (1u << 16); }
BFP8_DEV void umma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  umma_bf16(d_tmem, a_desc, b_desc, idesc, accumulate);   // the operands' type is in idesc
}

constexpr int kPrepThreads = 256;
constexpr int kPitch = 68, kPitchZ = 36;               // floats of a row of A or T, and of Z
constexpr int kGroup = 4;                              // value heads a block takes, at most
struct PrepShared {
  alignas(16) float A[kChunk * kPitch];                // A, zeros from its diagonal on; then block by block T
  // each token's gates, and the products of alphas from its half's first to it, and behind it
  float alpha[kGroup][kChunk], beta[kGroup][kChunk], within[kGroup][kChunk], behind[kGroup][kChunk];
  float factor[2 * kChunk];
  uint64_t full, gram, product;
  uint32_t tmem;
  int abort_flag;
};
constexpr int kPrepSharedAt = (kBlob + 15) / 16 * 16;   // the blob takes the K and Q rows' place
constexpr int kPrepSmem = kPrepSharedAt + static_cast<int>(sizeof(PrepShared));
static_assert(4 * (kPrepSmem + 1024) <= 228 * 1024 && 32 * kPitchZ * 4 <= kHalfTile, "four blocks an SM; Z in T's place");
static_assert(sizeof(StepShared<kPrepThreads / 32>) <= kPrepSharedAt, "the steps' rows fit the blob's place");

// Running products over the warp, of 32 values from the first to each lane's.
BFP8_DEV float scan_product(float v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v *= u;
  }
  return v;
}
// ... and of the values behind each lane's.
BFP8_DEV float scan_product_behind(float v, int lane) {
  float r = __shfl_down_sync(0xffffffffu, v, 1);
  if (lane == 31) r = 1.0f;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float u = __shfl_down_sync(0xffffffffu, r, o);
    if (lane + o < 32) r *= u;
  }
  return r;
}

// A warp's 16 x 8 piece of X (16 x K) Y (K x 8), all FP32 in shared memory, Y with rows PY apart: lane
// l has columns 2 (l % 4) and one more of rows l / 4 and l / 4 + 8. The operands are cut into two
// F16 parts; none exceeds 32 (a row of A by a column of T1), so that 2^8 of them stay in range,
// and the rests' smallest step is 2^-33. (On CUDA cores the two products of the 32-row block took
// 2,400 clocks, most of them reading shared memory; so they take 700. tcgen05 has no shape
// this small.)
template <int K, int PY = kPitch>
BFP8_DEV void small_product(const float* x, const float* y, int lane, float (&c)[4]) {
  constexpr float kUp = 256.0f;
  const int g = lane >> 2, t = lane & 3;
  c[0] = c[1] = c[2] = c[3] = 0.0f;
#pragma unroll
  for (int k = 0; k < K; k += 16) {
    uint32_t a[2][4], b[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = *reinterpret_cast<const float2*>(x + (g + 8 * (i & 1)) * kPitch + k + 2 * t + 8 * (i >> 1));
      split2(make_float2(f.x * kUp, f.y * kUp), a[0][i], a[1][i]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* f = y + (k + 2 * t + 8 * i) * PY + g;
      split2(make_float2(f[0] * kUp, f[PY] * kUp), b[0][i], b[1][i]);
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) {                      // rests by rests left out
      const uint32_t(&u)[4] = a[p >> 1];
      const uint32_t(&v)[2] = b[p & 1];
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
          : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
          : "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(v[0]), "r"(v[1]));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] *= 1.0f / (kUp * kUp);
}
// A piece written with a sign.
template <int P = kPitch>
BFP8_DEV void store_piece(float* at, int lane, const float (&c)[4], float sign) {
  float* const p = at + (lane >> 2) * P + 2 * (lane & 3);
  *reinterpret_cast<float2*>(p) = make_float2(sign * c[0], sign * c[1]);
  *reinterpret_cast<float2*>(p + 8 * P) = make_float2(sign * c[2], sign * c[3]);
}

// T and P T of one chunk, for up to four value heads of one key head. One product of the K rows
// and the Q rows with the K rows leaves row i of K K^T and of Q K^T in a lane of tensor memory;
// two threads share a lane's columns. (1 + A)^-1 is formed by blocks of 16: the diagonal ones
// column by column, then each lower one as -T_b A_ba T_a, of 16 rows and of 32. P T is a
// product on the tensor cores again. The grid's last blocks, up to four an SM, take the step's short
// requests, a token after the other, which so run beside the long ones' chunks (as its first
// blocks they kept the chunks waiting: 81 us against 60 for 12 requests of 1 to 141 tokens and 48
// heads; with a block for every part, 64 requests without a short one took 15 us of empty blocks).
//
// Bound by latency: a block passes a dozen barriers, and four to an SM, whose 64 registers spill 88
// bytes a thread, issue in 53% of the clocks.
// 129 chunks of 16 key and 32 value heads take 88 us (94 with three to an SM, 214 with one; 138
// with a thread a row solving against A from registers, whose unrolled code stalled on instruction
// fetches).
__global__ void __launch_bounds__(kPrepThreads, 4) delta_prepare_kernel(const __grid_constant__ CUtensorMap tq,
                                                                     const __grid_constant__ CUtensorMap tk,
                                                                     const ChunkParams p) {
  extern __shared__ __align__(1024) uint8_t prepare_smem[];
  uint8_t* const base = prepare_smem;
  PrepShared& sh = *reinterpret_cast<PrepShared*>(base + kPrepSharedAt);
  const uint32_t kq = smem_u32(base), blob = kq;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tq);
  }
  pdl_wait();
  if (blockIdx.x >= p.chunk_blocks) {
    pdl_launch_dependents();
    constexpr int kWarps = kPrepThreads / 32;
    const int64_t all = static_cast<int64_t>(p.d.req.batch) * p.d.v_heads * (kD / (8 * kWarps));
    for (int64_t part = blockIdx.x - p.chunk_blocks; part < all; part += gridDim.x - p.chunk_blocks) {
      delta_steps<kWarps>(p.d, part, *reinterpret_cast<StepShared<kWarps>*>(base));
      __syncthreads();
    }
    return;
  }
  const int block = static_cast<int>(blockIdx.x);
  const int hk = block % p.qk_heads, sub = block / p.qk_heads % p.subgroups;
  const int64_t slot = block / (p.qk_heads * p.subgroups);
  const int h0 = hk * p.d.group + sub * p.per_block, heads = min(p.per_block, p.d.group - sub * p.per_block);
  const int b = find_request(p.d.req, slot, kShift);
  if (b < 0) return;
  int64_t first;
  const int64_t len = chunked_len(p.d, b, first);
  const int64_t done = (slot - tile_key(p.d.req, b, kShift)) << kShift;
  if (done >= len) return;
  const int n = static_cast<int>(len - done < kChunk ? len - done : kChunk);
  const int64_t t0 = first + done;
  const int row = (warp & 3) * 32 + lane, i = row & 63, half = warp >> 2;
  const bool query = row >= kChunk;

  if (tid == 0) {
    mbar_init(smem_u32(&sh.full), 1);
    mbar_init(smem_u32(&sh.gram), 1);
    mbar_init(smem_u32(&sh.product), 1);
    sh.abort_flag = 0;
    mbar_fence_init();
    mbar_arrive_expect_tx(smem_u32(&sh.full), kKq);
    load_tile(kq, kTile, &tk, hk, static_cast<int>(t0), smem_u32(&sh.full));
    load_tile(kq + kHalfTile, kTile, &tq, hk, static_cast<int>(t0), smem_u32(&sh.full));
  }
  if (warp == 7) {
    tmem_alloc(smem_u32(&sh.tmem), 128);
    tmem_relinquish();
  }
  // the gates' inputs, of half of a value head's tokens a warp: asked for here, used while the
  // rows' product runs
  const int gate = warp >> 1, token = lane + 32 * (warp & 1);
  uint16_t ga = 0, gb = 0;
  float rate = 0.0f, dt_bias = 0.0f;
  if (gate < heads) {
    rate = __ldg(p.d.a_log + h0 + gate), dt_bias = __ldg(p.d.dt_bias + h0 + gate);
    if (token < n) {
      ga = *reinterpret_cast<const uint16_t*>(p.d.a + (t0 + token) * p.d.at + h0 + gate);
      gb = *reinterpret_cast<const uint16_t*>(p.d.b + (t0 + token) * p.d.bt + h0 + gate);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();   // with its tensor memory in hand: a kernel behind may take the rest
  const uint32_t tmem = sh.tmem, lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.full), 0, &sh.abort_flag));
  ok = __syncthreads_and(ok);

  if (ok) {
    // a thread's half of its row: its sum of squares and its largest entry, then F16
    const uint32_t at = kq + half * kTile + row * 128;
    uint4 raw[8];
    float2 ss = make_float2(0.0f, 0.0f);
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      raw[v] = lds128(at + ((v ^ (i & 7)) << 4));
      if (i >= n) raw[v] = make_uint4(0u, 0u, 0u, 0u);   // the next request's, or what lies behind
      float f[8];
      widen8(raw[v], f);
#pragma unroll
      for (int e = 0; e < 8; e += 2) ss = __ffma2_rn(make_float2(f[e], f[e + 1]), make_float2(f[e], f[e + 1]), ss);
      m = max_abs_bf16x2(max_abs_bf16x2(m, raw[v].x), raw[v].y);
      m = max_abs_bf16x2(max_abs_bf16x2(m, raw[v].z), raw[v].w);
    }
    float* const squares = sh.A;                       // of each half of a row, and the largest behind them
    float* const largest = sh.A + 4 * kChunk;
    squares[half * 2 * kChunk + row] = ss.x + ss.y;
    largest[half * 2 * kChunk + row] = max_bf16x2(m);
    __syncthreads();
    const float top = fmaxf(largest[row], largest[2 * kChunk + row]);
    const float to_one = top > 0.0f ? power_for(top, 0) : 1.0f;
    // rsqrt and the power taken back, in an order that does not overflow with it
    const float c = i < n ? rsqrtf(squares[row] + squares[2 * kChunk + row] + p.d.eps) / to_one : 0.0f;
    if (half == 0) sh.factor[row] = c;
    const float2 s2 = make_float2(to_one, to_one);
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      float f[8];
      widen8(raw[v], f);
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = __fmul2_rn(make_float2(f[2 * e], f[2 * e + 1]), s2);
        w[e] = pack_f16x2(x.x, x.y);
      }
      sts128(at + ((v ^ (i & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
    }
    fence_proxy_async_smem();
  }
  __syncthreads();
  if (ok && warp == 0 && elect_one()) {
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const uint64_t d = smem_desc_sw128(kq) + (s >> 2) * (kTile >> 4) + 2 * (s & 3);
      umma_f16(tmem, d, d, idesc_f16(128, 64), s > 0);
    }
    umma_commit(smem_u32(&sh.gram));
    if (sub == 0) {
      bulk_store(kq_at(p, slot, hk), kq, kKq);
      bulk_commit();
    }
  }
  __syncwarp();
  if (gate < heads) {
    const float alpha = token < n ? expf(log_decay(bf16_bits_to_f32(ga), dt_bias, expf(rate))) : 1.0f;
    const float product = scan_product(alpha, lane);
    sh.alpha[gate][token] = alpha;
    sh.beta[gate][token] = token < n ? beta_of(bf16_bits_to_f32(gb)) : 0.0f;
    sh.within[gate][token] = product;                  // of its half of the chunk
    sh.behind[gate][token] = scan_product_behind(alpha, lane);
  }
  ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.gram), 0, &sh.abort_flag));
  if (warp == 0) bulk_wait_read_all();                 // the K and Q rows have left shared memory
  ok = __syncthreads_and(ok);

  for (int g = 0; ok && g < heads; ++g) {
    const int h = h0 + g;
    if (g > 0) {                                       // the blob ahead has left shared memory
      if (warp == 0) bulk_wait_read_all();
      __syncthreads();
    }
    tc_fence_after();
    {
      // rows of A, and of P cut into its parts where P T will be; columns 32 half + 31 down to 32 half
      float w[32];
      tmem_ld32(tmem + lanes + 32 * half, w);
      const float c = sh.factor[row], f0 = query ? c * 64.0f : c * sh.beta[g][i];
      float ratio = half == 0 && i >= 32 ? sh.within[g][i] : 1.0f;   // Gamma_i / Gamma_j
#pragma unroll
      for (int jj = 31; jj >= 0; --jj) {
        const int j = 32 * half + jj;
        if (jj < 31 && j < i) ratio *= sh.alpha[g][j + 1];
        const float f = f0 * sh.factor[j] * ratio;
        w[jj] = (query ? j <= i : j < i) && i < n ? f * w[jj] : 0.0f;
      }
      if (query) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(make_float2(w[8 * v + 2 * e], w[8 * v + 2 * e + 1]), hi[e], lo[e]);
          const uint32_t at = blob + kHalfTile + i * 128 + (((4 * half + v) ^ (i & 7)) << 4);
          sts128(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
          sts128(at + kTile, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
      } else {
        float4* a = reinterpret_cast<float4*>(sh.A + i * kPitch + 32 * half);
#pragma unroll
        for (int v = 0; v < 8; ++v) a[v] = make_float4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
      }
    }
    __syncthreads();
    if (warp < 2) {
      // column j of a diagonal block: T_ij = 1_ij - sum_{l < i} A_il T_lj
      const int at = 16 * (tid >> 4), j = tid & 15;
      const float* a = sh.A + at * kPitch + at;
      float t[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float s = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int l = 0; l < r; l += 4) {
          const float4 x = *reinterpret_cast<const float4*>(a + r * kPitch + l);
          s = fmaf(x.x, t[l], s);
          if (l + 1 < r) s2 = fmaf(x.y, t[l + 1], s2);
          if (l + 2 < r) s = fmaf(x.z, t[l + 2], s);
          if (l + 3 < r) s2 = fmaf(x.w, t[l + 3], s2);
        }
        t[r] = (r == j ? 1.0f : 0.0f) - (s + s2);
      }
      __syncwarp();                                    // A's blocks have been read
#pragma unroll
      for (int r = 0; r < 16; ++r) sh.A[(at + r) * kPitch + at + j] = t[r];
    }
    __syncthreads();
    float c[4];
    float* const Z = reinterpret_cast<float*>(base);   // where T's parts will be
    {
      // the two lower blocks of 16 rows, next to the diagonal: four warps, half of one each
      const int a0 = 32 * (warp >> 1), b0 = a0 + 16, n0 = 8 * (warp & 1);
      float* const z = Z + 16 * (warp >> 1) * kPitchZ + n0;
      if (warp < 4) {
        small_product<16>(sh.A + b0 * kPitch + a0, sh.A + a0 * kPitch + a0 + n0, lane, c);
        store_piece<kPitchZ>(z, lane, c, 1.0f);
      }
      __syncthreads();
      if (warp < 4) {
        small_product<16, kPitchZ>(sh.A + b0 * kPitch + b0, z, lane, c);
        store_piece(sh.A + b0 * kPitch + a0 + n0, lane, c, -1.0f);
      }
    }
    __syncthreads();
    {
      // the lower block of 32 rows: 16 x 8 of it a warp
      const int r0 = 32 + 16 * (warp >> 2), n0 = 8 * (warp & 3);
      float* const z = Z + 16 * (warp >> 2) * kPitchZ + n0;
      small_product<32>(sh.A + r0 * kPitch, sh.A + n0, lane, c);
      store_piece<kPitchZ>(z, lane, c, 1.0f);
      __syncthreads();
      small_product<32, kPitchZ>(sh.A + r0 * kPitch + 32, Z + n0, lane, c);
      store_piece(sh.A + r0 * kPitch + n0, lane, c, -1.0f);
    }
    __syncthreads();
    {
      const int r = tid >> 2, c0 = 16 * (tid & 3);     // T's parts: 16 columns a thread
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 x = *reinterpret_cast<const float4*>(sh.A + r * kPitch + c0 + 8 * v + 4 * e);
          split2(make_float2(x.x * kTScale, x.y * kTScale), hi[2 * e], lo[2 * e]);
          split2(make_float2(x.z * kTScale, x.w * kTScale), hi[2 * e + 1], lo[2 * e + 1]);
        }
        const uint32_t at = blob + r * 128 + ((((c0 >> 3) + v) ^ (r & 7)) << 4);
        sts128(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        sts128(at + kTile, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      }
      float* scalars = reinterpret_cast<float*>(base + kScalars);
      if (tid < kChunk) {
        const float beta = sh.beta[g][tid], ck = sh.factor[tid];
        const float gamma = (tid >= 32 ? sh.within[g][31] : 1.0f) * sh.within[g][tid];
        const float rest = sh.behind[g][tid] * (tid >= 32 ? 1.0f : sh.within[g][kChunk - 1]);
        scalars[kBeta + tid] = beta;
        scalars[kKey + tid] = -beta * gamma * ck;
        scalars[kQuery + tid] = gamma * sh.factor[kChunk + tid] * kTScale;
        scalars[kUpdate + tid] = rest * ck * (1.0f / kTScale);
        if (tid == kChunk - 1) scalars[kGammaC] = gamma;
      }
      fence_proxy_async_smem();
    }
    __syncthreads();
    if (warp == 0 && elect_one()) {
      // rows 64 - 127 of the left operand are whatever lies behind P's: lanes that nothing reads
      const uint64_t dp = smem_desc_sw128(blob + kHalfTile), dt = smem_desc_sw128_mn(blob, kHalfTile);
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int t = 0; t < 2 - a; ++t)
#pragma unroll
          for (int s = 0; s < 4; ++s)                  // 16 rows of T a step
            umma_f16(tmem + 64, dp + a * (kTile >> 4) + 2 * s, dt + t * (kTile >> 4) + 128 * s, idesc_f16_mn(128, 64),
                     a || t || s);
      umma_commit(smem_u32(&sh.product));
    }
    __syncwarp();
    ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.product), g & 1, &sh.abort_flag));
    if (ok && !query) {
      tc_fence_after();
      float w[32];
      tmem_ld32(tmem + lanes + 64 + 32 * half, w);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          split2(make_float2(w[8 * v + 2 * e] * (1.0f / 64.0f), w[8 * v + 2 * e + 1] * (1.0f / 64.0f)), hi[e], lo[e]);
        const uint32_t at = blob + kHalfTile + i * 128 + (((4 * half + v) ^ (i & 7)) << 4);
        sts128(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        sts128(at + kTile, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      }
      fence_proxy_async_smem();
      tc_fence_before();
    }
    ok = __syncthreads_and(ok);
    if (ok && warp == 0 && elect_one()) {
      bulk_store(blob_at(p, slot, h), blob, kBlob);
      bulk_commit();
    }
    __syncwarp();
  }
  if (!ok) {
    sh.abort_flag = 1;
    if (tid == 0) atomicExch(&g_delta_err, static_cast<int>(BFP8_ERR_TIMEOUT));
  }
  if (warp == 0) bulk_wait_all();
  tc_fence_before();
  __syncthreads();
  if (warp == 7) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

// ---- the walk down a request's chunks. Lane r of tensor memory is row r of S (a value), its
// columns keys or tokens: what one product leaves in a lane is, scaled and cut, the next one's
// operand from tensor memory, so nothing passes between threads but the row's power of two. Two
// warpgroups share the columns: keys 0 - 63 and 64 - 127 of S (kept in registers), tokens 0 - 31
// and 32 - 63.
//
// A row's power of two brings the larger of its state's entries and of what its values write near
// 2^2: the chunk's largest beta times its largest |v|, as all that enters of a value is beta v. With
// both below 2^6, neither u nor S reaches 2^14 in the chunk: a row's length grows by beta |v| a
// token at most, |S| <= sqrt(128) 2^6 + 64 2^6, and |u| <= beta |v| + |S|. With the larger above 2^-3,
// the rests' 2^-25 is 2^-22 of it. (With |v| for beta |v|, a state of writes with beta about e^-10
// was right to 10 bits; looking for the largest beta takes 8192 tokens of 32 heads from 283 to 286
// us.) It is looked at once a chunk: Gamma_C times the state's largest
// at the chunk's begin, the largest update, and the next chunk's values stand for what the next
// chunk meets. So where a head forgets within a chunk, what comes after keeps 2^-22 of what was
// forgotten there, not of itself.
//
// What the chain of three products does not need runs beside it: S0 Q^T and the out rows of
// T behind the products that the chain waits for, the out rows' arithmetic in a third warpgroup,
// the values' turning (a row of S wants a value's tokens side by side) in two warps. Each product
// begins on the first half of its operand while the second is cut.
//
// Bound by the chain: 4,600 clocks a chunk and block, 2.4 us, one block an SM. The products the
// chain waits for are 1,410 of them at the tensor cores' rate (64 columns of 128 lanes by 16 take
// 32 clocks, 128 take 64); reading, cutting and handing over r, u and S are 500, 540 and 1,200,
// and each hand-over between threads and tensor cores costs 200 to 300 of waiting. On the way,
// 8192 tokens of 32 heads: 4.7 us a chunk with three BF16 parts a value (the cuts' masks and
// permutes run at half rate), 3.1 with two F16 parts, 2.5 with the out rows aside and the values
// turned. Sixteen warps of rows instead of eight: 2.9 us. Out rows by bulk copies of 256 bytes: 80
// clocks of the issuing warp each, which then was the bound.
//
// The sixteen warps' code does not fit what is fetched fast, and the SMs share what feeds it: with
// the loops below unrolled, 128 blocks that write rows of out took 3.4 us a chunk where 64 took 2.7
// (2.3 of 10 waiting warps without an instruction, against 0.4). So what the chain does not wait
// for is rolled (rows of out by 16 tokens, S0 Q^T, T's rows of out, the turning), and a change of a row's power
// stands apart: 2.85 and 2.55. The chain's own products rolled too cost it 150 clocks each.
constexpr int kRowWarps = 8, kOutWarps = 4;
constexpr int kWalkThreads = 32 * (kRowWarps + kOutWarps + 4);   // and a warp of products and one of loads
constexpr int kBlobAt = kKq;
constexpr int kStageBytes = kBlobAt + (kBlob + 1023) / 1024 * 1024;
constexpr int kStages = 2;
constexpr int kValuesAt = kStages * kStageBytes, kTurnedAt = kValuesAt + 2 * kTile, kOutAt = kTurnedAt + 2 * kTile;
constexpr int kOutPitch = 320;                         // of 64 rows of 128 BF16: two rows' banks apart
constexpr int kWalkSharedAt = kOutAt + kChunk * kOutPitch;
// A state on its way from and to memory, in a stage's place: 16 lanes copy 256 bytes of a row, and
// a lane's own row lies across the banks from its neighbours'. (Lanes that read their own rows
// from memory, 512 bytes apart, took 11,000 clocks for them.)
constexpr int kRowPitch = 528;
static_assert(kD * kRowPitch <= kStageBytes, "a state fits a stage's place");
// Columns of tensor memory. 16 keys or tokens of one part take 8. The parts of S lie where u K
// comes (read before they are written anew), those of r where S K^T came, those of u where u
// came; each warpgroup overwrites only columns that it alone has read.
constexpr uint32_t kColNew = 0, kColX = 128, kColY = 192, kColU = 256, kColO = 320;
BFP8_DEV uint32_t col_s(int part, int step) {          // step: 16 keys
  return kColNew + 64 * (step >> 2) + 32 * part + 8 * (step & 3);
}
BFP8_DEV uint32_t col_r(int part, int step) {          // step: 16 tokens
  return kColX + 32 * (step >> 1) + 16 * part + 8 * (step & 1);
}
BFP8_DEV uint32_t col_u(int part, int step) { return col_r(part, step) + (kColU - kColX); }

// 8 columns of this thread's lane written; complete after tmem_wait_st().
BFP8_DEV void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}

//
// Few heads' long prompts leave most SMs idle, so their chunks are walked in segments, all at
// once. What a segment makes of the state ahead of it is S -> S M + N, row by row of S: a walk
// from zeros leaves N, and one from the identity, without values, M. The first walk takes the
// first segment of each head (from the state itself, with its rows of out), and N and M of the
// others but the last; the states between the segments are then S M + N one behind another; and
// the second walk takes the other segments from those. Where the N and M do not all find an SM
// beside the first segments, they come in waves of shorter segments, and the first ones are as
// long as the waves. That is two segments' time, or a wave more, in place of the whole prompt's.
struct WalkShared {
  float most[2][2][kD];                                // what each half of a row offers for its power of two
  float power[2][kD];                                  // a chunk's, for its rows of out
  float2 beta[2];                                      // of the chunk whose values are turned: the largest of each 32 tokens
  uint64_t full[kStages], empty[kStages], v_full[2], v_empty[2], turned[2], taken[2];
  uint64_t s_full[2], x_done, r_full[2], u_done, p_full[2], o_done, y_free, new_done, told, out_full, begun, drained;
  uint32_t tmem;
  int abort_flag;
};
constexpr int kWalkSmem = 1024 + kWalkSharedAt + static_cast<int>(sizeof(WalkShared));

__global__ void __launch_bounds__(kWalkThreads, 1) delta_walk_kernel(const __grid_constant__ CUtensorMap tv,
                                                                     const ChunkParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  WalkShared& sh = *reinterpret_cast<WalkShared*>(base + kWalkSharedAt);
  const uint32_t stages = smem_u32(base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kMmaWarp = kRowWarps + kOutWarps;
  // The kernel ahead (the chunks' first one, or the join) waited for what came before it ahead of
  // letting this one begin: lengths, values and the requests' states are there already. What it
  // writes itself, the loads' warp waits for, and the rows' where they begin from a join's state.
  if (tid == 0) tma_prefetch_desc(&tv);
  const int pairs = p.d.req.batch * p.d.v_heads, job = blockIdx.x / pairs;
  const int h = blockIdx.x % pairs % p.d.v_heads;
  int b = blockIdx.x % pairs / p.d.v_heads;
  int slot_in, slot_out;
  if (p.longest_first) {
    // of its 32 requests the one with b % 32 ahead of it, by the power of two below its chunks; all
    // of their slots are asked for beside their lengths
    const int window = b & ~31, mine = window + lane;
    int64_t unused;
    const bool there = mine < p.d.req.batch;
    slot_in = there ? static_cast<int>(slot_of(p.d.req, p.d.req.slots_in, mine)) : -1;
    slot_out = there ? static_cast<int>(slot_of(p.d.req, p.d.req.slots_out, mine)) : -1;
    const int size = there ? 32 - __clz(static_cast<int>((chunked_len(p.d, mine, unused) + kChunk - 1) >> kShift)) : 0;
    uint32_t among = __ballot_sync(0xffffffffu, there);
    int rank = b & 31;
#pragma unroll
    for (int bit = 16; bit > 0; bit >>= 1) {
      const uint32_t larger = __ballot_sync(0xffffffffu, size & bit) & among;
      const int n = __popc(larger);
      among = rank < n ? larger : among & ~larger;
      rank -= rank < n ? 0 : n;
    }
    const bool it = (among >> lane & 1u) && __popc(among & ((1u << lane) - 1u)) == rank;
    const int found = __ffs(__ballot_sync(0xffffffffu, it)) - 1;
    b = window + found;
    slot_in = __shfl_sync(0xffffffffu, slot_in, found);
    slot_out = __shfl_sync(0xffffffffu, slot_out, found);
  } else {
    slot_in = static_cast<int>(slot_of(p.d.req, p.d.req.slots_in, b));
    slot_out = static_cast<int>(slot_of(p.d.req, p.d.req.slots_out, b));
  }
  const int pair = b * p.d.v_heads + h;
  // the first walk's jobs: the first segment with its rows of out, then N and M of each other but
  // the last (which so read the same chunks at about a time); the second's: the others
  const bool map = !p.second_walk && job && !(job & 1);
  const int segment = p.second_walk ? job + 1 : (job + 1) >> 1;
  const bool rows_out = p.second_walk || segment == 0;
  int64_t first;
  int64_t len = chunked_len(p.d, b, first);
  const int64_t segment_tokens = static_cast<int64_t>(p.segment_chunks) << kShift;
  const int begin = segment ? segment + p.lead : 0;    // in segments' lengths
  const bool last = len <= (segment + p.lead + 1) * segment_tokens;
  if (len <= begin * segment_tokens || (last && !rows_out)) {
    pdl_wait();                                        // nothing behind this grid runs ahead of the one before it
    return;
  }
  first += begin * segment_tokens;
  len = last ? len - begin * segment_tokens : (segment + p.lead + 1 - begin) * segment_tokens;
  float* const between = p.ends + (static_cast<int64_t>(pair) * (p.segments - 1) + segment) * (kD * kD);
  const int chunks = static_cast<int>((len + kChunk - 1) >> kShift);
  const int tail = static_cast<int>(len - (static_cast<int64_t>(chunks - 1) << kShift));

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), kRowWarps + (rows_out ? kOutWarps : 0) + 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sh.v_full[s]), 1);
      mbar_init(smem_u32(&sh.v_empty[s]), 2);
      mbar_init(smem_u32(&sh.turned[s]), 2);
      mbar_init(smem_u32(&sh.taken[s]), kRowWarps);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(smem_u32(&sh.s_full[q]), kRowWarps);
      mbar_init(smem_u32(&sh.r_full[q]), kRowWarps);
      mbar_init(smem_u32(&sh.p_full[q]), kRowWarps);
    }
    mbar_init(smem_u32(&sh.told), kRowWarps);
    mbar_init(smem_u32(&sh.begun), kRowWarps);
    mbar_init(smem_u32(&sh.y_free), kOutWarps);
    mbar_init(smem_u32(&sh.out_full), kOutWarps);
    mbar_init(smem_u32(&sh.x_done), 1);
    mbar_init(smem_u32(&sh.u_done), 1);
    mbar_init(smem_u32(&sh.o_done), 1);
    mbar_init(smem_u32(&sh.new_done), 1);
    mbar_init(smem_u32(&sh.drained), 1);
    sh.abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();   // with its tensor memory in hand, as a kernel behind may want it too
  const uint32_t tmem = sh.tmem;
  const volatile int* abort_flag = &sh.abort_flag;
  bool ok = true;
  auto wait = [&](uint64_t& bar, uint32_t parity) {
    ok = ok && __all_sync(0xffffffffu, warp < kRowWarps || warp == kMmaWarp
                                           ? mbar_wait(smem_u32(&bar), parity, abort_flag)
                                           : mbar_wait_sleep(smem_u32(&bar), parity, abort_flag));
    return ok;
  };
  auto tell_bar = [&](uint64_t& bar) {                 // one arrival a warp
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bar));
  };

  if (warp >= kMmaWarp) {
    warpgroup_reg_dealloc<64>();
    if (warp == kMmaWarp) {
      // ---------------------------------------------- products
      constexpr uint32_t kN64 = idesc_f16(128, 64), kKeys = idesc_f16_mn(128, 128);
      for (int c = 0; c < chunks; ++c) {
        const int s = c % kStages;
        const uint32_t at = stages + s * kStageBytes;
        const uint64_t dk = smem_desc_sw128(at), dt = smem_desc_sw128(at + kBlobAt), dn = smem_desc_sw128_mn(at, kTile);
        if (!wait(sh.full[s], (c / kStages) & 1)) break;
#pragma unroll
        for (int q = 0; q < 2; ++q) {                  // 32 keys of each warpgroup's
          if (!wait(sh.s_full[q], c & 1)) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int k = 4 * (e >> 1) + 2 * q + (e & 1);
                umma_f16_ts(tmem + kColX, tmem + col_s(part, k), dk + (k >> 2) * (kTile >> 4) + 2 * (k & 3), kN64,
                            q || part || e);
              }
            if (q == 1) umma_commit(smem_u32(&sh.x_done));
          }
          __syncwarp();
        }
        if (!ok || (rows_out && !wait(sh.y_free, (c & 1) ^ 1))) break;
        tc_fence_after();
        if (rows_out && elect_one()) {
#pragma unroll 1
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f16_ts(tmem + kColY, tmem + col_s(i >> 1, 4 * (i & 1) + k),
                          dk + ((kHalfTile + (i & 1) * kTile) >> 4) + 2 * k, kN64, i || k);
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 2; ++q) {                  // 16 tokens of each warpgroup's
          if (!wait(sh.r_full[q], c & 1)) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
              for (int t = 0; t < 2 - a; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int k = q + 2 * e;
                  umma_f16_ts(tmem + kColU, tmem + col_r(a, k), dt + t * (kTile >> 4) + 2 * k, kN64, q || a || t || e);
                }
            if (q == 1) umma_commit(smem_u32(&sh.u_done));
          }
          __syncwarp();
        }
        if (!ok) break;
        if (rows_out && elect_one()) {
#pragma unroll 1
          for (int i = 0; i < 3; ++i) {
            const int a = i >> 1, t = i & 1;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f16_ts(tmem + kColO, tmem + col_r(a, k), dt + ((kHalfTile + t * kTile) >> 4) + 2 * k, kN64, i || k);
          }
          umma_commit(smem_u32(&sh.o_done));
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (!wait(sh.p_full[q], c & 1)) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int e = 0; e < 2; ++e) {            // 16 tokens a step: 16 rows of 128 bytes
                const int k = q + 2 * e;
                umma_f16_ts(tmem + kColNew, tmem + col_u(part, k), dn + 128 * k, kKeys, q || part || e);
              }
            if (q == 1) {
              umma_commit(smem_u32(&sh.new_done));
              umma_commit(smem_u32(&sh.empty[s]));
            }
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      if (!ok) {   // products in flight end before tensor memory is given back
        const int none = 0;
        if (elect_one()) umma_commit(smem_u32(&sh.drained));
        __syncwarp();
        mbar_wait(smem_u32(&sh.drained), 0, &none);
      }
    } else if (warp == kMmaWarp + 1) {
      // ---------------------------------------------- loads, a chunk ahead; values two
      const int64_t key = tile_key(p.d.req, b, kShift) + static_cast<int64_t>(begin) * p.segment_chunks;
      int got = 0, values = map ? chunks : 0;          // chunks asked for; a map has no values
      auto load_values = [&]() {
        const int s = values % 2;
        if (values == chunks || !wait(sh.v_empty[s], ((values / 2) & 1) ^ 1)) return;
        if (elect_one()) {
          mbar_arrive_expect_tx(smem_u32(&sh.v_full[s]), kTile);
          load_tile(stages + kValuesAt + s * kTile, kHalfTile, &tv, h, static_cast<int>(first) + values * kChunk,
                    smem_u32(&sh.v_full[s]));
        }
        __syncwarp();
        ++values;
      };
      load_values();
      pdl_wait();
      while (ok && got < chunks) {
        const int s = got % kStages;
        if (got == 1 && !wait(sh.begun, 0)) break;     // the state that came through this stage's place is held
        if (!wait(sh.empty[s], ((got / kStages) & 1) ^ 1)) break;
        if (elect_one()) {
          const uint32_t dst = stages + s * kStageBytes, bar = smem_u32(&sh.full[s]);
          mbar_arrive_expect_tx(bar, kKq + kBlob);
          bulk_load(dst, kq_at(p, key + got, h / p.d.group), kKq, bar);
          bulk_load(dst + kBlobAt, blob_at(p, key + got, h), kBlob, bar);
        }
        __syncwarp();
        ++got;
        load_values();
      }
      if (!ok) {   // what was issued lands before the block ends
        const int none = 0;
        for (int d = got < kStages ? 0 : got - kStages; d < got; ++d)
          mbar_wait(smem_u32(&sh.full[d % kStages]), (d / kStages) & 1, &none);
        for (int d = values < 2 ? 0 : values - 2; !map && d < values; ++d)
          mbar_wait(smem_u32(&sh.v_full[d % 2]), (d / 2) & 1, &none);
      }
    } else {
      // ---------------------------------------------- values turned: of each value its tokens, two a word
      const int half = warp - kMmaWarp - 2;            // of the values
      // of tokens too: their gate b, whose largest has the largest beta
      const uint16_t* gate = reinterpret_cast<const uint16_t*>(p.d.b) + (first + 32 * half + lane) * p.d.bt + h;
      int left = static_cast<int>(len) - 32 * half - lane;
      for (int c = 0; !map && c < chunks; ++c) {
        const float b = left > 0 ? bf16_bits_to_f32(__ldcg(gate)) : -INFINITY;
        gate += kChunk * p.d.bt, left -= kChunk;
        if (!wait(sh.v_full[c & 1], (c >> 1) & 1) || !wait(sh.taken[c & 1], ((c >> 1) & 1) ^ 1)) break;
        // a lane's row of the four 8 x 8 pieces that the warp turns at once: 32 tokens of 8 values
        const uint32_t src = stages + kValuesAt + (c & 1) * kTile + half * kHalfTile + lane * 128;
        const uint32_t dst = stages + kTurnedAt + (c & 1) * kTile + (64 * half + (lane >> 2)) * 128 + (lane & 3) * 4;
#pragma unroll 1
        for (int g = 0; g < 2; ++g)
#pragma unroll 2
          for (int v = 0; v < 8; ++v) {
            uint32_t w[4];
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(src + 32 * g * 128 + ((v ^ (lane & 7)) << 4))
                         : "memory");
#pragma unroll
            for (int e = 0; e < 4; ++e)
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + 8 * v * 128 + (((4 * g + e) ^ (lane >> 2)) << 4)), "r"(w[e])
                           : "memory");
          }
        const float beta = sigmoid(fmaxf(warp_max(b), -87.0f));   // e^-87 bounds what is subnormal below it
        if (lane == 0) (half ? sh.beta[c & 1].y : sh.beta[c & 1].x) = beta;
        tell_bar(sh.turned[c & 1]);
        if (lane == 0) mbar_arrive(smem_u32(&sh.v_empty[c & 1]));
      }
    }
  } else if (warp >= kRowWarps) {
    // ------------------------------------------------ rows of out: a value a thread, 64 tokens
    warpgroup_reg_dealloc<112>();
    const int r = (warp & 3) * 32 + lane;
    const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const bool odd = lane & 1;
    for (int c = 0; rows_out && c < chunks; ++c) {
      const int s = c % kStages;
      const float* scalars = reinterpret_cast<const float*>(base + s * kStageBytes + kBlobAt + kScalars);
      if (!wait(sh.full[s], (c / kStages) & 1) || !wait(sh.o_done, c & 1)) break;
      tc_fence_after();
      const float back = p.d.scale * (1.0f / kTScale) / sh.power[c & 1][r];
      const float2 back2 = make_float2(back, back);
      // two values of one token make a word: even lanes have the pair's even tokens, odd ones the odd
      const uint32_t at = stages + kOutAt + (odd ? kOutPitch : 0) + (r & ~1) * 2;
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        uint32_t q[16], o[16], v[8];
        tmem_ld16(mine + kColY + 16 * g, q);
        tmem_ld16(mine + kColO + 16 * g, o);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 f = *reinterpret_cast<const float2*>(scalars + kQuery + 16 * g + j);
          const float2 w = __fmul2_rn(__ffma2_rn(f, make_float2(__uint_as_float(q[j]), __uint_as_float(q[j + 1])),
                                                 make_float2(__uint_as_float(o[j]), __uint_as_float(o[j + 1]))), back2);
          v[j / 2] = pack_bf16x2(w.x, w.y);
        }
        if (g == 3) {
          tc_fence_before();
          tell_bar(sh.y_free);
          if (lane == 0) mbar_arrive(smem_u32(&sh.empty[s]));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t w = __shfl_xor_sync(0xffffffffu, v[j], 1);
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + (16 * g + 2 * j) * kOutPitch),
                       "r"(odd ? __byte_perm(w, v[j], 0x7632) : __byte_perm(v[j], w, 0x5410))
                       : "memory");
        }
      }
      tell_bar(sh.out_full);
      if (!wait(sh.out_full, 0)) break;
      // a row of 256 bytes to 16 lanes
      const int n = c == chunks - 1 ? tail : kChunk;
      __nv_bfloat16* out = p.d.out + (first + static_cast<int64_t>(c) * kChunk) * p.d.ot + h * p.d.oh + (lane & 15) * 8;
#pragma unroll 4
      for (int e = 0; e < 8; ++e) {
        const int t = 8 * e + 2 * (warp & 3) + (lane >> 4);
        const uint4 w = lds128(stages + kOutAt + t * kOutPitch + (lane & 15) * 16);
        if (t < n) *reinterpret_cast<uint4*>(out + t * p.d.ot) = w;
      }
      tell_bar(sh.out_full);                           // the tile may be written again
      if (!wait(sh.out_full, 1)) break;
    }
  } else {
    // ------------------------------------------------ rows of S
    warpgroup_reg_alloc<168>();
    const int wg = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // where S comes from and goes to: the request's slots, or between the segments
    const float* from = nullptr;
    float* to = nullptr;
    const int64_t in_row = (r - lane) * kD + 64 * wg + (lane >> 4) * kD + 4 * (lane & 15);   // of two rows a copy
    if (segment == 0) {
      if (slot_in >= 0) from = p.d.state + slot_in * p.d.s_slot + h * p.d.s_head + in_row;
    } else if (p.second_walk) {
      pdl_wait();
      from = between - kD * kD + in_row;
    }
    if (last) {
      if (slot_out >= 0) to = p.d.state + slot_out * p.d.s_slot + h * p.d.s_head + in_row;
    } else if (!p.second_walk) {
      to = (map ? p.maps + (between - p.ends) : between) + in_row;
    }
    const uint32_t own = r * kRowPitch + 256 * wg;     // the thread's piece of its row, and where it copies
    const uint32_t copy = (r - lane + (lane >> 4)) * kRowPitch + 256 * wg + 16 * (lane & 15);
    float S[64], most = 0.0f;                          // S is the row times `power`
    if (from) {
      const uint32_t at = stages + kStageBytes;
#pragma unroll
      for (int k = 0; k < 16; ++k) cp_async16(at + copy + 2 * k * kRowPitch, from + 2 * k * kD);
      cp_async_wait_all();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint4 w = lds128(at + own + 16 * k);
        const float4 f = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
        S[4 * k] = f.x, S[4 * k + 1] = f.y, S[4 * k + 2] = f.z, S[4 * k + 3] = f.w;
        most = fmaxf(most, fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(f.z), fabsf(f.w))));
      }
      fence_proxy_async_smem();                        // read, before a load writes there
    } else {
#pragma unroll
      for (int k = 0; k < 64; ++k) S[k] = map && r == 64 * wg + k ? 1.0f : 0.0f;
      if (map) most = 1.0f;
    }
    tell_bar(sh.begun);
    uint32_t values[16];                               // the next chunk's: 32 tokens' BF16, two a word
    float written = 0.0f;                              // their largest times the chunk's largest beta
    auto load_values = [&](int c) {
      const int left = (c == chunks - 1 ? tail : kChunk) - 32 * wg;
      if (map) {
#pragma unroll
        for (int j = 0; j < 16; ++j) values[j] = 0u;
        return;
      }
      if (!wait(sh.turned[c & 1], (c >> 1) & 1)) return;
      const uint32_t row = stages + kTurnedAt + (c & 1) * kTile + r * 128;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint4 w = lds128(row + (((4 * wg + v) ^ (r & 7)) << 4));
        values[4 * v] = w.x, values[4 * v + 1] = w.y, values[4 * v + 2] = w.z, values[4 * v + 3] = w.w;
      }
      const float2 beta = sh.beta[c & 1];
      tell_bar(sh.taken[c & 1]);
      if (left < 32) {
#pragma unroll
        for (int j = 0; j < 32; j += 2)
          values[j / 2] = j >= left ? 0u : j + 1 >= left ? values[j / 2] & 0xFFFFu : values[j / 2];
      }
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) top = max_abs_bf16x2(top, values[j]);
      written = fmaxf(beta.x, beta.y) * max_bf16x2(top);
    };
    uint32_t largest = 0;                              // of the parts of S, as F16 pairs
    auto hand_over = [&](int q) {                      // 32 keys
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        split2(make_float2(S[32 * q + 2 * k], S[32 * q + 2 * k + 1]), hi[k], lo[k]);
        largest = max_abs_f16x2(q || k ? largest : 0u, hi[k]);
      }
      tmem_st16(mine + col_s(0, 4 * wg + 2 * q), hi);
      tmem_st16(mine + col_s(1, 4 * wg + 2 * q), lo);
      tmem_wait_st();
      tc_fence_before();
      tell_bar(sh.s_full[q]);
    };
    load_values(0);
    most = fmaxf(most, written);
    sh.most[1][wg][r] = most;
    if (ok) {
      tell_bar(sh.told);
      wait(sh.told, 0);
    }
    const float first_most = fmaxf(most, sh.most[1][wg ^ 1][r]);
    float power = first_most > 0.0f ? power_for(first_most, 2) : 1.0f;
#pragma unroll
    for (int k = 0; k < 64; ++k) S[k] *= power;
    for (int c = 0; ok && c < chunks; ++c) {
      hand_over(0);
      hand_over(1);
      const int s = c % kStages;
      const bool more = c + 1 < chunks;
      const float* scalars = reinterpret_cast<const float*>(base + s * kStageBytes + kBlobAt + kScalars);
      // while S meets K: this chunk's values
      if (wg == 0) sh.power[c & 1][r] = power;
      if (!wait(sh.full[s], (c / kStages) & 1)) break;
      float2 y[16];
      const float2 power2 = make_float2(power, power);
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 be = *reinterpret_cast<const float4*>(scalars + kBeta + 32 * wg + j);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t v = values[j / 2 + e];
          y[j / 2 + e] = __fmul2_rn(make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u)),
                                    __fmul2_rn(e ? make_float2(be.z, be.w) : make_float2(be.x, be.y), power2));
        }
      }
      if (!wait(sh.x_done, c & 1)) break;
      tc_fence_after();
      {
        float x[32];
        tmem_ld32(mine + kColX + 32 * wg, x);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const int j = 16 * q + e;
            const float4 kf = *reinterpret_cast<const float4*>(scalars + kKey + 32 * wg + j);
            split2(__ffma2_rn(make_float2(kf.x, kf.y), make_float2(x[j], x[j + 1]), y[j / 2]), hi[e / 2], lo[e / 2]);
            split2(__ffma2_rn(make_float2(kf.z, kf.w), make_float2(x[j + 2], x[j + 3]), y[j / 2 + 1]), hi[e / 2 + 1],
                   lo[e / 2 + 1]);
          }
          tmem_st8(mine + col_r(0, 2 * wg + q), hi);
          tmem_st8(mine + col_r(1, 2 * wg + q), lo);
          tmem_wait_st();
          tc_fence_before();
          tell_bar(sh.r_full[q]);
        }
      }
      // while r meets T: the next chunk's values
      const float gamma = scalars[kGammaC];
      const float back = 1.0f / power;                 // offers are sizes as they are, not as they are held
      float offer = gamma * max_f16x2(largest) * back;
      if (more) {
        load_values(c + 1);
        offer = fmaxf(offer, written);
      }
      if (!wait(sh.u_done, c & 1)) break;
      tc_fence_after();
      {
        float u[32];
        uint32_t m = 0;
        tmem_ld32(mine + kColU + 32 * wg, u);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const int j = 16 * q + e;
            const float4 f = *reinterpret_cast<const float4*>(scalars + kUpdate + 32 * wg + j);
            split2(__fmul2_rn(make_float2(u[j], u[j + 1]), make_float2(f.x, f.y)), hi[e / 2], lo[e / 2]);
            split2(__fmul2_rn(make_float2(u[j + 2], u[j + 3]), make_float2(f.z, f.w)), hi[e / 2 + 1], lo[e / 2 + 1]);
            m = max_abs_f16x2(max_abs_f16x2(m, hi[e / 2]), hi[e / 2 + 1]);
          }
          tmem_st8(mine + col_u(0, 2 * wg + q), hi);
          tmem_st8(mine + col_u(1, 2 * wg + q), lo);
          if (q == 1) sh.most[c & 1][wg][r] = offer = fmaxf(offer, max_f16x2(m) * back);   // read behind the product
          tmem_wait_st();
          tc_fence_before();
          tell_bar(sh.p_full[q]);
        }
      }
      if (lane == 0) mbar_arrive(smem_u32(&sh.empty[s]));
      if (!wait(sh.new_done, c & 1) || !wait(sh.p_full[1], c & 1)) break;   // (the second for the other half's offer)
      tc_fence_after();
      offer = fmaxf(offer, sh.most[c & 1][wg ^ 1][r]);
      // two factors, each a power of two that a float holds, where the power changes by up to 2^250
      float step[2] = {1.0f, 1.0f};
      const float held = offer * power;
      if (offer > 0.0f && !(held >= 0x1p-3f && held < 0x1p6f)) {
        const float next = power_for(offer, 2);
        const int e = static_cast<int>(__float_as_uint(next) >> 23) - static_cast<int>(__float_as_uint(power) >> 23);
        step[0] = __uint_as_float(static_cast<uint32_t>(127 + (e >> 1)) << 23);
        step[1] = __uint_as_float(static_cast<uint32_t>(127 + e - (e >> 1)) << 23);
        power = next;
      }
      const float2 keep = make_float2(gamma, gamma);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float d[32];
        tmem_ld32(mine + kColNew + 64 * wg + 32 * q, d);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const float2 f = __ffma2_rn(keep, make_float2(S[32 * q + k], S[32 * q + k + 1]), make_float2(d[k], d[k + 1]));
          S[32 * q + k] = f.x, S[32 * q + k + 1] = f.y;
        }
      }
      if (__any_sync(0xffffffffu, step[0] != 1.0f || step[1] != 1.0f)) {
#pragma unroll
        for (int k = 0; k < 64; ++k) S[k] = S[k] * step[0] * step[1];
      }
    }
    if (ok && to) {
      // through the place of the stage that the last chunk does not have
      const uint32_t at = stages + (chunks % kStages) * kStageBytes;
      const float back = 1.0f / power;
#pragma unroll
      for (int k = 0; k < 16; ++k)
        sts128(at + own + 16 * k, make_uint4(__float_as_uint(S[4 * k] * back), __float_as_uint(S[4 * k + 1] * back),
                                             __float_as_uint(S[4 * k + 2] * back), __float_as_uint(S[4 * k + 3] * back)));
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint4 w = lds128(at + copy + 2 * k * kRowPitch);
        *reinterpret_cast<uint4*>(to + 2 * k * kD) = w;
      }
    }
  }
  if (!ok) {
    sh.abort_flag = 1;
    if (lane == 0) atomicExch(&g_delta_err, static_cast<int>(BFP8_ERR_TIMEOUT));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The states between a head's segments, one behind another: the end of each but the first is its
// N and becomes S M + N. A warp has four rows of S; a block copies a map at a time to shared
// memory, the next one while it multiplies where there is a next one.
constexpr int kJoinThreads = 256, kJoinRows = 4 * kJoinThreads / 32, kMapBytes = kD * kD * 4;
__global__ void __launch_bounds__(kJoinThreads) delta_join_kernel(const ChunkParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ float4 S[kD][kJoinThreads / 32];          // of a key, each warp's rows
  __shared__ uint64_t full[2];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = (smem_u32(smem_raw) + 127) & ~127u;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&full[0]), 1);
    mbar_init(smem_u32(&full[1]), 1);
    abort_flag = 0;
    mbar_fence_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kParts = kD / kJoinRows;
  const int pair = blockIdx.x / kParts, b = pair / p.d.v_heads;
  int64_t first;
  const int64_t len = chunked_len(p.d, b, first), segment_tokens = static_cast<int64_t>(p.segment_chunks) << kShift;
  const int n = static_cast<int>((len + segment_tokens - 1) / segment_tokens) - p.lead;   // segments; maps 1 .. n - 2
  if (n <= 2) return;
  const int64_t at = static_cast<int64_t>(pair) * (p.segments - 1) * (kD * kD);
  const int row = (blockIdx.x % kParts) * kJoinRows + 4 * warp;
  float* const ends = p.ends + at + row * kD + 4 * lane;
  const int ahead = p.segments > 3 ? 2 : 1;            // maps that the shared memory holds
  auto ask = [&](int g) {
    if (threadIdx.x != 0 || g > n - 2) return;
    const uint32_t bar = smem_u32(&full[(g - 1) % ahead]);
    mbar_arrive_expect_tx(bar, kMapBytes);
    bulk_load(ring + (g - 1) % ahead * kMapBytes, p.maps + at + static_cast<int64_t>(g) * (kD * kD), kMapBytes, bar);
  };
  __syncthreads();
  for (int g = 1; g <= ahead; ++g) ask(g);
  float4 s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = *reinterpret_cast<const float4*>(ends + i * kD);
  bool ok = true;
  for (int g = 1; ok && g <= n - 2; ++g) {
    S[4 * lane][warp] = make_float4(s[0].x, s[1].x, s[2].x, s[3].x);
    S[4 * lane + 1][warp] = make_float4(s[0].y, s[1].y, s[2].y, s[3].y);
    S[4 * lane + 2][warp] = make_float4(s[0].z, s[1].z, s[2].z, s[3].z);
    S[4 * lane + 3][warp] = make_float4(s[0].w, s[1].w, s[2].w, s[3].w);
    __syncwarp();
    float* const end = ends + g * (kD * kD);
    float4 n4[4];                                      // N, added behind the product
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      n4[i] = *reinterpret_cast<const float4*>(end + i * kD);
    }
    ok = __syncthreads_and(mbar_wait(smem_u32(&full[(g - 1) % ahead]), (g - 1) / ahead & 1, &abort_flag));
    if (!ok) break;
    const uint32_t map = ring + (g - 1) % ahead * kMapBytes + lane * 16;
#pragma unroll 8
    for (int l = 0; l < kD; ++l) {
      const uint4 w = lds128(map + l * (kD * 4));
      const float4 m = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
      const float4 c = S[l][warp];
      const float row[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = make_float2(row[i], row[i]);
        const float2 lo = __ffma2_rn(f, make_float2(m.x, m.y), make_float2(s[i].x, s[i].y));
        const float2 hi = __ffma2_rn(f, make_float2(m.z, m.w), make_float2(s[i].z, s[i].w));
        s[i] = make_float4(lo.x, lo.y, hi.x, hi.y);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = make_float4(s[i].x + n4[i].x, s[i].y + n4[i].y, s[i].z + n4[i].z, s[i].w + n4[i].w);
      *reinterpret_cast<float4*>(end + i * kD) = s[i];
    }
    __syncthreads();                                   // the map's place is free
    ask(g + ahead);
  }
  if (!ok && threadIdx.x == 0) atomicExch(&g_delta_err, static_cast<int>(BFP8_ERR_TIMEOUT));
}

int64_t longest_chunks(int64_t tokens, int64_t max_q_len) {
  return ((max_q_len < tokens ? max_q_len : tokens) + kChunk - 1) / kChunk;
}

// How the longest request's chunks are walked in segments: the count with the least time, in
// tenths of a microsecond. A chunk takes 2.5 us; a join 4.5 us; the two launches and the blocks'
// beginnings 18 us, and 5 us those of a further wave, of the first walk or the second.
constexpr int kMostSegments = 16, kMostWaves = 4;
struct Split {
  int segments, lead;
};
Split split_walk(int64_t chunks, int64_t pairs, int sms) {
  Split best{1, 0};
  int64_t least = 25 * chunks;
  for (int n = 3; n <= kMostSegments && pairs < sms; ++n) {
    const int64_t beside = sms - pairs, waves = (2 * pairs * (n - 2) + beside - 1) / beside;
    if (waves > kMostWaves) break;
    const int64_t all = waves + (pairs * (n - 1) + sms - 1) / sms;
    const int64_t time = 25 * all * ((chunks + n + waves - 2) / (n + waves - 1)) + 45 * (n - 2) + 50 * (all - 2) + 180;
    if (time < least) least = time, best = {n, static_cast<int>(waves - 1)};
  }
  return best;
}

// Where no request has more new tokens than this, each takes them one after the other. Of 48
// heads, 16 / 24 / 32 tokens one after the other against the chunks' kernels: one request 9.0,
// 11.9, 14.9 and 14.6 us; 4 requests 21, 29, 38 and 27; 16 requests 57, 82, 107 and 82; 64 requests
// 206, 302, 395 and 268. They meet between 20 and 24 but for few heads, which lose 3 us.
constexpr int64_t kStepTokens = 20;
// Beside longer ones, which run the chunks' kernels anyway, up to this many do: requests of 1 to
// 141 tokens (12, of 48 heads) take 49.2, 47.5, 47.8, 47.3 and 50.2 us with 2, 4, 8, 12 and 20. (One
// mix of lengths, in which 4, 8 and 12 are within its noise.)
constexpr int64_t kStepTokensBeside = 12;
static_assert(kStepTokens <= kMostSteps, "a request's steps fit shared memory");

int64_t chunk_slots(int64_t batch, int64_t tokens) { return (tokens >> kShift) + batch; }

int tile_map(CUtensorMap* map, const void* x, int64_t heads, int64_t tokens, int64_t head_stride, int64_t token_stride) {
  return make_tmap_3d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, kD, static_cast<uint64_t>(heads),
                      static_cast<uint64_t>(tokens), static_cast<uint64_t>(head_stride) * 2,
                      static_cast<uint64_t>(token_stride) * 2, 64, 1, kChunk, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool off16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

}  // namespace

// The chunks' part of the workspace, and behind it the states between segments: n - 1 ends and
// maps a head. As 2 (n - 2) blocks a head fit the waves that the SMs beside the first segments
// take, they are fewer than half the waves' for each SM.
size_t chunk_bytes(int64_t batch, int64_t tokens, int64_t qk_heads, int64_t v_heads) {
  const size_t n = static_cast<size_t>(chunk_slots(batch, tokens)) *
                   (static_cast<size_t>(qk_heads) * kKq + static_cast<size_t>(v_heads) * kBlob);
  return (n + 255) / 256 * 256;
}
size_t delta_rule_workspace_bytes(int64_t batch, int64_t tokens, int64_t max_q_len, int64_t qk_heads,
                                  int64_t v_heads, int sms) {
  if (max_q_len <= kStepTokens) return 0;
  const size_t between = split_walk(longest_chunks(tokens, max_q_len), 1, sms).segments > 1
                             ? static_cast<size_t>(sms) * kMostWaves * kD * kD * sizeof(float)
                             : 0;
  return chunk_bytes(batch, tokens, qk_heads, v_heads) + between;
}

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
  int sms = 0;
  int rc = BFP8_OK;
  if (a.max_q_len > kStepTokens) rc = sm_count(&sms);
  if (rc != BFP8_OK) return rc;
  const size_t need = delta_rule_workspace_bytes(a.batch, a.tokens, a.max_q_len, a.qk_heads, a.v_heads, sms);
  if (need && (!a.workspace || a.ws_bytes < need)) return BFP8_ERR_INVALID_ARG;
  if (need && (reinterpret_cast<uintptr_t>(a.workspace) % 256 ||
               chunk_slots(a.batch, a.tokens) * a.v_heads > 0x5FFFFFFF))   // a grid, beside 2^29 blocks of steps
    return BFP8_ERR_UNSUPPORTED;
  rc = check_device_ptrs({a.q_bf16, a.k_bf16, a.v_bf16, a.a_bf16, a.b_bf16, a.a_log, a.dt_bias, a.state,
                              a.out_bf16, a.q_offsets, a.slots_in, a.slots_out, need ? a.workspace : nullptr});
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
  p.step_len = need ? kStepTokensBeside : kStepTokens;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!need)
    return launch_dependent(delta_step_kernel,
                            dim3(static_cast<unsigned>(a.batch * a.v_heads * (kD / (8 * kStepWarps)))), 32 * kStepWarps,
                            0, st, p);
  CUtensorMap tq, tk, tv;
  rc = tile_map(&tq, a.q_bf16, a.qk_heads, a.tokens, a.q_stride_head, a.q_stride_token);
  if (rc == BFP8_OK) rc = tile_map(&tk, a.k_bf16, a.qk_heads, a.tokens, a.k_stride_head, a.k_stride_token);
  if (rc == BFP8_OK) rc = tile_map(&tv, a.v_bf16, a.v_heads, a.tokens, a.v_stride_head, a.v_stride_token);
  if (rc == BFP8_OK) rc = set_max_dynamic_smem(reinterpret_cast<const void*>(delta_prepare_kernel), kPrepSmem);
  if (rc == BFP8_OK) rc = set_max_dynamic_smem(reinterpret_cast<const void*>(delta_walk_kernel), kWalkSmem);
  const int64_t chunks = longest_chunks(a.tokens, a.max_q_len), pairs = a.batch * a.v_heads;
  const Split split = split_walk(chunks, pairs, sms);
  if (rc == BFP8_OK && split.segments > 1)             // whatever can fail does so ahead of the first launch
    rc = set_max_dynamic_smem(reinterpret_cast<const void*>(delta_join_kernel), 2 * kMapBytes + 128);
  if (rc != BFP8_OK) return rc;
  // Value heads of one key head share a block, which norms and multiplies their rows once (14,000
  // of its 24,500 clocks for one head), unless the blocks of one head each fit the GPU at once,
  // four to an SM. (4 requests of 128 tokens, 48 heads on 16: 43 us shared, 39 apart; 12 of 1 to
  // 141 tokens 47 and 51; 64 of 128 tokens 354 and 418.)
  ChunkParams cp{};
  cp.d = p;
  cp.ws = static_cast<uint8_t*>(a.workspace);
  cp.qk_heads = static_cast<int32_t>(a.qk_heads);
  const int64_t apart = (a.tokens / kChunk + a.batch) * a.v_heads;
  cp.per_block = apart <= 4 * sms ? 1 : p.group < kGroup ? p.group : kGroup;
  cp.subgroups = (p.group + cp.per_block - 1) / cp.per_block;
  cp.chunk_blocks = static_cast<uint32_t>(chunk_slots(a.batch, a.tokens) * a.qk_heads * cp.subgroups);
  const int64_t step_parts = a.batch * a.v_heads * (kD / (8 * (kPrepThreads / 32)));
  const int64_t step_blocks = step_parts < 4 * sms ? step_parts : 4 * sms;
  rc = launch_dependent(delta_prepare_kernel, dim3(cp.chunk_blocks + static_cast<unsigned>(step_blocks)), kPrepThreads,
                        kPrepSmem, st, tq, tk, cp);
  if (rc != BFP8_OK) return rc;
  cp.segments = split.segments;
  // More heads than SMs: the longest requests' blocks first, so that none of them begins last. (48
  // heads: 12 requests of 1 to 1300 tokens 220 -> 202 us, 24 of 1 to 1121 203 -> 188; 64 of 40
  // tokens each 249 -> 253.)
  cp.longest_first = a.batch > 1 && pairs > sms;
  cp.lead = split.lead;
  cp.segment_chunks = static_cast<int32_t>((chunks + cp.segments + cp.lead - 1) / (cp.segments + cp.lead));
  cp.ends = reinterpret_cast<float*>(cp.ws + chunk_bytes(a.batch, a.tokens, a.qk_heads, a.v_heads));
  cp.maps = cp.ends + static_cast<int64_t>(sms) * (kMostWaves / 2) * kD * kD;
  const int jobs = cp.segments > 1 ? 2 * cp.segments - 3 : 1;
  rc = launch_dependent(delta_walk_kernel, dim3(static_cast<unsigned>(pairs * jobs)), kWalkThreads, kWalkSmem, st, tv, cp);
  if (rc != BFP8_OK || cp.segments == 1) return rc;
  const int join_smem = (cp.segments > 3 ? 2 : 1) * kMapBytes + 128;
  rc = launch_dependent(delta_join_kernel, dim3(static_cast<unsigned>(pairs * (kD / kJoinRows))), kJoinThreads,
                        join_smem, st, cp);
  if (rc != BFP8_OK) return rc;
  cp.second_walk = 1;
  return launch_dependent(delta_walk_kernel, dim3(static_cast<unsigned>(pairs * (cp.segments - 1))), kWalkThreads,
                          kWalkSmem, st, tv, cp);
}

int delta_read_clear_error() {
  int v = 0;
  const int zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_delta_err, sizeof(int)) != cudaSuccess) return BFP8_ERR_CUDA;
  if (v != 0 && cudaMemcpyToSymbol(g_delta_err, &zero, sizeof(int)) != cudaSuccess) return BFP8_ERR_CUDA;
  return v == 0 ? BFP8_OK : v;
}

}  // namespace bfp8
