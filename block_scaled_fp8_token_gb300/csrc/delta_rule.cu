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
  if (n <= 0 || n > p.step_len) return;
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

// ------------------------------------------------------------------ chunks of 64 tokens
//
// Within a chunk of C tokens that begins with the state S0, write Gamma_i = alpha_0 .. alpha_i,
// and k, q for the raw rows with ck, cq their factors (cq has the scale). Then
//   A_ij = beta_i ck_i ck_j (Gamma_i / Gamma_j) (k_i . k_j)      j < i
//   u = (1 + A)^-1 r,   r_i = beta_i (v_i - Gamma_i ck_i S0 k_i)
//   out_i = Gamma_i cq_i S0 q_i + sum_j P_ij u_j,   P_ij = cq_i ck_j (Gamma_i / Gamma_j) (q_i . k_j)   j <= i
//   S = Gamma_C S0 + sum_j (Gamma_C / Gamma_j) ck_j u_j k_j^T
// The first kernel forms T = (1 + A)^-1 and P T of every chunk at once, which need no state;
// the second walks down each request's chunks, three products one behind another a chunk:
//   [S0 K^T | S0 Q^T]  ->  r [T^T | (P T)^T] = [u | sum P u]  ->  u K
// Ratios of Gamma are running products of the alphas, so no difference of sums of logarithms
// loses digits and a decay to 0 gives 0.
//
// FP32 operands meet the tensor cores in BF16 parts whose sum they are: a value is cut into
// three of 8 bits each, exactly, and products of parts below 2^-24 are left out; K and Q are
// BF16 as they come and enter raw, so that their products are exact.
constexpr int kChunk = 64, kShift = 6;
constexpr int kHalfTile = kChunk * 128;                // 64 rows of 128 bytes: half the columns of a K, Q or V tile
constexpr int kTile = 2 * kHalfTile;
constexpr int kPart = kChunk * kChunk * 2;             // one BF16 part of T or P T
constexpr int kScalars = 5 * kPart;                    // behind T's three parts and P T's two
// beta, beta Gamma ck, Gamma cq, (Gamma_C / Gamma) ck of each token, then Gamma_C
constexpr int kBeta = 0, kKey = 64, kQuery = 128, kUpdate = 192, kGammaC = 256;
constexpr int kBlob = kScalars + 1152;

__device__ int g_delta_err;

struct ChunkParams {
  DeltaParams d;
  uint8_t* ws;
};

BFP8_DEV uint32_t cut_pair(float a, float b) {         // the upper halves of two floats, as a BF16 pair
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
// A pair's three parts; what is left after the first two has 8 bits.
BFP8_DEV void split3(float2 x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = cut_pair(x.x, x.y);
  x = __fadd2_rn(x, make_float2(__uint_as_float((__float_as_uint(x.x) & 0xFFFF0000u) ^ 0x80000000u),
                                __uint_as_float((__float_as_uint(x.y) & 0xFFFF0000u) ^ 0x80000000u)));
  mid = cut_pair(x.x, x.y);
  x = __fadd2_rn(x, make_float2(__uint_as_float((__float_as_uint(x.x) & 0xFFFF0000u) ^ 0x80000000u),
                                __uint_as_float((__float_as_uint(x.y) & 0xFFFF0000u) ^ 0x80000000u)));
  lo = cut_pair(x.x, x.y);
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
// A tile of 64 tokens of one head, each half of the columns in rows of 128 bytes with the
// 128-byte swizzle, the halves `apart` bytes apart. Rows past the tensor's are zeros.
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

constexpr int kPrepThreads = 128;
constexpr int kAtPitch = 68;
struct PrepShared {
  alignas(16) float at[kChunk * kAtPitch];             // A transposed: row j holds A_ij, i > j
  float alpha[kChunk], ck[kChunk];
  uint64_t full, done;
  uint32_t tmem;
  int abort_flag;
};
constexpr int kPrepSmem = 1024 + kBlob + 1024 + static_cast<int>(sizeof(PrepShared));

// x (1 + A) = w for one row in `w`, columns LIM - 1 down to 0: w_j -= sum_{l > j} w_l A_lj.
template <int LIM>
BFP8_DEV void solve_row(float (&w)[kChunk], const float* at) {
#pragma unroll
  for (int j = LIM - 2; j >= 0; --j) {
    float2 s = make_float2(0.0f, 0.0f), s2 = s;
#pragma unroll
    for (int l = (j + 1) & ~3; l < LIM; l += 4) {
      const float4 c = *reinterpret_cast<const float4*>(at + j * kAtPitch + l);
      if (l > j) {
        s = __ffma2_rn(make_float2(w[l], w[l + 1]), make_float2(c.x, c.y), s);
        s2 = __ffma2_rn(make_float2(w[l + 2], w[l + 3]), make_float2(c.z, c.w), s2);
      } else {
        if (l + 1 > j) s.y = fmaf(w[l + 1], c.y, s.y);
        if (l + 2 > j) s2.x = fmaf(w[l + 2], c.z, s2.x);
        s2.y = fmaf(w[l + 3], c.w, s2.y);
      }
    }
    w[j] -= (s.x + s2.x) + (s.y + s2.y);
  }
}

// T and P T of one chunk of one value head. Threads 0 - 63 have the chunk's key rows, 64 - 127
// its query rows: one product of both with the keys leaves row i of K K^T and of Q K^T in the
// threads' registers. Thread i forms row i of A, thread 64 + i row i of P; and as T (1 + A) = 1
// and (P T)(1 + A) = P, all 128 rows are then solved alike, each by a thread of its own, against
// A in shared memory.
__global__ void __launch_bounds__(kPrepThreads) delta_prepare_kernel(const __grid_constant__ CUtensorMap tq,
                                                                     const __grid_constant__ CUtensorMap tk,
                                                                     const ChunkParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  PrepShared& sh = *reinterpret_cast<PrepShared*>(base + (kBlob + 1023) / 1024 * 1024);
  const uint32_t tile = smem_u32(base);                // K and Q rows, then what goes to memory
  const int tid = threadIdx.x, warp = tid >> 5;
  pdl_wait();
  const int h = blockIdx.x % p.d.v_heads;
  const int64_t slot = blockIdx.x / p.d.v_heads;
  const int b = find_request(p.d.req, slot, kShift);
  if (b < 0) return;
  int64_t first;
  const int64_t len = chunked_len(p.d, b, first);
  const int64_t done = (slot - tile_key(p.d.req, b, kShift)) << kShift;
  if (done >= len) return;
  const int n = static_cast<int>(len - done < kChunk ? len - done : kChunk);
  const int64_t t0 = first + done;
  const int i = tid & 63;
  const bool query = tid >= 64;

  if (tid == 0) {
    mbar_init(smem_u32(&sh.full), 1);
    mbar_init(smem_u32(&sh.done), 1);
    sh.abort_flag = 0;
    mbar_fence_init();
    mbar_arrive_expect_tx(smem_u32(&sh.full), 2 * kTile);
    const int hk = h / p.d.group;
    load_tile(tile, kTile, &tk, hk, static_cast<int>(t0), smem_u32(&sh.full));
    load_tile(tile + kHalfTile, kTile, &tq, hk, static_cast<int>(t0), smem_u32(&sh.full));
  }
  if (warp == 0) {
    __syncwarp();
    tmem_alloc(smem_u32(&sh.tmem), 64);
    tmem_relinquish();
  }
  float beta = 0.0f;
  if (!query) {
    float alpha = 1.0f;
    if (i < n) {
      const float a = __bfloat162float(p.d.a[(t0 + i) * p.d.at + h]);
      alpha = expf(log_decay(a, __ldg(p.d.dt_bias + h), expf(__ldg(p.d.a_log + h))));
      beta = beta_of(__bfloat162float(p.d.b[(t0 + i) * p.d.bt + h]));
    }
    sh.alpha[i] = alpha;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();   // with its tensor memory in hand: a kernel behind may take the rest
  const uint32_t tmem = sh.tmem;
  bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.full), 0, &sh.abort_flag));
  float c = 0.0f;                                      // the row's factor
  if (ok) {
    if (warp == 0 && elect_one()) {
      const uint64_t da = smem_desc_sw128(tile);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const uint64_t d = da + (s >> 2) * (kTile >> 4) + 2 * (s & 3);
        umma_bf16(tmem, d, d, idesc_bf16(128, 64), s > 0);
      }
      umma_commit(smem_u32(&sh.done));
    }
    __syncwarp();
    float ss = 0.0f;
    const uint32_t row = tile + (query ? kHalfTile : 0) + i * 128;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      float f[8];
      widen8(lds128(row + (v >> 3) * kTile + (((v & 7) ^ (i & 7)) << 4)), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
    }
    if (i < n) c = rsqrtf(ss + p.d.eps) * (query ? p.d.scale : 1.0f);
    if (!query) sh.ck[i] = c;
  }
  __syncthreads();
  ok = ok && mbar_wait(smem_u32(&sh.done), 0, &sh.abort_flag);
  ok = __syncthreads_and(ok);
  float w[kChunk];
  if (ok) {
    tc_fence_after();
    tmem_ld64(tmem + (static_cast<uint32_t>(warp * 32) << 16), w);
    const float cb = query ? c : c * beta;
    float ratio = 1.0f, rest = 1.0f;                   // Gamma_i / Gamma_j, and Gamma_C / Gamma_i
#pragma unroll
    for (int j = kChunk - 1; j >= 0; --j) {
      const float next = j + 1 < kChunk ? sh.alpha[j + 1] : 1.0f;
      if (j < i) ratio *= next;
      else rest *= next;
      const float f = cb * sh.ck[j] * ratio;
      if (query) {
        w[j] = j <= i && i < n ? f * w[j] : 0.0f;
      } else {
        if (j < i) sh.at[j * kAtPitch + i] = i < n ? f * w[j] : 0.0f;
        w[j] = j == i ? 1.0f : 0.0f;
      }
    }
    const float gamma = ratio * sh.alpha[0];
    float* scalars = reinterpret_cast<float*>(base + kScalars);
    if (query) {
      scalars[kQuery + i] = gamma * c;
    } else {
      scalars[kBeta + i] = beta;
      scalars[kKey + i] = beta * gamma * c;
      scalars[kUpdate + i] = rest * c;
      if (i == kChunk - 1) scalars[kGammaC] = gamma;
    }
  }
  __syncthreads();                                     // A is there; the key and query rows have been read
  if (ok) {
    if (warp & 1) solve_row<64>(w, sh.at);             // rows 32 - 63 of T or P T
    else solve_row<32>(w, sh.at);                      // rows 0 - 31 end ahead of column 32
    const uint32_t row = tile + (query ? 3 * kPart : 0) + i * 128;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      uint32_t hi[4], mid[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split3(make_float2(w[8 * v + 2 * e], w[8 * v + 2 * e + 1]), hi[e], mid[e], lo[e]);
      const uint32_t at = row + ((v ^ (i & 7)) << 4);
      sts128(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
      sts128(at + kPart, make_uint4(mid[0], mid[1], mid[2], mid[3]));
      if (!query) sts128(at + 2 * kPart, make_uint4(lo[0], lo[1], lo[2], lo[3]));
    }
    fence_proxy_async_smem();
  } else {
    sh.abort_flag = 1;
    if (tid == 0) atomicExch(&g_delta_err, static_cast<int>(BFP8_ERR_TIMEOUT));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
  if (ok && tid == 0) {
    bulk_store(p.ws + (slot * p.d.v_heads + h) * static_cast<int64_t>(kBlob), tile, kBlob);
    bulk_commit();
    bulk_wait_all();
  }
}

// ---- the walk down a request's chunks. Lane r of tensor memory is row r of S (a value), its
// columns keys or tokens: what one product leaves in a lane is, scaled and cut, the next one's
// operand from tensor memory, so nothing passes between threads. Two warpgroups share the
// columns: keys 0 - 63 and 64 - 127 of S (kept in registers), tokens 0 - 31 and 32 - 63.
constexpr int kWalkThreads = 320;                      // 8 warps of rows, one of products, one of loads
constexpr int kRowWarps = 8;
constexpr int kStageBytes = 3 * kTile + (kBlob + 1023) / 1024 * 1024;
constexpr int kStages = 2;
// Columns of tensor memory. A chunk of 16 keys or tokens of one part takes 8. Parts 0 and 1
// of S lie where u K comes (read before they are written anew), those of r where S K^T came,
// those of u' where u came; each warpgroup overwrites only columns that it alone has read.
constexpr uint32_t kColNew = 0, kColS2 = 128, kColX = 192, kColY = 256, kColU = 320, kColO = 384, kColR2 = 448,
                   kColU2 = 480;
BFP8_DEV uint32_t col_s(int part, int step) {          // step: 16 keys
  return part < 2 ? kColNew + 64 * (step >> 2) + 32 * part + 8 * (step & 3) : kColS2 + 32 * (step >> 2) + 8 * (step & 3);
}
BFP8_DEV uint32_t col_r(int part, int step) {          // step: 16 tokens
  return part < 2 ? kColX + 32 * (step >> 1) + 16 * part + 8 * (step & 1) : kColR2 + 16 * (step >> 1) + 8 * (step & 1);
}
BFP8_DEV uint32_t col_u(int part, int step) {
  return part < 2 ? kColU + 32 * (step >> 1) + 16 * part + 8 * (step & 1) : kColU2 + 16 * (step >> 1) + 8 * (step & 1);
}

struct WalkShared {
  uint64_t full[kStages], empty[kStages];
  uint64_t s_full, x_done, r_full, u_done, p_full, o_done, new_done, drained;
  uint32_t tmem;
  int abort_flag;
};
constexpr int kWalkSmem = 1024 + kStages * kStageBytes + static_cast<int>(sizeof(WalkShared));

// D = A B: A from tensor memory, B a tile of N rows in shared memory, BF16.
BFP8_DEV void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  umma_f16_ts(d_tmem, a_tmem, b_desc, idesc, accumulate);   // the operands' type is in idesc
}

__global__ void __launch_bounds__(kWalkThreads, 1) delta_walk_kernel(const __grid_constant__ CUtensorMap tq,
                                                                     const __grid_constant__ CUtensorMap tk,
                                                                     const __grid_constant__ CUtensorMap tv,
                                                                     const ChunkParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  WalkShared& sh = *reinterpret_cast<WalkShared*>(base + kStages * kStageBytes);
  const uint32_t stages = smem_u32(base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  const int h = blockIdx.x % p.d.v_heads, b = blockIdx.x / p.d.v_heads;
  int64_t first;
  const int64_t len = chunked_len(p.d, b, first);
  if (len == 0) return;
  const int chunks = static_cast<int>((len + kChunk - 1) >> kShift);
  const int tail = static_cast<int>(len - (static_cast<int64_t>(chunks - 1) << kShift));

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), kRowWarps + 1);
    }
    mbar_init(smem_u32(&sh.s_full), kRowWarps);
    mbar_init(smem_u32(&sh.r_full), kRowWarps);
    mbar_init(smem_u32(&sh.p_full), kRowWarps);
    mbar_init(smem_u32(&sh.x_done), 1);
    mbar_init(smem_u32(&sh.u_done), 1);
    mbar_init(smem_u32(&sh.o_done), 1);
    mbar_init(smem_u32(&sh.new_done), 1);
    mbar_init(smem_u32(&sh.drained), 1);
    sh.abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == kRowWarps) {
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
    ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), parity, abort_flag));
    return ok;
  };

  if (warp == kRowWarps + 1) {
    // ------------------------------------------------ loads, a chunk ahead
    const int64_t key = tile_key(p.d.req, b, kShift);
    int c = 0;
    for (; c < chunks; ++c) {
      const int s = c % kStages;
      if (!wait(sh.empty[s], ((c / kStages) & 1) ^ 1)) break;
      if (elect_one()) {
        const uint32_t dst = stages + s * kStageBytes, bar = smem_u32(&sh.full[s]);
        const int t0 = static_cast<int>(first) + c * kChunk, hk = h / p.d.group;
        mbar_arrive_expect_tx(bar, 3 * kTile + kBlob);
        load_tile(dst, kHalfTile, &tk, hk, t0, bar);
        bulk_load(dst + 3 * kTile, p.ws + ((key + c) * p.d.v_heads + h) * static_cast<int64_t>(kBlob), kBlob, bar);
        load_tile(dst + 2 * kTile, kHalfTile, &tv, h, t0, bar);
        load_tile(dst + kTile, kHalfTile, &tq, hk, t0, bar);
      }
      __syncwarp();
    }
    if (!ok) {   // what was issued lands before the block ends
      const int none = 0;
      for (int d = c < kStages ? 0 : c - kStages; d < c; ++d)
        mbar_wait(smem_u32(&sh.full[d % kStages]), (d / kStages) & 1, &none);
    }
  } else if (warp == kRowWarps) {
    // ------------------------------------------------ products
    constexpr uint32_t kN64 = idesc_bf16(128, 64), kKeys = idesc_bf16(128, 128) | (1u << 16);
    for (int c = 0; c < chunks; ++c) {
      const int s = c % kStages;
      const uint32_t at = stages + s * kStageBytes;
      const uint64_t dk = smem_desc_sw128(at), dq = smem_desc_sw128(at + kTile), dt = smem_desc_sw128(at + 3 * kTile);
      const uint64_t dn = smem_desc_sw128_mn(at, kHalfTile);
      if (!wait(sh.full[s], (c / kStages) & 1) || !wait(sh.s_full, c & 1)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma_bf16_ts(tmem + kColX, tmem + col_s(part, k), dk + (k >> 2) * (kHalfTile >> 4) + 2 * (k & 3), kN64,
                         part || k);
        umma_commit(smem_u32(&sh.x_done));
#pragma unroll
        for (int part = 0; part < 2; ++part)           // out is rounded to BF16: two parts, 2^-16
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma_bf16_ts(tmem + kColY, tmem + col_s(part, k), dq + (k >> 2) * (kHalfTile >> 4) + 2 * (k & 3), kN64,
                         part || k);
      }
      __syncwarp();
      if (!wait(sh.r_full, c & 1)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int a = 0; a < 3; ++a)                    // parts of r and of T, down to 2^-24 of the product
#pragma unroll
          for (int t = 0; t < 3 - a; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16_ts(tmem + kColU, tmem + col_r(a, k), dt + t * (kPart >> 4) + 2 * k, kN64, a || t || k);
        umma_commit(smem_u32(&sh.u_done));
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int t = 0; t < 2 - a; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16_ts(tmem + kColO, tmem + col_r(a, k), dt + (3 + t) * (kPart >> 4) + 2 * k, kN64, a || t || k);
        umma_commit(smem_u32(&sh.o_done));
      }
      __syncwarp();
      if (!wait(sh.p_full, c & 1)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int k = 0; k < 4; ++k)                  // 16 tokens a step: 16 rows of 128 bytes
            umma_bf16_ts(tmem + kColNew, tmem + col_u(part, k), dn + 128 * k, kKeys, part || k);
        umma_commit(smem_u32(&sh.new_done));
        umma_commit(smem_u32(&sh.empty[s]));
      }
      __syncwarp();
    }
    if (!ok) {   // products in flight end before tensor memory is given back
      const int none = 0;
      if (elect_one()) umma_commit(smem_u32(&sh.drained));
      __syncwarp();
      mbar_wait(smem_u32(&sh.drained), 0, &none);
    }
  } else {
    // ------------------------------------------------ rows of S
    const int wg = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int64_t from = slot_of(p.d.req, p.d.req.slots_in, b), to = slot_of(p.d.req, p.d.req.slots_out, b);
    const int64_t in_head = h * p.d.s_head + r * kD + 64 * wg;
    float S[64];
    if (from >= 0) {
      const float4* src = reinterpret_cast<const float4*>(p.d.state + from * p.d.s_slot + in_head);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float4 f = src[k];
        S[4 * k] = f.x, S[4 * k + 1] = f.y, S[4 * k + 2] = f.z, S[4 * k + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 64; ++k) S[k] = 0.0f;
    }
    // S cut into its parts, and the word to the products' warp. The last chunk's rows past the
    // request are the next one's: zeros, before they meet weights of 0.
    auto hand_over = [&](int c) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t hi[16], mid[16], lo[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
          split3(make_float2(S[32 * half + 2 * k], S[32 * half + 2 * k + 1]), hi[k], mid[k], lo[k]);
        tmem_st16(mine + col_s(0, 4 * wg + 2 * half), hi);
        tmem_st16(mine + col_s(1, 4 * wg + 2 * half), mid);
        tmem_st16(mine + col_s(2, 4 * wg + 2 * half), lo);
      }
      tmem_wait_st();
      if (c == chunks - 1 && tail < kChunk) {
        if (!wait(sh.full[c % kStages], (c / kStages) & 1)) return;
        const uint32_t at = stages + (c % kStages) * kStageBytes;
        for (int v = tid; v < (kChunk - tail) * 16; v += 32 * kRowWarps) {
          const int row = tail + (v >> 4);
          sts128(at + ((v >> 3) & 1) * kHalfTile + row * 128 + ((v & 7) << 4), make_uint4(0u, 0u, 0u, 0u));
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.s_full));
    };
    hand_over(0);
    for (int c = 0; ok && c < chunks; ++c) {
      const int s = c % kStages;
      uint8_t* const at = base + s * kStageBytes;
      const float* scalars = reinterpret_cast<const float*>(at + 3 * kTile + kScalars);
      const int left = c == chunks - 1 ? tail : kChunk;
      if (!wait(sh.full[s], (c / kStages) & 1)) break;
      // column r of the values' tile, in rows of 128 bytes with the swizzle
      const uint8_t* vcol = at + 2 * kTile + (r >> 6) * kHalfTile;
      const uint32_t vbyte = (r & 63) * 2;
      if (!wait(sh.x_done, c & 1)) break;
      tc_fence_after();
      {
        float x[32];
        tmem_ld32(mine + kColX + 32 * wg, x);
        uint32_t hi[16], mid[16], lo[16];
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const int t = 32 * wg + j;
          const float2 be = *reinterpret_cast<const float2*>(scalars + kBeta + t);
          const float2 kf = *reinterpret_cast<const float2*>(scalars + kKey + t);
          const uint16_t v0 = *reinterpret_cast<const uint16_t*>(vcol + t * 128 + (vbyte ^ ((t & 7) << 4)));
          const uint16_t v1 = *reinterpret_cast<const uint16_t*>(vcol + (t + 1) * 128 + (vbyte ^ (((t + 1) & 7) << 4)));
          float2 y = __fmul2_rn(make_float2(bf16_bits_to_f32(v0), bf16_bits_to_f32(v1)), be);
          y = __ffma2_rn(make_float2(-x[j], -x[j + 1]), kf, y);
          if (t >= left) y.x = 0.0f;
          if (t + 1 >= left) y.y = 0.0f;
          split3(y, hi[j / 2], mid[j / 2], lo[j / 2]);
        }
        tmem_st16(mine + col_r(0, 2 * wg), hi);
        tmem_st16(mine + col_r(1, 2 * wg), mid);
        tmem_st16(mine + col_r(2, 2 * wg), lo);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.r_full));
      }
      if (!wait(sh.u_done, c & 1)) break;
      tc_fence_after();
      {
        float u[32];
        tmem_ld32(mine + kColU + 32 * wg, u);
        uint32_t hi[16], mid[16], lo[16];
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 f = *reinterpret_cast<const float2*>(scalars + kUpdate + 32 * wg + j);
          split3(__fmul2_rn(make_float2(u[j], u[j + 1]), f), hi[j / 2], mid[j / 2], lo[j / 2]);
        }
        tmem_st16(mine + col_u(0, 2 * wg), hi);
        tmem_st16(mine + col_u(1, 2 * wg), mid);
        tmem_st16(mine + col_u(2, 2 * wg), lo);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.p_full));
      }
      const float gamma = scalars[kGammaC];
      if (!wait(sh.o_done, c & 1)) break;
      tc_fence_after();
      {
        float y[32], o[32];
        tmem_ld32(mine + kColY + 32 * wg, y);
        tmem_ld32(mine + kColO + 32 * wg, o);
        __nv_bfloat16* out = p.d.out + (first + static_cast<int64_t>(c) * kChunk + 32 * wg) * p.d.ot + h * p.d.oh + r;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (32 * wg + j < left) out[j * p.d.ot] = __float2bfloat16_rn(fmaf(scalars[kQuery + 32 * wg + j], y[j], o[j]));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.empty[s]));
      if (!wait(sh.new_done, c & 1)) break;
      tc_fence_after();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float d[32];
        tmem_ld32(mine + kColNew + 64 * wg + 32 * half, d);
#pragma unroll
        for (int k = 0; k < 32; ++k) S[32 * half + k] = fmaf(gamma, S[32 * half + k], d[k]);
      }
      if (c + 1 < chunks) hand_over(c + 1);
    }
    if (ok && to >= 0) {
      float4* dst = reinterpret_cast<float4*>(p.d.state + to * p.d.s_slot + in_head);
#pragma unroll
      for (int k = 0; k < 16; ++k) dst[k] = make_float4(S[4 * k], S[4 * k + 1], S[4 * k + 2], S[4 * k + 3]);
    }
  }
  if (!ok) {
    sh.abort_flag = 1;
    if (lane == 0) atomicExch(&g_delta_err, static_cast<int>(BFP8_ERR_TIMEOUT));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kRowWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// A request of up to this many new tokens takes them one after the other.
constexpr int64_t kStepTokens = 16;

int64_t chunk_slots(int64_t batch, int64_t tokens) { return (tokens >> kShift) + batch; }

int tile_map(CUtensorMap* map, const void* x, int64_t heads, int64_t tokens, int64_t head_stride, int64_t token_stride) {
  return make_tmap_3d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, kD, static_cast<uint64_t>(heads),
                      static_cast<uint64_t>(tokens), static_cast<uint64_t>(head_stride) * 2,
                      static_cast<uint64_t>(token_stride) * 2, 64, 1, kChunk, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool off16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

}  // namespace

size_t delta_rule_workspace_bytes(int64_t batch, int64_t tokens, int64_t max_q_len, int64_t, int64_t v_heads) {
  if (max_q_len <= kStepTokens) return 0;
  return static_cast<size_t>(chunk_slots(batch, tokens)) * static_cast<size_t>(v_heads) * kBlob;
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
  const size_t need = delta_rule_workspace_bytes(a.batch, a.tokens, a.max_q_len, a.qk_heads, a.v_heads);
  if (need && (!a.workspace || a.ws_bytes < need)) return BFP8_ERR_INVALID_ARG;
  if (need && (reinterpret_cast<uintptr_t>(a.workspace) % 256 ||
               chunk_slots(a.batch, a.tokens) * a.v_heads > 0x7FFFFFFF))
    return BFP8_ERR_UNSUPPORTED;
  int rc = check_device_ptrs({a.q_bf16, a.k_bf16, a.v_bf16, a.a_bf16, a.b_bf16, a.a_log, a.dt_bias, a.state,
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
  p.step_len = kStepTokens;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned blocks = static_cast<unsigned>(a.batch * a.v_heads * (kD / (8 * kStepWarps)));
  rc = launch_dependent(delta_step_kernel, dim3(blocks), 32 * kStepWarps, 0, st, p);
  if (rc != BFP8_OK || !need) return rc;
  CUtensorMap tq, tk, tv;
  rc = tile_map(&tq, a.q_bf16, a.qk_heads, a.tokens, a.q_stride_head, a.q_stride_token);
  if (rc == BFP8_OK) rc = tile_map(&tk, a.k_bf16, a.qk_heads, a.tokens, a.k_stride_head, a.k_stride_token);
  if (rc == BFP8_OK) rc = tile_map(&tv, a.v_bf16, a.v_heads, a.tokens, a.v_stride_head, a.v_stride_token);
  if (rc == BFP8_OK) rc = set_max_dynamic_smem(reinterpret_cast<const void*>(delta_prepare_kernel), kPrepSmem);
  if (rc == BFP8_OK) rc = set_max_dynamic_smem(reinterpret_cast<const void*>(delta_walk_kernel), kWalkSmem);
  if (rc != BFP8_OK) return rc;
  const ChunkParams cp{p, static_cast<uint8_t*>(a.workspace)};
  rc = launch_dependent(delta_prepare_kernel, dim3(static_cast<unsigned>(chunk_slots(a.batch, a.tokens) * a.v_heads)),
                        kPrepThreads, kPrepSmem, st, tq, tk, cp);
  if (rc != BFP8_OK) return rc;
  return launch_dependent(delta_walk_kernel, dim3(static_cast<unsigned>(a.batch * a.v_heads)), kWalkThreads, kWalkSmem,
                          st, tq, tk, tv, cp);
}

int delta_read_clear_error() {
  int v = 0;
  const int zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_delta_err, sizeof(int)) != cudaSuccess) return BFP8_ERR_CUDA;
  if (v != 0 && cudaMemcpyToSymbol(g_delta_err, &zero, sizeof(int)) != cudaSuccess) return BFP8_ERR_CUDA;
  return v == 0 ? BFP8_OK : v;
}

}  // namespace bfp8
