// causal_conv.cu -- the short depthwise convolution ahead of a linear-attention layer, over
// the ragged tokens of a step, with each request's last inputs kept between steps:
//
//   y[t, c] = act(bias[c] + sum_j weight[c, j] x[t - (W - 1) + j, c]),   act = SiLU or none
//
// Inputs ahead of a request's first token come from its slot of the state, and the last
// W - 1 inputs go there. Bound by HBM: a row is read once and written once. 11,600 rows of 8192
// channels, 380 MB, take 63 us, 6.0 TB/s; with the next four rows under way in registers 69 us,
// without any 84, and with four channels a thread and twice the warps 93 (a row's addresses and
// predicates for half the work). A single token of 64 requests: 3.8 us of latency, two rounds of
// loads (which request, then its rows).
#include "hybrid_layer.cuh"

namespace bfp8 {
namespace {

using namespace dev;

constexpr int kConvThreads = 128;   // 8 channels each
constexpr int kConvAhead = 8;       // rows that a thread has under way

struct ConvParams {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  const void* weight;
  const void* bias;
  __nv_bfloat16* state;
  int64_t ldx, ldo, lds_slot, lds_row;
  Requests req;
  int32_t channels, w_f32, tile_shift;
};

// N consecutive weights from `at` on, N a multiple of 8, widened.
template <int N>
BFP8_DEV void load_weights(const void* w, int32_t f32, int64_t at, float (&v)[N]) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 f = __ldg(p + i);
      v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + at);
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      float f[8];
      widen8(__ldg(p + i), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[8 * i + e] = f[e];
    }
  }
}
BFP8_DEV void widen4x2(const uint4& r, float2 (&v)[4]) {
  float f[8];
  widen8(r, f);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = make_float2(f[2 * e], f[2 * e + 1]);
}

// A block takes 1024 channels of one tile of a request's tokens; a thread walks down its 8
// channels with the last W - 1 inputs in registers. It copies its 16 bytes of the next eight rows
// to places of its own in shared memory and waits for nobody else. The thread of a request's
// first tile also moves the state: it alone reads the old rows, before it writes the new ones, so
// one slot may be both.
template <int W, bool SILU>
__global__ void __launch_bounds__(kConvThreads, 4) causal_conv_kernel(const ConvParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int b = find_request(p.req, blockIdx.y, p.tile_shift);
  if (b < 0) return;
  const int c = (blockIdx.x * kConvThreads + threadIdx.x) * 8;
  if (c >= p.channels) return;
  const int64_t first = first_token(p.req, b), end = first_token(p.req, b + 1);
  const int64_t tile = static_cast<int64_t>(blockIdx.y) - tile_key(p.req, b, p.tile_shift);
  const int64_t t0 = first + (tile << p.tile_shift);
  if (t0 >= end) return;
  const int64_t left = end - t0, most = int64_t{1} << p.tile_shift;
  const int n = static_cast<int>(left < most ? left : most);

  __shared__ alignas(16) uint4 ring[kConvAhead][kConvThreads];   // a thread's own places
  const uint32_t place = smem_u32(&ring[0][threadIdx.x]);
  constexpr uint32_t kRow = sizeof(ring[0]);
  const __nv_bfloat16* x = p.x + t0 * p.ldx + c;
  const __nv_bfloat16* next = x;
  int asked = 0;
  auto ask = [&](int s) {
    if (asked < n) cp_async16(place + s * kRow, next);
    cp_async_commit();
    ++asked, next += p.ldx;
  };
#pragma unroll
  for (int s = 0; s < kConvAhead; ++s) ask(s);
  auto row = [&](int64_t t) { return __ldg(reinterpret_cast<const uint4*>(x + t * p.ldx)); };
  float2 w[W][4], h[W - 1][4], bias[4];
  {
    float flat[8 * W], flat_bias[8] = {};
    load_weights(p.weight, p.w_f32, static_cast<int64_t>(c) * W, flat);
    if (p.bias) load_weights(p.bias, p.w_f32, c, flat_bias);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][e] = make_float2(flat[2 * e * W + j], flat[(2 * e + 1) * W + j]);
      bias[e] = make_float2(flat_bias[2 * e], flat_bias[2 * e + 1]);
    }
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 past[W - 1];   // inputs t0 - (W - 1) .. t0 - 1
    if (tile > 0) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) past[j] = row(j - (W - 1));
    } else {
      const int64_t from = slot_of(p.req, p.req.slots_in, b), to = slot_of(p.req, p.req.slots_out, b);
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        past[j] = from < 0 ? zero
                           : *reinterpret_cast<const uint4*>(p.state + from * p.lds_slot + j * p.lds_row + c);
      if (to >= 0) {
        const int64_t len = end - first;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          uint4 v = zero;
          if (len + j >= W - 1) {
            v = row(len + j - (W - 1));
          } else {
#pragma unroll
            for (int i = 0; i < W - 1; ++i)   // a short request: row len + j of the old state
              if (i == len + j) v = past[i];
          }
          *reinterpret_cast<uint4*>(p.state + to * p.lds_slot + j * p.lds_row + c) = v;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) widen4x2(past[j], h[j]);
  }
  __nv_bfloat16* out = p.out + t0 * p.ldo + c;
  auto step = [&](const uint4& r) {
    float2 v[4], y[4];
    widen4x2(r, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[e] = bias[e];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) y[e] = __ffma2_rn(w[j][e], h[j][e], y[e]);
      y[e] = __ffma2_rn(w[W - 1][e], v[e], y[e]);
      if (SILU) y[e] = __fmul2_rn(y[e], make_float2(sigmoid(y[e].x), sigmoid(y[e].y)));
#pragma unroll
      for (int j = 0; j + 1 < W - 1; ++j) h[j][e] = h[j + 1][e];
      h[W - 2][e] = v[e];
    }
    *reinterpret_cast<uint4*>(out) = make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y),
                                                pack_bf16x2(y[2].x, y[2].y), pack_bf16x2(y[3].x, y[3].y));
    out += p.ldo;
  };
  for (int t = 0; t < n; t += kConvAhead) {
#pragma unroll
    for (int s = 0; s < kConvAhead; ++s) {
      if (t + s >= n) break;
      cp_async_wait_group<kConvAhead - 1>();
      const uint4 r = lds128(place + s * kRow);
      ask(s);
      step(r);
    }
  }
  cp_async_wait_group<0>();
}

bool off16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

}  // namespace

int launch_causal_conv(const bfp8_causal_conv_args& a, void* stream) {
  if (a.tokens < 0 || a.batch < 0 || a.channels < 0 || a.n_slots < 0) return BFP8_ERR_INVALID_ARG;
  if (a.width < 2 || a.width > 4) return BFP8_ERR_UNSUPPORTED;
  if (a.w_dtype != BFP8_DT_BF16 && a.w_dtype != BFP8_DT_F32) return BFP8_ERR_SCALE_DTYPE;
  if (a.tokens == 0 || a.batch == 0 || a.channels == 0) return BFP8_OK;
  if (!a.x_bf16 || !a.out_bf16 || !a.weight || !a.q_offsets || a.x_bf16 == a.out_bf16)
    return BFP8_ERR_INVALID_ARG;
  if (a.x_stride_token < a.channels || a.out_stride_token < a.channels) return BFP8_ERR_INVALID_ARG;
  if (a.state_bf16 ? a.state_stride_row < a.channels ||
                         a.state_stride_slot < a.state_stride_row * (a.width - 2) + a.channels
                   : a.slots_in || a.slots_out)
    return BFP8_ERR_INVALID_ARG;
  if (a.channels % 8 || a.channels > (1 << 24) || a.tokens > 0x7FFFFFFF || a.batch > (1 << 20) ||
      a.x_stride_token % 8 || a.out_stride_token % 8 || off16(a.x_bf16) || off16(a.out_bf16) ||
      off16(a.weight) || off16(a.bias) || off16(a.state_bf16) ||
      (a.state_bf16 && (a.state_stride_slot % 8 || a.state_stride_row % 8)))
    return BFP8_ERR_UNSUPPORTED;
  // Tiles of 32 tokens (16, 32, 64, 128 for 11,600 rows: 70, 63, 64, 76 us), or as many more as
  // keep them within the grid's second dimension.
  int shift = 5;
  while ((a.tokens >> shift) + a.batch > 65535 && shift < 30) ++shift;
  const int64_t tiles = (a.tokens >> shift) + a.batch;
  if (tiles > 65535) return BFP8_ERR_UNSUPPORTED;
  int rc = check_device_ptrs({a.x_bf16, a.out_bf16, a.weight, a.bias, a.state_bf16, a.q_offsets,
                              a.slots_in, a.slots_out});
  if (rc != BFP8_OK) return rc;
  ConvParams p{};
  p.x = static_cast<const __nv_bfloat16*>(a.x_bf16);
  p.out = static_cast<__nv_bfloat16*>(a.out_bf16);
  p.weight = a.weight;
  p.bias = a.bias;
  p.state = static_cast<__nv_bfloat16*>(a.state_bf16);
  p.ldx = a.x_stride_token;
  p.ldo = a.out_stride_token;
  p.lds_slot = a.state_stride_slot;
  p.lds_row = a.state_stride_row;
  p.req = {a.q_offsets, a.slots_in, a.slots_out, a.tokens, a.n_slots, static_cast<int32_t>(a.batch)};
  p.channels = static_cast<int32_t>(a.channels);
  p.w_f32 = a.w_dtype == BFP8_DT_F32;
  p.tile_shift = shift;
  const dim3 grid(static_cast<unsigned>((a.channels / 8 + kConvThreads - 1) / kConvThreads),
                  static_cast<unsigned>(tiles));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto kernel) { return launch_dependent(kernel, grid, kConvThreads, 0, st, p); };
  switch (a.width) {
    case 2: return a.silu ? go(causal_conv_kernel<2, true>) : go(causal_conv_kernel<2, false>);
    case 3: return a.silu ? go(causal_conv_kernel<3, true>) : go(causal_conv_kernel<3, false>);
    default: return a.silu ? go(causal_conv_kernel<4, true>) : go(causal_conv_kernel<4, false>);
  }
}

}  // namespace bfp8
