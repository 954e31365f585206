// kv_attention.cu -- attention over the paged 8-bit KV cache.
//
//   out[t, h] = softmax_i( scale * q[t, h] . k[i, g] ) v[i, g],   g = h / group
//   over the positions i a query sees: up to its own, at most `window` back.
//
// Arithmetic. A page's scales are powers of two, so they never touch the codes:
// the key scale is a factor of the score, and the value scale 2^ev joins the
// exponent. With x = score * log2(e) + ev the weights are w = 2^(x - M), M the
// running maximum of x, and
//   out = sum(w code_v) / sum(w 2^-ev),    lse = ln2 (M + log2 sum(w 2^-ev)).
// One running maximum bounds every product that is summed, whatever the pages'
// scales; scores, maxima, sums and outputs are FP32.
#include "bfp8_internal.h"
#include "kv_common.cuh"
#include "ptx.cuh"
#include "act_math.cuh"

namespace bfp8 {
namespace {

using namespace dev;

__device__ int g_kv_err;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -INFINITY;

struct AttnParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  const uint8_t* k_exp;
  const uint8_t* v_exp;
  const int32_t* table;
  const int32_t* q_offsets;
  const int32_t* kv_len;
  float* partial;            // split rows' partial sums
  uint64_t* schedule;        // [B + 1]: units before each request, and in all
  int64_t q_ldt, q_ldh, o_ldt, o_ldh, l_ldt, ld_table, exp_page, exp_head;
  int64_t T, n_pages;
  int32_t B, H, G, page_shift, max_blocks, window;
  float scale_log2;          // softmax scale * log2(e)
};

// ============================================================ few query rows
// A unit of work is 32 tokens of one segment; a segment is 16 query rows (the
// heads of a group, times the tokens of a draft) of one request and KV head.
// All units are numbered request by request and cut into equal contiguous
// ranges, one per block, so ragged lengths balance; a block's warps take its
// units in turn, each with its own ring of shared-memory stages and no barrier
// between them inside a segment.
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = 32;                 // tokens
constexpr int kRows = 16;                 // query rows of a segment
constexpr int kStages = 2;
constexpr int kStageBytes = 2 * kUnit * kHeadDim;            // keys, then values
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
constexpr int kMergeBytes = kWarps * kRows * kHeadDim * 4;
constexpr int kSmemBytes = kRingBytes + kMergeBytes + 1024;  // + alignment
constexpr int kPartialFloats = kRows * kHeadDim + 2 * kRows; // O, then M, then Z
// P is kept at 2^4 times the weight and the maximum moves only when a score
// passes it by 2^10, so F16 holds P up to 2^14 and, to full precision, down to
// 2^-18 of the maximum.
constexpr float kPBase = 4.0f;
constexpr float kLazy = 10.0f;

struct ReqUnits {
  int32_t q0, n, kv, lo;   // first row, new tokens, length, first unit
  uint32_t nt, nseg;       // units of a segment, segments
};
BFP8_DEV ReqUnits req_units(const AttnParams& p, int b) {
  ReqUnits r;
  r.q0 = max(__ldg(p.q_offsets + b), 0);
  const int64_t q1 = min(static_cast<int64_t>(__ldg(p.q_offsets + b + 1)), p.T);
  r.n = static_cast<int32_t>(max(q1 - r.q0, static_cast<int64_t>(0)));
  r.kv = max(__ldg(p.kv_len + b), 0);
  const int64_t held = min(static_cast<int64_t>(r.kv),
                           static_cast<int64_t>(p.max_blocks) << p.page_shift);
  int64_t lo = 0;
  if (p.window >= 0) lo = max(static_cast<int64_t>(r.kv) - r.n - p.window, static_cast<int64_t>(0));
  r.lo = static_cast<int32_t>(lo / kUnit);
  const int64_t hi = (held + kUnit - 1) / kUnit;
  r.nt = r.n > 0 && hi > r.lo ? static_cast<uint32_t>(hi - r.lo) : 0u;
  const int64_t rows = static_cast<int64_t>(r.n) * p.G;
  r.nseg = static_cast<uint32_t>((rows + kRows - 1) / kRows) * p.H;
  return r;
}
BFP8_DEV uint64_t units_of(const AttnParams& p, int b) {
  const ReqUnits r = req_units(p, b);
  return static_cast<uint64_t>(r.nt) * r.nseg;
}

// A warp's place in the sequence of units.
struct Cursor {
  uint64_t base;    // first unit of request b
  int b;
  ReqUnits r;
  uint32_t seg, u;  // segment of the request, unit of the segment
};
// Moves to unit g >= base. False past the last request.
BFP8_DEV bool locate(const AttnParams& p, Cursor& c, uint64_t g) {
  while (true) {
    const uint64_t cnt = static_cast<uint64_t>(c.r.nt) * c.r.nseg;
    if (g < c.base + cnt) break;
    c.base += cnt;
    if (++c.b >= p.B) return false;
    c.r = req_units(p, c.b);
  }
  const uint32_t rel = static_cast<uint32_t>(g - c.base);
  c.seg = rel / c.r.nt;
  c.u = rel - c.seg * c.r.nt;
  return true;
}

// Blocks that share U units: every warp of each gets one at least.
BFP8_DEV uint32_t used_blocks(uint64_t U, uint32_t grid) {
  const uint64_t want = (U + kWarps - 1) / kWarps;
  return static_cast<uint32_t>(want < grid ? (want ? want : 1) : grid);
}
BFP8_DEV uint64_t range_begin(uint64_t U, uint32_t c, uint32_t C) { return U * c / C; }
// The block whose range holds unit g.
BFP8_DEV uint32_t owner_of(uint64_t g, uint64_t U, uint32_t C) {
  return static_cast<uint32_t>(((g + 1) * C - 1) / U);
}

BFP8_DEV void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
BFP8_DEV uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
BFP8_DEV uint32_t f16_pair(uint32_t word, int half) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(half ? word >> 16 : word & 0xFFFFu));
}

// Row r of a segment: which query and head it is.
struct RowAt {
  int64_t token;
  int head;
  int pos;
  bool real;
};
BFP8_DEV RowAt row_at(const AttnParams& p, const ReqUnits& r, uint32_t seg, int row) {
  RowAt a;
  const uint32_t nrb = r.nseg / p.H;
  const uint32_t h = seg / nrb, rb = seg - h * nrb;
  const uint32_t i = rb * kRows + row;
  const uint32_t tok = i / p.G;
  a.real = tok < static_cast<uint32_t>(r.n);
  a.token = r.q0 + static_cast<int64_t>(a.real ? tok : 0);
  a.head = h * p.G + (i - tok * p.G);
  a.pos = r.kv - r.n + static_cast<int>(tok);
  return a;
}

// What a warp keeps of a unit between issuing its copies and using them.
// The scale bytes are loaded when the copies are issued and first looked at when
// those have landed, so their latency hides behind the copies'.
struct Pending {
  uint32_t k0, k1, v0, v1;   // scale bytes of the unit's two halves
  uint32_t valid;            // one bit per token that exists
};

BFP8_DEV void store_row16(__nv_bfloat16* dst, const float (&v)[16], float f) {
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v[2 * j + 1] * f), "f"(v[2 * j] * f));
  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(dst + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// out = O / Z and lse, from sums at maximum M; a row that saw nothing gives 0 and -inf.
BFP8_DEV float row_factor(float Z) { return Z == 0.0f ? 0.0f : __frcp_rn(Z); }
BFP8_DEV float row_lse(float M, float Z) {
  return Z == 0.0f ? kNegInf : kLn2 * (M - kPBase + log2f(Z));
}

__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_rows_kernel(const __grid_constant__ CUtensorMap tk,
                             const __grid_constant__ CUtensorMap tv, const AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[kWarps * kStages];
  __shared__ float sm_m[kWarps][kRows], sm_z[kWarps][kRows];
  __shared__ uint64_t scan[kWarps];
  __shared__ uint64_t start_base;
  __shared__ int start_b;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  float* merge = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)) + kRingBytes);
  if (tid < kWarps * kStages) mbar_init(smem_u32(&bars[tid]), 1);
  if (tid == 0) abort_flag = 0, start_b = 0, start_base = 0;
  mbar_fence_init();
  pdl_wait();
  pdl_launch_dependents();

  // ---- this block's range of units
  uint64_t U = 0;
  uint64_t mine = 0, before = 0;   // this thread's request in the last pass of the scan
  auto scan_pass = [&](int b0) {   // exclusive prefix of one request per thread; returns the total
    mine = b0 + tid < p.B ? units_of(p, b0 + tid) : 0;
    uint64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    uint64_t total = 0, off = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) off = total;
      total += scan[w];
    }
    before = off + inc - mine;
    return total;
  };
  for (int b0 = 0; b0 < p.B; b0 += kThreads) U += scan_pass(b0);
  const uint32_t C = used_blocks(U, gridDim.x);
  const bool idle = blockIdx.x >= C || U == 0;
  const uint64_t g0 = idle ? 0 : range_begin(U, blockIdx.x, C);
  const uint64_t g1 = idle ? 0 : range_begin(U, blockIdx.x + 1, C);
  {
    uint64_t run = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      const uint64_t total = p.B > kThreads ? scan_pass(b0) : U;   // one pass: still in registers
      const uint64_t at = run + before;
      if (!idle && mine && g0 >= at && g0 < at + mine) start_b = b0 + tid, start_base = at;
      if (blockIdx.x == 0 && b0 + tid < p.B) p.schedule[b0 + tid] = at;
      run += total;
    }
    if (blockIdx.x == 0 && tid == 0) p.schedule[p.B] = U;
  }
  __syncthreads();
  if (idle) return;

  const uint32_t bar0 = smem_u32(&bars[warp * kStages]);
  const uint32_t stage0 = ring + warp * kStages * kStageBytes;
  const int page = 1 << p.page_shift;
  const int box = min(page, kUnit);
  const int c = lane & 3, nrow = lane >> 2;
  const int ktok = nrow ^ ((nrow & 1) << 2);   // see "Fragments" below

  // ---- issuing: this warp's next unit
  Cursor pc;
  pc.b = start_b;
  pc.base = start_base;
  pc.r = req_units(p, pc.b);
  uint64_t pg = g0 + ((warp - g0) & (kWarps - 1));   // unit g belongs to warp g mod kWarps
  int32_t id0 = -1, id1 = -1;                        // its page numbers (two when pages hold 16)
  bool more = false;
  auto fetch_ids = [&] {
    more = pg < g1 && locate(p, pc, pg);
    if (!more) return;
    const int64_t t0 = static_cast<int64_t>(pc.r.lo + pc.u) * kUnit;
    const int32_t* row = p.table + pc.b * p.ld_table;
    const int64_t blk = t0 >> p.page_shift;
    id0 = __ldg(row + blk);   // blk < max_blocks: units stop at the table's width
    id1 = page < kUnit && blk + 1 < p.max_blocks && t0 + page < pc.r.kv ? __ldg(row + blk + 1) : -1;
  };
  Pending pend0{}, pend1{};             // of stages 0 and 1
  uint32_t armed = 0, phase_bits = 0;   // stages with copies in flight; their parities
  auto issue = [&](Pending& pd, const int s) __attribute__((always_inline)) {
    const uint32_t seg = pc.seg, nrb = pc.r.nseg / p.H;
    const int h = seg / nrb;
    const int64_t t0 = static_cast<int64_t>(pc.r.lo + pc.u) * kUnit;
    const int off = static_cast<int>(t0 & (page - 1));
    const bool ok0 = id0 >= 0 && id0 < p.n_pages, ok1 = id1 >= 0 && id1 < p.n_pages;
    const int64_t left = min(static_cast<int64_t>(pc.r.kv),
                             static_cast<int64_t>(p.max_blocks) << p.page_shift) - t0;
    uint32_t valid = left >= 32 ? 0xffffffffu : (1u << left) - 1u;   // left >= 1
    const uint32_t half0 = page < kUnit ? 0xffffu : 0xffffffffu;
    valid &= (ok0 ? half0 : 0u) | (page < kUnit && ok1 ? 0xffff0000u : 0u);
    pd.valid = valid;
    const int64_t e0 = id0 * p.exp_page + h * p.exp_head, e1 = id1 * p.exp_page + h * p.exp_head;
    pd.k0 = pd.k1 = pd.v0 = pd.v1 = 127u;
    if (ok0) pd.k0 = __ldg(p.k_exp + e0), pd.v0 = __ldg(p.v_exp + e0);
    if (page < kUnit && ok1) pd.k1 = __ldg(p.k_exp + e1), pd.v1 = __ldg(p.v_exp + e1);
    if (lane == 0) {
      const uint32_t bar = bar0 + 8 * s, dst = stage0 + s * kStageBytes;
      const uint32_t bytes = box * kHeadDim;
      mbar_arrive_expect_tx(bar, 2 * bytes * ((ok0 ? 1 : 0) + (ok1 ? 1 : 0)));
      if (ok0) {
        tma_load_4d(dst, &tk, 0, off, h, id0, bar);
        tma_load_4d(dst + kUnit * kHeadDim, &tv, 0, off, h, id0, bar);
      }
      if (ok1) {
        tma_load_4d(dst + bytes, &tk, 0, 0, h, id1, bar);
        tma_load_4d(dst + kUnit * kHeadDim + bytes, &tv, 0, 0, h, id1, bar);
      }
    }
    armed |= 1u << s;
    pg += kWarps;
    fetch_ids();
  };
  fetch_ids();
  if (more) issue(pend0, 0);
  if (more) issue(pend1, 1);

  // ---- segments of this block's range
  Cursor cc;
  cc.b = start_b;
  cc.base = start_base;
  cc.r = req_units(p, cc.b);
  int stage = 0;
  bool ok = true;
  for (uint64_t g = g0; g < g1;) {
    if (!locate(p, cc, g)) break;
    const uint64_t seg_begin = g - cc.u, seg_end = seg_begin + cc.r.nt;
    const uint64_t pe = seg_end < g1 ? seg_end : g1;
    const uint32_t seg = cc.seg;
    const int rows_left = [&] {
      const uint32_t nrb = cc.r.nseg / p.H, rb = seg - seg / nrb * nrb;
      const int64_t left = static_cast<int64_t>(cc.r.n) * p.G - static_cast<int64_t>(rb) * kRows;
      return static_cast<int>(left < kRows ? left : kRows);
    }();

    // Query rows nrow and nrow + 8 as F16 at a power of two that puts the row's
    // largest entry in [2^8, 2^9): a BF16 has 8 significant bits and F16 11, so
    // entries down to 2^-22 of the largest are exact.
    const RowAt ra = row_at(p, cc.r, seg, nrow), rb = row_at(p, cc.r, seg, nrow + 8);
    uint32_t qa[8][4];
    float fac[2];
    {
      uint4 raw[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const RowAt& r = i ? rb : ra;
        const __nv_bfloat16* src = p.q + r.token * p.q_ldt + r.head * p.q_ldh + 16 * c;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          raw[i][j] = make_uint4(0u, 0u, 0u, 0u);
          if (r.real) raw[i][j] = __ldg(reinterpret_cast<const uint4*>(src + 64 * (j >> 1) + 8 * (j & 1)));
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w[4] = {raw[i][j].x, raw[i][j].y, raw[i][j].z, raw[i][j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) m = max(m, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
        }
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int e = m ? min(max(8 - (static_cast<int>(m >> 7) - 127), -110), 110) : 0;
        const float up = exp2_int(e);
        fac[i] = exp2_int(-e) * p.scale_log2;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w[4] = {raw[i][j].x, raw[i][j].y, raw[i][j].z, raw[i][j].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t v = pack_f16x2(__uint_as_float(w[x] << 16) * up,
                                          __uint_as_float(w[x] & 0xFFFF0000u) * up);
            // 16 columns of chunk c + 4 (j >> 1): step s holds columns 4 (s & 3) .. + 3
            const int s = 4 * (j >> 1) + 2 * (j & 1) + (x >> 1);
            qa[s][i + 2 * (x & 1)] = v;
          }
        }
      }
    }
    const int lim0 = ra.real ? ra.pos + 1 : 0, lim1 = rb.real ? rb.pos + 1 : 0;
    const int win0 = p.window >= 0 ? max(ra.pos - p.window, 0) : 0;
    const int win1 = p.window >= 0 ? max(rb.pos - p.window, 0) : 0;

    float o[16][4];
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    float M[2] = {kNegInf, kNegInf}, Z[2] = {0.0f, 0.0f};

    // One unit, from stage ST. False when the wait for it ran out.
    auto unit = [&](const uint64_t x, Pending& pd, const int ST) __attribute__((always_inline)) {
      const uint32_t bar = bar0 + 8 * ST;
      const uint32_t kb = stage0 + ST * kStageBytes, vb = kb + kUnit * kHeadDim;
      if (!__all_sync(0xffffffffu, mbar_wait(bar, (phase_bits >> ST) & 1u, &abort_flag))) return false;
      armed &= ~(1u << ST);
      phase_bits ^= 1u << ST;
      const uint32_t two = page < kUnit ? 1u : 0u;   // the second half has a page of its own
      const int ek[2] = {static_cast<int>(pd.k0) - 127, static_cast<int>(two ? pd.k1 : pd.k0) - 127};
      const int ev[2] = {static_cast<int>(pd.v0) - 127, static_cast<int>(two ? pd.v1 : pd.v0) - 127};
      const uint32_t valid = pd.valid;
      const int t0 = static_cast<int>((cc.r.lo + static_cast<uint32_t>(x - seg_begin)) * kUnit);

      // Fragments. QK: rows x 8 tokens x 16 columns a step, and which column is
      // which does not matter as long as q agrees, so a lane reads its token's
      // 16-byte chunks c and c + 4 whole. PV: a lane reads 16 columns
      // (lane / 4) of four tokens, and O's columns come out as 32 in a row per
      // lane. Token n of a block of eight is n ^ 4(n & 1): with the 128-byte
      // swizzle both reads are then free of bank conflicts.
      float s[4][4];
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.0f;
        const uint32_t row = kb + (nb * 8 + ktok) * kHeadDim;
        const uint4 ka = lds128(row + ((c ^ ktok) << 4));
        const uint4 kc = lds128(row + (((c + 4) ^ ktok) << 4));
        const uint32_t w[8] = {ka.x, ka.y, ka.z, ka.w, kc.x, kc.y, kc.z, kc.w};
#pragma unroll
        for (int st = 0; st < 8; ++st) mma_f16(s[nb], qa[st], f16_pair(w[st], 0), f16_pair(w[st], 1));
      }
      // scores in units of log2, the value scale's exponent added; column e of
      // block nb is token nb * 8 + 2c + e, moved as above
      const float kf[2] = {exp2_int(ek[0]), exp2_int(ek[1])};
      const float lv[2] = {static_cast<float>(ev[0]), static_cast<float>(ev[1])};
      float mx[2] = {kNegInf, kNegInf};
      const bool masked = valid != 0xffffffffu || t0 + kUnit > min(lim0, lim1) ||
                          t0 < max(win0, win1);
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = e >> 1;
          s[nb][e] = fmaf(s[nb][e], fac[i] * kf[nb >> 1], lv[nb >> 1]);
        }
      }
      if (masked) {
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = e >> 1;
            const int tk_ = nb * 8 + ((2 * c + (e & 1)) ^ ((e & 1) << 2));
            const int at = t0 + tk_;
            const bool see = ((valid >> tk_) & 1u) && at < (i ? lim1 : lim0) &&
                             at >= (i ? win1 : win0);
            if (!see) s[nb][e] = kNegInf;
          }
        }
      }
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        mx[0] = fmaxf(mx[0], fmaxf(s[nb][0], s[nb][1]));
        mx[1] = fmaxf(mx[1], fmaxf(s[nb][2], s[nb][3]));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
      }
      const bool up0 = mx[0] > M[0] + kLazy, up1 = mx[1] > M[1] + kLazy;   // from -inf: any score
      if (__any_sync(0xffffffffu, up0 || up1)) {
        const float f0 = up0 ? (M[0] == kNegInf ? 0.0f : ex2_approx(M[0] - mx[0])) : 1.0f;
        const float f1 = up1 ? (M[1] == kNegInf ? 0.0f : ex2_approx(M[1] - mx[1])) : 1.0f;
        if (up0) M[0] = mx[0];
        if (up1) M[1] = mx[1];
        Z[0] *= f0;
        Z[1] *= f1;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          o[j][0] *= f0;
          o[j][1] *= f0;
          o[j][2] *= f1;
          o[j][3] *= f1;
        }
      }
      const float sub[2] = {M[0] == kNegInf ? 0.0f : M[0] - kPBase,
                            M[1] == kNegInf ? 0.0f : M[1] - kPBase};
      const float iv[2] = {exp2_int(-ev[0]), exp2_int(-ev[1])};
      uint32_t pa[2][4];   // P as the A operand of two 16-token steps
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nb][e] = ex2_approx(s[nb][e] - sub[e >> 1]);
        pa[nb >> 1][2 * (nb & 1)] = pack_f16x2(s[nb][0], s[nb][1]);
        pa[nb >> 1][2 * (nb & 1) + 1] = pack_f16x2(s[nb][2], s[nb][3]);
        Z[0] = fmaf(s[nb][0] + s[nb][1], iv[nb >> 1], Z[0]);
        Z[1] = fmaf(s[nb][2] + s[nb][3], iv[nb >> 1], Z[1]);
      }
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // tokens of fragment rows 2c, 2c + 1, 2c + 8, 2c + 9
          const int tk_ = 16 * h2 + 8 * (i >> 1) + ((2 * c + (i & 1)) ^ ((i & 1) << 2));
          v[i] = lds128(vb + tk_ * kHeadDim + ((nrow ^ (tk_ & 7)) << 4));
          // rows never written may hold NaN codes: 0 * NaN would reach every column
          if (masked && !((valid >> tk_) & 1u)) v[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        const uint32_t a0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, a1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
        const uint32_t a2[4] = {v[2].x, v[2].y, v[2].z, v[2].w}, a3[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t lo01 = __byte_perm(a0[w], a1[w], 0x5140), lo23 = __byte_perm(a0[w], a1[w], 0x7362);
          const uint32_t hi01 = __byte_perm(a2[w], a3[w], 0x5140), hi23 = __byte_perm(a2[w], a3[w], 0x7362);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma_f16(o[4 * w + e], pa[h2], f16_pair(e < 2 ? lo01 : lo23, e & 1),
                    f16_pair(e < 2 ? hi01 : hi23, e & 1));
        }
      }
      __syncwarp();   // every lane has read the stage
      if (more) issue(pd, ST);
      return true;
    };
    for (uint64_t x = g + ((warp - g) & (kWarps - 1)); ok && x < pe; x += kWarps) {
      ok = stage ? unit(x, pend1, 1) : unit(x, pend0, 0);
      stage ^= 1;
    }
    if (!ok) abort_flag = 1;

    // ---- the block's warps together: M, Z and O of rows nrow and nrow + 8
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      Z[i] += __shfl_xor_sync(0xffffffffu, Z[i], 1);
      Z[i] += __shfl_xor_sync(0xffffffffu, Z[i], 2);
      if (Z[i] != Z[i] && M[i] == kNegInf) M[i] = 0.0f;   // nothing but NaN scores: the row is NaN
      if (c == 0) {
        sm_m[warp][nrow + 8 * i] = M[i];
        sm_z[warp][nrow + 8 * i] = Z[i];
      }
    }
    // a lane's 32 columns 32c .. 32c + 31 as 16-byte chunks 8c .. 8c + 7,
    // chunk 8c + k kept at 8c + (k ^ 2c ^ (row & 1)): free of bank conflicts
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = nrow + 8 * i;
      if (row >= rows_left || M[i] == kNegInf) continue;
      float* dst = merge + (warp * kRows + row) * kHeadDim;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = 4 * e + j;
          *reinterpret_cast<float4*>(dst + 4 * (8 * c + (k ^ (2 * c) ^ (row & 1)))) =
              make_float4(o[4 * j][2 * i + e], o[4 * j + 1][2 * i + e], o[4 * j + 2][2 * i + e],
                          o[4 * j + 3][2 * i + e]);
        }
      }
    }
    __syncthreads();
    const bool whole = g == seg_begin && pe == seg_end;
    const uint32_t slot = 2 * blockIdx.x + (g == seg_begin ? 1 : 0);
    float* part = p.partial + static_cast<int64_t>(slot) * kPartialFloats;
    {
      const int row = tid >> 4, ch = tid & 15;   // 8 columns of a row per thread
      if (row < rows_left) {
        float m = kNegInf;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm_m[w][row]);
        float z = 0.0f, v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float mw = sm_m[w][row];
          if (mw == kNegInf) continue;
          const float f = ex2_approx(mw - m);
          z = fmaf(sm_z[w][row], f, z);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int chunk = 2 * ch + e, cg = chunk >> 3;
            const float4 x = *reinterpret_cast<const float4*>(
                merge + (w * kRows + row) * kHeadDim +
                4 * (8 * cg + ((chunk & 7) ^ (2 * cg) ^ (row & 1))));
            v[4 * e] = fmaf(x.x, f, v[4 * e]);
            v[4 * e + 1] = fmaf(x.y, f, v[4 * e + 1]);
            v[4 * e + 2] = fmaf(x.z, f, v[4 * e + 2]);
            v[4 * e + 3] = fmaf(x.w, f, v[4 * e + 3]);
          }
        }
        if (whole) {
          const RowAt r = row_at(p, cc.r, seg, row);
          const float f = row_factor(z);
          uint32_t w4[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                : "=r"(w4[j]) : "f"(v[2 * j + 1] * f), "f"(v[2 * j] * f));
          *reinterpret_cast<uint4*>(p.out + r.token * p.o_ldt + r.head * p.o_ldh + 8 * ch) =
              make_uint4(w4[0], w4[1], w4[2], w4[3]);
          if (p.lse && ch == 0) p.lse[r.token * p.l_ldt + r.head] = row_lse(m, z);
        } else {
          float4* dst = reinterpret_cast<float4*>(part + row * kHeadDim + 8 * ch);
          dst[0] = make_float4(v[0], v[1], v[2], v[3]);
          dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          if (ch == 0) {
            part[kRows * kHeadDim + row] = m;
            part[kRows * kHeadDim + kRows + row] = z;
          }
        }
      }
    }
    __syncthreads();   // before the next segment's rows replace these
    g = pe;
  }
  if (!ok && lane == 0) atomicExch(&g_kv_err, static_cast<int>(BFP8_ERR_TIMEOUT));
  // no copy may still be landing in shared memory when the block exits
  for (int s = 0; s < kStages; ++s)
    if ((armed >> s) & 1u) {
      const uint64_t t_start = globaltimer();
      while (!mbar_try_wait(bar0 + 8 * s, (phase_bits >> s) & 1u))
        if (globaltimer() - t_start > kWaitLimitNs) break;
    }
}

// Joins the partial sums of segments that several blocks shared, in block
// order, and writes the rows of segments that had no unit at all. One block
// per segment; a segment that one block finished is done.
__global__ void __launch_bounds__(128) kv_attention_join_kernel(const AttnParams p, uint32_t grid,
                                                                uint32_t max_rb) {
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t per_b = max_rb * p.H;
  const int b = blockIdx.x / per_b;
  const uint32_t rest = blockIdx.x - b * per_b;
  const uint32_t h = rest / max_rb, rb = rest - h * max_rb;
  const ReqUnits r = req_units(p, b);
  const uint32_t nrb = r.nseg / p.H;
  if (rb >= nrb) return;
  const uint32_t seg = h * nrb + rb;
  const uint64_t U = __ldg(p.schedule + p.B);
  const uint64_t a = __ldg(p.schedule + b) + static_cast<uint64_t>(seg) * r.nt, e = a + r.nt;
  uint32_t c0 = 0, c1 = 0, C = 1;
  if (r.nt) {
    C = used_blocks(U, grid);
    c0 = owner_of(a, U, C);
    c1 = owner_of(e - 1, U, C);
    if (c0 == c1) return;
  }
  const int row = threadIdx.x >> 3, ch = threadIdx.x & 7;   // 16 columns of a row per thread
  const RowAt at = row_at(p, r, seg, row);
  if (!at.real) return;
  float m = kNegInf, z = 0.0f, v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  if (r.nt) {
    auto slot_of = [&](uint32_t c) {
      return p.partial + static_cast<int64_t>(2 * c + (a >= range_begin(U, c, C) ? 1 : 0)) * kPartialFloats;
    };
    for (uint32_t c = c0; c <= c1; ++c) m = fmaxf(m, slot_of(c)[kRows * kHeadDim + row]);
    for (uint32_t c = c0; c <= c1; ++c) {
      const float* part = slot_of(c);
      const float mc = part[kRows * kHeadDim + row];
      if (mc == kNegInf) continue;
      const float f = ex2_approx(mc - m);
      z = fmaf(part[kRows * kHeadDim + kRows + row], f, z);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(part + row * kHeadDim + 16 * ch + 4 * i);
        v[4 * i] = fmaf(x.x, f, v[4 * i]);
        v[4 * i + 1] = fmaf(x.y, f, v[4 * i + 1]);
        v[4 * i + 2] = fmaf(x.z, f, v[4 * i + 2]);
        v[4 * i + 3] = fmaf(x.w, f, v[4 * i + 3]);
      }
    }
  }
  store_row16(p.out + at.token * p.o_ldt + at.head * p.o_ldh + 16 * ch, v, row_factor(z));
  if (p.lse && ch == 0) p.lse[at.token * p.l_ldt + at.head] = row_lse(m, z);
}

template <typename Kernel, typename... Args>
int launch_dependent(Kernel kernel, unsigned blocks, unsigned threads, size_t smem, cudaStream_t st,
                     Args... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? BFP8_OK : BFP8_ERR_CUDA;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t kv_attention_workspace_bytes(int64_t B, int64_t T, int64_t max_q, int64_t Hq, int64_t H,
                                    int sms) {
  (void)T;
  (void)max_q;
  (void)Hq;
  (void)H;
  return align256((B + 1) * 8) + static_cast<size_t>(sms) * 2 * kPartialFloats * 4;
}

int launch_kv_attention(const bfp8_kv_attention_args& a, const bfp8_kv_cache& c, void* stream) {
  int rc = check_kv_cache(c);
  if (rc != BFP8_OK) return rc;
  const int64_t H = c.n_kv_heads;
  if (a.batch < 0 || a.tokens < 0 || a.n_heads < 1 || a.n_heads % H || a.max_blocks < 0 ||
      a.max_q_len < 0 || a.ld_table < a.max_blocks)
    return BFP8_ERR_INVALID_ARG;
  if (a.batch == 0 || a.tokens == 0 || a.max_q_len == 0) return BFP8_OK;
  if (!a.q_bf16 || !a.out_bf16 || !a.q_offsets || !a.kv_len || (a.max_blocks > 0 && !a.block_table))
    return BFP8_ERR_INVALID_ARG;
  if (a.q_stride_token < 0 || a.q_stride_head < 0 || a.out_stride_token < kHeadDim ||
      a.out_stride_head < kHeadDim || (a.lse && a.lse_stride_token < a.n_heads))
    return BFP8_ERR_INVALID_ARG;
  if (!isfinite(a.softmax_scale)) return BFP8_ERR_INVALID_ARG;
  auto rows16 = [](const void* ptr, int64_t s, int64_t t) {
    return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && s % 8 == 0 && t % 8 == 0;
  };
  if (!rows16(a.q_bf16, a.q_stride_token, a.q_stride_head) ||
      !rows16(a.out_bf16, a.out_stride_token, a.out_stride_head) || a.batch > 0x7FFFFFFF ||
      a.max_blocks > 0x7FFFFFFF || a.n_heads > 65535 * 64 || a.tokens > 0x7FFFFFFF)
    return BFP8_ERR_UNSUPPORTED;
  rc = check_device_ptrs({a.q_bf16, a.out_bf16, a.lse, a.q_offsets, a.kv_len, a.block_table,
                          c.k_e4m3, c.v_e4m3, c.k_exp, c.v_exp, a.workspace});
  if (rc != BFP8_OK) return rc;
  int sms = 0;
  rc = sm_count(&sms);
  if (rc != BFP8_OK) return rc;
  const size_t need = kv_attention_workspace_bytes(a.batch, a.tokens, a.max_q_len, a.n_heads, H, sms);
  if (!a.workspace || a.ws_bytes < need || reinterpret_cast<uintptr_t>(a.workspace) % 256)
    return BFP8_ERR_INVALID_ARG;
  AttnParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q_bf16);
  p.out = static_cast<__nv_bfloat16*>(a.out_bf16);
  p.lse = a.lse;
  p.k_exp = c.k_exp;
  p.v_exp = c.v_exp;
  p.table = a.block_table;
  p.q_offsets = a.q_offsets;
  p.kv_len = a.kv_len;
  p.schedule = static_cast<uint64_t*>(a.workspace);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + align256((a.batch + 1) * 8));
  p.q_ldt = a.q_stride_token;
  p.q_ldh = a.q_stride_head;
  p.o_ldt = a.out_stride_token;
  p.o_ldh = a.out_stride_head;
  p.l_ldt = a.lse_stride_token;
  p.ld_table = a.ld_table;
  p.exp_page = c.exp_stride_page;
  p.exp_head = c.exp_stride_head;
  p.T = a.tokens;
  p.n_pages = c.n_pages;
  p.B = static_cast<int32_t>(a.batch);
  p.H = c.n_kv_heads;
  p.G = static_cast<int32_t>(a.n_heads / H);
  p.page_shift = kv_page_shift(c.page_size);
  p.max_blocks = static_cast<int32_t>(a.max_blocks);
  p.window = a.window < 0 ? -1 : a.window;
  p.scale_log2 = a.softmax_scale * kLog2e;
  CUtensorMap tk, tv;
  const uint32_t box = c.page_size < kUnit ? c.page_size : kUnit;
  rc = make_tmap_4d(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.k_e4m3, kHeadDim, c.page_size, H,
                    c.n_pages, c.k_stride_token, c.k_stride_head, c.k_stride_page, kHeadDim, box, 1,
                    1, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != BFP8_OK) return rc;
  rc = make_tmap_4d(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.v_e4m3, kHeadDim, c.page_size, H,
                    c.n_pages, c.v_stride_token, c.v_stride_head, c.v_stride_page, kHeadDim, box, 1,
                    1, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != BFP8_OK) return rc;
  rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kv_attention_rows_kernel), kSmemBytes);
  if (rc != BFP8_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = launch_dependent(kv_attention_rows_kernel, sms, kThreads, kSmemBytes, st, tk, tv, p);
  if (rc != BFP8_OK) return rc;
  const int64_t max_rb = (a.max_q_len * p.G + kRows - 1) / kRows;
  const int64_t blocks = a.batch * H * max_rb;
  if (blocks > 0x7FFFFFFF) return BFP8_ERR_UNSUPPORTED;
  rc = launch_dependent(kv_attention_join_kernel, static_cast<unsigned>(blocks), 128, 0, st, p,
                        static_cast<uint32_t>(sms), static_cast<uint32_t>(max_rb));
  if (rc != BFP8_OK) return rc;
  return check_launch();
}

int kv_read_clear_error() {
  int v = 0;
  const int zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv_err, sizeof(int)) != cudaSuccess) return BFP8_ERR_CUDA;
  if (v != 0 && cudaMemcpyToSymbol(g_kv_err, &zero, sizeof(int)) != cudaSuccess)
    return BFP8_ERR_CUDA;
  return v == 0 ? BFP8_OK : v;
}

}  // namespace bfp8
