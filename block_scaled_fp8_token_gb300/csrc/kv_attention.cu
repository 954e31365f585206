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
#include "attention_layer.cuh"
#include "kv_common.cuh"
#include "act_math.cuh"

#include <algorithm>

namespace bfp8 {
namespace {

using namespace dev;

__device__ int g_kv_err;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -INFINITY;

// Waits for copies or products in flight before a block ends, whatever else
// went wrong; bounded like every wait.
BFP8_DEV void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > kWaitLimitNs) break;
}

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
  uint64_t* schedule;        // [B + 1]: the rows kernel's units before each request, and in all
  int64_t q_ldt, q_ldh, o_ldt, o_ldh, l_ldt, ld_table, exp_page, exp_head;
  int64_t T, n_pages;
  int32_t max_q;             // rows of a request past this many are left alone
  int32_t B, H, G, page_shift, max_blocks, window;
  int32_t seg_rows;          // query rows of a segment of the rows kernel: 8 or 16
  int32_t few_rows;          // requests of at most this many rows of a KV head go to the rows kernel
  int32_t whole_items;       // the tiles kernel's blocks take whole items
  int32_t tiles_follow;      // it runs right behind the rows kernel
  struct TileDesc* tile_desc;   // [blocks]
  float* tile_partial;       // [blocks][2] of kTilePartialFloats
  float scale_log2;          // softmax scale * log2(e)
};

// ============================================================ few query rows
// A unit of work is 32 tokens of one segment; a segment is 8 or 16 query rows
// (the heads of a group, times the tokens of a draft) of one request and KV
// head. All units are numbered request by request and cut into equal contiguous
// ranges, one per block, so ragged lengths balance; a block's warps take its
// units in turn, each with its own ring of shared-memory stages and no barrier
// between them inside a segment.
//
// The products are transposed, tokens (and then columns of V) as the 16 rows of
// a matrix instruction and query rows as its 8 columns: a group of 8 heads fills
// one. S^T = K Q^T takes the codes as they are, an FP8 product with the query
// row split exactly into E5M2 + E4M3 (see query_terms); O^T += V^T P^T widens
// the codes to F16, two to an instruction, and rounds P to 11 bits.
//
// HBM bounds it. What kept it from that was copies in flight and warps to hide
// latencies: several small blocks an SM instead of one large one, so that one's
// merge and query loads overlap the others' products.
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = 32;                 // tokens
constexpr int kMaxRows = 16;              // query rows of a segment, at most
constexpr int kStageBytes = 2 * kUnit * kHeadDim;            // keys, then values
constexpr int kMergeBytes = kWarps * 8 * (kHeadDim / 2) * 4;
constexpr int kRowsPerSm = 2;             // blocks (three of two stages each: 130 us a pass, against 120)
constexpr int kStages = 3;
constexpr int kRowsSmem = kWarps * kStages * kStageBytes + kMergeBytes + 1024;   // + alignment
constexpr int kPartialFloats = kMaxRows * (kHeadDim + 2);    // O, then M, then Z
// Ending a segment costs a block about as long as this many units, which the
// schedule counts behind each segment's own.
constexpr uint32_t kPadUnits = 8;
// P is 2^(score - M), and M is taken 4 below the largest score and moves only when
// a score passes it by more than 14, so F16 holds P up to 2^14 and, to full
// precision, down to 2^-18 of the largest weight. Both steps are on M as it was
// rounded, not on the score it came from: at scores of 2^26 and more, where
// FP32's steps are 8 and up, M is a step away from what was meant, and the
// weights are within bounds all the same.
constexpr float kPBase = 4.0f;
constexpr float kReach = 14.0f;
// M of a row that has seen nothing: any score passes it.
constexpr float kNoMax = -3.40282347e38f;

// The first position that a row at `pos` sees; from a position below 0, which sees
// nothing, a large window would go past 32 bits.
BFP8_DEV int window_begin(const AttnParams& p, int pos) {
  return p.window >= 0 ? max(max(pos, 0) - p.window, 0) : 0;
}

// A request's rows: n of them from q0 on, the first at position pos0 (below 0 where
// the cache holds fewer tokens than there are new ones).
struct ReqRows {
  int32_t q0, n, pos0;
};
BFP8_DEV ReqRows req_rows(const AttnParams& p, int b, int kv) {
  ReqRows r;
  r.q0 = max(__ldg(p.q_offsets + b), 0);
  const int64_t q1 = min(static_cast<int64_t>(__ldg(p.q_offsets + b + 1)), p.T);
  const int32_t n = static_cast<int32_t>(max(q1 - r.q0, static_cast<int64_t>(0)));
  r.pos0 = kv - n;
  r.n = min(n, p.max_q);
  return r;
}

struct ReqUnits : ReqRows {
  int32_t kv;              // its length
  int32_t first, lo;       // first token that any row sees, and its unit
  uint32_t nt, nseg, nrb;  // units of a segment, segments, segments of a head
  BFP8_DEV uint32_t cost() const { return nt ? nt + kPadUnits : 0; }   // a segment's, in units
};
BFP8_DEV ReqUnits req_units(const AttnParams& p, int b) {
  ReqUnits r;
  r.kv = max(__ldg(p.kv_len + b), 0);
  static_cast<ReqRows&>(r) = req_rows(p, b, r.kv);
  const int64_t held = min(static_cast<int64_t>(r.kv),
                           static_cast<int64_t>(p.max_blocks) << p.page_shift);
  r.first = window_begin(p, r.pos0);
  r.lo = r.first / kUnit;
  const int64_t hi = (held + kUnit - 1) / kUnit;
  r.nt = r.n > 0 && hi > r.lo ? static_cast<uint32_t>(hi - r.lo) : 0u;
  const int64_t rows = static_cast<int64_t>(r.n) * p.G;
  r.nrb = static_cast<uint32_t>((rows + p.seg_rows - 1) / p.seg_rows);
  r.nseg = r.nrb * p.H;
  if (rows > p.few_rows) r.nt = 0;   // the tiles kernel's
  return r;
}
BFP8_DEV uint64_t units_of(const AttnParams& p, int b) {
  const ReqUnits r = req_units(p, b);
  return static_cast<uint64_t>(r.cost()) * r.nseg;
}

// A segment, and the part of it inside a block's range: `len` units from its
// u0-th on, `at` units into the range; the ones that exist are below nt.
struct SegPart {
  ReqUnits r;
  int b;
  uint32_t seg, h, u0, at, len;
  BFP8_DEV uint32_t units() const { return u0 < r.nt ? min(len, r.nt - u0) : 0; }
};
BFP8_DEV void next_segment(const AttnParams& p, SegPart& s, uint32_t range) {
  s.at += s.len;
  s.u0 = 0;
  if (++s.seg >= s.r.nseg) {
    s.seg = 0;
    do {
      if (++s.b >= p.B) {
        s.at = range;
        s.len = 0;
        return;
      }
      s.r = req_units(p, s.b);
    } while (s.r.nt == 0 || s.r.nseg == 0);
  }
  s.h = s.seg / s.r.nrb;
  s.len = min(s.r.cost(), range - s.at);
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

BFP8_DEV void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                      const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}
// E4M3 times E5M2, and E4M3 times E4M3.
BFP8_DEV void mma_e4m3_e5m2(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e5m2.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
BFP8_DEV void mma_e4m3_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
BFP8_DEV uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
BFP8_DEV uint32_t join16(uint16_t lo, uint16_t hi) {
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
// A query row as two FP8 terms, at a power of two that puts its largest entry
// in [2^11, 2^12). An entry of 2^e .. 2^(e+1) is a multiple of 2^(e-7) (a BF16
// has 8 significant bits); hi, E5M2, keeps 3 bits of it, so the rest is at most
// 16 of those steps, which E4M3's 4 bits hold, and 2^8 at most. hi + lo is exact
// for entries down to 2^-13 of the largest; below, it is within 2^-21 of it. (Rows
// below 2^-99 stay short of 2^11: at such sizes no score is of any weight.)
BFP8_DEV int query_exponent(uint32_t amax_bits) {
  return amax_bits ? min(11 - (static_cast<int>(amax_bits >> 7) - 127), 110) : 0;
}
// Largest |x| of each half, as BF16 bits with their sign cleared (a NaN stays one
// only where both operands are).
BFP8_DEV uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
  return r;
}
// Four entries (two BF16 pairs) times `up`: a word of codes of each term. F16
// holds every scaled entry down to 2^-26 of the largest exactly, and hi and the
// difference too. FP8 conversions saturate; an infinite entry's difference takes a
// NaN, x * 0, so that its row's scores are NaN.
BFP8_DEV void query_terms(uint32_t ab, uint32_t cd, float up, uint32_t& hi, uint32_t& lo) {
  const uint32_t in[2] = {ab, cd};
  uint16_t h[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = __fmul2_rn(make_float2(__uint_as_float(in[i] << 16), __uint_as_float(in[i] & 0xFFFF0000u)),
                                make_float2(up, up));
    const uint32_t x = pack_f16x2(f.x, f.y);
    h[i] = f16x2_to_e5m2x2(x);
    l[i] = f16x2_to_e4m3x2(fma_f16x2(x, 0u, sub_f16x2(x, e5m2x2_to_f16x2(h[i]))));
  }
  hi = join16(h[0], h[1]);
  lo = join16(l[0], l[1]);
}
BFP8_DEV uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
BFP8_DEV uint32_t f16_pair(uint32_t word, int half) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(half ? word >> 16 : word & 0xFFFFu));
}

// Row `row` of a segment: which query and head it is.
struct RowAt {
  int64_t token;
  int head;
  int pos;
  bool real;
};
BFP8_DEV RowAt row_at(const AttnParams& p, const ReqUnits& r, uint32_t h, uint32_t rb, int row) {
  RowAt a;
  const uint32_t i = rb * p.seg_rows + row;
  const uint32_t tok = i / p.G;
  a.real = tok < static_cast<uint32_t>(r.n);
  a.token = r.q0 + static_cast<int64_t>(a.real ? tok : 0);
  a.head = h * p.G + (i - tok * p.G);
  a.pos = r.pos0 + static_cast<int>(tok);
  return a;
}

// out = O / Z and lse, from sums of 2^(score - M); a row that saw nothing gives 0 and -inf.
BFP8_DEV float row_factor(float Z) { return Z == 0.0f ? 0.0f : __frcp_rn(Z); }
BFP8_DEV float row_lse(float M, float Z) {
  return Z == 0.0f ? kNegInf : kLn2 * (M + log2f(Z));
}
BFP8_DEV uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
BFP8_DEV void store_row16(__nv_bfloat16* dst, const float (&v)[16], float f) {
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = pack_bf16x2(v[2 * j] * f, v[2 * j + 1] * f);
  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(dst + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// NB: query rows of a segment, in eights.
template <int NB>
__global__ void __launch_bounds__(kThreads, kRowsPerSm)
    kv_attention_rows_kernel(const __grid_constant__ CUtensorMap tk,
                             const __grid_constant__ CUtensorMap tv, const AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[kWarps * kStages];
  __shared__ uint2 infos[kWarps][kStages];   // a unit's scale bytes (k, k, v, v of its halves) and valid tokens
  __shared__ float sm_m[kWarps][8 * NB], sm_z[kWarps][8 * NB];
  // each warp's places in the sequence of segments: computing, and loading
  __shared__ SegPart seg_at[kWarps][2], seg_next[kWarps];
  __shared__ uint64_t scan[kWarps];
  __shared__ uint64_t start_base;
  __shared__ int start_b;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  float* merge = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)) +
                                          kWarps * kStages * kStageBytes);
  if (tid < kWarps * kStages) mbar_init(smem_u32(&bars[tid]), 1);
  if (tid == 0) abort_flag = 0, start_b = 0, start_base = 0;
  mbar_fence_init();
  pdl_wait();
  // The tiles kernel needs nothing of this one: its blocks set themselves up as these
  // end, and wait there for whatever both read.
  if (p.tiles_follow) pdl_launch_dependents();

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
  const uint32_t range = idle ? 0 : static_cast<uint32_t>(range_begin(U, blockIdx.x + 1, C) - g0);
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
  if (range == 0) return;

  const uint32_t bar0 = smem_u32(&bars[warp * kStages]);
  const uint32_t stage0 = ring + warp * kStages * kStageBytes;
  const int page = 1 << p.page_shift;
  const int box = min(page, kUnit);
  const uint32_t two = page < kUnit ? 1u : 0u;   // a unit's second half has a page of its own
  const int c = lane & 3, g = lane >> 2;
  const int gtok = g ^ ((g & 1) << 2);           // see "Fragments" below

  SegPart& cs = seg_at[warp][0];
  SegPart& ps = seg_at[warp][1];
  {
    SegPart x;
    x.b = start_b;
    x.r = req_units(p, x.b);
    const uint32_t rel = static_cast<uint32_t>(g0 - start_base);
    x.seg = rel / x.r.cost();
    x.u0 = rel - x.seg * x.r.cost();
    x.h = x.seg / x.r.nrb;
    x.at = 0;
    x.len = min(x.r.cost() - x.u0, range);
    while (x.at < range && x.units() == 0) next_segment(p, x, range);
    if (lane == 0) cs = ps = x;
    __syncwarp();
  }

  // ---- issuing: this warp's next unit, the px-th of a segment's part; the
  // warps take a part's units in turn, from the one that its place gives
  uint32_t px = 0, p_units = 0;
  int32_t p_t0 = 0, p_held = 0, p_h = 0;         // of the segment: first token of the part, tokens, head
  const int32_t* p_row = nullptr;                // its request's row of the table
  int32_t id0 = -1, id1 = -1;                    // the unit's page numbers (two when pages hold 16)
  int32_t pt0 = 0;                               // its first token
  bool more = true;
  auto enter = [&](const SegPart& x) {
    px = (warp - x.at) & (kWarps - 1);
    p_units = x.units();
    p_t0 = (x.r.lo + static_cast<int32_t>(x.u0)) * kUnit;
    p_held = static_cast<int32_t>(min(static_cast<int64_t>(x.r.kv),
                                      static_cast<int64_t>(p.max_blocks) << p.page_shift));
    p_h = x.h;
    p_row = p.table + x.b * p.ld_table;
  };
  auto fetch_ids = [&] {
    if (px >= p_units) {
      SegPart x = ps;
      while (px >= p_units) {
        next_segment(p, x, range);
        if (x.at >= range) {
          more = false;
          return;
        }
        enter(x);
      }
      __syncwarp();
      if (lane == 0) ps = x;
      __syncwarp();
    }
    pt0 = p_t0 + static_cast<int32_t>(px) * kUnit;
    const int32_t* row = p_row + (pt0 >> p.page_shift);
    id0 = __ldg(row);   // inside the table: units stop at its width
    if (two) id1 = pt0 + page < p_held ? __ldg(row + 1) : -1;
  };
  uint32_t armed = 0, phase_bits = 0;   // stages with copies in flight; their parities
  // Scale bytes of the unit issued last. They are stored for its use only when
  // the next one is issued, so their latency hides behind a unit's products.
  uint32_t k0 = 127, k1 = 127, v0 = 127, v1 = 127, valid_next = 0;
  int pending = -1;
  auto flush = [&] {
    if (pending >= 0 && lane == 0)
      infos[warp][pending] = make_uint2(k0 | (k1 << 8) | (v0 << 16) | (v1 << 24), valid_next);
    pending = -1;
  };
  auto issue = [&](const int s) {
    // a page that ends ahead of the first token seen is as good as missing
    const int32_t ahead = ps.r.first - pt0;   // less than 32: the unit holds that token or follows it
    const bool ok0 = id0 >= 0 && id0 < p.n_pages && ahead < box, ok1 = two && id1 >= 0 && id1 < p.n_pages;
    if (lane == 0) {
      const uint32_t bar = bar0 + 8 * s, dst = stage0 + s * kStageBytes;
      const uint32_t bytes = box * kHeadDim;
      mbar_arrive_expect_tx(bar, 2 * bytes * ((ok0 ? 1 : 0) + (ok1 ? 1 : 0)));
      if (ok0) {
        tma_load_4d(dst, &tk, 0, pt0 & (page - 1), p_h, id0, bar);
        tma_load_4d(dst + kUnit * kHeadDim, &tv, 0, pt0 & (page - 1), p_h, id0, bar);
      }
      if (ok1) {
        tma_load_4d(dst + bytes, &tk, 0, 0, p_h, id1, bar);
        tma_load_4d(dst + kUnit * kHeadDim + bytes, &tv, 0, 0, p_h, id1, bar);
      }
    }
    const int32_t left = p_held - pt0;
    valid_next = left >= 32 ? 0xffffffffu : (1u << left) - 1u;   // left >= 1
    if (ahead > 0) valid_next &= 0xffffffffu << ahead;
    valid_next &= two ? (ok0 ? 0xffffu : 0u) | (ok1 ? 0xffff0000u : 0u) : (ok0 ? 0xffffffffu : 0u);
    k0 = k1 = v0 = v1 = 127u;
    if (ok0) {
      const int64_t e = id0 * p.exp_page + p_h * p.exp_head;
      k0 = __ldg(p.k_exp + e), v0 = __ldg(p.v_exp + e);
    }
    if (ok1) {
      const int64_t e = id1 * p.exp_page + p_h * p.exp_head;
      k1 = __ldg(p.k_exp + e), v1 = __ldg(p.v_exp + e);
    }
    armed |= 1u << s;
    pending = s;
    px += kWarps;
    fetch_ids();
  };
  enter(ps);
  fetch_ids();
  for (int s = 0; s < kStages && more; ++s) {
    flush();
    issue(s);
  }
  if (!more) flush();   // nothing may be issued any more that would do it

  // ---- query rows: lane (g, c) loads 16-byte chunks c and c + 4 of rows 8 nb + g
  uint4 raw[NB][4];
  auto load_q = [&](const SegPart& s) {
    const uint32_t rb = s.seg - s.h * s.r.nrb;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const RowAt r = row_at(p, s.r, s.h, rb, 8 * nb + g);
      const __nv_bfloat16* src = p.q + r.token * p.q_ldt + r.head * p.q_ldh + 16 * c;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        raw[nb][j] = make_uint4(0u, 0u, 0u, 0u);
        if (r.real) raw[nb][j] = __ldg(reinterpret_cast<const uint4*>(src + 64 * (j >> 1) + 8 * (j & 1)));
      }
    }
  };
  if (cs.at < range) load_q(cs);

  int stage = 0;
  bool ok = true;
  while (cs.at < range) {
    const uint32_t rb = cs.seg - cs.h * cs.r.nrb;
    const int rows_left = static_cast<int>(
        min(static_cast<int64_t>(8 * NB),
            static_cast<int64_t>(cs.r.n) * p.G - static_cast<int64_t>(rb) * (8 * NB)));

    uint32_t qh[NB][8], ql[NB][8];   // the two terms' codes: four columns a word
    float fac[NB][2];              // of rows 2c and 2c + 1: what a score is in log2 units
    int lim[NB][2], win[NB][2];    // they see [win, lim)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w[4] = {raw[nb][j].x, raw[nb][j].y, raw[nb][j].z, raw[nb][j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
      }
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = query_exponent(m);
      const float up = exp2_int(e), f = exp2_int(-e) * p.scale_log2;
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // eight columns: words 2j, 2j + 1
        query_terms(raw[nb][j].x, raw[nb][j].y, up, qh[nb][2 * j], ql[nb][2 * j]);
        query_terms(raw[nb][j].z, raw[nb][j].w, up, qh[nb][2 * j + 1], ql[nb][2 * j + 1]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        fac[nb][j] = __shfl_sync(0xffffffffu, f, (2 * c + j) * 4);
        const RowAt r = row_at(p, cs.r, cs.h, rb, 8 * nb + 2 * c + j);
        lim[nb][j] = r.real ? r.pos + 1 : 0x7FFFFFFF;   // rows that do not exist never ask for a mask
        win[nb][j] = r.real ? window_begin(p, r.pos) : 0;
      }
    }
    int lim_min = lim[0][0], win_max = win[0][0];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int j = 0; j < 2; ++j) lim_min = min(lim_min, lim[nb][j]), win_max = max(win_max, win[nb][j]);
    }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);
    win_max = __reduce_max_sync(0xffffffffu, win_max);

    float o[NB][8][4];
    float M[NB][2], Z[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[nb][i][0] = o[nb][i][1] = o[nb][i][2] = o[nb][i][3] = 0.0f;
      M[nb][0] = M[nb][1] = kNegInf;
      Z[nb][0] = Z[nb][1] = 0.0f;
    }

    const uint32_t units = cs.units();
    const int t_part = (cs.r.lo + static_cast<int32_t>(cs.u0)) * kUnit;
    for (uint32_t x = (warp - cs.at) & (kWarps - 1); ok && x < units; x += kWarps) {
      const uint32_t bar = bar0 + 8 * stage;
      const uint32_t kb = stage0 + stage * kStageBytes, vb = kb + kUnit * kHeadDim;
      ok = __all_sync(0xffffffffu, mbar_wait(bar, (phase_bits >> stage) & 1u, &abort_flag));
      if (!ok) break;
      __syncwarp();
      armed &= ~(1u << stage);
      phase_bits ^= 1u << stage;
      const uint2 info = infos[warp][stage];
      const int kx = static_cast<int>(info.x & 0xffu), vx = static_cast<int>((info.x >> 16) & 0xffu);
      const int ek[2] = {kx - 127, (two ? static_cast<int>((info.x >> 8) & 0xffu) : kx) - 127};
      const int ev[2] = {vx - 127, (two ? static_cast<int>(info.x >> 24) : vx) - 127};
      const uint32_t valid = info.y;
      const int t0 = t_part + static_cast<int>(x) * kUnit;

      // Fragments. S^T: 16 tokens x 32 columns of K a step, and which column is
      // which does not matter as long as q agrees, so a lane reads its tokens'
      // 16-byte chunks c and c + 4 whole. O^T: a lane reads 16 columns (chunk g)
      // of four tokens, and holds 16 columns in a row of O for rows 2c, 2c + 1.
      // Token n of a block of eight is n ^ 4(n & 1): with the 128-byte swizzle
      // both reads are then free of bank conflicts.
      float s[NB][2][4];
#pragma unroll
      for (int mb = 0; mb < 2; ++mb) {
        const uint32_t row = kb + (16 * mb + gtok) * kHeadDim;
        const uint32_t x0 = (c ^ gtok) << 4, x1 = ((c + 4) ^ gtok) << 4;
        const uint4 a = lds128(row + x0), b = lds128(row + x1);
        const uint4 d = lds128(row + 8 * kHeadDim + x0), e = lds128(row + 8 * kHeadDim + x1);
        const uint32_t w1[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const uint32_t w2[8] = {d.x, d.y, d.z, d.w, e.x, e.y, e.z, e.w};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          s[nb][mb][0] = s[nb][mb][1] = s[nb][mb][2] = s[nb][mb][3] = 0.0f;
#pragma unroll
          for (int st = 0; st < 4; ++st)
            mma_e4m3_e5m2(s[nb][mb], w1[2 * st], w2[2 * st], w1[2 * st + 1], w2[2 * st + 1],
                          qh[nb][2 * st], qh[nb][2 * st + 1]);
#pragma unroll
          for (int st = 0; st < 4; ++st)
            mma_e4m3_e4m3(s[nb][mb], w1[2 * st], w2[2 * st], w1[2 * st + 1], w2[2 * st + 1],
                          ql[nb][2 * st], ql[nb][2 * st + 1]);
        }
      }
      // s[nb][mb]: tokens 16 mb + gtok (entries 0, 1) and 8 on (2, 3), rows 2c
      // and 2c + 1. In log2 units, with the value scale's exponent:
      const bool masked = valid != 0xffffffffu || t0 + kUnit > lim_min || t0 < win_max;
      const float lv[2] = {static_cast<float>(ev[0]), static_cast<float>(ev[1])};
      const float kf[2] = {exp2_int(ek[0]), exp2_int(ek[1])};
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[nb][mb][e] = fmaf(s[nb][mb][e], fac[nb][e & 1] * kf[mb], lv[mb]);
        }
      }
      if (masked) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int mb = 0; mb < 2; ++mb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tok = 16 * mb + gtok + 8 * (e >> 1), at = t0 + tok;
              if (!((valid >> tok) & 1u) || at >= lim[nb][e & 1] || at < win[nb][e & 1])
                s[nb][mb][e] = kNegInf;
            }
          }
        }
      }
      float mx[NB][2];
      bool grow = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float m = fmaxf(fmaxf(s[nb][0][j], s[nb][0][2 + j]), fmaxf(s[nb][1][j], s[nb][1][2 + j]));
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
          mx[nb][j] = m;
          grow |= m - M[nb][j] > kReach;   // from -inf: any score
        }
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float f[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const bool up = mx[nb][j] - M[nb][j] > kReach;
            const float to = mx[nb][j] - kPBase;
            f[j] = !up ? 1.0f : M[nb][j] == kNegInf ? 0.0f : ex2_approx(M[nb][j] - to);
            if (up) M[nb][j] = to;
            Z[nb][j] *= f[j];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nb][i][e] *= f[e & 1];
          }
        }
      }
      const float iv[2] = {exp2_int(-ev[0]), exp2_int(-ev[1])};
      uint32_t pb[NB][2][2];   // P^T as the B operand of two 16-token steps
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float sub[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) sub[j] = M[nb][j] == kNegInf ? 0.0f : M[nb][j];
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nb][mb][e] = ex2_approx(s[nb][mb][e] - sub[e & 1]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            pb[nb][mb][j] = transpose8x8(pack_f16x2(s[nb][mb][2 * j], s[nb][mb][2 * j + 1]));
            Z[nb][j] = fmaf(s[nb][mb][j] + s[nb][mb][2 + j], iv[mb], Z[nb][j]);
          }
        }
      }
#pragma unroll
      for (int mb = 0; mb < 2; ++mb) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // the tokens of fragment columns 2c, 2c + 1, 2c + 8, 2c + 9
          const int tok = 16 * mb + 8 * (i >> 1) + ((2 * c + (i & 1)) ^ ((i & 1) << 2));
          v[i] = lds128(vb + tok * kHeadDim + ((g ^ (tok & 7)) << 4));
          // rows never written, or left to others behind the window, may hold NaN codes:
          // 0 * NaN would reach every column
          if (masked && !((valid >> tok) & 1u)) v[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        const uint32_t v0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, v1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
        const uint32_t v2[4] = {v[2].x, v[2].y, v[2].z, v[2].w}, v3[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {   // columns 4w + 2e and one on, of two tokens a word
            const uint32_t sel = e ? 0x7362 : 0x5140;
            const uint32_t ab = __byte_perm(v0[w], v1[w], sel), cd = __byte_perm(v2[w], v3[w], sel);
            const uint32_t a0 = f16_pair(ab, 0), a1 = f16_pair(ab, 1);
            const uint32_t a2 = f16_pair(cd, 0), a3 = f16_pair(cd, 1);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma_f16(o[nb][2 * w + e], a0, a1, a2, a3, pb[nb][mb]);
          }
        }
      }
      flush();
      __syncwarp();   // every lane has read the stage
      if (more) issue(stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    if (!ok) abort_flag = 1;

    // the next segment's query rows are on their way while this one is finished
    SegPart nx = cs;
    do next_segment(p, nx, range);
    while (nx.at < range && nx.units() == 0);
    if (nx.at < range) load_q(nx);
    __syncwarp();
    if (lane == 0) seg_next[warp] = nx;

    // ---- the block's warps together, eight rows and 64 columns at a time
    const bool whole = cs.u0 == 0 && units == cs.r.nt;
    float* part = p.partial +
                  static_cast<int64_t>(2 * blockIdx.x + (cs.u0 == 0 ? 1 : 0)) * kPartialFloats;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float z = Z[nb][j];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
        if (z != z && M[nb][j] == kNegInf) M[nb][j] = 0.0f;   // nothing but NaN scores: the row is NaN
        if (g == 0) {
          sm_m[warp][8 * nb + 2 * c + j] = M[nb][j];
          sm_z[warp][8 * nb + 2 * c + j] = z;
        }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        // a lane's 16 columns as 16-byte chunks 4 (g & 3) .. of its half, chunk k
        // of row r kept at k ^ (r / 2): free of bank conflicts
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = 2 * c + j;
          if ((g >> 2) == half && 8 * nb + row < rows_left && M[nb][j] != kNegInf) {
            float* dst = merge + (warp * 8 + row) * (kHeadDim / 2);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<float4*>(dst + 4 * ((4 * (g & 3) + k) ^ c)) =
                  make_float4(o[nb][2 * k][j], o[nb][2 * k][2 + j], o[nb][2 * k + 1][j],
                              o[nb][2 * k + 1][2 + j]);
          }
        }
        __syncthreads();
        const int row = tid >> 4, k = tid & 15, srow = 8 * nb + row;   // a 16-byte chunk per thread
        if (srow < rows_left) {
          const int col = 64 * half + 4 * k;
          float m = kNegInf;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm_m[w][srow]);
          float z = 0.0f;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float mw = sm_m[w][srow];
            if (mw == kNegInf) continue;
            const float f = ex2_approx(mw - m);
            z = fmaf(sm_z[w][srow], f, z);
            const float4 y = *reinterpret_cast<const float4*>(
                merge + (w * 8 + row) * (kHeadDim / 2) + 4 * (k ^ (row >> 1)));
            v.x = fmaf(y.x, f, v.x);
            v.y = fmaf(y.y, f, v.y);
            v.z = fmaf(y.z, f, v.z);
            v.w = fmaf(y.w, f, v.w);
          }
          if (whole) {
            const RowAt r = row_at(p, cs.r, cs.h, rb, srow);
            const float f = row_factor(z);
            *reinterpret_cast<uint2*>(p.out + r.token * p.o_ldt + r.head * p.o_ldh + col) =
                make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
            if (p.lse && col == 0) p.lse[r.token * p.l_ldt + r.head] = row_lse(m, z);
          } else {
            *reinterpret_cast<float4*>(part + srow * kHeadDim + col) = v;
            if (col == 0) {
              part[8 * NB * kHeadDim + srow] = m;
              part[8 * NB * (kHeadDim + 1) + srow] = z;
            }
          }
        }
        __syncthreads();   // before the next rows replace these
      }
    }
    if (lane == 0) cs = seg_next[warp];
    __syncwarp();
  }
  // Not earlier: blocks of the kernels behind that wait on an SM hold registers
  // and shared memory that this launch's or the next's need (130 -> 180 us a pass).
  pdl_launch_dependents();
  if (!ok && lane == 0) atomicExch(&g_kv_err, static_cast<int>(BFP8_ERR_TIMEOUT));
  // no copy may still be landing in shared memory when the block exits
  for (int s = 0; s < kStages; ++s)
    if ((armed >> s) & 1u) drain(bar0 + 8 * s, (phase_bits >> s) & 1u);
}

// ============================================================ many query rows
// An item is 256 query rows (two tiles of 128; the heads of a group times
// consecutive tokens) of one request and KV head, against its tokens in tiles
// of 128. S = Q K^T runs on the FP8 tensor cores with the codes of the keys as
// they lie in memory: a query row goes in as two terms, hi in E5M2 (3 of a
// BF16's 8 significant bits, and the range) and lo in E4M3 (the rest, exactly),
// at the cost of one BF16 product and half its operand bytes. O += P V runs on the
// F16 ones, P rounded to 11 significant bits and the codes of V widened exactly.
//   warp 0       loads pages by TMA into a ring of keys and one of values
//   warp 1       issues the products
//   warps 2, 3   widen the values' codes to F16, MN-major, in two buffers
//   warps 4..7   softmax of tile 0, one thread a row; warps 8..11 of tile 1
// While one tile's softmax runs, the tensor cores work on the other's. S is
// FP32 in tensor memory; P replaces it there, 64 tokens at a time, and is the PV
// product's A operand, so weights never touch shared memory. O stays in tensor
// memory and is scaled down only when a row's largest score has outgrown M.
// A weight's exponent is one fused step, y 2^ek + (ev - M), from a score that was
// never rounded, while M comes from one that was. That difference, half a step of
// the largest score, must stay small against kReach: from kBigScore on, where a
// step is 1/2, a row rounds its scores first (in pairs, for the registers: 238 us a
// pass of 4096 tokens, with or without this; one at a time it cost 8 more).
//
// One block an SM stays for the whole call. The items' tiles are cut into equal
// contiguous ranges, so that one long chunk does not hold the others up; an item
// cut by a range's end leaves FP32 partial sums that the join kernel adds. A
// single prompt with four items an SM or more keeps them whole, in rounds over
// the blocks of alternating direction, and needs no join. (Whole and cut, 64 heads on
// 8, from cold caches: prompts of 1200, 2600, 4000, 8192 tokens 40, 117, 229, 818 us and
// 52, 130, 249, 857; 1200, 2600, 4000 behind 6000 others 197, 507, 773 and 212, 467,
// 755; 640 and 2440 behind 30,000, with a last round that few blocks share, 794, 2046
// and 449, 1700. Fewer items would gain up to a quarter without a prefix, which
// the host cannot know, and lose up to 77 % behind a long one; from four an SM on
// either loss is a fifth at most.)
//
// What bounds it: 4096 tokens run at 1.19 PFLOP/s, counting the causal half of the
// scores. A pair of tiles takes 3,400 clocks, of which the products need 2,048 and
// their operands, with the widening and the copies, 2,300 of shared memory; a
// tile's scores wait for the PV product of the tile before, that for its softmax,
// and softmax of 64 tokens takes 900 to 1,200 clocks of latency. Tried: scores in
// halves of 64 tokens, made while softmax is still at work (273, and 238 with one
// thread that waits and issues) or one right behind the other (255), as N = 64
// products are bound by shared memory; two threads a row (303); weights taken
// before the maximum is known (275) or with no maximum unless their sum is too
// large (244); two issuing warps (279 when one took 263). One issuing thread, half
// the instructions in the widening, P stored in two parts: no change.
constexpr int kTileRows = 128, kTileTokens = 128;
constexpr int kItemRows = 2 * kTileRows;
constexpr int kHalf = kTileTokens / 2;
constexpr int kTileThreads = 384;
constexpr int kTileStages = 3;                           // of keys
constexpr int kValueStages = 2;                          // freed as soon as they are widened
constexpr int kInfos = kTileStages + 1;                  // see TileShared
constexpr int kQBytes = kTileRows * kHeadDim;            // one term of one query tile
constexpr int kKvBytes = kTileTokens * kHeadDim;
constexpr int kV16Bytes = 2 * kKvBytes;
constexpr int kQueryPairs = 2;                           // pairs of rows made into terms at a time
constexpr int kOutStage = 32 * 64;                        // a softmax warp's, for 32 columns of BF16
constexpr int kTileSmem =
    4 * kQBytes + (kTileStages + kValueStages) * kKvBytes + 2 * kV16Bytes + 8 * kOutStage + 1024;
// Queries' rows of an unfinished item: O as [column / 4][row][4], then M, then Z.
constexpr int kTilePartialFloats = kItemRows * kHeadDim + 2 * kItemRows;
constexpr uint32_t kColS = 0, kColO = 256;   // S of tile w at 128 w, O at 256 + 128 w
// Beginning and ending an item costs about as long as this many tiles, which
// the schedule counts behind each item's own; a block gets kTileShare at least.
constexpr uint32_t kTilePad = 3, kTileShare = 6;

constexpr float kBigScore = 4194304.0f;   // 2^22

struct TileReq : ReqRows {
  int32_t held;              // tokens inside the table
  uint32_t pairs;            // items of a KV head; 0: not this kernel's
};
BFP8_DEV TileReq tile_req(const AttnParams& p, int b) {
  TileReq r;
  const int32_t kv = max(__ldg(p.kv_len + b), 0);
  static_cast<ReqRows&>(r) = req_rows(p, b, kv);
  r.held = static_cast<int32_t>(min(static_cast<int64_t>(kv),
                                    static_cast<int64_t>(p.max_blocks) << p.page_shift));
  const int64_t rows = static_cast<int64_t>(r.n) * p.G;
  r.pairs = rows > p.few_rows ? static_cast<uint32_t>((rows + kItemRows - 1) / kItemRows) : 0u;
  return r;
}
// The first token that a row of pair `q` sees.
BFP8_DEV int pair_first(const AttnParams& p, const TileReq& r, uint32_t q) {
  return window_begin(p, r.pos0 + static_cast<int>(q * kItemRows / p.G));
}
// The tiles of tokens that the rows of pair `q` see: [x, y).
BFP8_DEV int2 pair_tiles(const AttnParams& p, const TileReq& r, uint32_t q) {
  const uint32_t row0 = q * kItemRows, rows = static_cast<uint32_t>(r.n) * p.G;
  const uint32_t last = min(rows, row0 + kItemRows) - 1;
  const int pos1 = r.pos0 + static_cast<int>(last / p.G);
  const int end = min(pos1 + 1, r.held);
  const int begin = pair_first(p, r, q);
  const int lo = begin / kTileTokens;
  return make_int2(lo, end > begin ? (end + kTileTokens - 1) / kTileTokens : lo);
}

// A block's next piece of work: an item, or a part of its tokens.
struct TileItem {
  int32_t b, h, q0, n, pos0, held;   // b < 0: there is no more
  int32_t row0;                    // first row of the item in its request
  int32_t lo, hi;                  // tiles of tokens
  int32_t first;                   // first token that any of its rows sees
  int32_t begins, ends;            // holds the item's first tile, its last
};

// What the join has to know of a block: its last item, when the block began it and
// others finish it, and whether its first part finishes another's.
struct TileDesc {
  int32_t open, closes, h, row0, q0, n, pos0, pad;
};

// Row `row` of an item.
BFP8_DEV RowAt tile_row(const AttnParams& p, const TileItem& x, int row) {
  RowAt a;
  const uint32_t i = x.row0 + row;
  const uint32_t tok = i / p.G;
  a.real = tok < static_cast<uint32_t>(x.n);
  a.token = x.q0 + static_cast<int64_t>(a.real ? tok : 0);
  a.head = x.h * p.G + (i - tok * p.G);
  a.pos = x.pos0 + static_cast<int>(tok);
  return a;
}

// Three-way maximum, one instruction.
BFP8_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// n FP32 columns of this lane's row of tensor memory times f. Rare, so kept
// small rather than fast.
BFP8_DEV void scale_columns(uint32_t taddr, int n, float f) {
#pragma unroll 1
  for (int i = 0; i < n; i += 16) {
    uint32_t r[16];
    tmem_ld16(taddr + i, r);
#pragma unroll
    for (int c = 0; c < 16; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * f);
    tmem_st16(taddr + i, r);
  }
}

struct TileShared {
  uint64_t k_full[kTileStages], k_empty[kTileStages], v_full[kValueStages], v_empty[kValueStages];
  uint64_t w_full[2], w_empty[2];      // the widened values' buffers
  uint64_t info_full[kInfos];
  uint64_t q_full[2], s_full[2], p_full[2][2], o_done[2][2], drained;   // p_full, o_done: of a tile's halves
  uint64_t item_full[2], item_empty[2];
  // What softmax needs of a tile. One slot more than there are stages: tile m's
  // keys are loaded once S of tile m - 3 is complete for both query tiles, which
  // follows their P of tile m - 4.
  float4 scale[kInfos][8];             // per 16 tokens: 2^ek, ev, 2^-ev
  uint16_t valid[kInfos][8];           // per 16 tokens: a bit for each that exists
  uint32_t tmem;
  uint64_t scan[kTileThreads / 32];
  TileItem item[2];                    // the one in work and the next
  uint64_t start_rel;                  // where the block's range begins: units into its request's
  int start_b;
  int abort_flag;
};

__global__ void __launch_bounds__(kTileThreads, 1)
    kv_attention_tiles_kernel(const __grid_constant__ CUtensorMap tk,
                              const __grid_constant__ CUtensorMap tv, const AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ TileShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = base;                         // [tile][hi, lo]
  const uint32_t sK = base + 4 * kQBytes;
  const uint32_t sV = sK + kTileStages * kKvBytes;
  const uint32_t sW = sV + kValueStages * kKvBytes;  // [buffer][64 columns][token]
  if (tid == 0) {
    for (int s = 0; s < kTileStages; ++s) {
      mbar_init(smem_u32(&sh.k_full[s]), 1);
      mbar_init(smem_u32(&sh.k_empty[s]), 1);
    }
    for (int s = 0; s < kValueStages; ++s) {
      mbar_init(smem_u32(&sh.v_full[s]), 1);
      mbar_init(smem_u32(&sh.v_empty[s]), 2);
    }
    for (int s = 0; s < kInfos; ++s) mbar_init(smem_u32(&sh.info_full[s]), 1);
    mbar_init(smem_u32(&sh.drained), 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_u32(&sh.w_full[w]), 2);
      mbar_init(smem_u32(&sh.w_empty[w]), 1);
      mbar_init(smem_u32(&sh.q_full[w]), 4);
      mbar_init(smem_u32(&sh.s_full[w]), 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_u32(&sh.p_full[w][b]), 4);
        mbar_init(smem_u32(&sh.o_done[w][b]), 1);
      }
      mbar_init(smem_u32(&sh.item_full[w]), 1);
      mbar_init(smem_u32(&sh.item_empty[w]), kTileThreads / 32 - 1);
    }
    sh.abort_flag = 0;
    sh.start_b = 0;
    sh.start_rel = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  // Behind the rows kernel too, which this one needs nothing of: what the calls before
  // it wrote is only sure to be seen by a grid that waits itself.
  pdl_wait();

  // ---- this block's range of units: an item has its tiles and kTilePad
  uint64_t range = 0;
  if (!p.whole_items) {
    uint64_t mine = 0, before = 0;   // this thread's request in the last pass of the scan
    auto scan_pass = [&](int b0) {   // exclusive prefix of one request per thread; returns the total
      TileReq r{};
      if (b0 + tid < p.B) r = tile_req(p, b0 + tid);
      mine = 0;
      for (uint32_t todo = __ballot_sync(0xffffffffu, r.pairs > 0); todo; todo &= todo - 1) {
        const int l = __ffs(todo) - 1;   // the warp counts this lane's request together
        TileReq o;
        o.n = __shfl_sync(0xffffffffu, r.n, l);
        o.pos0 = __shfl_sync(0xffffffffu, r.pos0, l);
        o.held = __shfl_sync(0xffffffffu, r.held, l);
        o.pairs = __shfl_sync(0xffffffffu, r.pairs, l);
        uint64_t sum = 0;
        for (uint32_t q = lane; q < o.pairs; q += 32) {
          const int2 t = pair_tiles(p, o, q);
          sum += t.y - t.x + kTilePad;
        }
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
        if (lane == l) mine = sum * p.H;
      }
      uint64_t inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      __syncthreads();
      if (lane == 31) sh.scan[warp] = inc;
      __syncthreads();
      uint64_t total = 0, off = 0;
#pragma unroll
      for (int w = 0; w < kTileThreads / 32; ++w) {
        if (w == warp) off = total;
        total += sh.scan[w];
      }
      before = off + inc - mine;
      return total;
    };
    uint64_t U = 0;
    for (int b0 = 0; b0 < p.B; b0 += kTileThreads) U += scan_pass(b0);
    const uint64_t want = (U + kTileShare - 1) / kTileShare;
    const uint32_t C = static_cast<uint32_t>(min(want, static_cast<uint64_t>(gridDim.x)));
    const uint64_t g0 = blockIdx.x < C ? range_begin(U, blockIdx.x, C) : 0;
    range = blockIdx.x < C ? range_begin(U, blockIdx.x + 1, C) - g0 : 0;
    uint64_t run = 0;
    for (int b0 = 0; b0 < p.B; b0 += kTileThreads) {
      const uint64_t total = p.B > kTileThreads ? scan_pass(b0) : U;   // one pass: still in registers
      const uint64_t at = run + before;
      if (mine && g0 >= at && g0 < at + mine) sh.start_b = b0 + tid, sh.start_rel = g0 - at;
      run += total;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const volatile int* abort_flag = &sh.abort_flag;
  // Tiles are counted on across the block's items (`tiles`), and so are the rings'
  // stages and the barriers' phases; so are the items (`items`).
  uint32_t tiles = 0, items = 0;

  if (warp < 4) {
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer
      const int page = 1 << p.page_shift;
      const uint32_t box_bytes = page * kHeadDim;
      bool ok = true;
      // where the walk over the items stands: request, pair from its last one, head,
      // units into the item; whole items come in rounds over the blocks instead, in
      // alternating directions, as the heaviest are first
      int b = sh.start_b;
      TileReq r = tile_req(p, b);
      uint32_t back = 0, h = 0, u0 = 0, round = 0;
      uint64_t left = range;
      if (left) {
        uint64_t rel = sh.start_rel;
        for (; back < r.pairs; back += 32) {   // the pair that holds it: 32 at a time
          const int2 t = back + lane < r.pairs ? pair_tiles(p, r, r.pairs - 1 - back - lane) : make_int2(0, 0);
          const uint64_t cost = back + lane < r.pairs ? static_cast<uint64_t>(t.y - t.x + kTilePad) * p.H : 0;
          uint64_t inc = cost;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint64_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
          }
          const uint32_t past = __ballot_sync(0xffffffffu, inc > rel);
          if (past) {
            const int l = __ffs(past) - 1;
            rel -= __shfl_sync(0xffffffffu, inc - cost, l);
            const uint32_t one = static_cast<uint32_t>(__shfl_sync(0xffffffffu, cost, l) / p.H);
            back += l;
            h = static_cast<uint32_t>(rel / one);
            u0 = static_cast<uint32_t>(rel - static_cast<uint64_t>(h) * one);
            break;
          }
          rel -= __shfl_sync(0xffffffffu, inc, 31);
        }
      }
      auto next_item = [&] {
        TileItem x{};
        x.b = -1;
        if (p.whole_items) {
          const uint32_t at = round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
          ++round;
          if (at >= r.pairs * p.H) return x;
          back = at / p.H;
          h = at - back * p.H;
        }
        while (p.whole_items || left) {
          if (!p.whole_items && back >= r.pairs) {   // the next request with items: 32 at a time
            back = 0;
            uint32_t has = 0;
            for (++b; b < p.B; b += 32) {
              has = __ballot_sync(0xffffffffu, b + lane < p.B && tile_req(p, b + lane).pairs > 0);
              if (has) break;
            }
            if (!has) return x;
            b += __ffs(has) - 1;
            r = tile_req(p, b);
          }
          const uint32_t pair = r.pairs - 1 - back;
          const int2 t = pair_tiles(p, r, pair);
          const uint32_t nt = t.y - t.x, begin = u0;
          uint32_t end = nt + kTilePad;
          if (!p.whole_items) {
            end = static_cast<uint32_t>(min(static_cast<uint64_t>(end), u0 + left));
            left -= end - u0;
          }
          x.h = h;
          if (!p.whole_items) {
            u0 = 0;
            if (++h >= static_cast<uint32_t>(p.H)) h = 0, ++back;
          }
          if (begin >= nt && !(nt == 0 && begin == 0)) continue;   // nothing but the padding
          x.b = b;
          x.q0 = r.q0, x.n = r.n, x.pos0 = r.pos0, x.held = r.held;
          x.row0 = pair * kItemRows;
          x.lo = t.x + begin;
          x.hi = t.x + min(end, nt);
          x.first = pair_first(p, r, pair);
          x.begins = begin == 0;
          x.ends = end >= nt;
          return x;
        }
        return x;
      };
      TileDesc desc{};
      while (true) {
        TileItem x = next_item();
        const int slot = items & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_sleep(smem_u32(&sh.item_empty[slot]),
                                                     ((items >> 1) & 1) ^ 1u, abort_flag));
        if (!ok) break;
        if (lane == 0) {
          sh.item[slot] = x;
          mbar_arrive(smem_u32(&sh.item_full[slot]));
        }
        __syncwarp();
        ++items;
        if (x.b < 0) break;
        if (!x.begins && x.ends) desc.closes = 1;
        if (x.begins && !x.ends) {
          desc.open = 1;
          desc.h = x.h, desc.row0 = x.row0, desc.q0 = x.q0, desc.n = x.n, desc.pos0 = x.pos0;
        }
        const int nt = x.hi - x.lo;
        const int32_t* row = p.table + x.b * p.ld_table;
        auto page_id = [&](int j) {   // lane l < 8: the page of tokens 16 l .. of tile j
          const int t = (x.lo + j) * kTileTokens + 16 * lane;
          return j < nt && lane < 8 && t < x.held ? __ldg(row + (t >> p.page_shift)) : -1;
        };
        int32_t id = page_id(0);
        for (int j = 0; j < nt; ++j, ++tiles) {
          const int s = tiles % kTileStages;
          const uint32_t ph = (tiles / kTileStages) & 1;
          const int vs = tiles % kValueStages;
          const uint32_t vph = (tiles / kValueStages) & 1;
          const uint32_t kf = smem_u32(&sh.k_full[s]), vf = smem_u32(&sh.v_full[vs]);
          if (!__all_sync(0xffffffffu,
                          mbar_wait_sleep(smem_u32(&sh.k_empty[s]), ph ^ 1u, abort_flag) &&
                              mbar_wait_sleep(smem_u32(&sh.v_empty[vs]), vph ^ 1u, abort_flag))) {
            ok = false;
            break;
          }
          const int t = (x.lo + j) * kTileTokens + 16 * lane;
          // a page that ends ahead of the first token seen is as good as missing: it may
          // be another request's by now
          const bool there = lane < 8 && id >= 0 && id < p.n_pages && (t | (page - 1)) >= x.first;
          const bool leads = there && (t & (page - 1)) == 0;
          const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, leads));
          if (lane == 0) {
            mbar_expect_tx(kf, boxes * box_bytes);
            mbar_expect_tx(vf, boxes * box_bytes);
          }
          __syncwarp();
          if (leads) {
            const uint32_t at = 16 * lane * kHeadDim;
            tma_load_4d(sK + s * kKvBytes + at, &tk, 0, 0, x.h, id, kf);
            tma_load_4d(sV + vs * kKvBytes + at, &tv, 0, 0, x.h, id, vf);
          }
          int ek = 127, ev = 127;
          if (there) {
            const int64_t at = id * p.exp_page + x.h * p.exp_head;
            ek = __ldg(p.k_exp + at);
            ev = __ldg(p.v_exp + at);
          }
          id = page_id(j + 1);
          if (lane < 8) {
            const int left_here = there ? min(x.held - t, 16) : 0;
            const int unseen = min(max(x.first - t, 0), 16);
            sh.scale[tiles % kInfos][lane] = make_float4(exp2_int(ek - 127), static_cast<float>(ev - 127),
                                                         exp2_int(127 - ev), 0.0f);
            sh.valid[tiles % kInfos][lane] = static_cast<uint16_t>(((1u << left_here) - 1u) & (0xffffu << unseen));
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(kf);
            mbar_arrive(vf);
            mbar_arrive(smem_u32(&sh.info_full[tiles % kInfos]));
          }
        }
        if (!ok) break;
      }
      if (!p.whole_items && lane == 0) p.tile_desc[blockIdx.x] = desc;
      if (!ok) sh.abort_flag = 1;
      // every stage's last load has landed before the block may end
      const int loaded = static_cast<int>(tiles);
      for (int j = max(loaded - kTileStages, 0); j < loaded; ++j)
        drain(smem_u32(&sh.k_full[j % kTileStages]), (j / kTileStages) & 1);
      for (int j = max(loaded - kValueStages, 0); j < loaded; ++j)
        drain(smem_u32(&sh.v_full[j % kValueStages]), (j / kValueStages) & 1);
      if (!ok && lane == 0) atomicExch(&g_kv_err, static_cast<int>(BFP8_ERR_TIMEOUT));
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t kQk[2] = {idesc_e5m2_e4m3(kTileRows, kTileTokens),
                                   idesc_e4m3(kTileRows, kTileTokens)};
      constexpr uint32_t kPv = idesc_f16_bmn(kTileRows, kHeadDim);
      bool ok = true;
      auto wait = [&](uint64_t& bar, uint32_t parity) {
        if (ok && !__all_sync(0xffffffffu, mbar_wait_sleep(smem_u32(&bar), parity, abort_flag))) ok = false;
      };
      auto qk = [&](uint32_t j, int w) {
        const int s = j % kTileStages;
        if (elect_one()) {
          const uint64_t db = smem_desc_sw128(sK + s * kKvBytes);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint64_t da = smem_desc_sw128(sQ + (2 * w + t) * kQBytes);
#pragma unroll
            for (int k = 0; k < 4; ++k)   // 32 columns a step: 32 bytes
              umma_e4m3(tmem + kColS + 128 * w, da + 2 * k, db + 2 * k, kQk[t], t || k);
          }
          umma_commit(smem_u32(&sh.s_full[w]));
          if (w == 1) umma_commit(smem_u32(&sh.k_empty[s]));
        }
        __syncwarp();
      };
      auto pv = [&](uint32_t j, int w, int b, bool add) {   // half b of the tile's tokens
        if (elect_one()) {
          const uint64_t db = smem_desc_sw128_mn(sW + (j & 1) * kV16Bytes + b * kHalf * 128, kKvBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k)   // 16 tokens a step: 16 rows of 128 bytes
            umma_f16_ts(tmem + kColO + 128 * w, tmem + kColS + 128 * w + kHalf * b + 8 * k,
                        db + 128 * k, kPv, add || k);
          umma_commit(smem_u32(&sh.o_done[w][b]));
          if (w == 1 && b == 1) umma_commit(smem_u32(&sh.w_empty[j & 1]));
        }
        __syncwarp();
      };
      for (uint32_t queries = 0; ok; ++items) {
        const int slot = items & 1;
        wait(sh.item_full[slot], (items >> 1) & 1);
        if (!ok || sh.item[slot].b < 0) break;
        const uint32_t nt = sh.item[slot].hi - sh.item[slot].lo;
        if (nt > 0) {
          wait(sh.k_full[tiles % kTileStages], (tiles / kTileStages) & 1);
          for (int w = 0; w < 2; ++w) {
            wait(sh.q_full[w], queries & 1);
            tc_fence_after();
            if (ok) qk(tiles, w);
          }
          ++queries;
        }
        for (uint32_t j = 0; ok && j < nt; ++j, ++tiles) {
          wait(sh.w_full[tiles & 1], (tiles >> 1) & 1);
          for (int w = 0; w < 2; ++w) {
            for (int b = 0; b < 2; ++b) {
              wait(sh.p_full[w][b], tiles & 1);
              if (!ok) break;
              tc_fence_after();
              pv(tiles, w, b, j > 0 || b);
            }
            if (!ok) break;
            if (j + 1 == nt) continue;
            if (w == 0) wait(sh.k_full[(tiles + 1) % kTileStages], ((tiles + 1) / kTileStages) & 1);
            if (!ok) break;
            qk(tiles + 1, w);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.item_empty[slot]));
      }
      if (!ok) {
        sh.abort_flag = 1;
        if (lane == 0) atomicExch(&g_kv_err, static_cast<int>(BFP8_ERR_TIMEOUT));
        // products in flight end before tensor memory is given back
        if (elect_one()) umma_commit(smem_u32(&sh.drained));
        __syncwarp();
        drain(smem_u32(&sh.drained), 0);
      }
    } else {
      // ------------------------------------------- values' codes widened to F16
      // A lane takes 16 columns (chunk c) of a row a step; its 32 bytes go to
      // columns 64 (c / 4) .. of that half's tile. Values of tokens that do not
      // exist become zeros: what lies there may be NaN codes, and a weight of 0
      // does not silence those.
      const int c = lane & 7, r0 = 4 * (warp - 2) + (lane >> 3);
      bool ok = true;
      uint32_t nt = 0;   // tiles left of the item
      for (;; ++tiles, --nt) {
        while (nt == 0) {
          __syncwarp();
          if (items > 0 && lane == 0) mbar_arrive(smem_u32(&sh.item_empty[(items - 1) & 1]));
          const int slot = items & 1;
          ok = __all_sync(0xffffffffu, mbar_wait_sleep(smem_u32(&sh.item_full[slot]),
                                                       (items >> 1) & 1, abort_flag));
          if (!ok || sh.item[slot].b < 0) break;
          nt = sh.item[slot].hi - sh.item[slot].lo;
          ++items;
        }
        if (nt == 0) break;
        const uint32_t j = tiles;
        const int s = j % kValueStages;
        if (!__all_sync(0xffffffffu,
                        mbar_wait_sleep(smem_u32(&sh.w_empty[j & 1]), ((j >> 1) & 1) ^ 1, abort_flag) &&
                            mbar_wait_sleep(smem_u32(&sh.v_full[s]), (j / kValueStages) & 1, abort_flag))) {
          ok = false;
          break;
        }
        const uint32_t src = sV + s * kKvBytes + r0 * kHeadDim;
        const uint32_t dst = sW + (j & 1) * kV16Bytes + (c >> 2) * kKvBytes + r0 * 128;
        const uint16_t* valid = sh.valid[j % kInfos];
        const uint4 vw = *reinterpret_cast<const uint4*>(valid);
        const bool full = (vw.x & vw.y & vw.z & vw.w) == 0xffffffffu;
        // the two halves' lanes store their two chunks in opposite order, which
        // keeps the stores free of bank conflicts; rows 8 apart swizzle alike
        const int first = c >> 2, x = r0 & 7;
        const uint32_t at = src + ((c ^ x) << 4);
        const uint32_t to0 = dst + (((2 * (c & 3) + first) ^ x) << 4);
        const uint32_t to1 = dst + (((2 * (c & 3) + 1 - first) ^ x) << 4);
#pragma unroll 4
        for (int i = 0; i < kTileTokens; i += 8) {
          uint4 v = lds128(at + i * kHeadDim);
          if (!full && !((valid[(i + r0) >> 4] >> ((i + r0) & 15)) & 1u)) v = make_uint4(0u, 0u, 0u, 0u);
          const uint4 lo = make_uint4(f16_pair(v.x, 0), f16_pair(v.x, 1), f16_pair(v.y, 0), f16_pair(v.y, 1));
          const uint4 hi = make_uint4(f16_pair(v.z, 0), f16_pair(v.z, 1), f16_pair(v.w, 0), f16_pair(v.w, 1));
          sts128(to0 + i * 128, first ? hi : lo);
          sts128(to1 + i * 128, first ? lo : hi);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sh.v_empty[s]));
          mbar_arrive(smem_u32(&sh.w_full[j & 1]));
        }
      }
      if (!ok) {
        sh.abort_flag = 1;
        if (lane == 0) atomicExch(&g_kv_err, static_cast<int>(BFP8_ERR_TIMEOUT));
      }
    }
  } else {
    // ------------------------------------------------- softmax, one thread a row
    const int w = (warp >> 2) - 1;                 // query tile
    const int r = tid & 127;                       // row of the tile = TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp & 3) << 21);   // lane 32 (warp mod 4)
    const uint32_t o_col = lane_base + kColO + 128 * w;
    const uint32_t stage = sW + 2 * kV16Bytes + (warp - 4) * kOutStage;
    bool ok = true, open = false;
    float M = 0.0f, Z = 0.0f;
    // where the open item's row goes: elements into out and lse, or a partial sum's slot
    int64_t out_at = -1, lse_at = -1;
    int part = -1;
    bool any = false;    // the item had tiles
    // Each round makes the queries of the next item, so that its first products can
    // run, writes out the item before it, and then works through the next one.
    while (true) {
      const int slot = items & 1;
      ok = __all_sync(0xffffffffu, mbar_wait_sleep(smem_u32(&sh.item_full[slot]), (items >> 1) & 1, abort_flag));
      if (!ok) break;
      const TileItem& x = sh.item[slot];
      const bool more = x.b >= 0;
      const int nt = more ? x.hi - x.lo : 0;
      float fac = 0.0f;
      RowAt at{};
      if (more) at = tile_row(p, x, w * kTileRows + r);
      if (nt > 0) {
        // The queries as two FP8 terms. The BF16 rows are copied to where the terms go
        // (the first 64 columns of a row to its row of hi, the others to that of lo)
        // and replaced row by row, a half-warp each: all of them are in flight at once,
        // and the loop stays small, for instructions that are not in the cache cost
        // more than the arithmetic (unrolled 16 times: 13,000 clocks; this: 6,000, and
        // 4,000 of them the terms).
        // The lane that owns a row keeps its factor. A negative softmax scale turns the
        // queries round, so that the factor is positive.
        const int64_t mine = at.real ? at.token * p.q_ldt + at.head * p.q_ldh : -1;
        const int half = lane >> 4, c = lane & 15;
        const uint32_t rows_at = sQ + 2 * w * kQBytes + 32 * (warp & 3) * kHeadDim;
#pragma unroll 4
        for (int i = half; i < 32; i += 2) {
          const int64_t off = __shfl_sync(0xffffffffu, mine, i);
          const __nv_bfloat16* src = p.q + (off >= 0 ? off : 0) + 8 * c;
          cp_async16_zfill(rows_at + (c >> 3) * kQBytes + i * kHeadDim + (((c & 7) ^ (i & 7)) << 4), src, off >= 0);
        }
        cp_async_wait_all();
#pragma unroll 1
        for (int i0 = 0; i0 < 32; i0 += 2 * kQueryPairs) {
          uint4 v[kQueryPairs];
          int e[kQueryPairs][2];
#pragma unroll
          for (int k = 0; k < kQueryPairs; ++k) {
            const int i = i0 + 2 * k + half;
            v[k] = lds128(rows_at + (c >> 3) * kQBytes + i * kHeadDim + (((c & 7) ^ (i & 7)) << 4));
          }
#pragma unroll
          for (int k = 0; k < kQueryPairs; ++k) {
            uint32_t m = max_abs_bf16x2(max_abs_bf16x2(v[k].x, v[k].y), max_abs_bf16x2(v[k].z, v[k].w));
            m = max(m & 0xFFFFu, m >> 16);
            e[k][0] = query_exponent(__reduce_max_sync(0xffffffffu, half ? 0u : m));
            e[k][1] = query_exponent(__reduce_max_sync(0xffffffffu, half ? m : 0u));
          }
#pragma unroll
          for (int k = 0; k < kQueryPairs; ++k) {
            const int i = i0 + 2 * k + half;
            if ((lane & ~1) == i0 + 2 * k) fac = exp2_int(-(lane & 1 ? e[k][1] : e[k][0])) * fabsf(p.scale_log2);
            const float up = copysignf(exp2_int(half ? e[k][1] : e[k][0]), p.scale_log2);
            uint2 hi, lo;
            query_terms(v[k].x, v[k].y, up, hi.x, lo.x);
            query_terms(v[k].z, v[k].w, up, hi.y, lo.y);
            const uint32_t to = rows_at + i * kHeadDim + (((c >> 1) ^ (i & 7)) << 4) + 8 * (c & 1);
            sts64(to, hi);   // every lane has its row's 16 bytes: the maximum needed them
            sts64(to + kQBytes, lo);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.q_full[w]));
      }
      if (open) {
        if (any) {
          ok = __all_sync(0xffffffffu, mbar_wait_sleep(smem_u32(&sh.o_done[w][1]), (tiles - 1) & 1, abort_flag));
          if (!ok) break;
          tc_fence_after();
        }
        float* dst = p.tile_partial + (2 * static_cast<int64_t>(blockIdx.x) + part) * kTilePartialFloats;
        const int row = w * kTileRows + r;
        if (part >= 0) {
          dst[kItemRows * kHeadDim + row] = M;
          dst[kItemRows * kHeadDim + kItemRows + row] = Z;
        } else if (lse_at >= 0) {
          p.lse[lse_at] = row_lse(M, Z);
        }
        const float f = row_factor(Z);
#pragma unroll 1
        for (int c = 0; c < kHeadDim; c += 32) {
          float o[32];
          if (any) {
            tmem_ld32(o_col + c, o);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0.0f;
          }
          if (part >= 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              reinterpret_cast<float4*>(dst)[(c / 4 + k) * kItemRows + row] =
                  make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          } else {
            // through 2 KB of the warp's own, so that four lanes store a row's 64 bytes;
            // chunk k of row r is kept at k ^ (r / 2 % 4)
            uint32_t p2[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) p2[k] = pack_bf16x2(o[2 * k] * f, o[2 * k + 1] * f);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              sts128(stage + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4),
                     make_uint4(p2[4 * k], p2[4 * k + 1], p2[4 * k + 2], p2[4 * k + 3]));
            __syncwarp();
            const int k = lane & 3;
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              const int from = i + (lane >> 2);
              const int64_t off = __shfl_sync(0xffffffffu, out_at, from);
              const uint4 v = lds128(stage + from * 64 + ((k ^ ((from >> 1) & 3)) << 4));
              if (off >= 0) *(reinterpret_cast<uint4*>(p.out + off + c) + k) = v;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.item_empty[slot ^ 1]));
      }
      if (!more) break;
      open = true;
      any = nt > 0;
      part = x.begins && x.ends ? -1 : x.begins ? 1 : 0;
      out_at = at.real ? at.token * p.o_ldt + at.head * p.o_ldh : -1;
      lse_at = at.real && p.lse ? at.token * p.l_ldt + at.head : -1;

      // the positions that the row sees; rows that do not exist never ask for a
      // mask, and what they compute is not stored
      const int first = at.real ? window_begin(p, at.pos) : 0;
      const int last = at.real ? at.pos : 0x7FFFFFFE;
      const int last_warp = __reduce_min_sync(0xffffffffu, last);
      const int first_warp = __reduce_max_sync(0xffffffffu, first);

      M = kNoMax;   // weights of scores of -inf are 0
      Z = 0.0f;
      // The loop is kept short: unrolled over 128 tokens, softmax ran at half the
      // speed, out of instructions.
#pragma unroll 1
      for (int u = 0; u < 2 * nt; ++u) {
        const int b = u & 1, t0 = (x.lo + (u >> 1)) * kTileTokens + kHalf * b;
        const uint32_t j = tiles + (u >> 1);
        const uint32_t s_col = lane_base + kColS + 128 * w + kHalf * b;
        if (b == 0) {
          ok = __all_sync(0xffffffffu,
                          mbar_wait_sleep(smem_u32(&sh.info_full[j % kInfos]), (j / kInfos) & 1, abort_flag) &&
                              mbar_wait_sleep(smem_u32(&sh.s_full[w]), j & 1, abort_flag));
          if (!ok) break;
          tc_fence_after();
        }
        uint32_t y[64];
        tmem_ld64_bits(s_col, y);
        float4 info[4];   // 2^ek, ev, 2^-ev per 16 tokens
#pragma unroll
        for (int g = 0; g < 4; ++g) info[g] = sh.scale[j % kInfos][4 * b + g];
        const uint2 vw = *reinterpret_cast<const uint2*>(&sh.valid[j % kInfos][4 * b]);
        if ((vw.x & vw.y) != 0xffffffffu || t0 + kHalf - 1 > last_warp || t0 < first_warp) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = t0 + 32 * k;
            const int hi = min(max(last + 1 - t, 0), 32), lo = min(max(first - t, 0), 32);
            const uint32_t below = hi == 32 ? 0xffffffffu : (1u << hi) - 1u;
            const uint32_t under = lo == 32 ? 0xffffffffu : (1u << lo) - 1u;
            const uint32_t see = (k ? vw.y : vw.x) & below & ~under;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((see >> c) & 1u)) y[32 * k + c] = 0xFF800000u;   // -inf
          }
        }
        // the maximum of x = y * fac * 2^ek + ev
        float ck[4], top = kNegInf;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          ck[g] = fmaxf(fac * info[g].x, 1e-37f);
          auto v = [&](int c) { return __uint_as_float(y[16 * g + c]); };
          const float m0 = max3(max3(v(0), v(1), v(2)), v(3), v(4));
          const float m1 = max3(max3(v(5), v(6), v(7)), v(8), v(9));
          const float m2 = max3(max3(v(10), v(11), v(12)), v(13), max3(v(14), v(15), m0));
          top = fmaxf(top, fmaf(fmaxf(m1, m2), ck[g], info[g].y));
        }
        const bool grow = top - M > kReach;
        const bool big = fabsf(top) >= kBigScore && top > kNegInf;
        if (__any_sync(0xffffffffu, grow || big)) {   // rare but for the first tokens
          const float to = top - kPBase, f = grow ? ex2_approx(M - to) : 1.0f;
          if (grow) M = to;
          Z *= f;
          if (big) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
#pragma unroll
              for (int c = 16 * g; c < 16 * g + 16; c += 2) {
                const float2 x2 = __ffma2_rn(make_float2(__uint_as_float(y[c]), __uint_as_float(y[c + 1])),
                                             make_float2(ck[g], ck[g]), make_float2(info[g].y, info[g].y));
                y[c] = __float_as_uint(x2.x), y[c + 1] = __float_as_uint(x2.y);
              }
              ck[g] = 1.0f;
              info[g].y = 0.0f;
            }
          }
          if (u > 0) {
            // the product before this one: the half ahead, or the last of the tile ahead
            ok = __all_sync(0xffffffffu, mbar_wait_sleep(smem_u32(&sh.o_done[w][b ^ 1]), (j - 1 + b) & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
            scale_columns(o_col, kHeadDim, f);
          }
        }
        uint32_t pw[32];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float cb = info[g].y - M;
          const float2 ck2 = make_float2(ck[g], ck[g]), cb2 = make_float2(cb, cb);
          float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float2 x2 = __ffma2_rn(make_float2(__uint_as_float(y[16 * g + 2 * c]),
                                                     __uint_as_float(y[16 * g + 2 * c + 1])), ck2, cb2);
            const float2 e = make_float2(ex2_approx(x2.x), ex2_approx(x2.y));
            sum = __fadd2_rn(sum, e);
            pw[8 * g + c] = pack_f16x2(e.x, e.y);
          }
          Z = fmaf(sum.x + sum.y, info[g].z, Z);
        }
        tmem_st32(s_col, pw);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[w][b]));
      }
      if (!ok) break;
      tiles += nt;
      ++items;
    }
    if (!ok) {
      sh.abort_flag = 1;
      if (lane == 0) atomicExch(&g_kv_err, static_cast<int>(BFP8_ERR_TIMEOUT));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partial sums of segments and items that several blocks shared, in
// block order, and writes the rows of segments that had no unit at all. The
// first `seg_blocks` blocks take a segment each (one that one block finished
// is done), then come 16 blocks for each block of the tiles kernel: the item
// that it began and others finished, 128 rows and 16 columns each.
__global__ void __launch_bounds__(128) kv_attention_join_kernel(const AttnParams p, uint32_t grid,
                                                                uint32_t max_rb, uint32_t seg_blocks) {
  pdl_wait();
  // Sums so far at maximum m. Every part's numbers are loaded before the maximum is
  // known, so that parts' loads overlap.
  float m = kNoMax, z = 0.0f, v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  auto add = [&](float mc, float zc, const float4 (&x)[4]) {
    const float top = fmaxf(m, mc), a = ex2_approx(m - top), f = ex2_approx(mc - top);
    m = top;
    z = fmaf(zc, f, z * a);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[4 * e] = fmaf(x[e].x, f, v[4 * e] * a);
      v[4 * e + 1] = fmaf(x[e].y, f, v[4 * e + 1] * a);
      v[4 * e + 2] = fmaf(x[e].z, f, v[4 * e + 2] * a);
      v[4 * e + 3] = fmaf(x[e].w, f, v[4 * e + 3] * a);
    }
  };
  if (blockIdx.x >= seg_blocks) {
    const uint32_t i = blockIdx.x - seg_blocks, c0 = i >> 4;
    const int row = 128 * (i & 1) + threadIdx.x, c = 16 * ((i & 15) >> 1);
    const TileDesc d = p.tile_desc[c0];
    if (!d.open) return;
    const uint32_t blocks = (gridDim.x - seg_blocks) / 16;
    TileItem x{};
    x.h = d.h, x.row0 = d.row0, x.q0 = d.q0, x.n = d.n, x.pos0 = d.pos0;
    const RowAt at = tile_row(p, x, row);
    if (!at.real) return;
    for (uint32_t k = c0;; ++k) {   // to the block that finished it
      const float* part = p.tile_partial + static_cast<int64_t>(2 * k + (k == c0)) * kTilePartialFloats;
      float4 o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = reinterpret_cast<const float4*>(part)[(c / 4 + e) * kItemRows + row];
      const bool last = k + 1 >= blocks || (k > c0 && p.tile_desc[k].closes);
      add(part[kItemRows * kHeadDim + row], part[kItemRows * kHeadDim + kItemRows + row], o);
      if (last) break;
    }
    store_row16(p.out + at.token * p.o_ldt + at.head * p.o_ldh + c, v, row_factor(z));
    if (p.lse && c == 0) p.lse[at.token * p.l_ldt + at.head] = row_lse(m, z);
    return;
  }
  const uint32_t per_b = max_rb * p.H;
  const int b = blockIdx.x / per_b;
  const uint32_t rest = blockIdx.x - b * per_b;
  const uint32_t h = rest / max_rb, rb = rest - h * max_rb;
  const uint64_t U = p.schedule[p.B], unit0 = p.schedule[b];
  const ReqUnits r = req_units(p, b);
  if (rb >= r.nrb || static_cast<int64_t>(r.n) * p.G > p.few_rows) return;
  const uint32_t seg = h * r.nrb + rb;
  // partial sums: `count` of them, M and Z behind the rows. The segment begins
  // inside the first block's range (its second slot) and before the others'
  // (their first slot).
  const float* first = nullptr;
  uint32_t count = 0;
  if (r.nt) {
    const uint64_t a = unit0 + static_cast<uint64_t>(seg) * r.cost(), e = a + r.nt;
    const uint32_t C = used_blocks(U, grid);
    const uint32_t c0 = owner_of(a, U, C), c1 = owner_of(e - 1, U, C);
    if (c0 == c1) return;
    first = p.partial + static_cast<int64_t>(2 * c0 + 1) * kPartialFloats;
    count = c1 - c0 + 1;
  }
  const int row = threadIdx.x >> 3, ch = threadIdx.x & 7;   // 16 columns of a row per thread
  if (row >= p.seg_rows) return;
  const RowAt at = row_at(p, r, h, rb, row);
  if (!at.real) return;
  const int64_t m_at = static_cast<int64_t>(p.seg_rows) * kHeadDim + row;
#pragma unroll 4
  for (uint32_t c = 0; c < count; ++c) {
    const float* part = first + (2 * c - (c ? 1 : 0)) * static_cast<int64_t>(kPartialFloats);
    float4 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = *reinterpret_cast<const float4*>(part + row * kHeadDim + 16 * ch + 4 * e);
    add(part[m_at], part[m_at + p.seg_rows], x);
  }
  store_row16(p.out + at.token * p.o_ldt + at.head * p.o_ldh + 16 * ch, v, row_factor(z));
  if (p.lse && ch == 0) p.lse[at.token * p.l_ldt + at.head] = row_lse(m, z);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Requests whose rows of a KV head (new tokens times the group) are at most
// this many go to the rows kernel, which goes over their tokens once for every 16
// (from L2 but for the first). A call from cold caches, 64 heads on 8, all requests
// there against all in the tiles kernel, in us:
//   8 tokens (64 rows) of 4, 16, 64 requests behind 8000: 87, 302, 1133 against 52, 124, 406
//   5 tokens (40 rows) of 32 behind 300, 2000, 16000: 51, 139, 841 against 51, 90, 395
//   the same of 1 and of 2 behind 2000: 25 and 27 against 29 and 34
//   4 tokens (32 rows) of 32 behind 300, 2000, 16000: 41, 103, 570 against 51, 88, 395
//   the same of 1, 2 and 8 behind 2000: 25, 26 and 40 against 29, 34 and 41
// Above 32 rows the tiles kernel is up to 2.8 times as fast, and slower by less than 10
// us on one or two requests; below, it gains 1.4 times at most, on long caches only.
constexpr int32_t kFewRows = 32;

// What the host knows of a call's shape, from upper bounds alone: max_q is the most
// rows of a request, and no more than T.
struct Shape {
  bool tiles;   // some request may have more than kFewRows rows
  bool whole;   // the tiles kernel's blocks take whole items
};
Shape shape_of(int64_t B, int64_t max_q, int64_t G, int64_t H, int sms) {
  Shape s{};
  s.tiles = max_q * G > kFewRows;
  s.whole = s.tiles && B == 1 && (max_q * G + kItemRows - 1) / kItemRows * H >= 4 * sms;
  return s;
}

struct Workspace {
  size_t partial, tile_desc, tile_partial, bytes;   // offsets; the schedule is at 0
};
Workspace workspace_of(int64_t B, const Shape& s, int sms) {
  Workspace w{};
  w.partial = align256((B + 1) * 8);
  w.tile_desc = w.partial + align256(static_cast<size_t>(sms) * kRowsPerSm * 2 * kPartialFloats * 4);
  w.tile_partial = w.tile_desc + align256(sms * sizeof(TileDesc));
  w.bytes = w.tile_partial;
  // whole items need none of these, but a workspace that holds a long prompt has to
  // hold its shorter chunks too
  if (s.tiles) w.bytes += static_cast<size_t>(sms) * 2 * kTilePartialFloats * 4;
  return w;
}

}  // namespace

// What a call needs falls as its KV heads rise, for their groups shrink. The size that
// users ask for is one KV head's, so that it grows with every argument and one
// workspace serves layers of other head counts too.
size_t kv_attention_workspace_bytes(int64_t B, int64_t T, int64_t max_q, int64_t Hq, int sms) {
  return workspace_of(B, shape_of(B, std::min(max_q, T), Hq, 1, sms), sms).bytes;
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
      a.max_blocks > 0x7FFFFFFF || a.tokens > 0x7FFFFFFF / a.n_heads)
    return BFP8_ERR_UNSUPPORTED;
  rc = check_device_ptrs({a.q_bf16, a.out_bf16, a.lse, a.q_offsets, a.kv_len, a.block_table,
                          c.k_e4m3, c.v_e4m3, c.k_exp, c.v_exp, a.workspace});
  if (rc != BFP8_OK) return rc;
  int sms = 0;
  rc = sm_count(&sms);
  if (rc != BFP8_OK) return rc;
  const int64_t max_q = std::min(a.max_q_len, a.tokens);
  const Shape shape = shape_of(a.batch, max_q, a.n_heads / H, H, sms);
  const Workspace ws = workspace_of(a.batch, shape, sms);
  if (!a.workspace || a.ws_bytes < ws.bytes || reinterpret_cast<uintptr_t>(a.workspace) % 256)
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
  uint8_t* scratch = static_cast<uint8_t*>(a.workspace);
  p.schedule = reinterpret_cast<uint64_t*>(scratch);
  p.partial = reinterpret_cast<float*>(scratch + ws.partial);
  p.tile_desc = reinterpret_cast<TileDesc*>(scratch + ws.tile_desc);
  p.tile_partial = reinterpret_cast<float*>(scratch + ws.tile_partial);
  p.q_ldt = a.q_stride_token;
  p.q_ldh = a.q_stride_head;
  p.o_ldt = a.out_stride_token;
  p.o_ldh = a.out_stride_head;
  p.l_ldt = a.lse_stride_token;
  p.ld_table = a.ld_table;
  p.exp_page = c.exp_stride_page;
  p.exp_head = c.exp_stride_head;
  p.T = a.tokens;
  p.max_q = static_cast<int32_t>(max_q);
  p.n_pages = c.n_pages;
  p.B = static_cast<int32_t>(a.batch);
  p.H = c.n_kv_heads;
  p.G = static_cast<int32_t>(a.n_heads / H);
  p.page_shift = kv_page_shift(c.page_size);
  p.max_blocks = static_cast<int32_t>(a.max_blocks);
  p.window = a.window < 0 ? -1 : a.window;
  p.scale_log2 = a.softmax_scale * kLog2e;
  p.whole_items = shape.whole;
  p.tiles_follow = shape.tiles && a.batch > 1;
  // one request has only one kernel to go to; of several, each is looked at on the device
  p.few_rows = !shape.tiles ? 0x7FFFFFFF : a.batch > 1 ? kFewRows : 0;
  const int64_t most_rows = max_q * p.G;
  // what goes to the rows kernel next to prompts is single tokens for the most part
  // (6, 24 and 64 requests of up to 900 new tokens behind up to 6000, groups of 8: 54, 151
  // and 545 us with 8 rows, 60, 163 and 556 with 16; groups of 4: 45, 103, 321 and 50,
  // 116, 333; of 5: 47, 120, 383 and 53, 131, 394)
  p.seg_rows = most_rows <= 8 || (shape.tiles && p.G <= 8) ? 8 : kMaxRows;
  const int64_t max_rb = (most_rows + p.seg_rows - 1) / p.seg_rows;
  const int64_t few_rb = kFewRows / p.seg_rows;
  const bool rows_kernel = p.few_rows > 0, join_items = shape.tiles && !shape.whole;
  const int64_t join_rb = shape.tiles && max_rb > few_rb ? few_rb : max_rb;
  const int64_t segs = rows_kernel ? a.batch * H * join_rb : 0, joins = segs + (join_items ? 16 * sms : 0);
  if (joins > 0x7FFFFFFF) return BFP8_ERR_UNSUPPORTED;
  auto maps = [&](uint32_t rows, CUtensorMap* tk, CUtensorMap* tv) {
    const int r = make_tmap_4d(tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.k_e4m3, kHeadDim, c.page_size, H,
                               c.n_pages, c.k_stride_token, c.k_stride_head, c.k_stride_page,
                               kHeadDim, rows, 1, 1, CU_TENSOR_MAP_SWIZZLE_128B);
    if (r != BFP8_OK) return r;
    return make_tmap_4d(tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.v_e4m3, kHeadDim, c.page_size, H,
                        c.n_pages, c.v_stride_token, c.v_stride_head, c.v_stride_page, kHeadDim,
                        rows, 1, 1, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap tk, tv;
  const unsigned rows_grid = static_cast<unsigned>(sms) * kRowsPerSm;
  if (rows_kernel) {
    rc = maps(c.page_size < kUnit ? c.page_size : kUnit, &tk, &tv);
    if (rc != BFP8_OK) return rc;
    auto kernel = p.seg_rows == 8 ? kv_attention_rows_kernel<1> : kv_attention_rows_kernel<2>;
    rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), kRowsSmem);
    if (rc != BFP8_OK) return rc;
    rc = launch_dependent(kernel, rows_grid, kThreads, kRowsSmem, st, tk, tv, p);
    if (rc != BFP8_OK) return rc;
  }
  if (shape.tiles) {
    rc = maps(c.page_size, &tk, &tv);
    if (rc != BFP8_OK) return rc;
    rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kv_attention_tiles_kernel), kTileSmem);
    if (rc != BFP8_OK) return rc;
    rc = launch_dependent(kv_attention_tiles_kernel, static_cast<unsigned>(sms), kTileThreads,
                          kTileSmem, st, tk, tv, p);
    if (rc != BFP8_OK) return rc;
  }
  if (joins) {
    rc = launch_dependent(kv_attention_join_kernel, static_cast<unsigned>(joins), 128, 0, st, p,
                          rows_grid, static_cast<uint32_t>(join_rb), static_cast<uint32_t>(segs));
    if (rc != BFP8_OK) return rc;
  }
  return BFP8_OK;
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
