// kv_cache.cu -- the two steps that keep a paged 8-bit KV cache:
//   * the block plan of one step: new pages taken from a free list, the block
//     tables extended, and every new token's slot, position and offsets, from
//     the requests' lengths alone;
//   * the append: new keys and values quantized into their pages with one
//     power-of-two scale per page and head.
#include "attention_layer.cuh"
#include "kv_common.cuh"

#include <algorithm>

namespace bfp8 {
namespace {

using namespace dev;

// ------------------------------------------------------------------ block plan
constexpr int kPlanThreads = 512;
constexpr int64_t kPlanMaxBatch = 16384;   // two uint32 prefixes per request in shared memory
constexpr uint32_t kMaxCount = 0x7FFFFFFFu;

struct PlanParams {
  const int32_t* ctx;
  const int32_t* q_len;
  const int32_t* free_pages;
  int32_t* table;
  int32_t* q_offsets;
  int32_t* kv_len;
  int64_t* slots;
  int32_t* positions;
  int32_t* counts;
  int64_t ld_table, n_free, T;
  int32_t B, max_blocks, shift;
};

// Sums of lengths stay in [0, 2^31): two such values cannot wrap a uint32.
BFP8_DEV uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kMaxCount); }

// Exclusive prefixes of one value pair per thread over the block, plus the
// block's totals. Saturating addition of non-negative numbers is associative,
// so any order of the scan gives the same prefixes.
BFP8_DEV void block_scan2(uint32_t a, uint32_t b, uint32_t (*part)[2], uint32_t& ea, uint32_t& eb,
                          uint32_t& ta, uint32_t& tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t ua = __shfl_up_sync(0xffffffffu, ia, o), ub = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) ia = sat_add(ia, ua), ib = sat_add(ib, ub);
  }
  __syncthreads();   // the previous scan's totals have been read
  if (lane == 31) part[warp][0] = ia, part[warp][1] = ib;
  __syncthreads();
  uint32_t wa = 0, wb = 0;
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w == warp) wa = ta, wb = tb;
    ta = sat_add(ta, part[w][0]);
    tb = sat_add(tb, part[w][1]);
  }
  const uint32_t pa = __shfl_up_sync(0xffffffffu, ia, 1), pb = __shfl_up_sync(0xffffffffu, ib, 1);
  ea = lane ? sat_add(wa, pa) : wa;
  eb = lane ? sat_add(wb, pb) : wb;
}

// Largest b in [0, n) with pre[b] <= v; pre is non-decreasing and pre[0] == 0.
BFP8_DEV int find_owner(const uint32_t* pre, int n, uint32_t v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

struct Request {
  uint32_t ctx, q, before, after;   // lengths; pages held before and needed after
};
BFP8_DEV Request load_request(const PlanParams& p, int b) {
  Request r;
  r.ctx = static_cast<uint32_t>(max(__ldg(p.ctx + b), 0));
  r.q = min(static_cast<uint32_t>(max(__ldg(p.q_len + b), 0)), kMaxCount - r.ctx);
  const uint32_t round = (1u << p.shift) - 1u, cap = static_cast<uint32_t>(p.max_blocks);
  r.before = min((r.ctx + round) >> p.shift, cap);
  r.after = r.q ? min((r.ctx + r.q + round) >> p.shift, cap) : r.before;
  return r;
}

// Every block scans all requests' lengths (a few thousand integers, read from
// L2), keeps the prefixes in shared memory and takes its share of the tokens
// and of the new pages; owners are found by binary search. No block waits for
// another: a new page's number comes from the free list by its rank, not from
// the table that some other block is writing.
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanParams p) {
  extern __shared__ uint32_t pre[];   // [B] tokens before request b, then [B] pages before it
  __shared__ uint32_t part[kPlanThreads / 32][2];
  __shared__ uint32_t lost[kPlanThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  uint32_t* pre_tok = pre;
  uint32_t* pre_page = pre + p.B;
  // the first block writes the requests' offsets and lengths, the last one counts the
  // tokens that have no page
  const bool first = blockIdx.x == 0, counts = blockIdx.x + 1 == gridDim.x;
  uint32_t tok = 0, page = 0, missing = 0;
  if (counts) {
    // tokens that continue a page which is not there; no block writes its entry, and
    // several requests' loads are in flight at once
#pragma unroll 4
    for (int b = threadIdx.x; b < p.B; b += kPlanThreads) {
      const Request r = load_request(p, b);
      const uint32_t used = r.ctx & ((1u << p.shift) - 1u), held = r.ctx >> p.shift;
      const bool continues = r.q && used && held < r.before;
      const int32_t pg = continues ? p.table[b * p.ld_table + held] : 0;
      if (pg < 0) missing = sat_add(missing, min(r.q, (1u << p.shift) - used));
    }
  }
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    Request r{};
    if (b < p.B) r = load_request(p, b);
    uint32_t et, ep, tt, tp;
    block_scan2(r.q, r.after - r.before, part, et, ep, tt, tp);
    if (b < p.B) {
      pre_tok[b] = sat_add(tok, et);
      pre_page[b] = sat_add(page, ep);
      if (first) {
        p.q_offsets[b] = static_cast<int32_t>(pre_tok[b]);
        p.kv_len[b] = static_cast<int32_t>(r.ctx + r.q);
      }
      if (counts) {
        // tokens from the first block on that has no page: past the table's
        // width, or past the end of the free list
        const uint64_t have = p.n_free > pre_page[b] ? p.n_free - pre_page[b] : 0;
        const uint64_t blocks = min(static_cast<uint64_t>(r.after), r.before + have);
        const uint64_t place = max(blocks << p.shift, static_cast<uint64_t>(r.ctx));
        const uint64_t end = static_cast<uint64_t>(r.ctx) + r.q;
        if (end > place) missing = sat_add(missing, static_cast<uint32_t>(end - place));
      }
    }
    tok = sat_add(tok, tt);
    page = sat_add(page, tp);
  }
  __syncthreads();
  if (first && threadIdx.x == 0) {
    p.q_offsets[p.B] = static_cast<int32_t>(tok);
    const uint32_t have = static_cast<uint32_t>(min(p.n_free, static_cast<int64_t>(kMaxCount)));
    p.counts[0] = static_cast<int32_t>(min(page, have));
    p.counts[1] = static_cast<int32_t>(page - min(page, have));
  }
  if (counts) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      missing = sat_add(missing, __shfl_xor_sync(0xffffffffu, missing, o));
    if ((threadIdx.x & 31) == 0) lost[threadIdx.x >> 5] = missing;
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t m = 0;
      for (int w = 0; w < kPlanThreads / 32; ++w) m = sat_add(m, lost[w]);
      p.counts[2] = static_cast<int32_t>(m);
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
  const uint32_t in_page = (1u << p.shift) - 1u;
  for (int64_t t = at; t < p.T; t += step) {
    int64_t slot = -1;
    int32_t pos = -1;
    if (t < tok) {
      const int b = find_owner(pre_tok, p.B, static_cast<uint32_t>(t));
      const Request r = load_request(p, b);
      const uint32_t x = r.ctx + (static_cast<uint32_t>(t) - pre_tok[b]);
      const uint32_t blk = x >> p.shift;
      pos = static_cast<int32_t>(x);
      int32_t pg = -1;
      if (blk < r.before) {
        pg = p.table[b * p.ld_table + blk];   // the page it continues: no block writes this entry
      } else if (blk < r.after) {
        const int64_t i = static_cast<int64_t>(pre_page[b]) + (blk - r.before);
        if (i < p.n_free) pg = __ldg(p.free_pages + i);
      }
      if (pg >= 0) slot = (static_cast<int64_t>(pg) << p.shift) + (x & in_page);
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
  for (int64_t i = at; i < page; i += step) {
    const int b = find_owner(pre_page, p.B, static_cast<uint32_t>(i));
    const Request r = load_request(p, b);
    p.table[b * p.ld_table + r.before + (i - pre_page[b])] =
        i < p.n_free ? __ldg(p.free_pages + i) : -1;
  }
}

// ------------------------------------------------------------------ append
struct AppendParams {
  const __nv_bfloat16* x[2];   // keys, values: [T, heads, 128]
  int64_t ldt[2], ldh[2];      // their token and head strides, in elements
  uint8_t* codes[2];
  uint8_t* exps[2];
  int64_t sp[2], sh[2], st[2];   // page, head and token strides of the codes, in bytes
  int64_t ep, eh;                // page and head strides of the scale bytes
  const int64_t* slots;
  int64_t T, n_slots;
  int32_t heads, window;
};

constexpr int kRowsInRegs = 16;   // rows of a run that a warp holds between its two passes

// Largest |x| so far per half, as BF16 bits; a NaN counts as nothing (max takes
// the other operand, and m is never one).
BFP8_DEV uint32_t amax8(const uint4& r, uint32_t m) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[j] & 0x7FFF7FFFu));
  return m;
}

BFP8_DEV uint2 quant8(const uint4& r, float inv) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
    const float2 x = __fmul2_rn(v, make_float2(inv, inv));
    c[j] = f32x2_to_e4m3x2(x.x, x.y);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Eight codes times a power of two, rounded again where they leave the normal
// range (exact above it).
BFP8_DEV uint2 rescale8(const uint2& v, float f) {
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = j < 2 ? v.x : v.y;
    const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(w >> (16 * (j & 1))));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    o[j] = f32x2_to_e4m3x2(x.x * f, x.y * f);
  }
  return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

// A team of WARPS warps owns one (window of tokens, head, K or V) and quantizes
// every run that begins in its window: a run is the consecutive rows that fill
// consecutive slots of one page, so one team sees all new tokens of a page and
// head, and the page's scale needs no atomics. A half-warp holds a row (8
// elements a lane), a load covers two rows.
//
// WARPS = 1 (four teams a block) is for calls whose every (token, head) can have
// a warp, such as a decode step's, whose runs are one row each: bound by latency.
// Otherwise a team has a warp for every 16 rows of a page, so that a page's rows
// are read once and stay in registers until its scale is known: bound by HBM on
// prompts. Runs short enough for one warp are dealt out to the team's in turn.
// 16,000 prompt tokens of 8 heads (99 MB moved): 20 us, 4.8 TB/s, where one warp
// for every run took 27; a decode step of 128 tokens: 4.4 us.
template <int PAGE, int WARPS>
__global__ void __launch_bounds__(WARPS == 1 ? 128 : 32 * WARPS)
    kv_append_kernel(const AppendParams p) {
  constexpr int kTeams = WARPS == 1 ? 4 : 1;
  __shared__ uint32_t team_max[2][WARPS];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = WARPS == 1 ? 0 : threadIdx.x >> 5;
  const int sub = lane >> 4, chunk = lane & 15;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kTeams + (WARPS == 1 ? threadIdx.x >> 5 : 0);
  const int64_t win = id / (2 * p.heads);
  const int rest = static_cast<int>(id - win * (2 * p.heads));
  const int head = rest >> 1, kv = rest & 1;
  const int64_t t_end = min((win + 1) * p.window, p.T);
  const __nv_bfloat16* x = p.x[kv] + head * p.ldh[kv] + 8 * chunk;
  const int64_t ldt = p.ldt[kv];
  int turn = 0, buf = 0;
  for (int64_t t = win * p.window; t < t_end;) {
    // the run's slots, as far as a page goes, and the one before it, in one round of loads
    int64_t next[(PAGE + 31) / 32];
#pragma unroll
    for (int c = 0; c < PAGE; c += 32)
      next[c / 32] = t + c + lane < p.T ? __ldg(p.slots + t + c + lane) : -1;
    const int64_t before = t > 0 ? __ldg(p.slots + t - 1) : -1;
    const int64_t slot = __shfl_sync(0xffffffffu, next[0], 0);
    if (slot < 0 || slot >= p.n_slots) {
      ++t;
      continue;
    }
    const int64_t page = slot / PAGE;
    const int off = static_cast<int>(slot - page * PAGE);
    int n = 0;   // rows of this run: the lanes compare the slots with the ones expected
#pragma unroll
    for (int c = 0; c < PAGE; c += 32) {
      const int i = c + lane;
      const bool in = i < PAGE - off && next[c / 32] == slot + i;
      const uint32_t gap = ~__ballot_sync(0xffffffffu, in);
      const int k = gap ? __ffs(gap) - 1 : 32;
      if (n == c) n += k;
    }
    const bool inside = off > 0 && before == slot - 1;
    const int64_t t0 = t;
    t += n;
    if (inside) continue;   // the run began in an earlier window
    // a long run is shared by the team, 16 rows a warp from `first` on
    const bool together = WARPS > 1 && n > kRowsInRegs;
    if (WARPS > 1 && !together) {
      const bool mine = turn == warp;
      turn = turn + 1 < WARPS ? turn + 1 : 0;
      if (!mine) continue;
    }
    const int first = together ? kRowsInRegs * warp : 0;
    uint8_t* exp_at = p.exps[kv] + page * p.ep + head * p.eh;
    uint8_t* base = p.codes[kv] + page * p.sp[kv] + head * p.sh[kv] + 8 * chunk;
    const int held = off > 0 ? static_cast<int>(*exp_at) - 127 : -128;
    uint4 r[kRowsInRegs / 2];
    uint32_t am = 0;
    for (int i0 = first; i0 < (WARPS > 1 ? first + 1 : n); i0 += kRowsInRegs) {
#pragma unroll
      for (int i = 0; i < kRowsInRegs / 2; ++i) {
        const int row = i0 + 2 * i + sub;
        r[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row < n) r[i] = __ldg(reinterpret_cast<const uint4*>(x + (t0 + row) * ldt));
      }
#pragma unroll
      for (int i = 0; i < kRowsInRegs / 2; ++i) am = amax8(r[i], am);
    }
    am = __reduce_max_sync(0xffffffffu, max(am & 0xFFFFu, am >> 16));
    if (together) {
      if (lane == 0) team_max[buf][warp] = am;
      __syncthreads();   // also: every warp has read the page's scale before it changes
#pragma unroll
      for (int w = 0; w < WARPS; ++w) am = max(am, team_max[buf][w]);
      buf ^= 1;
    }
    const int fit = scale_exponent(__uint_as_float(am << 16)), e = max(fit, held);
    if (off > 0 && fit > held) {
      // a louder token than the page has seen: its older codes move to the new scale
      const float f = exp2_int(held - e);
      for (int row = sub + (together ? 2 * warp : 0); row < off; row += together ? 2 * WARPS : 2) {
        uint2* at = reinterpret_cast<uint2*>(base + row * p.st[kv]);
        *at = rescale8(*at, f);
      }
    }
    __syncwarp();
    if (lane == 0 && first == 0) *exp_at = static_cast<uint8_t>(e + 127);
    const float inv = exp2_int(-e);
    for (int i0 = first; i0 < (WARPS > 1 ? first + 1 : n); i0 += kRowsInRegs) {
      if (WARPS == 1 && n > kRowsInRegs) {   // more rows than one warp holds: read again (L1 or L2)
#pragma unroll
        for (int i = 0; i < kRowsInRegs / 2; ++i) {
          const int row = i0 + 2 * i + sub;
          if (row < n) r[i] = __ldg(reinterpret_cast<const uint4*>(x + (t0 + row) * ldt));
        }
      }
#pragma unroll
      for (int i = 0; i < kRowsInRegs / 2; ++i) {
        const int row = i0 + 2 * i + sub;
        if (row < n)
          *reinterpret_cast<uint2*>(base + static_cast<int64_t>(off + row) * p.st[kv]) =
              quant8(r[i], inv);
      }
    }
  }
}

}  // namespace

int launch_kv_plan(const int32_t* ctx, const int32_t* q_len, int64_t B, const int32_t* free_pages,
                   int64_t n_free, int32_t* table, int64_t ld_table, int64_t max_blocks,
                   int32_t page_size, int32_t* q_offsets, int32_t* kv_len, int64_t* slots,
                   int32_t* positions, int64_t T, int32_t* counts, void* stream) {
  if (B < 0 || n_free < 0 || max_blocks < 0 || T < 0 || ld_table < max_blocks)
    return BFP8_ERR_INVALID_ARG;
  if (!q_offsets || !counts || (T > 0 && (!slots || !positions)) || (n_free > 0 && !free_pages) ||
      (B > 0 && (!ctx || !q_len || !kv_len)) || (B > 0 && max_blocks > 0 && !table))
    return BFP8_ERR_INVALID_ARG;
  if (!kv_page_size_ok(page_size) || B > kPlanMaxBatch || max_blocks > 0x7FFFFFFF)
    return BFP8_ERR_UNSUPPORTED;
  int rc = check_device_ptrs({ctx, q_len, n_free ? free_pages : nullptr, table, q_offsets, kv_len,
                              slots, positions, counts});
  if (rc != BFP8_OK) return rc;
  int sms = 0;
  rc = sm_count(&sms);
  if (rc != BFP8_OK) return rc;
  PlanParams p{};
  p.ctx = ctx;
  p.q_len = q_len;
  p.free_pages = free_pages;
  p.table = table;
  p.q_offsets = q_offsets;
  p.kv_len = kv_len;
  p.slots = slots;
  p.positions = positions;
  p.counts = counts;
  p.ld_table = ld_table;
  p.n_free = n_free;
  p.T = T;
  p.B = static_cast<int32_t>(B);
  p.max_blocks = static_cast<int32_t>(max_blocks);
  p.shift = kv_page_shift(page_size);
  const size_t smem = static_cast<size_t>(B) * 8;
  if (smem > 40 * 1024) {   // the 48 KB that need no asking count the kernel's own arrays too
    rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kv_plan_kernel),
                              static_cast<int>(kPlanMaxBatch * 8));
    if (rc != BFP8_OK) return rc;
  }
  const int64_t items = T > B ? T : B;
  const int64_t want = (items + kPlanThreads - 1) / kPlanThreads;
  const unsigned blocks = static_cast<unsigned>(want < 1 ? 1 : want < sms ? want : sms);
  return launch_dependent(kv_plan_kernel, dim3(blocks), kPlanThreads, smem,
                          static_cast<cudaStream_t>(stream), p);
}

int launch_kv_append(const void* k, int64_t k_ldt, int64_t k_ldh, const void* v, int64_t v_ldt,
                     int64_t v_ldh, const int64_t* slots, int64_t T, const bfp8_kv_cache& c,
                     void* stream) {
  int rc = check_kv_cache(c);
  if (rc != BFP8_OK) return rc;
  if (T < 0) return BFP8_ERR_INVALID_ARG;
  if (T == 0) return BFP8_OK;
  if (!k || !v || !slots || k_ldt < 0 || k_ldh < 0 || v_ldt < 0 || v_ldh < 0)
    return BFP8_ERR_INVALID_ARG;
  auto rows16 = [](const void* ptr, int64_t a, int64_t b) {
    return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && a % 8 == 0 && b % 8 == 0;
  };
  if (!rows16(k, k_ldt, k_ldh) || !rows16(v, v_ldt, v_ldh)) return BFP8_ERR_UNSUPPORTED;
  rc = check_device_ptrs({k, v, slots, c.k_e4m3, c.v_e4m3, c.k_exp, c.v_exp});
  if (rc != BFP8_OK) return rc;
  int sms = 0;
  rc = sm_count(&sms);
  if (rc != BFP8_OK) return rc;
  AppendParams p{};
  p.x[0] = static_cast<const __nv_bfloat16*>(k);
  p.x[1] = static_cast<const __nv_bfloat16*>(v);
  p.ldt[0] = k_ldt, p.ldt[1] = v_ldt;
  p.ldh[0] = k_ldh, p.ldh[1] = v_ldh;
  p.codes[0] = static_cast<uint8_t*>(c.k_e4m3);
  p.codes[1] = static_cast<uint8_t*>(c.v_e4m3);
  p.exps[0] = c.k_exp, p.exps[1] = c.v_exp;
  p.sp[0] = c.k_stride_page, p.sh[0] = c.k_stride_head, p.st[0] = c.k_stride_token;
  p.sp[1] = c.v_stride_page, p.sh[1] = c.v_stride_head, p.st[1] = c.v_stride_token;
  p.ep = c.exp_stride_page, p.eh = c.exp_stride_head;
  p.slots = slots;
  p.T = T;
  p.n_slots = c.n_pages * c.page_size;
  p.heads = c.n_kv_heads;
  const int64_t pairs = 2 * static_cast<int64_t>(p.heads);
  const int64_t warps = static_cast<int64_t>(sms) * 32;
  auto go = [&](auto kernel, int team, int block_warps) {
    // a team's window: one token while the GPU's warps suffice, then as many as fill
    // them once, up to a page
    const int64_t w = std::clamp<int64_t>(T * pairs * team / warps, 1, c.page_size);
    const int64_t teams = (T + w - 1) / w * pairs, per = block_warps / team;
    const int64_t blocks = (teams + per - 1) / per;
    if (blocks > 0x7FFFFFFF) return static_cast<int>(BFP8_ERR_UNSUPPORTED);
    p.window = static_cast<int32_t>(w);
    return launch_dependent(kernel, dim3(static_cast<unsigned>(blocks)), 32 * block_warps, 0,
                            static_cast<cudaStream_t>(stream), p);
  };
  const bool few = T * pairs <= warps;
  switch (c.page_size) {
    case 16: return go(kv_append_kernel<16, 1>, 1, 4);
    case 32: return few ? go(kv_append_kernel<32, 1>, 1, 4) : go(kv_append_kernel<32, 2>, 2, 2);
    case 64: return few ? go(kv_append_kernel<64, 1>, 1, 4) : go(kv_append_kernel<64, 4>, 4, 4);
    default: return few ? go(kv_append_kernel<128, 1>, 1, 4) : go(kv_append_kernel<128, 8>, 8, 8);
  }
}

}  // namespace bfp8
