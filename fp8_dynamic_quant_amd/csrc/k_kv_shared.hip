// Attention over the paged 8-bit cache of sequences that begin with the same pages.
//
// Neighbouring sequences of one group id share their first tokens.  A softmax over [shared | own]
// splits into one over each, joined by their maxima and sums, so that the shared tokens are taken
// once for all rows of the group: its rows are one run of rows (row * R + query head, as in
// attention of one sequence) in tiles, all of which see all of those tokens.  Each sequence's own
// tokens are taken for its rows alone.
//
// Items are (sequence, head, row tile) over own tokens and (group, head, row tile) over shared ones.
// Of up to 16 rows they are narrow: a wave takes one alone, straight from memory.  Of more they are
// wide: a workgroup of eight waves takes one (Wide).  The items of either kind lie on an axis of
// their own, in units of a step of 64 tokens and a constant for an item's beginning and end, which
// is cut into equal runs: of narrow ones one a wave, of wide ones one a workgroup.  Workgroups take
// one kind or the other, as many of either as their units ask for.  A row's parts, of both items
// where it shares and of as many runs as cut them, go to the workspace in f32 and are joined by a
// second kernel in the order of the axes: results do not depend on timing.
//
// What a call takes, and of it the join, in us:
//   8 sequences of 50 own tokens behind 1000, 32 heads of 128 on 8   14.9   4  launches, the plan (2.5), steps in turn
//   64 of 500 behind 8192, the same heads, int8                        40   6  short runs: beginnings, parts
//   256 of 1500 behind 32768, the same heads                          236  10  the wide kernel's arithmetic
//   24 of 4 rows and 300 tokens behind four documents of 32768,
//   16 heads of 256 on one                                             72   8  chains of reads and products, a row tile a wave
// A wide run of the second begins its first step 9 us after the launch: plan 2.7, its item found 1.9,
// rows and limits 1.5, page numbers 1, addresses 1.1, the first step 0.7 (latency, and code that is
// fetched as it runs); seven steps take 17, their parts 3.
// Beside attention of each sequence alone, E4M3, one token each, 32 query heads of 128 on 8: 64 sequences of
// up to 200 own tokens behind 4096 35 and 73, of 2000 behind 512 42 and 48.  Where little is shared the plan
// and the parts cost more than it saves: 64 of 200 behind 512 28.6 and 20.5, behind 1024 29.6 and 36.1;
// 8 of 50 15.2 and 13.3, 15.5 and 17.8; 200 of 500 less from 64 on (42 and 50), but with 64 heads of 64 on 8
// 39 and 35 behind 512, 45 and 55 behind 1024.
#include "wq_kernels.h"
#include "wq_kv_plan.h"
#include "wq_kv_wide.h"
#include "wq_layer.h"

namespace wq {

namespace {

constexpr int kThreads = 64 * kWideWaves;
static_assert(kWideWaves == kShareWaves, "the plan's workgroups are the wide kernel's");

struct ShareArgs {
  KvAttnArgs a;            // part, stat: [share_slots] rows
  const int32_t* group;    // [B]
  const int32_t* shared;   // [B]
  uint4* desc;             // [keys], keys = T * Hq
};

struct ShareLds {
  uint32_t pre[2][kShareSeqs + 1];  // by kind: units before sequence b, for one head
  int row0[kShareSeqs + 1];
  int len[kShareSeqs];
  int id[kShareSeqs];
  int lead[kShareSeqs];    // the first sequence of each one's group
  int steps[kShareSeqs];   // by first sequence: the steps that the group shares,
  int end[kShareSeqs];     // where its rows end,
  int many[kShareSeqs];    // how many sequences have rows,
  int holder[kShareSeqs];  // the first that does: its table names the shared pages
  uint32_t carry[2][kWideWaves];
  int last[kWideWaves], most[kWideWaves];
};

// steps that the group led by sequence `lead` shares
__device__ __forceinline__ uint32_t shared_steps(const ShareLds& l, int lead) {
  return l.many[lead] > 1 ? (uint32_t)l.steps[lead] : 0u;
}
// steps of a sequence behind them (one also where none is left: its rows are stored)
__device__ __forceinline__ uint32_t own_steps(const KvArgs& c, int len, uint32_t shared) {
  return (uint32_t)max((int)steps_of(c, len) - (int)shared, 1);
}
__device__ __forceinline__ uint32_t own_rows(const ShareLds& l, int b) { return (uint32_t)(l.row0[b + 1] - l.row0[b]); }
// (of a group that shares steps: some of its sequences have rows)
__device__ __forceinline__ uint32_t group_rows(const ShareLds& l, int lead) { return (uint32_t)(l.end[lead] - l.row0[lead]); }

// Every thread of the workgroup takes part.  Offsets are read as their running maximum, which is what they
// are where they do not decrease: whatever they hold, sequences have rows of their own, side by side, no
// more than T in all, so that units stay in 32 bits and what tell_row says lies in the workspace.
template <int D>
__device__ __forceinline__ SharePlan make_share_plan(const ShareArgs& s, ShareLds& l) {
  const KvAttnArgs& a = s.a;
  const KvArgs& c = a.c;
  const int b = threadIdx.x, lane = b & 63, wv = b >> 6;
  const bool in = b < c.B;
  static_assert(kShareSeqs == kThreads, "a thread for each sequence");
  int row0 = 0, next = 0, len = 0, wants = 0, id = -1;
  if (in) {
    row0 = (int)seq_offset(c, b);
    next = (int)seq_offset(c, b + 1);
    len = c.lens[b];
    id = s.group[b];
    wants = s.shared[b];
    l.len[b] = len;
    l.id[b] = id;
    l.steps[b] = INT32_MAX;
    l.end[b] = 0;
    l.many[b] = 0;
    l.holder[b] = INT32_MAX;
  }
  __syncthreads();
  // the last sequence up to b that begins a group
  int lead = in && b > 0 && (id < 0 || id != l.id[b - 1]) ? b : 0;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(lead, o, 64), v = __shfl_up(row0, o, 64);
    if (lane >= o) {
      lead = max(lead, u);
      row0 = max(row0, v);
    }
  }
  if (lane == 63) {
    l.last[wv] = lead;
    l.most[wv] = row0;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWideWaves; ++w)
    if (w < wv) {
      lead = max(lead, l.last[w]);
      row0 = max(row0, l.most[w]);
    }
  const int rows = max(next - row0, 0);
  if (in) {
    l.row0[b] = row0;
    if (b == c.B - 1) l.row0[c.B] = row0 + rows;
    l.lead[b] = lead;
    if (rows > 0) {
      // the whole pages that all of its rows see, in whole steps
      int64_t own = min((int64_t)len - (a.causal ? rows : 0), (int64_t)c.max_pages * c.P);
      own = max(min((int64_t)wants, own), (int64_t)0);
      atomicMin(&l.steps[lead], (int)((uint32_t)own / (uint32_t)c.P * (uint32_t)c.P / kTokTile));
      atomicMax(&l.end[lead], row0 + rows);
      atomicAdd(&l.many[lead], 1);
      atomicMin(&l.holder[lead], b);
    }
  }
  __syncthreads();
  uint32_t v[2] = {0, 0};
  if (in) {
    auto add = [&](const Kind& k) __attribute__((always_inline)) {
      v[kNarrow] += k.kind == kNarrow ? k.tiles * k.units : 0u;
      v[kWide] += k.kind == kWide ? k.tiles * k.units : 0u;
    };
    const uint32_t sh = shared_steps(l, lead);
    add(kind_of<D>((uint32_t)rows * (uint32_t)a.R, own_steps(c, len, sh)));
    if (lead == b && sh > 0) add(kind_of<D>(group_rows(l, b) * (uint32_t)a.R, sh));
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t u = (uint32_t)__shfl_up((int)v[k], o, 64);
      if (lane >= o) v[k] += u;
    }
    if (lane == 63) l.carry[k][wv] = v[k];
  }
  __syncthreads();
  uint32_t total[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t base = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kWideWaves; ++w) {
      base += w < wv ? l.carry[k][w] : 0u;
      sum += l.carry[k][w];
    }
    if (in) l.pre[k][b + 1] = base + v[k];
    if (b == 0) l.pre[k][0] = 0;
    total[k] = (uint32_t)uniform((int)(sum * (uint32_t)c.H));
  }
  const SharePlan p = cut_axes(total[kNarrow], total[kWide], gridDim.x);
  __syncthreads();
  return p;
}

// The item of a kind that unit u of its axis is in.  Of a sequence's units those of its own tokens'
// items come first, then, of a group's first sequence, the shared ones'.
struct ShareItem {
  int b;             // the sequence, or the one whose table the group takes
  bool of_group;
  uint32_t h, tile;
  Kind k;
  uint32_t shared;   // steps that the group shares: own tokens' steps begin there
  int row0, rows;    // tokens
  uint32_t i0;       // the item's first unit
};
template <int D, int KIND>
__device__ __forceinline__ ShareItem share_item(const ShareArgs& s, const ShareLds& l, uint32_t u, int lane) {
  const KvArgs& c = s.a.c;
  const uint32_t* pre = l.pre[KIND];
  // the last sequence that begins at or before u (of equal ones the one with work): eight at a time, then one
  const uint32_t H = (uint32_t)c.H;
  const int far = 8 * (__popcll(__ballot(8 * lane < c.B && pre[min(8 * lane, c.B)] * H <= u)) - 1);
  const int lo = uniform(far + __popcll(__ballot(lane < 8 && far + lane < c.B && pre[min(far + lane, c.B)] * H <= u)) - 1);
  ShareItem it;
  const int lead = uniform(l.lead[lo]);
  it.shared = (uint32_t)uniform((int)shared_steps(l, lead));
  it.b = lo;
  it.row0 = uniform(l.row0[lo]);
  it.rows = uniform((int)own_rows(l, lo));
  it.k = kind_of<D>((uint32_t)it.rows * (uint32_t)s.a.R, own_steps(c, uniform(l.len[lo]), it.shared));
  uint32_t first = (uint32_t)uniform((int)pre[lo]) * H;
  const uint32_t own = it.k.kind == KIND ? it.k.tiles * it.k.units * H : 0u;
  it.of_group = u - first >= own;
  if (it.of_group) {
    first += own;
    it.rows = uniform((int)group_rows(l, lo));
    it.b = uniform(l.holder[lo]);
    it.k = kind_of<D>((uint32_t)it.rows * (uint32_t)s.a.R, it.shared);
  }
  const uint32_t item = (u - first) / it.k.units;
  it.i0 = first + item * it.k.units;
  it.h = item / it.k.tiles;
  it.tile = item - it.h * it.k.tiles;
  return it;
}
// What a run has of an item, and where its rows' output or part goes
struct Share {
  const ShareArgs& s;
  const KvAttnArgs& a;
  ShareItem it;
  Seq q;             // the item's rows and tokens
  uint32_t from, to; // steps of the sequence
  bool whole;        // all of them, and nobody shares
  uint32_t run;

  // (token, query head) of row rr
  __device__ __forceinline__ int64_t key(uint32_t rr) const {
    const uint32_t i = rr / (uint32_t)a.R;
    return (q.row0 + i) * (int64_t)(a.c.H * a.R) + (it.h * (uint32_t)a.R + (rr - i * (uint32_t)a.R));
  }
  __device__ __forceinline__ bool begins() const { return from == (it.of_group ? 0u : it.shared); }  // has the item's first step
  // the row of its part: by key where the run begins the item, else by the run, which begins inside no
  // other item
  template <int D>
  __device__ __forceinline__ int64_t slot(uint32_t rr, int64_t key) const {
    const int64_t keys = a.c.T * a.c.H * a.R;
    if (begins()) return first_slot(keys, key, it.of_group);
    return run_slot<D>(keys, gridDim.x, it.k.kind, run, rr - it.tile * it.k.tile);
  }
};
template <int D, int KIND>
__device__ __forceinline__ bool take_share(Share& r, const SharePlan& p, const ShareLds& l, uint32_t u, uint32_t end, int lane) {
  const ShareArgs& s = r.s;
  r.it = share_item<D, KIND>(s, l, u, lane);
  const ShareItem& it = r.it;
  r.from = step_at(it.k, u - it.i0);
  r.to = step_at(it.k, min(end - it.i0, it.k.units));
  if (r.from >= r.to) return false;
  r.whole = !it.of_group && it.shared == 0 && r.from == 0 && r.to == it.k.steps;
  r.q.row0 = it.row0;
  r.q.rows = it.rows;
  r.q.nrows = (int64_t)it.rows * s.a.R;
  r.q.len = uniform(l.len[it.b]);
  r.q.seen = (uint32_t)min((int64_t)max(r.q.len, 0), (int64_t)s.a.c.max_pages * s.a.c.P);
  r.q.table = s.a.c.table + it.b * s.a.c.table_stride;
  if (it.of_group) {  // all of its rows see all of it (limit_of, causal or not)
    r.q.seen = it.shared * kTokTile;
    r.q.len = (int)r.q.seen;
    r.q.rows = 0;
  } else {  // steps of the sequence
    r.from += it.shared;
    r.to += it.shared;
  }
  return true;
}

// The join of row rr of an own item, told by the run that has the item's first step: of its own
// tokens' item and of the shared ones' item the first run, how many, and the row's place in the tile.
template <int D>
__device__ __forceinline__ void tell_row(const Share& r, const SharePlan& p, const ShareLds& l, uint32_t rr, int64_t key) {
  const ShareItem& it = r.it;
  uint4 d{0, 0, 0, 0};
  if (!r.whole) {
    auto parts = [&](const Kind& k, uint32_t i0, uint32_t row) {
      const Parts t = parts_of(k, p, i0, row);
      return uint2{t.run | t.count << 16, t.at};
    };
    const uint2 own = parts(it.k, it.i0, rr);
    d.x = own.x;
    d.z = own.y;
    if (it.shared > 0) {
      const int lead = l.lead[it.b];
      const uint32_t R = (uint32_t)r.a.R, H = (uint32_t)r.a.c.H;
      const uint32_t gr = (uint32_t)(it.row0 - l.row0[lead]) * R + rr;
      const Kind k = kind_of<D>(group_rows(l, lead) * R, it.shared);
      // the group's units lie behind the own ones of its first sequence
      const Kind kl = kind_of<D>(own_rows(l, lead) * R, own_steps(r.a.c, l.len[lead], it.shared));
      const uint32_t ahead = kl.kind == k.kind ? kl.tiles * kl.units : 0u;
      const uint2 all = parts(k, (l.pre[k.kind][lead] + ahead) * H + (it.h * k.tiles + gr / k.tile) * k.units, gr);
      d.y = all.x;
      d.z |= all.y << 16;
    }
  }
  r.s.desc[key] = d;
}

// A wave's own rows, to the output if nothing else has a part of them, else to the workspace: lane
// (j, g) holds of row j the elements 16 i + 4 g .. + 3.  total: the sum of the weights, kept: of the
// weights that o was made with, total itself where the largest of them is 1.
//
// Wide's are rounded, the largest too, which may be anything in (1/2, 2^8].  Over their own sum that rounding
// cancels as far as it is common to what a row sees, so that a row of one token is that token's value; over
// the other sum it would leave up to 2^-8 of everything (rows of a few large weights: 0.0023 off against 64
// bits, 0.0017 so, which is the output's own rounding; of many 0.0024 and 0.0021).  A part is brought to the
// scale of `total`, which lse and the join go by.
template <int D>
__device__ __forceinline__ void store_share(const Share& r, const SharePlan& p, const ShareLds& l, const v4f (&o)[D / 16], float mx,
                                            float total, float kept, uint32_t rr, int g) {
  if (rr >= (uint32_t)r.q.nrows) return;
  const int64_t key = r.key(rr);
  if (r.whole) {
    const int64_t hq = r.a.c.H * r.a.R, token = r.q.row0 + rr / (uint32_t)r.a.R;
    uint16_t* out = r.a.out + token * r.a.ldo + (key - token * hq) * D + 4 * g;
    const float inv = inverse_sum(kept);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const v4f v = o[i] * inv;
      *reinterpret_cast<v2u*>(out + 16 * i) = v2u{f32_to_bf16_nan(v[0]) | f32_to_bf16_nan(v[1]) << 16,
                                                  f32_to_bf16_nan(v[2]) | f32_to_bf16_nan(v[3]) << 16};
    }
    if (r.a.lse && g == 0) r.a.lse[key] = log_sum(mx, total);
  } else {
    const int64_t slot = r.template slot<D>(rr, key);
    float* to = r.a.part + slot * D + 4 * g;
    const float back = kept > 0.0f ? total / kept : 1.0f;  // (rows that saw nothing: zeros; NaN is in o as well)
#pragma unroll
    for (int i = 0; i < D / 16; ++i) *reinterpret_cast<v4f*>(to + 16 * i) = o[i] * back;
    if (g == 0) r.a.stat[slot] = float2{mx, total};
  }
  if (g == 0 && !r.it.of_group && r.begins()) tell_row<D>(r, p, l, rr, key);
}

// the steps that the rows up to `row` see
__device__ __forceinline__ uint32_t steps_to(const Share& r, int64_t row, uint32_t tokens) {
  return (uint32_t)uniform((int)((limit_of(r.a, r.q, (int)(min(row, r.q.nrows) - 1) / r.a.R) + tokens - 1) / tokens));
}

template <int D, bool I8>
__device__ __forceinline__ void narrow_runs(const ShareArgs& s, const SharePlan& p, const ShareLds& l, uint32_t run, int lane) {
  const int j = lane & 15, g = lane >> 4;
  const uint32_t per = p.axis[kNarrow].per, end = min((run + 1) * per, p.axis[kNarrow].units);
  for (uint32_t u = run * per; u < end;) {
    Share r{s, s.a};
    r.run = run;
    const bool some = take_share<D, kNarrow>(r, p, l, u, end, lane);
    u = r.it.i0 + r.it.k.units;
    if (!some) continue;
    const int64_t r0 = (int64_t)r.it.tile * kNarrowRows;
    Rows<D, I8, 1> w;
    w.run(r.a, r.q, (int)r.it.h, r0, r.from, min(r.to, steps_to(r, r0 + kNarrowRows, kTokTile)), 1, j, g);
    const float total = groups_sum(w.sum[0]);
    store_share<D>(r, p, l, w.o[0], w.mx[0], total, total, (uint32_t)r0 + j, g);
  }
}

template <int D, bool I8, int RT>
__device__ __forceinline__ void take_wide(const Share& r, const SharePlan& p, const ShareLds& l, uint8_t* smem, int wv, int lane) {
  using W = Wide<D, I8, RT>;
  constexpr uint32_t kSub = kTokTile / W::T;  // its steps to one of 64 tokens
  const int j = lane & 15, g = lane >> 4;
  const int64_t t0 = (int64_t)r.it.tile * wide_rows(D), r0 = t0 + wv * 16 * RT;
  W w;
  w.begin(r.a, r.q, (int)r.it.h, r0, j, g);
  w.run(r.a, r.q, (int)r.it.h, r.from * kSub, min(r.to * kSub, steps_to(r, t0 + W::kRows, W::T)),
        r0 < r.q.nrows, smem, wv, lane);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
    store_share<D>(r, p, l, w.o[rt], w.mx[rt], groups_sum(w.sum[rt]), w.kept[rt][0], (uint32_t)r0 + 16 * rt + j, g);
}

template <int D, bool I8>
__device__ __forceinline__ void wide_runs(const ShareArgs& s, const SharePlan& p, const ShareLds& l, uint32_t run, uint8_t* smem, int wv,
                                          int lane) {
  const uint32_t per = p.axis[kWide].per, end = min((run + 1) * per, p.axis[kWide].units);
  for (uint32_t u = run * per; u < end;) {
    Share r{s, s.a};
    r.run = run;
    const bool some = take_share<D, kWide>(r, p, l, u, end, lane);
    u = r.it.i0 + r.it.k.units;
    if (!some) continue;
    if constexpr (D < 256) {
      if ((uint32_t)r.q.nrows - r.it.tile * wide_rows(D) > 128u) {
        take_wide<D, I8, 2>(r, p, l, smem, wv, lane);
        continue;
      }
    }
    take_wide<D, I8, 1>(r, p, l, smem, wv, lane);
  }
}

template <int D, bool I8>
__global__ __launch_bounds__(kThreads, 2) void k_kv_shared(ShareArgs s) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ ShareLds lds;
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const SharePlan plan = make_share_plan<D>(s, lds);
  const uint32_t wide = plan.axis[kWide].runs;  // workgroups that take wide runs; the waves of the others narrow ones
  if (blockIdx.x < wide) {
    wide_runs<D, I8>(s, plan, lds, blockIdx.x, smem, wv, lane);
  } else if constexpr (D < 256) {
    narrow_runs<D, I8>(s, plan, lds, blockIdx.x - wide + (uint32_t)wv * (gridDim.x - wide), lane);
  }
}

// The parts of a row, found by its descriptor
struct JoinParts {
  const ShareArgs& s;
  int64_t key, keys;
  uint4 d;
  int own, all;  // parts of its own tokens; with the shared ones'
  __device__ __forceinline__ JoinParts(const ShareArgs& s, int64_t key, int64_t keys, uint4 d)
      : s(s), key(key), keys(keys), d(d), own((int)(d.x >> 16)), all((int)(d.x >> 16) + (int)(d.y >> 16)) {}
  template <int D>
  __device__ __forceinline__ int64_t slot(int p) const {
    const bool mine = p < own;
    const int k = mine ? p : p - own;
    if (k == 0) return first_slot(keys, key, !mine);
    const uint32_t run = ((mine ? d.x : d.y) & 0xFFFFu) + k, at = mine ? d.z & 0xFFFFu : d.z >> 16;
    return run_slot<D>(keys, s.a.runs, at & 0x8000u ? kWide : kNarrow, run, at & 0x7FFFu);
  }
};
template <int D>
__device__ __forceinline__ void store_joined(const ShareArgs& s, int64_t key, int64_t hq, int col, v4f acc, float M, float L) {
  const float inv = inverse_sum(L);
  const int64_t token = key / hq;
  uint16_t* out = s.a.out + token * s.a.ldo + (key - token * hq) * D + col;
  *reinterpret_cast<v2u*>(out) = v2u{f32_to_bf16_nan(acc[0] * inv) | f32_to_bf16_nan(acc[1] * inv) << 16,
                                     f32_to_bf16_nan(acc[2] * inv) | f32_to_bf16_nan(acc[3] * inv) << 16};
  if (col == 0 && s.a.lse) s.a.lse[key] = log_sum(M, L);
}

// A wave for each row: D / 4 lanes of four columns take a part, 256 / D parts at once, kAhead times in
// flight; the running maximum and sum go with them.
template <int D>
__global__ __launch_bounds__(256) void k_kv_shared_join(ShareArgs s) {
  constexpr int kLanes = D / 4, kAtOnce = 64 / kLanes, kAhead = 4;
  const KvAttnArgs& a = s.a;
  const int lane = threadIdx.x & 63, mine = lane / kLanes, col = lane % kLanes * 4;
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t hq = (int64_t)a.c.H * a.R, keys = a.c.T * hq;
  const int64_t end = seq_offset(a.c, a.c.B) * hq;
  for (int64_t key = seq_offset(a.c, 0) * hq + (int64_t)blockIdx.x * 4 + wv; key < end; key += (int64_t)gridDim.x * 4) {
    const JoinParts j(s, key, keys, s.desc[key]);
    float M = -INFINITY, L = 0.0f;
    v4f acc{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p0 = 0; p0 < j.all; p0 += kAtOnce * kAhead) {
      v4f v[kAhead];
      float2 st[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int64_t slot = j.template slot<D>(min(p0 + x * kAtOnce + mine, j.all - 1));
        v[x] = *reinterpret_cast<const v4f*>(a.part + slot * D + col);
        st[x] = a.stat[slot];
        if (p0 + x * kAtOnce + mine >= j.all) st[x] = float2{-INFINITY, 0.0f};
      }
      float top = M;
#pragma unroll
      for (int x = 0; x < kAhead; ++x) top = fmaxf(top, st[x].x);
      const float base = top == -INFINITY ? 0.0f : top, old = __builtin_amdgcn_exp2f(M - base);
      L *= old;
      acc *= old;
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        if (p0 + x * kAtOnce + mine >= j.all) continue;
        const float w = __builtin_amdgcn_exp2f(st[x].x - base);
        L += w * st[x].y;
        acc += w * v[x];
      }
      M = top;
    }
    if (j.all == 0) continue;
    // the lanes that took parts beside each other
#pragma unroll
    for (int o = kLanes; o < 64; o <<= 1) {
      const float m = __shfl_xor(M, o, 64), top = fmaxf(M, m), base = top == -INFINITY ? 0.0f : top;
      const float w0 = __builtin_amdgcn_exp2f(M - base), w1 = __builtin_amdgcn_exp2f(m - base);
      L = w0 * L + w1 * __shfl_xor(L, o, 64);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = w0 * acc[e] + w1 * __shfl_xor(acc[e], o, 64);
      M = top;
    }
    if (mine == 0) store_joined<D>(s, key, hq, col, acc, M, L);
  }
}

// A workgroup for each row, where rows are few and may have hundreds of parts.
template <int D>
__global__ __launch_bounds__(256) void k_kv_shared_join_wide(ShareArgs s) {
  constexpr int kLanes = D / 4, kAtOnce = 256 / kLanes, kAhead = 4;
  __shared__ float top_of[kAtOnce], sum_of[kAtOnce];
  __shared__ v4f acc_of[kAtOnce][kLanes];
  const KvAttnArgs& a = s.a;
  const int t = threadIdx.x, mine = t / kLanes, col = t % kLanes * 4;
  const int64_t hq = (int64_t)a.c.H * a.R, keys = a.c.T * hq;
  const int64_t end = seq_offset(a.c, a.c.B) * hq;
  for (int64_t key = seq_offset(a.c, 0) * hq + blockIdx.x; key < end; key += gridDim.x) {
    const JoinParts j(s, key, keys, s.desc[key]);
    if (j.all == 0) continue;
    float M = -INFINITY, L = 0.0f;
    v4f acc{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p0 = mine; p0 < j.all; p0 += kAtOnce * kAhead) {
      v4f v[kAhead];
      float2 st[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int64_t slot = j.template slot<D>(min(p0 + x * kAtOnce, j.all - 1));
        v[x] = *reinterpret_cast<const v4f*>(a.part + slot * D + col);
        st[x] = a.stat[slot];
        if (p0 + x * kAtOnce >= j.all) st[x] = float2{-INFINITY, 0.0f};
      }
      float top = M;
#pragma unroll
      for (int x = 0; x < kAhead; ++x) top = fmaxf(top, st[x].x);
      const float base = top == -INFINITY ? 0.0f : top, old = __builtin_amdgcn_exp2f(M - base);
      L *= old;
      acc *= old;
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        if (p0 + x * kAtOnce >= j.all) continue;
        const float w = __builtin_amdgcn_exp2f(st[x].x - base);
        L += w * st[x].y;
        acc += w * v[x];
      }
      M = top;
    }
    if (col == 0) {
      top_of[mine] = M;
      sum_of[mine] = L;
    }
    acc_of[mine][t % kLanes] = acc;
    __syncthreads();
    if (mine == 0) {
      float top = top_of[0];
#pragma unroll
      for (int w = 1; w < kAtOnce; ++w) top = fmaxf(top, top_of[w]);
      const float base = top == -INFINITY ? 0.0f : top;
      L = 0.0f;
      acc = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kAtOnce; ++w) {
        const float x = __builtin_amdgcn_exp2f(top_of[w] - base);
        L += x * sum_of[w];
        acc += x * acc_of[w][t];
      }
      store_joined<D>(s, key, hq, col, acc, top, L);
    }
    __syncthreads();  // the next row's sums go where these were
  }
}

// How a call runs.  Sequences of many rows fill row tiles of their own, which read the shared tokens
// once for each: attention as it is does that, with no parts to join.  What is shared decides which is
// quicker, and the host does not know it: the rule lies where either gains about what the other would, an
// average of 512 new tokens here.  (32 heads of 128 in groups of four, E4M3, attention as it is and this, by
// the new tokens of the longest sequence, the average being 0.63 of that with 16 and 0.68 with 4 sequences:
//   16 behind 4096:  128 228 and 150 us, 256 389 and 282, 512 634 and 525, 768 899 and 771
//   16 behind 512:    64 44 and 50,      128 48 and 71,   256 83 and 117,  768 227 and 363
//   4 behind 4096:   128 76 and 60,      256 122 and 95,  512 231 and 160, 768 348 and 241
//   4 behind 512:    128 38 and 38,      256 47 and 51,   512 62 and 79,   768 76 and 113)
// So do sizes whose units are not counted in 32 bits.
struct ShareShape {
  bool own;
  int64_t keys, slots;  // output rows; rows of the workspace
};
ShareShape share_shape(const KvArgs& c, int R, int num_cu) {
  ShareShape s{};
  const double tiles = 2.0 * ((double)c.T * R / kNarrowRows + c.B) * c.H, steps = (double)c.max_pages * c.P / kTokTile + 8;
  s.own = c.T * R < 2048 * (int64_t)c.B && tiles * steps < 2147483648.0;
  s.keys = c.T * c.H * R;
  s.slots = share_slots(s.keys, max(num_cu, 2), c.D);
  return s;
}

template <int D, bool I8>
hipError_t shared_of(ShareArgs s, int64_t keys, hipStream_t st) {
  constexpr int lds = Wide<D, I8, 1>::kBytes;
  hipError_t e = set_lds_limit(reinterpret_cast<const void*>(k_kv_shared<D, I8>), lds);
  if (e != hipSuccess) return e;
  const ShareArgs all = s;
  const int cus = s.a.runs;
  for (int b = 0; b < all.a.c.B; b += kShareSeqs) {  // the launches of one stream use the workspace in turn
    s.a.c.B = min(all.a.c.B - b, kShareSeqs);
    s.a.c.offsets = all.a.c.offsets + b;
    s.a.c.lens = all.a.c.lens + b;
    s.a.c.table = all.a.c.table + b * all.a.c.table_stride;
    s.group = all.group + b;
    s.shared = all.shared + b;
    hipLaunchKernelGGL((k_kv_shared<D, I8>), dim3((unsigned)cus), dim3(kThreads), lds, st, s);
    // a wave a row once that fills the chip (rows have few parts then): 2048 rows of 128 in up to 22
    // parts 41.0 us with what comes before, a workgroup a row 41.7; 1536 rows of 256 77.2 and 75.0
    if (keys >= 8 * cus)
      hipLaunchKernelGGL(k_kv_shared_join<D>, dim3((unsigned)min((keys + 3) / 4, (int64_t)8 * cus)), dim3(256), 0, st, s);
    else
      hipLaunchKernelGGL(k_kv_shared_join_wide<D>, dim3((unsigned)keys), dim3(256), 0, st, s);
  }
  return hipGetLastError();
}

}  // namespace

size_t kv_shared_workspace(const KvArgs& c, int R, int num_cu) {
  const ShareShape s = share_shape(c, R, num_cu);
  if (!s.own) return kv_attention_workspace(c, R, num_cu);
  return (size_t)s.slots * (c.D * sizeof(float) + sizeof(float2)) + (size_t)s.keys * sizeof(uint4);
}

int kv_shared_path(const KvArgs& c, int R, int num_cu) {
  return share_shape(c, R, num_cu).own ? 16 : kv_attention_path(c, R, num_cu);
}

hipError_t launch_kv_attention_shared(KvAttnArgs a, bool i8, const int32_t* group, const int32_t* shared, int num_cu,
                                      void* ws, hipStream_t st) {
  const ShareShape sh = share_shape(a.c, a.R, num_cu);
  if (!sh.own) return launch_kv_attention(a, i8, num_cu, ws, st);
  a.runs = max(num_cu, 2);  // workgroups: some for either kind
  ShareArgs s{a, group, shared, static_cast<uint4*>(ws)};
  s.a.part = reinterpret_cast<float*>(s.desc + sh.keys);
  s.a.stat = reinterpret_cast<float2*>(s.a.part + sh.slots * a.c.D);
  auto go = [&](auto d) {
    constexpr int D = decltype(d)::value;
    return i8 ? shared_of<D, true>(s, sh.keys, st) : shared_of<D, false>(s, sh.keys, st);
  };
  if (a.c.D == 64) return go(std::integral_constant<int, 64>{});
  return a.c.D == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 256>{});
}

}  // namespace wq
