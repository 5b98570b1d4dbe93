// Attention over the paged 8-bit cache of sequences that begin with the same pages.
//
// Neighbouring sequences of one group id share their first tokens.  A softmax over [shared | own]
// splits into one over each, joined by their maxima and sums, so that the shared tokens are taken
// once for all rows of the group: its rows are one run of rows (row * R + query head, as in
// attention of one sequence) in tiles of up to 128, all of which see all of those tokens.  Each
// sequence's own tokens are taken for its rows alone.
//
// The work of both kinds, (sequence, head, row tile) items over own tokens and (group, head, row
// tile) items over shared ones, is laid on one axis in units of cost and cut into equal runs, one a
// workgroup.  A row's parts, of at least two items where it shares and of as many runs as cut them,
// go to the workspace in f32 and are joined by a second kernel, in the order of the axis: results
// do not depend on timing.
#include "wq_kernels.h"
#include "wq_kv_attn.h"
#include "wq_layer.h"

namespace wq {

namespace {

constexpr int kShareSeqs = 512;  // sequences of one launch (their plan is held in LDS)
constexpr int kMaxParts = 1024;  // parts of an item: no more than runs

struct ShareArgs {
  KvAttnArgs a;            // part, stat: [2 T Hq + runs * tile] rows; runs, least
  const int32_t* group;    // [B]
  const int32_t* shared;   // [B]
  uint4* desc;             // [T * Hq]
};

// Where the parts of a row are: of its own tokens' item and of the shared ones' item the first run,
// how many, and the row's place in the tile.  Part 0 of an item has a slot by (token, query head),
// part p > 0 one by its run, which begins inside no other item.
__device__ __forceinline__ uint4 pack_desc(int run0, int parts0, int tile_row0, int run1, int parts1, int tile_row1) {
  return uint4{(uint32_t)run0 | (uint32_t)parts0 << 16, (uint32_t)run1 | (uint32_t)parts1 << 16,
               (uint32_t)tile_row0 | (uint32_t)tile_row1 << 16, 0u};
}

// Rows of a tile, the units that a step of 64 tokens costs, and an item besides its steps.
struct Cost {
  int tile, step, fixed;
};
template <int D>
__device__ __forceinline__ Cost cost_of(int64_t rows) {
  if (D < 256 && rows <= 16) return Cost{16, 1, 2 * kAttnWaves};
  if (D == 256 || rows <= 64) return Cost{64, 2, 8};
  return Cost{128, 3, 12};
}

struct ShareLds {
  int64_t pre[kShareSeqs + 1];  // units before sequence b, for one head
  int row0[kShareSeqs + 1];
  int len[kShareSeqs];
  int id[kShareSeqs];
  int lead[kShareSeqs];    // the first sequence of each one's group
  int steps[kShareSeqs];   // by first sequence: the steps that the group shares,
  int end[kShareSeqs];     // where its rows end,
  int many[kShareSeqs];    // how many sequences have rows,
  int holder[kShareSeqs];  // the first that does: its table names the shared pages
  int64_t carry[kAttnWaves];
  int last[kAttnWaves];
};

// steps that the group led by sequence `lead` shares
__device__ __forceinline__ uint32_t shared_steps(const ShareLds& l, int lead) {
  return l.many[lead] > 1 ? (uint32_t)l.steps[lead] : 0u;
}
// steps of a sequence behind them (one also where none is left: its rows are stored)
__device__ __forceinline__ uint32_t own_steps(const KvArgs& c, int len, uint32_t shared) {
  return (uint32_t)max((int)steps_of(c, len) - (int)shared, 1);
}

__device__ __forceinline__ int64_t group_rows(const ShareLds& l, int lead) { return max(l.end[lead] - l.row0[lead], 0); }

struct SharePlan {
  int64_t units, per;
  int runs;
};
__device__ __forceinline__ int64_t item_units(const Cost& k, uint32_t steps) { return k.fixed + (int64_t)k.step * steps; }
__device__ __forceinline__ int tiles_of(const Cost& k, int64_t rows) { return (int)((rows + k.tile - 1) / k.tile); }

// Every thread of the workgroup takes part.
template <int D>
__device__ __forceinline__ SharePlan make_share_plan(const ShareArgs& s, ShareLds& l) {
  const KvAttnArgs& a = s.a;
  const KvArgs& c = a.c;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  constexpr int kThreads = 64 * kAttnWaves;
  for (int b = t; b < c.B; b += kThreads) {
    const int64_t lo = seq_offset(c, b), rows = max(seq_offset(c, b + 1) - lo, (int64_t)0);
    l.row0[b] = (int)lo;
    l.len[b] = c.lens[b];
    l.id[b] = s.group[b];
    l.steps[b] = INT32_MAX;
    l.end[b] = 0;
    l.many[b] = 0;
    l.holder[b] = INT32_MAX;
    if (b == c.B - 1) l.row0[c.B] = (int)(lo + rows);
  }
  __syncthreads();
  int before = 0;
  for (int b0 = 0; b0 < c.B; b0 += kThreads) {
    // the last sequence up to b that begins a group
    const int b = b0 + t;
    int lead = b < c.B && b > 0 && (l.id[b] < 0 || l.id[b] != l.id[b - 1]) ? b : 0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(lead, o, 64);
      if (lane >= o) lead = max(lead, u);
    }
    if (lane == 63) l.last[wv] = lead;
    __syncthreads();
    lead = max(lead, before);
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      if (w < wv) lead = max(lead, l.last[w]);
      before = max(before, l.last[w]);
    }
    if (b < c.B) {
      l.lead[b] = lead;
      const int row0 = l.row0[b], rows = l.row0[b + 1] - row0;
      if (rows > 0) {
        // the whole pages that all of its rows see, in whole steps
        int64_t own = min((int64_t)l.len[b] - (a.causal ? rows : 0), (int64_t)c.max_pages * c.P);
        own = max(min((int64_t)s.shared[b], own), (int64_t)0);
        atomicMin(&l.steps[lead], (int)(own / c.P * c.P / kTokTile));
        atomicMax(&l.end[lead], row0 + rows);
        atomicAdd(&l.many[lead], 1);
        atomicMin(&l.holder[lead], b);
      }
    }
    __syncthreads();
  }
  int64_t sum = 0;
  for (int b0 = 0; b0 < c.B; b0 += kThreads) {
    const int b = b0 + t;
    int64_t v = 0;
    if (b < c.B) {
      const int row0 = l.row0[b], lead = l.lead[b];
      const int64_t rows = (int64_t)max(l.row0[b + 1] - row0, 0) * a.R;
      const uint32_t sh = shared_steps(l, lead);
      const Cost k = cost_of<D>(rows);
      v = tiles_of(k, rows) * item_units(k, own_steps(c, l.len[b], sh));
      if (lead == b && sh > 0) {
        const int64_t all = group_rows(l, b) * a.R;
        const Cost kg = cost_of<D>(all);
        v += tiles_of(kg, all) * item_units(kg, sh);
      }
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t u = __shfl_up(v, o, 64);
      if (lane >= o) v += u;
    }
    if (lane == 63) l.carry[wv] = v;
    __syncthreads();
    int64_t base = sum;
    for (int w = 0; w < wv; ++w) base += l.carry[w];
    if (b < c.B) l.pre[b + 1] = base + v;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) sum += l.carry[w];
    if (b == 0) l.pre[0] = 0;
    __syncthreads();
  }
  SharePlan p;
  p.units = sum * c.H;
  p.per = max(quotient(p.units + a.runs - 1, a.runs), (int64_t)a.least);
  p.runs = (int)quotient(p.units + p.per - 1, p.per);
  return p;
}

// The item that unit u is in.  Of a sequence's units, those of its own tokens' items come first,
// then, of a group's first sequence, the shared ones'.
struct ShareItem {
  int b;             // the sequence, or the one whose table the group takes
  bool of_group;
  int h, tile;
  Cost cost;
  uint32_t shared;   // steps that the group shares: own tokens' steps begin there
  uint32_t steps;    // of the item
  int64_t row0;      // token rows
  int rows;
  int64_t i0, units; // the item's units
};
template <int D>
__device__ __forceinline__ ShareItem share_item(const ShareArgs& s, const ShareLds& l, int64_t u) {
  const KvArgs& c = s.a.c;
  int lo = 0, hi = c.B - 1;
  while (lo < hi) {  // the last sequence that begins at or before u (of equal ones the one with work)
    const int mid = (lo + hi + 1) >> 1;
    if (l.pre[mid] * c.H <= u) lo = mid;
    else hi = mid - 1;
  }
  ShareItem it;
  it.b = lo = uniform(lo);
  const int lead = uniform(l.lead[lo]);
  it.shared = (uint32_t)uniform((int)shared_steps(l, lead));
  it.row0 = uniform(l.row0[lo]);
  it.rows = uniform(max(l.row0[lo + 1] - l.row0[lo], 0));
  it.steps = own_steps(c, uniform(l.len[lo]), it.shared);
  it.cost = cost_of<D>((int64_t)it.rows * s.a.R);
  it.units = item_units(it.cost, it.steps);
  int64_t first = l.pre[lo] * c.H;
  const int64_t own = (int64_t)tiles_of(it.cost, (int64_t)it.rows * s.a.R) * it.units * c.H;
  it.of_group = u - first >= own;
  if (it.of_group) {
    first += own;
    it.rows = uniform((int)group_rows(l, lo));
    it.b = uniform(l.holder[lo]);
    it.steps = it.shared;
    it.cost = cost_of<D>((int64_t)it.rows * s.a.R);
    it.units = item_units(it.cost, it.steps);
  }
  const int64_t item = quotient(u - first, it.units);
  it.i0 = first + item * it.units;
  const int tiles = tiles_of(it.cost, (int64_t)it.rows * s.a.R);
  it.h = uniform((int)quotient(item, tiles));
  it.tile = uniform((int)(item - (int64_t)it.h * tiles));
  return it;
}
// Step p of an item lies at unit fixed + p * step of it: a run that begins in front of that and ends
// behind it takes the step.
__device__ __forceinline__ uint32_t step_at(const ShareItem& it, int64_t x) {
  if (x <= it.cost.fixed) return 0;
  if (x >= it.units) return it.steps;
  return (uint32_t)uniform((int)quotient(x - it.cost.fixed + it.cost.step - 1, it.cost.step));
}
__device__ __forceinline__ int run_of(const SharePlan& p, int64_t unit) { return uniform((int)quotient(unit, p.per)); }

// What a run has of a row: where its output or its part goes
struct Share {
  const ShareArgs& s;
  ShareItem it;
  Seq q;             // the item's rows and tokens
  KvAttnArgs a;      // (rows of a group are not masked)
  bool first, whole; // the run has the item's first step; all of them, and nobody shares
  int run;

  __device__ __forceinline__ int64_t key(int64_t rr) const {  // (token, query head) of row rr
    const int i = (int)rr / a.R;
    return (q.row0 + i) * (int64_t)(a.c.H * a.R) + it.h * a.R + ((int)rr - i * a.R);
  }
  __device__ __forceinline__ int64_t slot(int64_t rr) const {
    const int64_t keys = a.c.T * a.c.H * a.R;
    if (first) return (it.of_group ? keys : 0) + key(rr);
    return 2 * keys + (int64_t)run * a.tile_rows + (rr - (int64_t)it.tile * it.cost.tile);
  }
};

// The join of row rr of an own item: told by the run that has the item's first step.
template <int D>
__device__ __forceinline__ void tell_row(const Share& r, const SharePlan& p, const ShareLds& l, int64_t rr) {
  const ShareItem& it = r.it;
  if (r.whole) {
    r.s.desc[r.key(rr)] = uint4{0, 0, 0, 0};
    return;
  }
  auto at = [&](const Cost& k, int64_t i0, uint32_t step) { return (int)quotient(i0 + k.fixed + (int64_t)step * k.step, p.per); };
  const int run0 = at(it.cost, it.i0, 0), parts0 = at(it.cost, it.i0, it.steps - 1) - run0 + 1;
  int run1 = 0, parts1 = 0, row1 = 0;
  if (it.shared > 0) {
    const int lead = l.lead[it.b];
    const int64_t ahead = (int64_t)l.row0[lead];
    const int64_t all = group_rows(l, lead) * r.a.R, gr = (it.row0 - ahead) * r.a.R + rr;
    const Cost k = cost_of<D>(all);
    const int64_t units = item_units(k, it.shared);
    const int tiles = tiles_of(k, all), tile = (int)(gr / k.tile);
    // the group's units lie behind the own ones of its first sequence
    const int64_t lr = (int64_t)max(l.row0[lead + 1] - l.row0[lead], 0) * r.a.R;
    const Cost kl = cost_of<D>(lr);
    const int64_t own = (int64_t)tiles_of(kl, lr) * item_units(kl, own_steps(r.a.c, l.len[lead], it.shared));
    const int64_t i1 = (l.pre[lead] + own) * r.a.c.H + ((int64_t)it.h * tiles + tile) * units;
    run1 = at(k, i1, 0);
    parts1 = at(k, i1, it.shared - 1) - run1 + 1;
    row1 = (int)(gr - (int64_t)tile * k.tile);
  }
  r.s.desc[r.key(rr)] = pack_desc(run0, parts0, (int)(rr - (int64_t)it.tile * it.cost.tile), run1, parts1, row1);
}

// A wave's own rows: to the output if nothing else has a part of them, else to the workspace
template <int D, bool I8, int RT>
__device__ __forceinline__ void store_share(const Share& r, Rows<D, I8, RT>& w, const SharePlan& p, const ShareLds& l, int64_t r0,
                                            int j, int g) {
  if (r.whole) {
    store_rows(r.a, r.q, w, r.it.h, r0, j, g);
  } else {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float sum = groups_sum(w.sum[rt]);
      const int64_t rr = r0 + 16 * rt + j;
      if (rr >= r.q.nrows) continue;
      const int64_t slot = r.slot(rr);
      float* to = r.a.part + slot * D + 4 * g;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) *reinterpret_cast<v4f*>(to + 16 * i) = w.o[rt][i];
      if (g == 0) r.a.stat[slot] = float2{w.mx[rt], sum};
    }
  }
  if (r.first && !r.it.of_group && g == 0) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      if (r0 + 16 * rt + j < r.q.nrows) tell_row<D>(r, p, l, r0 + 16 * rt + j);
  }
}

// 64 RT rows, whose waves share the keys through LDS
template <int D, bool I8, int RT, int S>
__device__ __forceinline__ void take_wide(const Share& r, const SharePlan& p, const ShareLds& l, uint32_t lo, uint32_t hi, uint8_t* smem,
                                          int wv, int lane) {
  const int j = lane & 15, g = lane >> 4;
  const int64_t t0 = (int64_t)r.it.tile * 64 * RT, r0 = t0 + wv * 16 * RT;
  auto steps_to = [&](int64_t row) {
    return (uint32_t)uniform((int)((limit_of(r.a, r.q, (int)(row / r.a.R)) + kTokTile - 1) / kTokTile));
  };
  Rows<D, I8, RT> w;
  w.limits(r.a, r.q, r0, j);
  w.load_q(r.a, r.q, r.it.h, r0, j, g);
  SharedRows<D, I8, RT, S>::run(w, r.a, r.q, r.it.h, lo, min(hi, steps_to(min(t0 + 64 * RT, r.q.nrows) - 1)),
                                r0 < r.q.nrows ? steps_to(min(r0 + 16 * RT, r.q.nrows) - 1) : 0, smem, wv, lane);
  store_share(r, w, p, l, r0, j, g);
}

// 16 rows, whose waves take steps in turn and are joined in LDS
template <int D, bool I8>
struct NarrowLds {
  float o[kAttnWaves][16][D + 4], m[kAttnWaves][16], l[kAttnWaves][16];
};
template <int D, bool I8>
__device__ __forceinline__ void take_narrow(const Share& r, const SharePlan& p, const ShareLds& l, uint32_t lo, uint32_t hi,
                                            NarrowLds<D, I8>& n, int wv, int lane) {
  const int j = lane & 15, g = lane >> 4;
  const int64_t r0 = (int64_t)r.it.tile * 16;
  const uint32_t most = (uint32_t)uniform((int)((limit_of(r.a, r.q, (int)((min(r0 + 16, r.q.nrows) - 1) / r.a.R)) + kTokTile - 1) / kTokTile));
  {
    Rows<D, I8, 1> w;
    w.run(r.a, r.q, r.it.h, r0, lo + wv, min(hi, most), kAttnWaves, j, g);
    const float sum = groups_sum(w.sum[0]);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) *reinterpret_cast<v4f*>(&n.o[wv][j][16 * i + 4 * g]) = w.o[0][i];
    if (g == 0) {
      n.m[wv][j] = w.mx[0];
      n.l[wv][j] = sum;
    }
  }
  __syncthreads();
  // join the waves: 16 threads a row, D / 16 elements each
  constexpr int E = D / 16;
  typedef float vE __attribute__((ext_vector_type(E)));
  const int row = threadIdx.x >> 4, q4 = (threadIdx.x & 15) * E;
  const int64_t rr = r0 + row;
  if (rr < r.q.nrows) {
    float M = n.m[0][row];
#pragma unroll
    for (int x = 1; x < kAttnWaves; ++x) M = fmaxf(M, n.m[x][row]);
    const float Mb = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
    vE v = 0.0f;
#pragma unroll
    for (int x = 0; x < kAttnWaves; ++x) {
      const float wgt = __builtin_amdgcn_exp2f(n.m[x][row] - Mb);
      L += wgt * n.l[x][row];
      v += wgt * *reinterpret_cast<const vE*>(&n.o[x][row][q4]);
    }
    if (r.whole) {
      v *= inverse_sum(L);
      const int64_t key = r.key(rr), hq = r.a.c.H * r.a.R, token = r.q.row0 + (int)rr / r.a.R;
      uint16_t* out = r.a.out + token * r.a.ldo + (key - token * hq) * D + q4;
#pragma unroll
      for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(out + e) = f32_to_bf16_nan(v[e]) | f32_to_bf16_nan(v[e + 1]) << 16;
      if (q4 == 0 && r.a.lse) r.a.lse[key] = log_sum(M, L);
    } else {
      const int64_t slot = r.slot(rr);
      *reinterpret_cast<vE*>(r.a.part + slot * D + q4) = v;
      if (q4 == 0) r.a.stat[slot] = float2{M, L};
    }
    if (q4 == 0 && r.first && !r.it.of_group) tell_row<D>(r, p, l, rr);
  }
  __syncthreads();  // the next item's waves write where this one's were read
}

template <int D, bool I8, int S>
__global__ __launch_bounds__(64 * kAttnWaves, 2) void k_kv_shared(ShareArgs s) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ ShareLds lds;
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const SharePlan plan = make_share_plan<D>(s, lds);
  const int64_t end = min((blockIdx.x + 1) * plan.per, plan.units);
  for (int64_t u = blockIdx.x * plan.per; u < end;) {
    Share r{s, share_item<D>(s, lds, u)};
    const ShareItem& it = r.it;
    const uint32_t from = step_at(it, u - it.i0), to = step_at(it, end - it.i0);
    u = it.i0 + it.units;
    if (from >= to) continue;
    r.a = s.a;
    r.run = blockIdx.x;
    r.first = from == 0;
    r.whole = !it.of_group && it.shared == 0 && from == 0 && to == it.steps;
    r.q.row0 = it.row0;
    r.q.rows = it.rows;
    r.q.nrows = (int64_t)it.rows * s.a.R;
    r.q.len = uniform(lds.len[it.b]);
    r.q.seen = (uint32_t)min((int64_t)max(r.q.len, 0), (int64_t)s.a.c.max_pages * s.a.c.P);
    r.q.table = s.a.c.table + it.b * s.a.c.table_stride;
    uint32_t base = it.shared;
    if (it.of_group) {
      r.q.seen = it.shared * kTokTile;
      r.a.causal = 0;
      base = 0;
    }
    if constexpr (D < 256) {
      if (it.cost.tile == 16) {
        take_narrow<D, I8>(r, plan, lds, base + from, base + to, *reinterpret_cast<NarrowLds<D, I8>*>(smem), wv, lane);
        continue;
      }
      if (it.cost.tile == 128) {
        take_wide<D, I8, 2, S>(r, plan, lds, base + from, base + to, smem, wv, lane);
        continue;
      }
    }
    take_wide<D, I8, 1, S>(r, plan, lds, base + from, base + to, smem, wv, lane);
  }
}

// One workgroup for each row with parts: D / 4 lanes of four columns take a part, 1024 / D parts go
// at a time, and the sums are added in order.
template <int D>
__global__ __launch_bounds__(256) void k_kv_shared_join(ShareArgs s) {
  constexpr int kLanes = D / 4, kAtOnce = 256 / kLanes, kAhead = 4;
  __shared__ float wgt[2 * kMaxParts], red[8];
  __shared__ v4f sums[kAtOnce][kLanes];
  const KvAttnArgs& a = s.a;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  const int64_t hq = (int64_t)a.c.H * a.R, keys = a.c.T * hq;
  const int64_t end = seq_offset(a.c, a.c.B) * hq;
  for (int64_t key = seq_offset(a.c, 0) * hq + blockIdx.x; key < end; key += gridDim.x) {
    const uint4 d = s.desc[key];
    const int parts0 = (int)(d.x >> 16), parts = parts0 + (int)(d.y >> 16);
    if (parts == 0) continue;
    auto slot = [&](int p) __attribute__((always_inline)) {
      const bool own = p < parts0;
      const int k = own ? p : p - parts0;
      if (k == 0) return (own ? 0 : keys) + key;
      const uint32_t run = ((own ? d.x : d.y) & 0xFFFFu) + k, row = own ? d.z & 0xFFFFu : d.z >> 16;
      return 2 * keys + (int64_t)run * a.tile_rows + row;
    };
    // the first parts' sums are on their way while the weights are made
    const int mine = t / kLanes, col = (t % kLanes) * 4;
    v4f v[kAhead];
    auto load = [&](int p0) __attribute__((always_inline)) {
#pragma unroll
      for (int x = 0; x < kAhead; ++x)
        v[x] = *reinterpret_cast<const v4f*>(a.part + slot(min(p0 + x * kAtOnce + mine, parts - 1)) * D + col);
    };
    load(0);
    float M = -INFINITY;
    for (int p = t; p < parts; p += 256) {
      const float m = a.stat[slot(p)].x;
      wgt[p] = m;
      M = fmaxf(M, m);
    }
    M = wave_max(M);
    if (lane == 0) red[wv] = M;
    __syncthreads();
    M = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float Mb = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
    for (int p = t; p < parts; p += 256) {
      const float x = __builtin_amdgcn_exp2f(wgt[p] - Mb);
      wgt[p] = x;
      L += x * a.stat[slot(p)].y;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) L += __shfl_xor(L, o, 64);
    if (lane == 0) red[4 + wv] = L;
    __syncthreads();
    L = (red[4] + red[5]) + (red[6] + red[7]);
    v4f acc{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p0 = 0;;) {
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int p = p0 + x * kAtOnce + mine;
        if (p < parts) acc += wgt[p] * v[x];
      }
      p0 += kAhead * kAtOnce;
      if (p0 >= parts) break;
      load(p0);
    }
    sums[mine][t % kLanes] = acc;
    __syncthreads();
    if (t < kLanes) {
#pragma unroll
      for (int w = 1; w < kAtOnce; ++w) acc += sums[w][t];
      const float inv = inverse_sum(L);
      const int64_t token = key / hq;
      uint16_t* out = a.out + token * a.ldo + (key - token * hq) * D + col;
      *reinterpret_cast<v2u*>(out) = v2u{f32_to_bf16_nan(acc[0] * inv) | f32_to_bf16_nan(acc[1] * inv) << 16,
                                         f32_to_bf16_nan(acc[2] * inv) | f32_to_bf16_nan(acc[3] * inv) << 16};
      if (t == 0 && a.lse) a.lse[key] = log_sum(M, L);
    }
    __syncthreads();  // the next row's weights and sums go where these were
  }
}

// How a call runs.  Sequences of many rows fill row tiles of their own, which read the shared
// tokens once for each: attention as it is does that, with no parts to join.
struct ShareShape {
  bool own;
  int runs, tile, least;
};
ShareShape share_shape(const KvArgs& c, int R, int num_cu) {
  ShareShape s{};
  s.own = c.T * R < 64 * (int64_t)c.B;
  s.runs = (c.D == 256 ? 1 : 2) * num_cu;
  s.tile = c.D == 256 ? 64 : 128;
  s.least = 16;
  return s;
}

template <int D, bool I8>
hipError_t shared_of(ShareArgs s, hipStream_t st) {
  constexpr int S = D == 256 ? 2 : 3;
  constexpr int ring = SharedRows<D, I8, D == 256 ? 1 : 2, S>::kBytes;
  constexpr int lds = ring > (int)sizeof(NarrowLds<D, I8>) || D == 256 ? ring : (int)sizeof(NarrowLds<D, I8>);
  hipError_t e = set_lds_limit(reinterpret_cast<const void*>(k_kv_shared<D, I8, S>), lds);
  if (e != hipSuccess) return e;
  const ShareArgs all = s;
  const int64_t keys = all.a.c.T * all.a.c.H * all.a.R;
  for (int b = 0; b < all.a.c.B; b += kShareSeqs) {  // the launches of one stream use the workspace in turn
    s.a.c.B = min(all.a.c.B - b, kShareSeqs);
    s.a.c.offsets = all.a.c.offsets + b;
    s.a.c.lens = all.a.c.lens + b;
    s.a.c.table = all.a.c.table + b * all.a.c.table_stride;
    s.group = all.group + b;
    s.shared = all.shared + b;
    hipLaunchKernelGGL((k_kv_shared<D, I8, S>), dim3((unsigned)s.a.runs), dim3(64 * kAttnWaves), lds, st, s);
    hipLaunchKernelGGL(k_kv_shared_join<D>, dim3((unsigned)min(keys, (int64_t)1 << 16)), dim3(256), 0, st, s);
  }
  return hipGetLastError();
}

}  // namespace

size_t kv_shared_workspace(const KvArgs& c, int R, int num_cu) {
  const ShareShape s = share_shape(c, R, num_cu);
  if (!s.own) return kv_attention_workspace(c, R, num_cu);
  const size_t keys = (size_t)c.T * c.H * R;
  return (2 * keys + (size_t)s.runs * s.tile) * (c.D * sizeof(float) + sizeof(float2)) + keys * sizeof(uint4);
}

int kv_shared_path(const KvArgs& c, int R, int num_cu) {
  return share_shape(c, R, num_cu).own ? 16 : kv_attention_path(c, R, num_cu);
}

hipError_t launch_kv_attention_shared(KvAttnArgs a, bool i8, const int32_t* group, const int32_t* shared, int num_cu,
                                      void* ws, hipStream_t st) {
  const ShareShape sh = share_shape(a.c, a.R, num_cu);
  if (!sh.own) return launch_kv_attention(a, i8, num_cu, ws, st);
  const size_t keys = (size_t)a.c.T * a.c.H * a.R, slots = 2 * keys + (size_t)sh.runs * sh.tile;
  a.runs = sh.runs;
  a.least = sh.least;
  a.tile_rows = sh.tile;
  ShareArgs s{a, group, shared, static_cast<uint4*>(ws)};
  s.a.part = reinterpret_cast<float*>(s.desc + keys);
  s.a.stat = reinterpret_cast<float2*>(s.a.part + slots * a.c.D);
  if (a.c.D == 64) return i8 ? shared_of<64, true>(s, st) : shared_of<64, false>(s, st);
  if (a.c.D == 128) return i8 ? shared_of<128, true>(s, st) : shared_of<128, false>(s, st);
  return i8 ? shared_of<256, true>(s, st) : shared_of<256, false>(s, st);
}

}  // namespace wq
