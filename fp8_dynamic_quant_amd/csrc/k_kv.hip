// A paged cache of keys and values in 8 bits, and attention over it.
//
// A page holds P tokens of every head, as codes (E4M3, or int8) and one UE8M0 byte for each
// (page, head) of keys and of values: x = code * 2^(byte - 127).  Keys lie [page][H][P][D],
// values [page][H][D][P]: the matrix instruction contracts q k over D and p v over tokens,
// and wants eight consecutive terms of a contraction from each lane, so with this layout both
// come from memory in operand order and nothing is transposed when they are read.
#include "wq_kernels.h"
#include "wq_kv_attn.h"

namespace wq {

namespace {

constexpr int kPlanSeqs = 1024;  // sequences of one launch of runs (their work is summed up in LDS)
constexpr int kMaxRuns = 1024;   // workgroups of one

// ---- append -------------------------------------------------------------------------------

// One workgroup for the new rows of one sequence in one page of one head, keys (side 0) or
// values (side 1): append_rows.
// Latency bounds it where rows are few: the sequence, its page, the page's scale, the codes in turn;
// one token to each of 64 sequences of 8 x 128 heads takes 7.8 us (10.7 with a search by halves and a
// workgroup for every two pages a sequence can touch).  2000 rows to each of three sequences: 12.2 us,
// 24 MB, 2.0 TB/s (15.6 when values were stored a byte at a time and rows read twice).
template <bool I8>
__global__ __launch_bounds__(256) void k_kv_append(KvArgs c, int64_t first_slot, int div, int per_seq, const uint16_t* k_new, int64_t ldk, const uint16_t* v_new,
                                                   int64_t ldv) {
  __shared__ int count[4];
  __shared__ Found told;
  __shared__ uint32_t red[4];
  const int t = threadIdx.x, h = blockIdx.y, side = blockIdx.z;
  const Found s = find_slot_256(c, first_slot + blockIdx.x, div, per_seq, &told, count);
  append_rows<I8>(c, s, h, side, side ? v_new : k_new, side ? ldv : ldk, red);
}

// ---- attention -----------------------------------------------------------------------------

// Many rows: a workgroup takes 64 RT rows of one sequence and cache head over all their keys.  A
// sequence's last rows, which see most, come first.  The arithmetic around the matrix instructions
// bounds it: for each 16 x 16 of scores a lane widens codes, scales, takes maximum, power of two and
// rounding of four, beside 2 x D / 32 instructions of 16 clocks.  Two prompts of 2000 behind 2099, 32
// query heads on 8 of 128: E4M3 255 to 260 us, 630 TFLOP/s of the 1376 that a bf16 product of 8192^3
// reaches (vector instructions 46 % of the SIMDs' cycles, matrix instructions 26 %); int8, whose
// codes take twelve instructions for eight where E4M3's take four, 334 us (57 and 20 %); heads of 64
// 172 / 216 us, of 256 497 / 729.
template <int D, bool I8, int RT, int S>
__global__ __launch_bounds__(64 * kAttnWaves, 2) void k_kv_attention_rows(KvAttnArgs a) {
  using W = SharedRows<D, I8, RT, S>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  constexpr int kRows = 16 * RT * kAttnWaves;
  const uint32_t block = blockIdx.x + (blockIdx.y << kGridXLog);  // < 2^31 + 2^22
  const int h = block % (uint32_t)a.c.H;
  const SeqSlot sl = find_slot(a.c, block / (uint32_t)a.c.H, a.R, kRows, 1);
  const Seq s = seq_of(a, sl.b, sl.row0, max(sl.rows, (int64_t)0));
  const int64_t tiles = (s.nrows + kRows - 1) / kRows;
  if (sl.j >= tiles) return;
  const int64_t t0 = (tiles - 1 - sl.j) * kRows, r0 = t0 + wv * 16 * RT;
  auto steps_to = [&](int64_t row) {
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)((limit_of(a, s, (int)(row / a.R)) + kTokTile - 1) / kTokTile));
  };
  Rows<D, I8, RT> w;
  w.limits(a, s, r0, j);
  w.load_q(a, s, h, r0, j, g);
  W::run(w, a, s, h, 0, steps_to(min(t0 + kRows, s.nrows) - 1),
         r0 < s.nrows ? steps_to(min(r0 + 16 * RT, s.nrows) - 1) : 0, smem, wv, lane);
  store_rows(a, s, w, h, r0, j, g);
}

// Few rows: the work, the 64-token steps of all (sequence, head, row tile) items in a row, is cut
// into equal runs, one for each workgroup, whatever the lengths.  An item also counts `fixed` steps
// for its beginning and end (without them the workgroups that got many short sequences came in
// last: 64 sequences of 700 to 8192 tokens, the median done after 99 us, the last after 138); a cut
// inside those lies in front of the item.  An item that lies in one run is stored; of one that is
// cut the parts go to the workspace, and k_kv_join adds them.  Where a table holds few tokens a run
// is one item, and nothing is cut.
struct Plan {
  int64_t units;  // steps, the fixed ones among them, or items
  int64_t per;    // of a run
  int runs;       // workgroups that take some
};
struct PlanLds {
  int64_t pre[kPlanSeqs + 1];  // units of the sequences before b, for one head
  int row0[kPlanSeqs + 1];     // their rows
  int len[kPlanSeqs];
  int64_t carry[kAttnWaves];
};
__device__ __forceinline__ uint32_t units_of(const KvAttnArgs& a, uint32_t steps) { return a.cut ? steps + a.fixed : 1; }
// Every thread of the workgroup takes part.
template <int kRows>
__device__ __forceinline__ Plan make_plan(const KvAttnArgs& a, PlanLds& l) {
  const KvArgs& c = a.c;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  constexpr int kThreads = 64 * kAttnWaves;
  int64_t before = 0;
  for (int b0 = 0; b0 < c.B; b0 += kThreads) {
    const int b = b0 + t;
    int64_t v = 0;
    if (b < c.B) {
      const int64_t lo = seq_offset(c, b), rows = max(seq_offset(c, b + 1) - lo, (int64_t)0);
      const int len = c.lens[b];
      v = (rows * a.R + kRows - 1) / kRows * units_of(a, steps_of(c, len));
      l.row0[b] = (int)lo;
      l.len[b] = len;
      if (b == c.B - 1) l.row0[c.B] = (int)(lo + rows);
    }
    if (b0 + wv * 64 < c.B) {
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int64_t u = __shfl_up(v, o, 64);
        if (lane >= o) v += u;
      }
    }
    if (lane == 63) l.carry[wv] = v;
    __syncthreads();
    int64_t base = before;
    for (int w = 0; w < wv; ++w) base += l.carry[w];
    if (b < c.B) l.pre[b + 1] = base + v;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) before += l.carry[w];
    if (b == 0) l.pre[0] = 0;
    __syncthreads();
  }
  Plan p;
  p.units = before * c.H;
  p.per = max(quotient(p.units + a.runs - 1, a.runs), (int64_t)a.least);
  p.runs = (int)quotient(p.units + p.per - 1, p.per);
  return p;
}
struct Item {
  int b, h, tile;
  uint32_t steps, step;  // of the item; where the unit is in it
  int64_t i0;            // its first unit
};
__device__ __forceinline__ Item item_of(const KvAttnArgs& a, const PlanLds& l, int64_t u) {
  const KvArgs& c = a.c;
  int lo = 0, hi = c.B - 1;
  while (lo < hi) {  // the last sequence that begins at or before u (of equal ones the one with work)
    const int mid = (lo + hi + 1) >> 1;
    if (l.pre[mid] * c.H <= u) lo = mid;
    else hi = mid - 1;
  }
  Item it;
  lo = uniform(lo);
  it.b = lo;
  it.steps = (uint32_t)uniform((int)steps_of(c, l.len[lo]));
  const uint32_t units = units_of(a, it.steps);
  const int64_t first = l.pre[lo] * c.H;
  const int64_t item = quotient(u - first, units);
  it.i0 = first + item * units;
  const int64_t in = u - it.i0;
  it.step = a.cut && in > a.fixed ? (uint32_t)uniform((int)(in - a.fixed)) : 0u;
  const int64_t tiles = quotient(l.pre[lo + 1] - l.pre[lo], units);
  it.h = uniform((int)quotient(item, tiles));
  it.tile = uniform((int)(item - it.h * tiles));
  return it;
}
__device__ __forceinline__ Seq seq_of(const KvAttnArgs& a, const PlanLds& l, int b) {
  Seq s;
  s.row0 = uniform(l.row0[b]);
  s.rows = uniform(l.row0[b + 1]) - (int)s.row0;
  s.nrows = (int64_t)s.rows * a.R;
  s.len = uniform(l.len[b]);
  s.seen = (uint32_t)min((int64_t)max(s.len, 0), (int64_t)a.c.max_pages * a.c.P);
  s.table = a.c.table + b * a.c.table_stride;
  return s;
}
// A run's share of an item, and where its part goes
struct Run {
  Item it;
  uint32_t n;    // steps of it: 0 behind the run's last
  bool whole;
  int64_t slot;  // first row of its part in the workspace
};
__device__ __forceinline__ Run next_run(const KvAttnArgs& a, const PlanLds& l, int64_t u, int64_t end, int part, int krows) {
  Run r;
  r.it = item_of(a, l, u);
  const int64_t to = a.cut ? min(max(end - r.it.i0 - a.fixed, (int64_t)0), (int64_t)r.it.steps) : (int64_t)r.it.steps;
  r.n = (uint32_t)uniform((int)max(to - (int64_t)r.it.step, (int64_t)0));
  r.whole = r.n == r.it.steps;
  r.slot = ((int64_t)blockIdx.x * 2 + part) * krows;
  return r;
}
// What k_kv_join needs of the item that run w begins inside, if it is the first run to do so
// (parts = 0 otherwise): it stands for the item.
__device__ __forceinline__ void tell_join(const KvAttnArgs& a, const Plan& p, const PlanLds& l, int w) {
  if (threadIdx.x != 0) return;
  KvJoin d{};
  if (w > 0 && w < p.runs) {
    const Item it = item_of(a, l, w * p.per);
    const int64_t before = (w - 1) * p.per;
    if (it.step > 0 && before <= it.i0 + a.fixed) {
      const int last = (int)quotient(it.i0 + a.fixed + it.steps - 1, p.per);  // the last run that begins in it
      d.parts = last - w + 2;
      d.first_slot = 2 * (w - 1) + (before < it.i0 ? 1 : 0);  // its second part if the item begins inside it
      d.h = it.h;
      d.tile = it.tile;
      d.row0 = l.row0[it.b];
      d.rows = l.row0[it.b + 1] - d.row0;
    }
  }
  a.joins[w] = d;
}

// 64-row tiles, each wave 16 rows of its own, keys shared through LDS.  64 rows over 131072 tokens of
// one head of 256: 33 us and 8 for the join, a third of the rate at which the codes could be read: a
// CU has one run of eight steps, whose loads, widening and matrix instructions wait for each other.
template <int D, bool I8, int S>
__global__ __launch_bounds__(64 * kAttnWaves, 2) void k_kv_attention_runs64(KvAttnArgs a) {
  using W = SharedRows<D, I8, 1, S>;
  constexpr int kRows = 64;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ PlanLds plan_lds;
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const Plan plan = make_plan<kRows>(a, plan_lds);
  if (a.cut) tell_join(a, plan, plan_lds, blockIdx.x);
  if ((int)blockIdx.x >= plan.runs) return;
  int64_t u = blockIdx.x * plan.per;
  const int64_t end = min(u + plan.per, plan.units);
  for (int part = 0; u < end; part = 1) {
    const Run r = next_run(a, plan_lds, u, end, part, kRows);
    if (r.n == 0) break;
    u = r.it.i0 + units_of(a, r.it.steps);
    const Seq s = seq_of(a, plan_lds, r.it.b);
    const int64_t t0 = (int64_t)r.it.tile * kRows, r0 = t0 + wv * 16;
    auto steps_to = [&](int64_t row) {
      return (uint32_t)__builtin_amdgcn_readfirstlane((int)((limit_of(a, s, (int)(row / a.R)) + kTokTile - 1) / kTokTile));
    };
    Rows<D, I8, 1> w;
    w.limits(a, s, r0, j);
    w.load_q(a, s, r.it.h, r0, j, g);
    W::run(w, a, s, r.it.h, r.it.step, min(r.it.step + r.n, steps_to(min(t0 + kRows, s.nrows) - 1)),
           r0 < s.nrows ? steps_to(min(r0 + 16, s.nrows) - 1) : 0, smem, wv, lane);
    if (r.whole) {
      store_rows(a, s, w, r.it.h, r0, j, g);
    } else {
      const float l = groups_sum(w.sum[0]);
      float* to = a.part + (r.slot + wv * 16 + j) * D + 4 * g;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) *reinterpret_cast<v4f*>(to + 16 * i) = w.o[0][i];
      if (g == 0) a.stat[r.slot + wv * 16 + j] = float2{w.mx[0], l};
    }
  }
}

// 16-row tiles: the waves share the rows and take steps in turn, and are joined in LDS.  Reading the
// cache bounds it: 64 sequences of 8192 tokens, int8, 8 heads of 128, 584 MB in 123 us, 4.75 TB/s
// with the joins; one sequence of 1000 takes 12.5 us, latencies of plan, page numbers and codes.
template <int D, bool I8>
__global__ __launch_bounds__(64 * kAttnWaves, 2) void k_kv_attention_runs16(KvAttnArgs a) {
  constexpr int kRows = 16;
  __shared__ float o_lds[kAttnWaves][kRows][D + 4];
  __shared__ float m_lds[kAttnWaves][kRows], l_lds[kAttnWaves][kRows];
  __shared__ PlanLds plan_lds;
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const Plan plan = make_plan<kRows>(a, plan_lds);
  if (a.cut) tell_join(a, plan, plan_lds, blockIdx.x);
  if ((int)blockIdx.x >= plan.runs) return;
  int64_t u = blockIdx.x * plan.per;
  const int64_t end = min(u + plan.per, plan.units);
  for (int part = 0; u < end; part = 1) {
    const Run r = next_run(a, plan_lds, u, end, part, kRows);
    if (r.n == 0) break;
    u = r.it.i0 + units_of(a, r.it.steps);
    const Seq s = seq_of(a, plan_lds, r.it.b);
    const int64_t r0 = (int64_t)r.it.tile * kRows;
    const uint32_t most = __builtin_amdgcn_readfirstlane(
        (int)((limit_of(a, s, (int)((min(r0 + kRows, s.nrows) - 1) / a.R)) + kTokTile - 1) / kTokTile));
    Rows<D, I8, 1> w;
    w.run(a, s, r.it.h, r0, r.it.step + wv, min(r.it.step + r.n, most), kAttnWaves, j, g);
    const float l = groups_sum(w.sum[0]);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) *reinterpret_cast<v4f*>(&o_lds[wv][j][16 * i + 4 * g]) = w.o[0][i];
    if (g == 0) {
      m_lds[wv][j] = w.mx[0];
      l_lds[wv][j] = l;
    }
    __syncthreads();
    // join the waves: 16 threads a row, D / 16 elements each
    constexpr int E = D / 16;
    typedef float vE __attribute__((ext_vector_type(E)));
    const int row = threadIdx.x >> 4, q4 = (threadIdx.x & 15) * E;
    const int64_t rr = r0 + row;
    if (rr < s.nrows) {
      float M = m_lds[0][row];
#pragma unroll
      for (int x = 1; x < kAttnWaves; ++x) M = fmaxf(M, m_lds[x][row]);
      const float Mb = M == -INFINITY ? 0.0f : M;
      float L = 0.0f, wgt[kAttnWaves];
#pragma unroll
      for (int x = 0; x < kAttnWaves; ++x) {
        wgt[x] = __builtin_amdgcn_exp2f(m_lds[x][row] - Mb);
        L += wgt[x] * l_lds[x][row];
      }
      const float inv = inverse_sum(L);
      const int i = (int)rr / a.R, head = r.it.h * a.R + (int)rr % a.R;
      vE v = 0.0f;
#pragma unroll
      for (int x = 0; x < kAttnWaves; ++x) v += wgt[x] * *reinterpret_cast<const vE*>(&o_lds[x][row][q4]);
      if (r.whole) {
        v *= inv;
        uint16_t* out = a.out + (s.row0 + i) * a.ldo + (int64_t)head * D + q4;
#pragma unroll
        for (int e = 0; e < E; e += 2)
          *reinterpret_cast<uint32_t*>(out + e) = f32_to_bf16_nan(v[e]) | f32_to_bf16_nan(v[e + 1]) << 16;
      } else {
        *reinterpret_cast<vE*>(a.part + (r.slot + row) * D + q4) = v;
      }
      if (q4 == 0) {
        if (!r.whole) a.stat[r.slot + row] = float2{M, L};
        else if (a.lse) a.lse[(s.row0 + i) * (int64_t)(a.c.H * a.R) + head] = log_sum(M, L);
      }
    }
    __syncthreads();  // the next item's waves write where this one's were read
  }
}

// The items that runs cut: the parts of one row, weighted by their maxima, over the weighted sum.
struct JoinRow {
  const KvAttnArgs& a;
  KvJoin d;
  int run, row;  // the run that stands for the item; row of the tile
  __device__ __forceinline__ int64_t tile_row() const { return (int64_t)d.tile * a.tile_rows + row; }
  __device__ __forceinline__ bool there() const { return d.parts > 0 && tile_row() < (int64_t)d.rows * a.R; }
  __device__ __forceinline__ int64_t slot(int p) const {
    return (int64_t)(p == 0 ? d.first_slot : 2 * (run - 1 + p)) * a.tile_rows + row;
  }
  // the parts' weights into LDS, their maximum and the sum, by W waves
  template <int W>
  __device__ __forceinline__ float2 weigh(float* wgt, float* red) const {
    const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
    float M = -INFINITY;
    for (int p = t; p < d.parts; p += 64 * W) {
      const float m = a.stat[slot(p)].x;
      wgt[p] = m;
      M = fmaxf(M, m);
    }
    M = wave_max(M);
    if constexpr (W > 1) {
      if (lane == 0) red[wv] = M;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, red[w]);
      __syncthreads();
    }
    const float Mb = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
    for (int p = t; p < d.parts; p += 64 * W) {
      const float x = __builtin_amdgcn_exp2f(wgt[p] - Mb);
      wgt[p] = x;
      L += x * a.stat[slot(p)].y;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) L += __shfl_xor(L, o, 64);
    if (lane == 0) red[wv] = L;
    __syncthreads();
    L = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) L += red[w];
    return float2{M, L};
  }
  __device__ __forceinline__ int64_t token() const { return (int64_t)d.row0 + (int)tile_row() / a.R; }
  __device__ __forceinline__ int head() const { return d.h * a.R + (int)tile_row() % a.R; }
  __device__ __forceinline__ void store_lse(float2 ml) const {
    if (threadIdx.x == 0 && a.lse) a.lse[token() * (int64_t)(a.c.H * a.R) + head()] = log_sum(ml.x, ml.y);
  }
};

// Few parts to an item: one wave for each (run, row), which goes over the parts in order.
template <int D>
__global__ __launch_bounds__(64) void k_kv_join(KvAttnArgs a) {
  constexpr int kAhead = 8, E = D / 64;  // parts in flight; elements of a lane
  __shared__ float wgt[kMaxRuns + 1], red[1];
  const JoinRow r{a, a.joins[blockIdx.x + 1], (int)blockIdx.x + 1, (int)blockIdx.y};
  if (!r.there()) return;
  const int lane = threadIdx.x;
  const float2 ml = r.template weigh<1>(wgt, red);
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
  for (int p0 = 0; p0 < r.d.parts; p0 += kAhead) {
    float v[kAhead][E];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const float* from = a.part + r.slot(min(p0 + x, r.d.parts - 1)) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) v[x][e] = from[e];
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x)
      if (p0 + x < r.d.parts) {
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += wgt[p0 + x] * v[x][e];
      }
  }
  const float inv = inverse_sum(ml.y);
  uint16_t* out = a.out + r.token() * a.ldo + (int64_t)r.head() * D;
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane * E + e] = (uint16_t)f32_to_bf16_nan(acc[e] * inv);
  r.store_lse(ml);
}

// Many parts to an item: blockIdx.x counts the items that were cut, blockIdx.y rows, blockIdx.z
// slices of 64 columns.  16 lanes of four columns take a part, 16 parts go at a time, and the 16
// sums are added in order.
template <int D>
__global__ __launch_bounds__(256) void k_kv_join_wide(KvAttnArgs a) {
  constexpr int kAhead = 8;
  __shared__ float wgt[kMaxRuns + 1], red[4];
  __shared__ v4f sums[16][16];
  __shared__ int count[4], found;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  if (t == 0) found = 0;
  int before = 0;
  for (int w0 = 1; w0 < a.runs; w0 += 256) {  // the blockIdx.x-th run that stands for an item
    const bool one = w0 + t < a.runs && a.joins[w0 + t].parts > 0;
    const uint64_t votes = __ballot(one);
    if (lane == 0) count[wv] = __popcll(votes);
    __syncthreads();
    int rank = before + __popcll(votes & (((uint64_t)1 << lane) - 1));
    for (int w = 0; w < wv; ++w) rank += count[w];
    if (one && rank == (int)blockIdx.x) found = w0 + t;
    before += count[0] + count[1] + count[2] + count[3];
    __syncthreads();
  }
  if (before <= (int)blockIdx.x) return;
  const JoinRow r{a, a.joins[found], found, (int)blockIdx.y};
  if (!r.there()) return;
  const float2 ml = r.template weigh<4>(wgt, red);
  const int col = blockIdx.z * 64 + (t & 15) * 4, mine = t >> 4;
  v4f acc{0.0f, 0.0f, 0.0f, 0.0f};
  for (int p0 = mine; p0 < r.d.parts; p0 += 16 * kAhead) {
    v4f v[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x)
      v[x] = *reinterpret_cast<const v4f*>(a.part + r.slot(min(p0 + 16 * x, r.d.parts - 1)) * D + col);
#pragma unroll
    for (int x = 0; x < kAhead; ++x)
      if (p0 + 16 * x < r.d.parts) acc += wgt[p0 + 16 * x] * v[x];
  }
  sums[mine][t & 15] = acc;
  __syncthreads();
  if (t < 16) {
    for (int w = 1; w < 16; ++w) acc += sums[w][t];
    const float inv = inverse_sum(ml.y);
    uint16_t* out = a.out + r.token() * a.ldo + (int64_t)r.head() * D + col;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = (uint16_t)f32_to_bf16_nan(acc[e] * inv);
  }
  if (blockIdx.z == 0) r.store_lse(ml);
}

}  // namespace

hipError_t launch_kv_append(const KvArgs& c, bool i8, const uint16_t* k_new, int64_t ldk, const uint16_t* v_new,
                            int64_t ldv, hipStream_t st) {
  // rows / P + 2 pages hold a sequence's rows, and no more than its rows: the host knows the sums only
  const int64_t by_pages = c.T / c.P + 2 * (int64_t)c.B;
  const bool by_rows = c.T <= by_pages;
  const int div = by_rows ? 1 : c.P, per = by_rows ? 0 : 2;
  const int64_t slots = by_rows ? c.T : by_pages;
  for (int64_t first = 0; first < slots; first += kGridX) {
    const dim3 grid((unsigned)min(slots - first, (int64_t)kGridX), (unsigned)c.H, 2);
    if (i8)
      hipLaunchKernelGGL(k_kv_append<true>, grid, dim3(256), 0, st, c, first, div, per, k_new, ldk, v_new, ldv);
    else
      hipLaunchKernelGGL(k_kv_append<false>, grid, dim3(256), 0, st, c, first, div, per, k_new, ldk, v_new, ldv);
  }
  return hipGetLastError();
}

bool kv_head_dim_ok(int64_t D) { return D == 64 || D == 128 || D == 256; }

namespace {

constexpr size_t kJoinBytes = 64u << 20;

// How a call runs: row tiles of `rows` rows, whole (many rows), or in equal runs of the work.
struct Shape {
  bool whole;
  int rows, runs, least, cut, fixed, items;
  bool wide_join;
};

int rows_of_whole(int D) { return D == 256 ? 64 : 128; }

Shape shape_of(const KvArgs& c, int R, int num_cu) {
  Shape s{};
  const int big = rows_of_whole(c.D);
  const int64_t cap = ((int64_t)c.max_pages * c.P + kTokTile - 1) / kTokTile;  // steps of the longest sequence
  // 16-row tiles for sequences that have no more on average (16 against 64: one token of a sequence of
  // 1000, 12.5 / 16.1 us; of each of 64 of 8192, 123 / 158), where the registers hold a head
  const int64_t avg = (c.T * R + c.B - 1) / c.B;
  s.rows = avg <= 16 && c.D < 256 ? 16 : 64;
  // Whole row tiles once they fill the chip (runs against whole tiles, us, 8 heads of 128, R = 4: at a
  // tile a CU 1024 rows over 2048 tokens 84 / 70, over 16384 501 / 456; at half of that, 512 rows,
  // over 2048 61 / 67, over 16384 283 / 449).  Single tokens leave most of such a tile empty and stay
  // with 16-row tiles, unless their tables are short or they need many launches (16-row against
  // whole tiles: 256 sequences of 2000, R = 16, 134 / 200, of 300 53 / 60; 1024 of 4000, R = 4, 826 / 1129,
  // of 600 267 / 271, of 400 241 / 221; 3000 of 4000 2358 / 3179; 4096 of 1000 1495 / 1448).  Of more
  // rows than sequences the host does not know whose they are: four tokens to each of 512 sequences
  // of 2000 take 258 / 354, but a prompt of 4000 among 3000 single tokens over 1000 1915 / 1762.
  const bool singles = s.rows == 16 && c.T <= c.B && cap > 8 && c.B <= 4 * kPlanSeqs;
  if (c.T * R / big * c.H >= num_cu && !singles) {
    s.whole = true;
    s.rows = big;
    return s;
  }
  const int64_t B = min((int64_t)c.B, (int64_t)kPlanSeqs);
  const int64_t items = (c.T * R / s.rows + B) * c.H;
  // a sequence of few steps is not worth cutting: a run is an item then.  Heads of 256 get one run a
  // CU: two workgroups' rings and plans (84,528 bytes each) do not fit a CU's LDS together, and a
  // second run would wait for the first (131072 tokens, 64 rows: 56 us with two runs a CU, 43 with
  // one; 8 sequences of 9000: 73 / 56)
  s.cut = cap > (s.rows == 16 ? 4 * kAttnWaves : 8);
  s.least = !s.cut ? 1 : s.rows == 16 ? 2 * kAttnWaves : 4;
  s.fixed = s.rows == 16 ? 2 * kAttnWaves : 4;
  const int most = (int)min((int64_t)min(kMaxRuns, (c.D == 256 ? 1 : 2) * num_cu), (int64_t)(kJoinBytes / ((size_t)2 * s.rows * (c.D * 4 + 8) + sizeof(KvJoin))));
  if (!s.cut) {
    s.runs = (int)min(items, (int64_t)kGridX);  // of more, a run takes several
  } else {
    s.runs = (int)min((int64_t)most, (items * (cap + s.fixed) + s.least - 1) / s.least);
    s.wide_join = items * 8 < s.runs;  // many parts to an item
    s.items = (int)min(items, (int64_t)s.runs);
  }
  return s;
}

template <int D, bool I8>
hipError_t attention_of(KvAttnArgs a, const Shape& s, hipStream_t st) {
  const dim3 block(64 * kAttnWaves);
  constexpr int S = D == 256 ? 2 : 3;
  if (s.whole) {
    constexpr int RT = D == 256 ? 1 : 2;
    const int64_t tiles = a.c.T * a.R / (16 * RT * kAttnWaves) + a.c.B;
    constexpr int lds = SharedRows<D, I8, RT, S>::kBytes;
    hipError_t e = set_lds_limit(reinterpret_cast<const void*>(k_kv_attention_rows<D, I8, RT, S>), lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_kv_attention_rows<D, I8, RT, S>), folded_grid(tiles * a.c.H), block, lds, st, a);
    return hipGetLastError();
  }
  const KvAttnArgs all = a;
  for (int b = 0; b < all.c.B; b += kPlanSeqs) {  // the launches of one stream use the workspace in turn
    a.c.B = min(all.c.B - b, kPlanSeqs);
    a.c.offsets = all.c.offsets + b;
    a.c.lens = all.c.lens + b;
    a.c.table = all.c.table + b * all.c.table_stride;
    if (s.rows == 16) {
      // (a head of 256 elements does not fit the registers that leave two waves to a SIMD)
      if constexpr (D < 256)
        hipLaunchKernelGGL((k_kv_attention_runs16<D, I8>), dim3((unsigned)s.runs), dim3(64 * kAttnWaves), 0, st, a);
    } else {
      constexpr int lds = SharedRows<D, I8, 1, S>::kBytes;
      hipError_t e = set_lds_limit(reinterpret_cast<const void*>(k_kv_attention_runs64<D, I8, S>), lds);
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL((k_kv_attention_runs64<D, I8, S>), dim3((unsigned)s.runs), block, lds, st, a);
    }
    if (s.cut && s.runs > 1) {
      const dim3 grid((unsigned)(s.runs - 1), (unsigned)s.rows);
      if (s.wide_join)
        hipLaunchKernelGGL(k_kv_join_wide<D>, dim3((unsigned)s.items, (unsigned)s.rows, D / 64), dim3(256), 0, st, a);
      else
        hipLaunchKernelGGL(k_kv_join<D>, grid, dim3(64), 0, st, a);
    }
  }
  return hipGetLastError();
}

}  // namespace

size_t kv_attention_workspace(const KvArgs& c, int R, int num_cu) {
  const Shape s = shape_of(c, R, num_cu);
  return s.cut ? (size_t)s.runs * ((size_t)2 * s.rows * (c.D * 4 + 8) + sizeof(KvJoin)) : 0;
}

int kv_attention_path(const KvArgs& c, int R, int num_cu) {
  const Shape s = shape_of(c, R, num_cu);
  return s.whole ? 1 : (s.cut ? 4 : 2) + (s.rows == 64) + (s.wide_join ? 8 : 0);
}

hipError_t launch_kv_attention(KvAttnArgs a, bool i8, int num_cu, void* ws, hipStream_t st) {
  const Shape s = shape_of(a.c, a.R, num_cu);
  a.runs = s.runs;
  a.least = s.least;
  a.cut = s.cut;
  a.fixed = s.fixed;
  a.tile_rows = s.rows;
  if (s.cut) {
    const size_t slots = (size_t)2 * s.runs * s.rows;
    a.part = static_cast<float*>(ws);
    a.stat = reinterpret_cast<float2*>(a.part + slots * a.c.D);
    a.joins = reinterpret_cast<KvJoin*>(a.stat + slots);
  }
  if (a.c.D == 64) return i8 ? attention_of<64, true>(a, s, st) : attention_of<64, false>(a, s, st);
  if (a.c.D == 128) return i8 ? attention_of<128, true>(a, s, st) : attention_of<128, false>(a, s, st);
  return i8 ? attention_of<256, true>(a, s, st) : attention_of<256, false>(a, s, st);
}

}  // namespace wq
