// Rows appended to the paged 8-bit cache with their keys turned by position on the way, and the
// queries of the same rows turned.
//
// Elements (a, b) of a pair at a position whose angle has cosine c and sine s become
//   (a c - b s, b c + a s)
// in 32 bits: two products, each rounded, and their sum.  Keys go from there to their 8-bit codes
// with no rounding between; queries are rounded once to bf16, what attention takes.
//
// One launch for all three.  3900 rows (2000, 1300 and 600) of 32 heads on 8 of 128, int8: 23.8 to 25.4 us with
// pages of 32 tokens, 20.1 of 64 (3.5 to 3.8 and 4.5 TB/s read and written; a copy 5.2), where values leave
// in words of four tokens; a token of one sequence 5.6, of 64 sequences 7.6: the launch, and offsets, length, page number, rows
// and the old scale in turn.
#include "wq_kv_device.h"
#include "wq_layer.h"

namespace wq {

namespace {

// Exponent of a block with the largest magnitude a (a finite f32 pattern): the smallest e with
// 2^e >= a / c, at least -127.  c = 448 = 1.75 * 2^8 (E4M3), 127 = 1.984375 * 2^6 (int8).
template <bool I8>
__device__ __forceinline__ int block_exp32(uint32_t a) {
  const int E = (int)(a >> 23);
  const uint32_t F = a & 0x7FFFFFu;
  return max(I8 ? E - 133 + (F > 0x7E0000u ? 1 : 0) : E - 135 + (F > 0x600000u ? 1 : 0), -127);
}

// A unit is two pieces of eight elements of one head: of the turned elements the two that hold both
// of each pair (halves: eight of either half; neighbours: sixteen in a row), behind them any two.
// Its angles are eight consecutive frequencies in either case.
struct Unit {
  int at0, at1;  // first elements of the pieces
  bool turns;
};
template <bool PAIRS>
__device__ __forceinline__ Unit unit_of(int i, int rot) {
  if (PAIRS || 16 * i >= rot) return Unit{16 * i, 16 * i + 8, 16 * i < rot};
  return Unit{8 * i, 8 * i + rot / 2, true};
}
// the pieces, and where they are turned the angles of position pos: NaN outside the table
template <bool PAIRS>
struct Turned {
  v4u x0, x1;
  v4f c[2], s[2];
  __device__ __forceinline__ void load(const uint16_t* x, const Unit& u, int i, const TurnArgs& r, int64_t pos) {
    pieces(x, u);
    angles(u, i, r, pos);
  }
  __device__ __forceinline__ void pieces(const uint16_t* x, const Unit& u) {
    x0 = *reinterpret_cast<const v4u*>(x + u.at0);
    x1 = *reinterpret_cast<const v4u*>(x + u.at1);
  }
  __device__ __forceinline__ void angles(const Unit& u, int i, const TurnArgs& r, int64_t pos) {
    const float nan = __uint_as_float(0x7FC00000u);
    c[0] = c[1] = v4f{nan, nan, nan, nan};
    s[0] = s[1] = c[0];
    if (u.turns && (uint64_t)pos < (uint64_t)r.positions) {
      const float* at = r.angles + pos * r.rot + 8 * i;
      c[0] = *reinterpret_cast<const v4f*>(at);
      c[1] = *reinterpret_cast<const v4f*>(at + 4);
      s[0] = *reinterpret_cast<const v4f*>(at + r.rot / 2);
      s[1] = *reinterpret_cast<const v4f*>(at + r.rot / 2 + 4);
    }
  }
  __device__ __forceinline__ void values(const Unit& u, float (&y0)[8], float (&y1)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y0[e] = half_of(x0, e);
      y1[e] = half_of(x1, e);
    }
    if (!u.turns) return;
    auto turn = [](float& a, float& b, float cc, float ss) __attribute__((always_inline)) {
      const float t = __fsub_rn(__fmul_rn(a, cc), __fmul_rn(b, ss));
      b = __fadd_rn(__fmul_rn(b, cc), __fmul_rn(a, ss));
      a = t;
    };
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (PAIRS) turn(e < 4 ? y0[2 * e] : y1[2 * e - 8], e < 4 ? y0[2 * e + 1] : y1[2 * e - 7], c[e >> 2][e & 3], s[e >> 2][e & 3]);
      else turn(y0[e], y1[e], c[e >> 2][e & 3], s[e >> 2][e & 3]);
    }
  }
};

// The new keys of one sequence (s) in one page of one head, by a workgroup of 256: two units a
// thread and round, the first round's values held between the two passes (the largest magnitude,
// the codes).
template <bool I8, bool PAIRS>
__device__ __forceinline__ void append_turned(const KvArgs& c, const Found& s, int h, const uint16_t* rows, int64_t ld,
                                              const TurnArgs& tr, uint32_t* red) {
  if (s.rows <= 0) return;
  const int t = threadIdx.x;
  const int64_t len = s.len, start = len - s.rows;
  const int64_t pg = max(start, (int64_t)0) / c.P + s.j;
  const int64_t lo = max(start, pg * c.P), hi = min(len, (pg + 1) * c.P);
  if (lo >= hi || pg >= c.max_pages) return;
  const int page = c.table[s.b * c.table_stride + pg];
  const int D = c.D, P = c.P, s0 = (int)(lo - pg * P), n = (int)(hi - lo), per = D / 16, units = n * per;
  const uint16_t* x = rows + (s.row0 + (lo - start)) * ld + (int64_t)h * D;
  constexpr int kUnits = 2;
  struct Share {
    float y[kUnits][2][8];
  };
  auto load = [&](int k, Share& v) __attribute__((always_inline)) {
    Turned<PAIRS> w[kUnits];
    Unit u[kUnits];
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
      const int i = min((k * kUnits + e) * 256 + t, units - 1), r = i / per;
      u[e] = unit_of<PAIRS>(i - r * per, tr.rot);
      w[e].load(x + r * ld, u[e], i - r * per, tr, lo + r);
    }
#pragma unroll
    for (int e = 0; e < kUnits; ++e) w[e].values(u[e], v.y[e][0], v.y[e][1]);
  };
  const int rounds = (units + 256 * kUnits - 1) / (256 * kUnits);
  Share first;
  load(0, first);
  if (page < 0 || page >= c.pages) return;
  uint8_t* scale = c.k_scale + (int64_t)page * c.H + h;
  const int old = s0 > 0 ? *scale : 0;
  uint32_t a = 0;
  auto largest = [&](const Share& v) __attribute__((always_inline)) {  // (units past the last repeat it)
#pragma unroll
    for (int e = 0; e < kUnits; ++e)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(v.y[e][p][j]) & 0x7FFFFFFFu);
  };
  largest(first);
  for (int k = 1; k < rounds; ++k) {
    Share v;
    load(k, v);
    largest(v);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) a = max(a, (uint32_t)__shfl_xor((int)a, o, 64));
  if ((t & 63) == 0) red[t >> 6] = a;
  __syncthreads();  // and every thread has read the old byte
  a = max(max(red[0], red[1]), max(red[2], red[3]));
  const int byte = max(old, a < 0x7F800000u ? block_exp32<I8>(a) + 127 : 255);
  if (t == 0) *scale = (uint8_t)byte;
  uint8_t* codes = static_cast<uint8_t*>(c.k) + ((int64_t)page * c.H + h) * P * D;
  if (s0 > 0 && old < byte && byte != 255) {
    for (int i = t; i < s0 * D; i += 256) codes[i] = (uint8_t)rescale<I8>(codes[i], old - byte);
  }
  const float f = byte == 255 ? 0.0f : ldexpf(1.0f, 127 - byte);  // a power of two: products are exact
  auto store = [&](int k, const Share& v) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
      const int i = (k * kUnits + e) * 256 + t;
      if (i >= units) continue;
      const int r = i / per;
      const Unit u = unit_of<PAIRS>(i - r * per, tr.rot);
      uint8_t* to = codes + (s0 + r) * D;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float* y = v.y[e][p];
        v2u w{0u, 0u};  // NaN and infinities: codes of zero
        if (byte != 255)
          w = v2u{encode4<I8>(y[0] * f, y[1] * f, y[2] * f, y[3] * f), encode4<I8>(y[4] * f, y[5] * f, y[6] * f, y[7] * f)};
        *reinterpret_cast<v2u*>(to + (p ? u.at1 : u.at0)) = w;
      }
    }
  };
  store(0, first);
  for (int k = 1; k < rounds; ++k) {
    Share v;
    load(k, v);
    store(k, v);
  }
}

// The queries of heads h R .. h R + R - 1 of rows from row0 on; pos[r] their positions, none: a row of
// no sequence, left as it is.  A thread reads both pieces of a unit before it writes them, so
// that the rows may be turned in place.
constexpr int kNoRow = INT32_MIN;
template <bool PAIRS>
__device__ __forceinline__ void store_turned(const Turned<PAIRS>& w, const Unit& u, uint16_t* to) {
  float y0[8], y1[8];
  w.values(u, y0, y1);
  auto pack = [](const float (&y)[8]) __attribute__((always_inline)) {
    v4u o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = f32_to_bf16_nan(y[2 * e]) | f32_to_bf16_nan(y[2 * e + 1]) << 16;
    return o;
  };
  *reinterpret_cast<v4u*>(to + u.at0) = pack(y0);
  *reinterpret_cast<v4u*>(to + u.at1) = pack(y1);
}
// of one row, a thread a unit of a head
template <bool PAIRS>
__device__ __forceinline__ void turn_row(const KvArgs& c, int64_t row, int h, const TurnArgs& tr, int64_t pos) {
  const int per = c.D / 16;
  for (int i = threadIdx.x; i < tr.R * per; i += 256) {
    const int head = i / per, at = i - head * per;
    const int64_t col = ((int64_t)h * tr.R + head) * c.D;
    const Unit u = unit_of<PAIRS>(at, tr.rot);
    Turned<PAIRS> w;
    w.load(tr.q + row * tr.ldq + col, u, at, tr, pos);
    store_turned(w, u, tr.q_out + row * tr.ldo + col);
  }
}
// of many, a thread a unit of kHeads heads, whose angles are the same
constexpr int kHeads = 4;
template <bool PAIRS>
__device__ __forceinline__ void turn_rows(const KvArgs& c, int64_t row0, int n, int h, const TurnArgs& tr, const int* pos) {
  const int per = c.D / 16, all = (tr.R + kHeads - 1) / kHeads * per;
  for (int i = threadIdx.x; i < n * all; i += 256) {
    const int r = i / all, k = i - r * all, h0 = k / per, at = k - h0 * per, heads = min(tr.R - kHeads * h0, kHeads);
    if (pos[r] == kNoRow) continue;
    const int64_t col = ((int64_t)h * tr.R + kHeads * h0) * c.D;
    const uint16_t* from = tr.q + (row0 + r) * tr.ldq + col;
    uint16_t* to = tr.q_out + (row0 + r) * tr.ldo + col;
    const Unit u = unit_of<PAIRS>(at, tr.rot);
    Turned<PAIRS> w[kHeads];
    w[0].angles(u, at, tr, pos[r]);
#pragma unroll
    for (int e = 0; e < kHeads; ++e) w[e].pieces(from + min(e, heads - 1) * c.D, u);
#pragma unroll
    for (int e = 0; e < kHeads; ++e) {
      if (e >= heads) break;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        w[e].c[x] = w[0].c[x];
        w[e].s[x] = w[0].s[x];
      }
      store_turned(w[e], u, to + e * c.D);
    }
  }
}

// Rows of a workgroup: one unit of kHeads heads for each of its threads.  (A page's rows for each, units
// one after another: 8000 rows of 16 heads of 256 on one head of keys 137 us, so 30.)
__host__ __device__ __forceinline__ int query_rows(const KvArgs& c, int R) {
  const int all = (R + kHeads - 1) / kHeads * (c.D / 16);
  return all >= 256 ? 1 : min(256 / all, c.P);
}

// Workgroups (slot, head, 0 and 1): keys and values of a sequence's rows in one page, as in
// append.  (slot, head, 2 and on): the head's queries of one row where slots are rows, otherwise of
// P rows, some of them each (query_rows: so that a head has workgroups enough, whatever P and R are).
template <bool I8, bool PAIRS>
__global__ __launch_bounds__(256) void k_kv_append_rotated(KvArgs c, int64_t first_slot, int div, int per_seq, const uint16_t* k_new,
                                                           int64_t ldk, const uint16_t* v_new, int64_t ldv, TurnArgs tr) {
  __shared__ int count[4];
  __shared__ Found told;
  __shared__ uint32_t red[4];
  __shared__ int pos[256];
  const int h = blockIdx.y, side = blockIdx.z;
  const int64_t slot = first_slot + blockIdx.x;
  if (side < 2 || div == 1) {
    const Found s = find_slot_256(c, slot, div, per_seq, &told, count);
    if (side == 0) {
      append_turned<I8, PAIRS>(c, s, h, k_new, ldk, tr, red);
    } else if (side == 1) {
      append_rows<I8>(c, s, h, 1, v_new, ldv, red);
    } else {
      if (s.rows <= 0 || s.j >= s.rows) return;
      turn_row<PAIRS>(c, slot, h, tr, s.len - s.rows + s.j);
    }
    return;
  }
  const int each = query_rows(c, tr.R), in = (side - 2) * each;
  const int64_t row0 = slot * c.P + in;
  if (row0 >= c.T) return;
  const int n = (int)min((int64_t)min(each, c.P - in), c.T - row0);
  if ((int)threadIdx.x < n) {
    const int64_t row = row0 + threadIdx.x;
    const SeqSlot s = find_slot(c, row, 1, 1, 0);
    const int64_t p = (int64_t)c.lens[s.b] - s.rows + s.j;
    pos[threadIdx.x] = s.rows <= 0 || s.j >= s.rows ? kNoRow : (int)max(p, (int64_t)-1);
  }
  __syncthreads();
  turn_rows<PAIRS>(c, row0, n, h, tr, pos);
}

}  // namespace

hipError_t launch_kv_append_rotated(const KvArgs& c, bool i8, bool pairs, const uint16_t* k_new, int64_t ldk,
                                    const uint16_t* v_new, int64_t ldv, const TurnArgs& r, hipStream_t st) {
  // slots as in append
  const int64_t by_pages = c.T / c.P + 2 * (int64_t)c.B;
  const bool by_rows = c.T <= by_pages;
  const int div = by_rows ? 1 : c.P, per = by_rows ? 0 : 2;
  const int64_t slots = by_rows ? c.T : by_pages;
  for (int64_t first = 0; first < slots; first += kGridX) {
    const int queries = !r.q ? 0 : by_rows ? 1 : (c.P + query_rows(c, r.R) - 1) / query_rows(c, r.R);
    const dim3 grid((unsigned)min(slots - first, (int64_t)kGridX), (unsigned)c.H, 2 + queries);
    auto go = [&](auto i, auto p) {
      hipLaunchKernelGGL((k_kv_append_rotated<decltype(i)::value, decltype(p)::value>), grid, dim3(256), 0, st, c, first, div, per,
                         k_new, ldk, v_new, ldv, r);
    };
    if (i8) pairs ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
    else pairs ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
  }
  return hipGetLastError();
}

}  // namespace wq
