// A paged cache of keys and values in 8 bits, and attention over it.
//
// A page holds P tokens of every head, as codes (E4M3, or int8) and one UE8M0 byte for each
// (page, head) of keys and of values: x = code * 2^(byte - 127).  Keys lie [page][H][P][D],
// values [page][H][D][P]: the matrix instruction contracts q k over D and p v over tokens,
// and wants eight consecutive terms of a contraction from each lane, so with this layout both
// come from memory in operand order and nothing is transposed when they are read.
#include <type_traits>

#include "wq_dma.h"
#include "wq_kernels.h"
#include "wq_mx4_kv.h"

namespace wq {

namespace {

typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kTokTile = 64;     // tokens of a step
constexpr int kAttnWaves = 4;    // waves of an attention workgroup
constexpr int kPlanSeqs = 1024;  // sequences of one launch of runs (their work is summed up in LDS)
constexpr int kMaxRuns = 1024;   // workgroups of one

// The sequence of slot `item` when sequence b owns the slots from offsets[b] * mul / div +
// per * b on (the host knows neither a sequence's rows nor its length, so every sequence gets
// as many slots as it can need): the last b whose first slot is not behind `item`.  Offsets are
// read as 0 .. T, whatever they hold.
struct SeqSlot {
  int b;
  int64_t row0, rows;  // its rows
  int64_t j;           // the slot's place among its slots
};
__device__ __forceinline__ int64_t seq_offset(const KvArgs& c, int b) {
  return min(max(c.offsets[b], (int64_t)0), c.T);
}
__device__ __forceinline__ SeqSlot find_slot(const KvArgs& c, int64_t item, int mul, int div, int per) {
  int lo = 0, hi = c.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_offset(c, mid) * mul / div + (int64_t)per * mid <= item) lo = mid;
    else hi = mid - 1;
  }
  SeqSlot s;
  s.b = lo;
  s.row0 = seq_offset(c, lo);
  s.rows = seq_offset(c, lo + 1) - s.row0;
  s.j = item - (s.row0 * mul / div + (int64_t)per * lo);
  if (s.j < 0) s.j = s.rows = 0;  // offsets that do not begin at 0: rows before the first sequence
  return s;
}

// ---- append -------------------------------------------------------------------------------

// Exponent of a block with the largest magnitude a (a finite bf16 pattern): the smallest e with
// 2^e >= a / c, at least -127.  c = 448 = 1.75 * 2^8 (E4M3), 127 = 1.984375 * 2^6 (int8).
template <bool I8>
__device__ __forceinline__ int block_exp(uint32_t a) {
  const int E = (int)(a >> 7);
  const uint32_t F = a & 0x7Fu;  // a = 2^(E-127) (1 + F/128)
  const int e = I8 ? E - 133 + (F > 0x7Eu ? 1 : 0) : E - 135 + (F > 0x60u ? 1 : 0);
  return e < -127 ? -127 : e;
}

template <bool I8>
__device__ __forceinline__ uint32_t encode(float y) {
  if constexpr (I8) {
    return (uint32_t)(int)rintf(y) & 0xFFu;
  } else {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y, y, 0, false) & 0xFFu;
  }
}
// the codes of four numbers, the first in the lowest byte
template <bool I8>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if constexpr (I8) {
    return encode<true>(a) | encode<true>(b) << 8 | encode<true>(c) << 16 | encode<true>(d) << 24;
  } else {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true);
  }
}
__device__ __forceinline__ float half_of(const v4u& u, int j) {  // element j of eight bf16
  return __uint_as_float((j & 1) ? u[j / 2] & 0xFFFF0000u : u[j / 2] << 16);
}

// a held code at a larger scale: its value times 2^d, d < 0, rounded once more.  int8 codes stay
// within a unit of the exact quotient however often a page's scale grows: each growth at least
// halves what the earlier roundings left (1/2 + 1/4 + ...).
template <bool I8>
__device__ __forceinline__ uint32_t rescale(uint32_t code, int d) {
  if constexpr (I8) {
    return (uint32_t)(int)rintf(ldexpf((float)(int8_t)code, d)) & 0xFFu;
  } else {
    if ((code & 0x7Fu) == 0x7Fu) return code;  // E4M3's NaN
    return encode<false>(ldexpf(__builtin_amdgcn_cvt_f32_fp8((int)code, 0), d)) & 0xFFu;
  }
}

// find_slot by a workgroup of 256, and the sequence's length: each round asks for 256 sequences at
// once, and the thread that has the one sought tells the others
struct Found {
  int b;
  int64_t row0, rows, j, len;
};
__device__ __forceinline__ Found find_slot_256(const KvArgs& c, int64_t item, int div, int per, Found* told, int* count) {
  const int t = threadIdx.x;
  int lo = 0, span = c.B;
  for (;;) {
    const int step = (span + 255) / 256, i = t * step;
    const bool mine = i < span;
    const int64_t row0 = mine ? seq_offset(c, lo + i) : 0, base = row0 / div + (int64_t)per * (lo + i);
    int64_t end = 0, len = 0;
    if (step == 1 && mine) {
      end = seq_offset(c, lo + i + 1);
      len = c.lens[lo + i];
    }
    const uint64_t votes = __ballot(mine && base <= item);
    if ((t & 63) == 0) count[t >> 6] = __popcll(votes);
    __syncthreads();
    const int at = max(count[0] + count[1] + count[2] + count[3] - 1, 0);
    if (step == 1) {
      // j < 0: offsets that do not begin at 0, rows before the first sequence
      if (t == at) *told = Found{lo + i, row0, item < base ? 0 : end - row0, max(item - base, (int64_t)0), len};
      __syncthreads();
      return *told;
    }
    __syncthreads();  // the counts have been read
    lo += at * step;
    span = min(step, span - at * step);
  }
}

// One workgroup for the new rows of one sequence in one page of one head, keys (side 0) or
// values (side 1).  A thread's share is four pieces of eight elements: of keys 256 pieces apart in
// the order of memory, of values the four slots of an aligned group, whose codes are then whole
// words of the value rows.  The first share stays in registers between the two passes (the
// largest magnitude, the codes); larger pages read the others again.  The codes are products with a
// power of two, exact but for the one rounding to 8 bits.
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
  if (s.rows <= 0) return;
  const int64_t len = s.len, start = len - s.rows;
  const int64_t pg = max(start, (int64_t)0) / c.P + s.j;
  const int64_t lo = max(start, pg * c.P), hi = min(len, (pg + 1) * c.P);
  if (lo >= hi || pg >= c.max_pages) return;
  const int page = c.table[s.b * c.table_stride + pg];
  const int D = c.D, P = c.P, s0 = (int)(lo - pg * P), n = (int)(hi - lo), per = D / 8;
  const int64_t ld = side ? ldv : ldk;
  const uint16_t* x = (side ? v_new : k_new) + (s.row0 + (lo - start)) * ld + (int64_t)h * D;
  const int q0 = s0 / 4, nq = (s0 + n - 1) / 4 + 1 - q0;  // groups of four slots
  const int units = side ? nq * per : (n * per + 3) / 4;
  // piece e of unit i: its row (of the new ones here) and eighth of D; false if there is none
  auto piece = [&](int i, int e, int& r, int& d8) __attribute__((always_inline)) {
    if (side) {
      r = 4 * (q0 + i % nq) + e - s0;
      d8 = i / nq;
      return i < units && r >= 0 && r < n;
    }
    const int at = (i & ~255) * 4 + e * 256 + (i & 255);
    r = at / per;
    d8 = at % per;
    return r < n;
  };
  auto load = [&](int i, v4u (&u)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int r, d8;
      u[e] = v4u{0, 0, 0, 0};
      if (piece(i, e, r, d8)) u[e] = *reinterpret_cast<const v4u*>(x + r * ld + d8 * 8);
    }
  };
  const int rounds = side ? (units + 255) / 256 : (n * per + 1023) / 1024;
  v4u first[4];
  load(t, first);
  if (page < 0 || page >= c.pages) return;
  uint8_t* scale = (side ? c.v_scale : c.k_scale) + (int64_t)page * c.H + h;
  const int old = s0 > 0 ? *scale : 0;
  // largest magnitude of the new rows
  uint32_t a = 0;
  auto largest = [&](const v4u (&u)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < 4; ++j) a = max(a, max(u[e][j] & 0x7FFFu, (u[e][j] >> 16) & 0x7FFFu));
  };
  largest(first);
  for (int k = 1; k < rounds; ++k) {
    v4u u[4];
    load(256 * k + t, u);
    largest(u);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) a = max(a, (uint32_t)__shfl_xor((int)a, o, 64));
  if ((t & 63) == 0) red[t >> 6] = a;
  __syncthreads();  // and every thread has read the old byte
  a = max(max(red[0], red[1]), max(red[2], red[3]));
  const int byte = max(old, a < 0x7F80u ? block_exp<I8>(a) + 127 : 255);
  if (t == 0) *scale = (uint8_t)byte;
  uint8_t* codes = static_cast<uint8_t*>(side ? c.v : c.k) + ((int64_t)page * c.H + h) * P * D;
  // keys: slot-major rows of D; values: D rows of P slots
  if (s0 > 0 && old < byte && byte != 255) {
    for (int i = t; i < s0 * D; i += 256) {
      uint8_t* at = side ? codes + (int64_t)(i / s0) * P + i % s0 : codes + i;
      *at = (uint8_t)rescale<I8>(*at, old - byte);
    }
  }
  const float f = byte == 255 ? 0.0f : ldexpf(1.0f, 127 - byte);  // a power of two: products are exact
  auto store = [&](int i, v4u (&u)[4]) __attribute__((always_inline)) {
    if (byte == 255) {
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = v4u{0, 0, 0, 0};  // NaN and infinities too: codes of zero
    }
    if (!side) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int r, d8;
        if (!piece(i, e, r, d8)) continue;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = half_of(u[e], j) * f;
        *reinterpret_cast<v2u*>(codes + (s0 + r) * D + d8 * 8) =
            v2u{encode4<I8>(y[0], y[1], y[2], y[3]), encode4<I8>(y[4], y[5], y[6], y[7])};
      }
      return;
    }
    if (i >= units) return;
    const int q = 4 * (q0 + i % nq);  // the group's first slot
    uint8_t* at = codes + (int64_t)(i / nq) * 8 * P + q;
    const bool whole = q >= s0 && q + 4 <= s0 + n;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t w = encode4<I8>(half_of(u[0], j) * f, half_of(u[1], j) * f, half_of(u[2], j) * f, half_of(u[3], j) * f);
      if (whole) {
        *reinterpret_cast<uint32_t*>(at + j * P) = w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (q + e >= s0 && q + e < s0 + n) at[j * P + e] = (uint8_t)(w >> (8 * e));
      }
    }
  };
  store(t, first);
  for (int k = 1; k < rounds; ++k) {
    v4u u[4];
    load(256 * k + t, u);
    store(256 * k + t, u);
  }
}

// ---- attention -----------------------------------------------------------------------------
//
// Lane l of a wave: j = l % 16, g = l / 16.  A wave takes 16-row tiles of one sequence and cache
// head (a row is new token * R + query head of the group, so the R heads that share the keys share
// their reads) and steps of 64 tokens, in 16-token groups g = 0 .. 3, each inside one page.
//  * s^T = k q^T in four 16-token instructions t: the lane that supplies k row i takes token
//    16 (i / 4) + 4 t + i % 4, so that the results, rows 4 g + r of column j, are tokens
//    16 g + 4 t + r of row j: lane group g ends with the 16 consecutive tokens of its group.
//  * o^T += v^T p^T: the lane supplies p of exactly those 16 tokens, from its own registers, and v
//    of the same 16 tokens, 16 consecutive bytes of a value row.  Nothing crosses lanes but the
//    running maximum.
//  * the scales are one number for the lane's 16 tokens: the keys' multiplies s, the values' goes
//    into the widening of v (E4M3) or multiplies p (int8).

// eight codes -> eight bf16, exact (E4M3 has 4 significant bits, int8 at most 7); E4M3 times
// `scale`, a power of two
template <bool I8>
__device__ __forceinline__ v8bf widen8(uint32_t lo, uint32_t hi, float scale) {
  v4u o;
  if constexpr (I8) {
    const uint32_t w[2] = {lo, hi};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = w[i / 2] >> (16 * (i & 1));
      const uint32_t f0 = __float_as_uint((float)(int8_t)(x & 0xFF)), f1 = __float_as_uint((float)(int8_t)((x >> 8) & 0xFF));
      o[i] = __builtin_amdgcn_perm(f1, f0, 0x07060302u);  // the high halves: exact
    }
  } else {
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
  }
  return __builtin_bit_cast(v8bf, o);
}

// 2^(byte - 127), byte 0 the subnormal 2^-127; byte 255 is NaN
__device__ __forceinline__ float scale_of(uint32_t byte) {
  const float f = ldexpf(1.0f, (int)byte - 127);
  return byte == 255u ? __uint_as_float(0x7FC00000u) : f;
}

// max / sum over the four lane groups that share a row (lanes j, j + 16, j + 32, j + 48): the swaps
// of both registers' halves leave the two halves of v in two registers
__device__ __forceinline__ float groups_max(float v) {
  const v2u a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const v2u b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float groups_sum(float v) {
  const v2u a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const v2u b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// a value that every lane of the wave has, as one scalar
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}

// One sequence as the rows of a cache head see it, in scalars.
struct Seq {
  int64_t row0;      // its first row
  int64_t nrows;     // rows * R
  int len;           // tokens (as given)
  int rows;
  uint32_t seen;     // tokens that the table can hold, >= 0
  const int32_t* table;
};
__device__ __forceinline__ Seq seq_of(const KvAttnArgs& a, int b, int64_t row0, int64_t rows) {
  Seq s;
  b = uniform(b);
  s.row0 = uniform64(row0);
  s.rows = uniform((int)rows);
  s.nrows = (int64_t)s.rows * a.R;
  s.len = uniform(a.c.lens[b]);
  s.seen = (uint32_t)min((int64_t)max(s.len, 0), (int64_t)a.c.max_pages * a.c.P);
  s.table = a.c.table + b * a.c.table_stride;
  return s;
}
// tokens 0 .. limit - 1 are what a row of new token i sees
__device__ __forceinline__ uint32_t limit_of(const KvAttnArgs& a, const Seq& s, int i) {
  return a.causal ? (uint32_t)min((int64_t)max((int64_t)s.len - s.rows + i + 1, (int64_t)0), (int64_t)s.seen) : s.seen;
}
// page of a token group: group / per by per's rounded-up reciprocal (exact below 2^28 for per to
// 16); at per = 1 the reciprocal is 0 and `one` all ones
__device__ __forceinline__ uint32_t by_page(uint32_t group, uint32_t recip, uint32_t one) {
  return __umulhi(group, recip) + (group & one);
}

// slots of the lane's 16 that hold tokens: from the sequence's end on they hold anything
__device__ __forceinline__ int there_slots(const Seq& s, bool there, uint32_t gt) {
  return !there || gt >= s.seen ? 0 : (int)min(s.seen - gt, 16u);
}
__device__ __forceinline__ v4u keep_bytes(v4u v, int n) {  // the first n bytes, the others zero
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int keep = n - 4 * w;
    v[w] = keep >= 4 ? v[w] : keep <= 0 ? 0u : v[w] & ((1u << (8 * keep)) - 1u);
  }
  return v;
}

// |scale| (1 for a zero scale, at which q is zero)
__device__ __forceinline__ float score_scale(const KvAttnArgs& a) { return a.scale == 0.0f ? 1.0f : fabsf(a.scale); }
// |scale| 2^(byte - 127) log2(e), with which a page's scores become powers of two, kept within the
// positive finite numbers: scores of -inf (hidden) and 0 stay what they are.  Products of f32 with
// what lies below the least of them are below 2^-21, with nothing to tell between them.
__device__ __forceinline__ float log2_scale(float scale, uint32_t byte) {
  const float f = ldexpf(scale, (int)byte - 127) * 1.44269504088896340736f;
  return fminf(fmaxf(f, __uint_as_float(1u)), __uint_as_float(0x7F7FFFFFu));
}

// RT row tiles of a wave over steps [lo, hi) with stride TW, keys and values straight from memory
// in operand order.  The next step's keys load as soon as this one's scores are made, its values as
// soon as this one's are used, so that each has a whole step's time; page numbers load two ahead.
template <int D, bool I8, int RT>
struct Rows {
  static constexpr int ND = D / 16, NC = D / 64;
  v8bf qf[RT][NC][2];
  v4f o[RT][ND];
  float mx[RT], sum[RT];  // running maximum (in log2 units) and this lane group's part of the sum
  uint32_t limit[RT];

  // r0: the first row; rows past the sequence's last repeat it (and are not stored)
  __device__ __forceinline__ void limits(const KvAttnArgs& a, const Seq& s, int64_t r0, int j) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      limit[rt] = limit_of(a, s, (int)min(r0 + 16 * rt + j, s.nrows - 1) / a.R);
      mx[rt] = -INFINITY;
      sum[rt] = 0.0f;
#pragma unroll
      for (int i = 0; i < ND; ++i) o[rt][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }
  __device__ __forceinline__ void load_q(const KvAttnArgs& a, const Seq& s, int h, int64_t r0, int j, int g) {
    // the sign goes into q, and a zero, so that scores scale by a positive number (log2_scale)
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u, keep = a.scale == 0.0f ? 0u : ~0u;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int rc = (int)min(r0 + 16 * rt + j, s.nrows - 1);
      const uint16_t* q = a.q + (s.row0 + rc / a.R) * a.ldq + (int64_t)(h * a.R + rc % a.R) * D + 16 * g;
#pragma unroll
      for (int cc = 0; cc < NC; ++cc)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          qf[rt][cc][m] = __builtin_bit_cast(v8bf, (*reinterpret_cast<const v4u*>(q + 64 * cc + 8 * m) ^ flip) & keep);
    }
  }

  // Scores of the lane's 16 tokens from gt on that a row does not see become -inf; of a page marked
  // NaN (bad) those it sees become NaN, and the caller's scales one.
  __device__ __forceinline__ void hide(v4f (&sc)[RT][4], bool there, bool bad, uint32_t gt) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int left = there ? (int)min(limit[rt], 0x7FFFFFFFu) - (int)min(gt, 0x7FFFFFFFu) : 0;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          sc[rt][t][r] = 4 * t + r >= left ? -INFINITY : bad ? __uint_as_float(0x7FC00000u) : sc[rt][t][r];
    }
  }
  // scores -> weights, the running maximum and sum
  __device__ __forceinline__ void weights(v4f (&sc)[RT][4], v8bf (&pf)[RT][2], float ks, float vs) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) top = fmaxf(top, sc[rt][t][r]);
      top = groups_max(top * ks);
      if (__any(top > mx[rt])) {
        const float mn = fmaxf(mx[rt], top);
        const float alpha = __builtin_amdgcn_exp2f(mx[rt] - (mn == -INFINITY ? 0.0f : mn));
        mx[rt] = mn;
        sum[rt] *= alpha;
#pragma unroll
        for (int i = 0; i < ND; ++i) o[rt][i] *= alpha;
      }
      const float base = mx[rt] == -INFINITY ? 0.0f : mx[rt];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[rt][t][r], ks, -base));
          sum[rt] += e;
          // rounded to bf16, with an int8 page's scale on it (a power of two: no further rounding).  By
          // at most 2^-8 of each weight, as the output itself is: against 64 bits outputs are off by 0.0019
          // to 0.0020 (relative, over all) where f32 weights give 0.0017.  The instruction takes bf16;
          // keeping the weights' other bits would take a second one for each.
          pf[rt][t >> 1][(t & 1) * 4 + r] = (__bf16)(I8 ? e * vs : e);
        }
    }
  }

  __device__ __forceinline__ void run(const KvAttnArgs& a, const Seq& s, int h, int64_t r0, uint32_t lo, uint32_t hi,
                                      uint32_t TW, int j, int g) {
    limits(a, s, r0, j);
    if (lo >= hi) return;
    auto begin_rows = [&]() __attribute__((always_inline)) { load_q(a, s, h, r0, j, g); };
    const KvArgs& c = a.c;
    const uint32_t per = (uint32_t)c.P >> 4, recip = c.page_recip, one = per == 1 ? ~0u : 0u, H = (uint32_t)c.H;
    const float abs_scale = score_scale(a);
    const uint32_t page_bytes = (uint32_t)c.P * D;
    const uint8_t* K = static_cast<const uint8_t*>(c.k) + (uint32_t)h * page_bytes;
    const uint8_t* V = static_cast<const uint8_t*>(c.v) + (uint32_t)h * page_bytes;
    const int64_t page_step = (int64_t)H * page_bytes;
    const int kg = j >> 2;  // the token group that this lane reads keys of
    const uint32_t first = __builtin_amdgcn_readfirstlane((int)limit[0]);  // the least of the wave's limits
    struct Page {
      uint32_t at, slot;
      bool there;
    };
    auto number = [&](uint32_t step, uint32_t grp) -> int {  // the table's entry
      const uint32_t tg = 4 * step + grp;
      return 16 * tg < s.seen ? s.table[by_page(tg, recip, one)] : -1;
    };
    // a group past the end, or a page number that is none, reads page 0 and is masked
    auto place = [&](uint32_t step, uint32_t grp, int page) -> Page {
      const uint32_t tg = 4 * step + grp;
      const bool there = (uint32_t)page < (uint32_t)c.pages;
      return Page{there ? (uint32_t)page : 0u, (tg - by_page(tg, recip, one) * per) * 16, there};
    };
    v4u kk[4][NC];
    auto load_k = [&](const Page& p) {
      const uint8_t* kp = K + p.at * page_step + (p.slot + (j & 3)) * D + 16 * g;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int cc = 0; cc < NC; ++cc) kk[t][cc] = *reinterpret_cast<const v4u*>(kp + 4 * t * D + 64 * cc);
    };
    const int n0 = number(lo, g), n1 = number(lo, kg);
    begin_rows();  // (the rows' own loads behind the page numbers', which are waited for first)
    Page pv = place(lo, g, n0);
    load_k(place(lo, kg, n1));
    uint32_t kb = c.k_scale[(int64_t)pv.at * H + h], vb;
    v4u vv[ND];
    auto load_v = [&](const Page& p) {
      const uint8_t* vp = V + p.at * page_step + (uint32_t)j * c.P + p.slot;
      vb = c.v_scale[(int64_t)p.at * H + h];
#pragma unroll
      for (int i = 0; i < ND; ++i) vv[i] = *reinterpret_cast<const v4u*>(vp + 16 * i * c.P);
    };
    load_v(pv);
    uint32_t nstep = min(lo + TW, hi - 1);  // the last step's "next" is a repeat, loaded and not used
    int nk = number(nstep, kg), nv = number(nstep, g);
    for (uint32_t step = lo; step < hi; step += TW) {
      const uint32_t tok0 = step * kTokTile, gt = tok0 + 16 * g;
      // ---- scores
      v4f sc[RT][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) sc[rt][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int cc = 0; cc < NC; ++cc)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const v8bf kf = widen8<I8>(kk[t][cc][2 * m], kk[t][cc][2 * m + 1], 1.0f);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) sc[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[rt][cc][m], sc[rt][t], 0, 0, 0);
          }
      }
      const uint32_t kbyte = kb;
      // ---- the next step's keys
      const Page npv = place(nstep, g, nv);
      load_k(place(nstep, kg, nk));
      kb = c.k_scale[(int64_t)npv.at * H + h];
      nstep = min(nstep + TW, hi - 1);
      nk = number(nstep, kg);
      nv = number(nstep, g);
      // ---- weights and values
      const bool tail = tok0 + kTokTile > s.seen || !__all(pv.there), bad = kbyte == 255u || vb == 255u;
      if (tail || tok0 + kTokTile > first || __any(bad)) hide(sc, pv.there, bad, gt);
      const float ks = bad || !pv.there ? 1.0f : log2_scale(abs_scale, kbyte), vs = bad || !pv.there ? 1.0f : scale_of(vb);
      v8bf pf[RT][2];
      weights(sc, pf, ks, vs);
#pragma unroll
      for (int i = 0; i < ND; ++i) {
        // E4M3 codes behind the sequence's end may be NaN (an int8 times a zero weight is zero)
        if (!I8 && tail) vv[i] = keep_bytes(vv[i], there_slots(s, pv.there, gt));
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const v8bf vf = widen8<I8>(vv[i][2 * m], vv[i][2 * m + 1], vs);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) o[rt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[rt][m], o[rt][i], 0, 0, 0);
        }
      }
      // ---- the next step's values
      pv = npv;
      load_v(pv);
    }
  }
};

// The same for the four waves of a workgroup, 64 RT rows that read the same keys: a step's keys
// (64 token rows of D bytes) and values (D rows of 64 tokens) go global -> LDS by DMA, S - 1 steps
// ahead in a ring, each byte read once by the workgroup.  Chunks of 16 bytes are XORed so that the
// sixteen rows that are read at one chunk meet sixteen different bank groups: a key read takes
// tokens 16 a + 4 t + b (a, b = 0 .. 3), a value read sixteen consecutive rows of 64 bytes.
// Wave w sends the keys of token group w, and of the values every fourth run of 16 rows; page
// numbers come by DMA too, so that no other vector load is in flight and the count of DMAs tells
// when a step has landed.
template <int D, bool I8, int RT, int S>
struct SharedRows {
  using R = Rows<D, I8, RT>;
  static constexpr int ND = D / 16, NC = D / 64;
  static constexpr int kTile = 64 * D, kStage = 2 * kTile + 256;  // keys, values, scale bytes (a word each)
  static constexpr int kDma = 2 * NC + 2;
  static constexpr int kPages = S * kStage;  // page numbers of eight steps, a word a lane
  static constexpr int kBytes = kPages + 8 * 256;
  static __device__ __forceinline__ int k_swz(int token) {
    return NC == 1 ? (token >> 4) & 3 : NC == 2 ? ((token >> 4) & 3) * 2 + ((token >> 1) & 1) : ((token >> 4) & 3) * 4 + (token & 3);
  }
  static __device__ __forceinline__ int v_swz(int d) { return (d >> 2) & 3; }

  // every wave of the workgroup calls this with the same lo, hi; a wave whose rows see only steps
  // below `most` skips the others' arithmetic
  static __device__ __forceinline__ void run(R& w, const KvAttnArgs& a, const Seq& s, int h, uint32_t lo, uint32_t hi,
                                             uint32_t most, uint8_t* smem, int wv, int lane) {
    if (lo >= hi) return;
    const KvArgs& c = a.c;
    const int j = lane & 15, g = lane >> 4;
    const uint32_t per = (uint32_t)c.P >> 4, recip = c.page_recip, one = per == 1 ? ~0u : 0u, H = (uint32_t)c.H;
    const float abs_scale = score_scale(a);
    const uint32_t page_bytes = (uint32_t)c.P * D;
    const uint8_t* K = static_cast<const uint8_t*>(c.k) + (uint32_t)h * page_bytes;
    const uint8_t* V = static_cast<const uint8_t*>(c.v) + (uint32_t)h * page_bytes;
    const uint32_t page_step = H * page_bytes;  // < 2^32: 65535 heads of 256 x 256
    const uint32_t first = __builtin_amdgcn_readfirstlane((int)w.limit[0]);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_u8)smem;
    // This lane's places.  Keys: position wv * NC * 64 + lane of the tile is (token, chunk).  Values:
    // row wv * 16 + lane / 4 (then 64 rows on), chunk lane % 4, which holds token group vg.  Page
    // numbers are held for token group vg (lanes 0 .. 3: groups 0 .. 3).
    const uint32_t vg = (uint32_t)((lane & 3) ^ ((lane >> 4) & 3));
    auto entry = [&](uint32_t step) __attribute__((always_inline)) {  // of the table; past the end the first
      const uint32_t tg = 4 * step + vg;
      return s.table + (16 * tg < s.seen ? by_page(tg, recip, one) : 0u);
    };
    // page of token group vg of a step, -1 where there is none
    auto checked = [&](uint32_t step, int page) __attribute__((always_inline)) {
      return 16 * (4 * step + vg) < s.seen && (uint32_t)page < (uint32_t)c.pages ? page : -1;
    };
    auto slot_of = [&](uint32_t tg) __attribute__((always_inline)) { return (tg - by_page(tg, recip, one) * per) * 16; };
    uint32_t koff[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int pos = (wv * NC + i) * 64 + lane, tok = pos / (D / 16), ch = (pos % (D / 16)) ^ k_swz(tok);
      koff[i] = (uint32_t)((tok & 15) * D + ch * 16);
    }
    const uint8_t* vrow = V + (uint32_t)(wv * 16 + (lane >> 2)) * c.P;
    const uint8_t* scales = (lane & 4 ? c.v_scale : c.k_scale) + h;
    auto issue = [&](uint32_t step, int page, int stage) __attribute__((always_inline)) {
      const uint32_t st = lds0 + stage * kStage;
      const uint32_t held = (uint32_t)max(page, 0);  // a group without a page reads page 0 and is masked
      const uint8_t* kb = K + (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)held, wv) * page_step + slot_of(4 * step + wv) * D;
#pragma unroll
      for (int i = 0; i < NC; ++i) dma16_at(kb + koff[i], st + (wv * NC + i) * 1024);
      const uint8_t* vb = vrow + (uint64_t)held * page_step + slot_of(4 * step + vg);
#pragma unroll
      for (int i = 0; i < NC; ++i) dma16_at(vb + (uint32_t)(64 * i * c.P), st + kTile + (wv + 4 * i) * 1024);
      // scale bytes: word x of the stage's last 256 bytes is the keys' of token group x, word 4 + x
      // the values' (each wave writes the same)
      dma1_at(scales + (uint64_t)held * H, st + 2 * kTile);
    };
    auto send_page = [&](uint32_t step) __attribute__((always_inline)) {
      dma4_at(entry(min(step, hi - 1)), lds0 + kPages + (step & 7) * 256);
    };
    static_assert(S == 2 || S == 3, "page numbers of three steps");
    // p0, p1(, p2): pages of this step and the next; step + S - 1's are read when its data are sent,
    // two steps after they were sent for themselves
    int p0 = checked(lo, *entry(lo)), p1 = checked(lo + 1, *entry(min(lo + 1, hi - 1)));
    int p2 = S == 3 ? checked(lo + 2, *entry(min(lo + 2, hi - 1))) : 0;
    send_page(lo + S);
    issue(lo, p0, 0);
    if (S == 3 && lo + 1 < hi) issue(lo + 1, p1, 1);
    int stage = 0;
    for (uint32_t step = lo; step < hi; ++step) {
      if (S > 2 && step + S - 2 < hi && step > lo) wait_vm<kDma*(S - 2)>();
      else wait_vm<0>();
      lds_barrier();  // the step has landed for all, and the one before it has been read by all
      if (step > lo) {
        const int got = *reinterpret_cast<const int*>(smem + kPages + ((step + S - 1) & 7) * 256 + lane * 4);
        (S == 3 ? p2 : p1) = checked(step + S - 1, got);
      }
      send_page(step + S + 1);
      if (step + S - 1 < hi) issue(step + S - 1, S == 3 ? p2 : p1, stage == 0 ? S - 1 : stage - 1);
      const uint32_t none = (uint32_t)__ballot(p0 < 0) & 15u;
      p0 = p1;
      if (S == 3) p1 = p2;
      const uint8_t* sk = smem + stage * kStage;
      const uint8_t* sv = sk + kTile;
      const uint32_t* sb = reinterpret_cast<const uint32_t*>(sv + kTile);
      stage = stage + 1 == S ? 0 : stage + 1;
      if (step >= most) continue;  // uniform in the wave
      // operands are read one ahead of their use
      v4f sc[RT][4];
      auto key = [&](int x) __attribute__((always_inline)) {
        const int tok = 16 * (j >> 2) + 4 * (x / NC) + (j & 3), ch = 4 * (x % NC) + g;
        return *reinterpret_cast<const v4u*>(sk + tok * D + ((ch ^ k_swz(tok)) << 4));
      };
      v4u kk = key(0);
#pragma unroll
      for (int x = 0; x < 4 * NC; ++x) {
        const int t = x / NC, cc = x % NC;
        const v4u next = x + 1 < 4 * NC ? key(x + 1) : kk;
        if (cc == 0)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) sc[rt][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const v8bf kf = widen8<I8>(kk[2 * m], kk[2 * m + 1], 1.0f);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) sc[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, w.qf[rt][cc][m], sc[rt][t], 0, 0, 0);
        }
        kk = next;
      }
      const uint32_t kbyte = sb[g], vbyte = sb[4 + g];
      const uint32_t tok0 = step * kTokTile, gt = tok0 + 16 * g;
      const bool there = !(none >> g & 1u), tail = tok0 + kTokTile > s.seen || none != 0, bad = kbyte == 255u || vbyte == 255u;
      if (tail || tok0 + kTokTile > first || __any(bad)) w.hide(sc, there, bad, gt);
      const float ks = bad || !there ? 1.0f : log2_scale(abs_scale, kbyte), vs = bad || !there ? 1.0f : scale_of(vbyte);
      auto value = [&](int i) __attribute__((always_inline)) {
        return *reinterpret_cast<const v4u*>(sv + (16 * i + j) * 64 + ((g ^ v_swz(j)) << 4));
      };
      v4u vv = value(0);
      v8bf pf[RT][2];
      w.weights(sc, pf, ks, vs);
#pragma unroll
      for (int i = 0; i < ND; ++i) {
        const v4u next = i + 1 < ND ? value(i + 1) : vv;
        // E4M3 codes behind the sequence's end may be NaN (an int8 times a zero weight is zero)
        if (!I8 && tail) vv = keep_bytes(vv, there_slots(s, there, gt));
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const v8bf vf = widen8<I8>(vv[2 * m], vv[2 * m + 1], vs);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) w.o[rt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[rt][m], w.o[rt][i], 0, 0, 0);
        }
        vv = next;
      }
    }
    wait_vm<0>();   // no page number is still on its way
    lds_barrier();  // the ring may be filled again
  }
};

// The log-sum-exp of maximum m (log2) and sum l, and what the weighted values are multiplied by.  A
// row that saw no token has l = 0 and gets -inf and zeros.  The maximum does not tell: it passes
// over NaN, so that it stays -inf too where all that a row saw was NaN.  The sum keeps NaN.
__device__ __forceinline__ float log_sum(float m, float l) {
  return (m + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f;
}
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

// A wave's own rows, whole: lane (j, g) holds of row j the elements 16 i + 4 g .. + 3
template <int D, bool I8, int RT>
__device__ __forceinline__ void store_rows(const KvAttnArgs& a, const Seq& s, Rows<D, I8, RT>& w, int h, int64_t r0, int j,
                                           int g) {
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const float l = groups_sum(w.sum[rt]);
    const int64_t rr = r0 + 16 * rt + j;
    if (rr >= s.nrows) continue;
    const int i = (int)rr / a.R, head = h * a.R + (int)rr % a.R;
    const float inv = inverse_sum(l);
    uint16_t* out = a.out + (s.row0 + i) * a.ldo + (int64_t)head * D + 4 * g;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      const v4f v = w.o[rt][d] * inv;
      *reinterpret_cast<v2u*>(out + 16 * d) = v2u{f32_to_bf16_nan(v[0]) | f32_to_bf16_nan(v[1]) << 16,
                                                  f32_to_bf16_nan(v[2]) | f32_to_bf16_nan(v[3]) << 16};
    }
    if (a.lse && g == 0) a.lse[(s.row0 + i) * (int64_t)(a.c.H * a.R) + head] = log_sum(w.mx[rt], l);
  }
}

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
// n / d for 0 <= n < 2^52 (what the call accepts stays below), d > 0; integer divisions of 64 bits
// are hundreds of instructions
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  int64_t q = (int64_t)((double)n / (double)d);
  const int64_t r = n - q * d;
  return r < 0 ? q - 1 : r >= d ? q + 1 : q;
}
__device__ __forceinline__ uint32_t steps_of(const KvArgs& c, int len) {
  const int64_t seen = min((int64_t)max(len, 0), (int64_t)c.max_pages * c.P);
  return (uint32_t)max((seen + kTokTile - 1) / kTokTile, (int64_t)1);  // rows that see nothing are stored too
}
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
