// The paged 8-bit cache on the device: the sequence of a workgroup's share, codes and their scales,
// and the appending of one sequence's rows in one page.
#pragma once

#include "wq_dma.h"
#include "wq_mx4_kv.h"

namespace wq {

namespace {

typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

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

// The new rows of one sequence (s) in one page of one head, keys (side 0) or values (side 1), by a
// workgroup of 256.  A thread's share is four pieces of eight elements: of keys 256 pieces apart in
// the order of memory, of values the four slots of an aligned group, whose codes are then whole
// words of the value rows.  The first share stays in registers between the two passes (the
// largest magnitude, the codes); larger pages read the others again.  The codes are products with a
// power of two, exact but for the one rounding to 8 bits.
template <bool I8>
__device__ __forceinline__ void append_rows(const KvArgs& c, const Found& s, int h, int side, const uint16_t* rows, int64_t ld,
                                            uint32_t* red) {
  if (s.rows <= 0) return;
  const int t = threadIdx.x;
  const int64_t len = s.len, start = len - s.rows;
  const int64_t pg = max(start, (int64_t)0) / c.P + s.j;
  const int64_t lo = max(start, pg * c.P), hi = min(len, (pg + 1) * c.P);
  if (lo >= hi || pg >= c.max_pages) return;
  const int page = c.table[s.b * c.table_stride + pg];
  const int D = c.D, P = c.P, s0 = (int)(lo - pg * P), n = (int)(hi - lo), per = D / 8;
  const uint16_t* x = rows + (s.row0 + (lo - start)) * ld + (int64_t)h * D;
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

}  // namespace

}  // namespace wq
