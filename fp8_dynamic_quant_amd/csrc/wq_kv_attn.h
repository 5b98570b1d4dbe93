// Attention over the paged 8-bit cache on the device: row tiles that step through a sequence's
// tokens, in a wave of their own or in a workgroup that shares the keys.
#pragma once

#include <type_traits>

#include "wq_kv_device.h"

namespace wq {

namespace {

constexpr int kTokTile = 64;     // tokens of a step
constexpr int kAttnWaves = 4;    // waves of an attention workgroup

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

}  // namespace

}  // namespace wq
