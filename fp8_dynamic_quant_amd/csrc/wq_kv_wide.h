// Attention over the paged 8-bit cache for many rows of one head: a workgroup of eight waves, 16 RT
// rows each, that share keys and values through LDS, widened once for all of them.
#pragma once

#include "wq_kv_attn.h"

namespace wq {

namespace {

constexpr int kWideWaves = 8;

// A step's keys (T token rows of D bytes) and values (D rows of T tokens) go global -> LDS by DMA, two
// steps ahead, in a ring; the workgroup widens them to bf16 a step ahead, each thread one piece of
// sixteen codes of either, into one of two buffers that the matrix instructions read.  Widening in each
// wave for itself, as attention of one sequence's rows does (SharedRows), is a third of that kernel's
// vector instructions with E4M3 codes and more than half with int8.
//
// What bounds it.  1024 rows of 8 heads of 128 over 32768 tokens, E4M3: 187 us, 735 TFLOP/s (int8 196);
// with each wave widening for itself 257 and 320.  Of the SIMDs' cycles matrix instructions take 41 %,
// other vector instructions 40 %, and two waves a SIMD do not hide each other: half of the waves of a
// workgroup reach the barrier a quarter of a step before the others.  (The later four waves half a step
// behind, products with values beside scores: 2 % slower.)  Heads of 64, 8 to a cache head: 233.  Heads of
// 256, 4 to each of 4: 281, one row tile a wave: a step of 32 tokens 2700 cycles, LDS 40 % of them, matrix
// instructions 22 %, the others 27 %, waves waiting for reads and barriers 42 % of their time; registers
// do not hold a second row tile.
// The row of ones (below) costs 1 to 2 % of that, of heads of 64, whose products are fewest, 3.5 %: 184, 193,
// 226 and 276 without.  Two-element dot products instead: 264 with heads of 64, and with heads of 128 453, whose
// registers do not hold them.
//
// Lane (j, g) = (l % 16, l / 16).  s^T = k q^T in instructions t of 16 tokens: the lane that supplies key
// row i takes token (T / 4) (i / 4) + 4 t + i % 4, so that lane group g ends with the T / 4 consecutive
// tokens from (T / 4) g on of row j, the operand of o^T += v^T p^T from its own registers.
//
// Pieces of 16 bytes are XORed with their row so that the sixteen lanes of a read meet sixteen different
// places of 256 bytes: key rows by the lane that reads them, value rows by their number.
// A step's token groups of 16 each have a page of their own to look up; taking one for the whole step
// where pages hold whole ones, with scalar addresses, was 1 % quicker at best.
template <int D, bool I8, int RT>
struct Wide {
  static constexpr int T = D == 256 ? 32 : 64;  // tokens of a step: two buffers of 32 KiB
  static constexpr int kGroups = T / 16, NT = T / 16, NK = D / 32, NV = D / 16, NM = T / 32;
  static constexpr int kTile = T * D, kRaw = 2 * kTile, kBuf = 2 * kTile, kRing = 3;
  static constexpr int kKeys = kRing * kRaw, kValues = kKeys + 2 * kBuf, kScales = kValues + 2 * kBuf;
  static constexpr int kTable = kScales + 4 * 256, kBytes = kTable + 512;
  static constexpr int kDma = D == 64 ? 1 : 2;  // of a wave and step, and the first wave's scale bytes
  static constexpr int kRows = 16 * RT * kWideWaves;

  v8bf qf[RT][NK];
  v4f o[RT][NV];
  float mx[RT], sum[RT];  // what weights are relative to (log2), and this lane group's part of their sum
  v4f kept[RT];           // in each element the whole sum of the weights as they are rounded for o
  float down[RT];         // what a score is lowered by
  uint32_t limit[RT];

  static __device__ __forceinline__ int key_place(int token) {  // the lane j that reads it
    const int j = T == 64 ? 4 * ((token >> 4) & 3) + (token & 3) : 4 * ((token >> 3) & 3) + (token & 3);
    return D == 64 ? j >> 1 : j;
  }
  static __device__ __forceinline__ int value_place(int row) {
    return T == 64 ? (row & 2) << 1 ^ (row & 4) >> 1 ^ ((row & 8) >> 3) * 3 : -(row >> 2) & 3;
  }

  // r0: the first row of the wave; rows past the last repeat it (and are not stored)
  __device__ __forceinline__ void begin(const KvAttnArgs& a, const Seq& s, int h, int64_t r0, int j, int g) {
    // the sign of the scale goes into q, and a zero, so that scores scale by a positive number (log2_scale)
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u, keep = a.scale == 0.0f ? 0u : ~0u;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int rc = (int)min(r0 + 16 * rt + j, s.nrows - 1);
      const uint16_t* q = a.q + (s.row0 + rc / a.R) * a.ldq + (int64_t)(h * a.R + rc % a.R) * D + 8 * g;
#pragma unroll
      for (int k = 0; k < NK; ++k) qf[rt][k] = __builtin_bit_cast(v8bf, (*reinterpret_cast<const v4u*>(q + 32 * k) ^ flip) & keep);
      limit[rt] = limit_of(a, s, rc / a.R);
      mx[rt] = -INFINITY;
      down[rt] = INFINITY;
      sum[rt] = 0.0f;
      kept[rt] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i) o[rt][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }

  // sixteen codes -> bf16, exact (a power of two times int8's seven bits or E4M3's four): pieces `piece`
  // and `piece + apart` of a row
  static __device__ __forceinline__ void widen16(v4u c, float scale, uint8_t* row, int piece, int apart, int place) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      v4u w;
      if constexpr (I8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = c[2 * m + i / 2] >> (16 * (i & 1));
          const float f0 = (float)(int8_t)(x & 0xFF) * scale, f1 = (float)(int8_t)((x >> 8) & 0xFF) * scale;
          w[i] = __builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u);
        }
      } else {
        w = __builtin_bit_cast(v4u, widen8<false>(c[2 * m], c[2 * m + 1], scale));
      }
      *reinterpret_cast<v4u*>(row + (((piece + m * apart) ^ place) << 4)) = w;
    }
  }

  // Of the lane's scores of instruction t, whose tokens lie from at on: those that a row does not see
  // become -inf; of a page marked NaN (bad) those it sees become NaN, and the caller's scale one.
  __device__ __forceinline__ void hide(v4f (&sc)[RT], bool there, bool bad, uint32_t at) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int left = there ? (int)min(limit[rt], 0x7FFFFFFFu) - (int)min(at, 0x7FFFFFFFu) : 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) sc[rt][r] = r >= left ? -INFINITY : bad ? __uint_as_float(0x7FC00000u) : sc[rt][r];
    }
  }

  // Every wave of the workgroup calls this with the same lo, hi (in steps of T); `active`: the wave
  // has rows.
  __device__ __forceinline__ void run(const KvAttnArgs& a, const Seq& s, int h, uint32_t lo, uint32_t hi, bool active,
                                      uint8_t* smem, int wv, int lane) {
    if (lo >= hi) return;
    const KvArgs& c = a.c;
    const int j = lane & 15, g = lane >> 4, t = threadIdx.x;
    const uint32_t per = (uint32_t)c.P >> 4, recip = c.page_recip, one = per == 1 ? ~0u : 0u, H = (uint32_t)c.H;
    const float abs_scale = score_scale(a);
    const uint32_t page_bytes = (uint32_t)c.P * D;
    const uint8_t* K = static_cast<const uint8_t*>(c.k) + (uint32_t)h * page_bytes;
    const uint8_t* V = static_cast<const uint8_t*>(c.v) + (uint32_t)h * page_bytes;
    const uint32_t page_step = H * page_bytes;  // < 2^32: 65535 heads of 256 x 256
    const uint32_t first = (uint32_t)uniform((int)limit[0]);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_u8)smem;
    const uint32_t n = hi - lo;
    // This lane's share of a step's DMA.  Keys: piece 64 w + lane of the tile, of one token group a wave.
    // Values: row and piece likewise, the piece its token group.  Page numbers are held for token group
    // lane % kGroups.
    constexpr int kPer = D / 16;                                   // pieces of a key row
    const int kw = wv, vw = D == 64 ? wv - 4 : wv;                 // (heads of 64: four waves for each)
    const int ktok = kw * (64 / kPer) + lane / kPer, kgroup = kw * (64 / kPer) / 16;
    const uint32_t koff = (uint32_t)((ktok & 15) * D + (lane % kPer) * 16);
    const uint32_t mine = (uint32_t)(lane % kGroups);
    const uint32_t voff = (uint32_t)((vw * (64 / kGroups) + lane / kGroups) * c.P);
    const uint8_t* scales = (lane & 4 ? c.v_scale : c.k_scale) + h;
    auto slot_of = [&](uint32_t tg) __attribute__((always_inline)) { return (tg - by_page(tg, recip, one) * per) * 16; };
    auto entry = [&](uint32_t tg) __attribute__((always_inline)) {  // (a choice, no branch: loads of several go together)
      uint32_t at = by_page(tg, recip, one);
      asm volatile("" : "+v"(at));
      return 16 * tg < s.seen ? at : 0u;
    };
    // page of a step's token group `mine`; -1 where there is none
    auto checked = [&](uint32_t step, int page) __attribute__((always_inline)) {
      return 16 * (kGroups * (lo + step) + mine) < s.seen && (uint32_t)page < (uint32_t)c.pages ? page : -1;
    };
    auto none_of = [&](int page) __attribute__((always_inline)) {
      return (uint32_t)__ballot(page < 0) & ((1u << kGroups) - 1u);
    };
    // step b at the group's page (page 0 where there is none: it is masked)
    auto issue = [&](uint32_t b, int page_of, int slot) __attribute__((always_inline)) {
      const uint32_t raw = lds0 + slot * kRaw, held = (uint32_t)max(page_of, 0);
      if (D != 64 || wv < 4) {
        const uint32_t page = (uint32_t)__builtin_amdgcn_readlane((int)held, kgroup);
        dma16(K + (uint64_t)page * page_step + slot_of(kGroups * (lo + b) + kgroup) * D, koff, raw + kw * 1024);
      }
      if (D != 64 || wv >= 4)
        dma16_at(V + (uint64_t)held * page_step + (voff + slot_of(kGroups * (lo + b) + mine)), raw + kTile + vw * 1024);
      // scale bytes: word x the keys' of token group x, word 4 + x the values'
      if (wv == 0) dma1_at(scales + (uint64_t)held * H, lds0 + kScales + (b & 3) * 256);
    };
    const uint32_t* words = reinterpret_cast<const uint32_t*>(smem + kScales);
    // the thread's pieces of a step: read, and widened
    v4u kraw{0, 0, 0, 0}, vraw{0, 0, 0, 0};
    uint32_t vword = 0;
    auto fetch = [&](uint32_t b, uint32_t none, int slot) __attribute__((always_inline)) {
      const uint8_t* raw = smem + slot * kRaw;
      if (D != 64 || t < 256) kraw = *reinterpret_cast<const v4u*>(raw + 16 * t);
      if (D != 64 || t >= 256) {
        const int u = D == 64 ? t - 256 : t, x = u % kGroups;
        vraw = *reinterpret_cast<const v4u*>(raw + kTile + 16 * u);
        vword = words[(b & 3) * 64 + 4 + x];
        const uint32_t step = lo + b;
        // codes behind the sequence's end and of pages that are none may be anything, E4M3's NaN too
        if (__builtin_expect(none != 0 || (step + 1) * T > s.seen, 0)) {
          uint32_t at = step * T + 16 * x;
          asm volatile("" : "+v"(at));  // (all of it in the branch)
          vraw = keep_bytes(vraw, there_slots(s, !(none >> x & 1u), at));
        }
      }
    };
    auto widen_keys = [&](uint32_t b) __attribute__((always_inline)) {
      const int tok = t / kPer;
      if (D != 64 || t < 256) widen16(kraw, 1.0f, smem + kKeys + (b & 1) * kBuf + tok * 2 * D, 2 * (t % kPer), 1, key_place(tok));
    };
    auto widen_values = [&](uint32_t b) __attribute__((always_inline)) {
      const int u = D == 64 ? t - 256 : t, row = u / kGroups, x = u % kGroups;
      if (D != 64 || t >= 256)
        widen16(vraw, vword == 255u ? 1.0f : scale_of(vword), smem + kValues + (b & 1) * kBuf + row * 2 * T, T == 64 ? x : 2 * x, T == 64 ? 4 : 1, value_place(row));
    };
    // ---- steps 0, 1, 2 on their way (of a step in any case)
    const int* table = s.table;
    auto read = [&](uint32_t step) __attribute__((always_inline)) { return table[entry(kGroups * (lo + min(step, n - 1)) + mine)]; };
    int e0 = read(0), e1 = read(1), e2 = read(2);
    asm volatile("" : "+v"(e0), "+v"(e1), "+v"(e2));  // all of them are here before the first DMA, which waits would count
    const int p0 = checked(0, e0), p1 = checked(min(1u, n - 1), e1), p2 = checked(min(2u, n - 1), e2);
    // the queries have come with them: from here on the waits count DMAs alone
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        v4u q = __builtin_bit_cast(v4u, qf[rt][k]);
        asm volatile("" : "+v"(q));
        qf[rt][k] = __builtin_bit_cast(v8bf, q);
      }
    // table entries of 64 token groups at a time, by DMA: half (q & 1) of 512 bytes holds those from 64 q on
    auto send_entries = [&](uint32_t q) __attribute__((always_inline)) {
      dma4_at(s.table + entry(kGroups * lo + min(64 * q + lane, kGroups * n - 1)), lds0 + kTable + (q & 1) * 256);
    };
    auto told = [&](uint32_t step) __attribute__((always_inline)) {
      return *reinterpret_cast<const int*>(smem + kTable + ((kGroups * step + mine) & 127) * 4);
    };
    if (wv == 0) send_entries(0);
    issue(0, p0, 0);
    if (n > 1) issue(1, p1, 1);
    if (n > 2) issue(2, p2, 2);
    uint32_t none = none_of(p0) | none_of(p1) << 4 | none_of(p2) << 8;  // of step b on, four bits each
    // step 0 has landed (16 KB a workgroup of 48, and the chip's memory in a third of the time)
    if (n <= 2) wait_vm<0>();
    else if (wv == 0) wait_vm<2 * (kDma + 1)>();
    else wait_vm<2 * kDma>();
    lds_barrier();
    fetch(0, none & 15u, 0);
    widen_keys(0);
    widen_values(0);
    const int kj = D == 64 ? j >> 1 : j;
    const uint8_t* kread = smem + kKeys + ((T / 4) * (j >> 2) + (j & 3)) * 2 * D;
    const uint32_t kpiece = (uint32_t)((g ^ kj) << 4);
    const uint8_t* vread = smem + kValues + j * 2 * T;
    const uint32_t vpiece = (uint32_t)((g ^ value_place(j)) << 4);
    const int x = T == 64 ? g : g >> 1;  // the lane's token group
    int slot = 0, next_page = checked(3, told(3));
    // the next step has landed for all; this one is widened; the one before has been read by all
    auto meet = [&](uint32_t b) __attribute__((always_inline)) {
      if (b + 2 >= n) wait_vm<0>();
      else if (wv == 0) wait_vm<kDma + 1>();
      else wait_vm<kDma>();
      lds_barrier();
    };
    // step b + 3 on its way, in the place of step b, which has been widened
    auto send = [&](uint32_t b) __attribute__((always_inline)) {
      if (b + 3 < n) {
        issue(b + 3, next_page, slot);
        none |= none_of(next_page) << 12;
        if (wv == 0 && (b * kGroups) % 64 == 0 && b * kGroups + 64 < kGroups * n) send_entries(b * kGroups / 64 + 1);
      }
      slot = slot == 2 ? 0 : slot + 1;
      none >>= 4;
    };
    // step b + 1 is widened by all (behind the last step, what the ring happens to hold: nothing reads it)
    if (!active) {
      for (uint32_t b = 0; b < n; ++b) {
        meet(b);
        send(b);
        fetch(b + 1, none & 15u, slot);
        next_page = checked(b + 4, told(b + 4));
        widen_keys(b + 1);
        widen_values(b + 1);
      }
      lds_barrier();  // the ring and the buffers may be filled again
      return;
    }
    for (uint32_t b = 0; b < n; ++b) {
      meet(b);
      const uint8_t* kp = kread + (b & 1) * kBuf;
      const uint8_t* vp = vread + (b & 1) * kBuf;
      auto key = [&](int i) __attribute__((always_inline)) {
        return *reinterpret_cast<const v8bf*>(kp + i / NK * 4 * 2 * D + (kpiece ^ (uint32_t)(i % NK << 6)));
      };
      auto value = [&](int i) __attribute__((always_inline)) {
        return *reinterpret_cast<const v8bf*>(vp + i % NV * 16 * 2 * T + (vpiece ^ (uint32_t)(i / NV << 6)));
      };
      // pieces are read kAhead ahead of their use, the step's first ones here (heads of 256: 72 us, four ahead 75)
      constexpr int kAhead = D == 64 ? 4 : 8;
      v8bf frag[kAhead];
      const uint32_t kbyte = words[(b & 3) * 64 + x], vbyte = words[(b & 3) * 64 + 4 + x];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) frag[i] = key(i);
      const uint32_t gone = none & 15u;
      // The step in sections: the scores of 16 tokens beside the weights of the 16 before.  The weights are
      // relative to a base that follows the scores only where they pass it far (weights up to 2^8 are as
      // exact as those up to 1), and to a whole number, so that what is summed is scaled by a power of two.
      // So no maximum is taken: a lane's weights whose sum passes 2^8, or is infinite or NaN where there is
      // no base yet, tell that the step is made again with another.  That sum bounds each of them, and only
      // passes 2^8 where one of at most 16 passes 2^4: rows with such a score get a new base, and the others'
      // weights are small enough without.  So none is ever used that is larger than 2^8.
      const uint32_t tok0 = (lo + b) * T, gt = tok0 + (T / 4) * g;
      const bool there = !(gone >> x & 1u), bad = kbyte == 255u || vbyte == 255u;
      const bool mask = uniform(gone != 0 || tok0 + T > s.seen || tok0 + T > first || __any(bad)) != 0;
      const float ks = bad || !there ? 1.0f : log2_scale(abs_scale, kbyte);
      v8bf pf[RT][NM];
      v4f sc[2][RT];
      float part[RT];
      auto scores = [&](int y) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          const int i = y * NK + k;
          const v8bf now = frag[i % kAhead];
          frag[i % kAhead] = i + kAhead < NT * NK ? key(i + kAhead) : value(i + kAhead - NT * NK);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            sc[y & 1][rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(now, qf[rt][k], k == 0 ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : sc[y & 1][rt], 0, 0, 0);
        }
      };
      auto masked = [&](int y) __attribute__((always_inline)) {
        if (__builtin_expect(mask, 0)) {
          uint32_t at = gt + 4 * y;
          asm volatile("" : "+v"(at));  // a branch, and all of it there: it is rare
          hide(sc[y & 1], there, bad, at);
        }
      };
      // the weights of instruction y's tokens
      auto weights = [&](int y) __attribute__((always_inline)) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          v4f e;
#pragma unroll
          for (int r = 0; r < 4; ++r) e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[y & 1][rt][r], ks, down[rt]));
          const float four = (e[0] + e[1]) + (e[2] + e[3]);
          part[rt] = y == 0 ? four : part[rt] + four;
          // rounded to bf16, by at most 2^-8 of each weight, as the output itself is: the instruction's type
#pragma unroll
          for (int r = 0; r < 4; ++r) pf[rt][y >> 1][(y & 1) * 4 + r] = (__bf16)e[r];
          // (made here, beside the matrix instructions of this section)
          v4u w = __builtin_bit_cast(v4u, pf[rt][y >> 1]);
          uint32_t w0 = w[(y & 1) * 2], w1 = w[(y & 1) * 2 + 1];
          asm volatile("" : "+v"(w0), "+v"(w1), "+v"(part[rt]));
          w[(y & 1) * 2] = w0;
          w[(y & 1) * 2 + 1] = w1;
          pf[rt][y >> 1] = __builtin_bit_cast(v8bf, w);
        }
      };
      float alpha[RT];  // what the sums so far are scaled by (behind the loop, whose registers stay few)
      int tries = 0;
      for (;; ++tries) {
#pragma unroll
        for (int y = 0; y < NT; ++y) {
          if (y > 0) masked(y - 1);
          scores(y);
          if (y > 0) weights(y - 1);
#pragma unroll
          for (int k = 0; k < NK; ++k) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // a read,
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a matrix instruction,
              if (y > 0) {
                __builtin_amdgcn_sched_group_barrier(0x002, 12 / NK, 0);  // vector instructions,
                __builtin_amdgcn_sched_group_barrier(0x400, 1, 0);        // a power of two
              }
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        masked(NT - 1);
        weights(NT - 1);
        bool far = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) far |= !(part[rt] <= 256.0f);
        // (once: rows that hold NaN, or see nothing yet, stay as they are)
        if (__builtin_expect(tries != 0 || __any(far) == 0, 1)) break;
        asm volatile("");
        float top[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) top[rt] = -INFINITY;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) frag[i] = key(i);
#pragma unroll
        for (int y = 0; y < NT; ++y) {
          scores(y);
          masked(y);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const v4f z = sc[y & 1][rt];
            top[rt] = fmaxf(top[rt], fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])));
          }
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const float row = groups_max(top[rt] * ks), mn = row > mx[rt] + 4.0f ? ceilf(row) : mx[rt];
          const float base = mn == -INFINITY ? 0.0f : mn;
          alpha[rt] = __builtin_amdgcn_exp2f(mx[rt] - base);  // a power of two
          mx[rt] = mn;
          down[rt] = -base;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) frag[i] = key(i);
      }
      if (__builtin_expect(tries != 0, 0)) {
        asm volatile("");
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          sum[rt] *= alpha[rt];
          kept[rt] *= alpha[rt];
#pragma unroll
          for (int d = 0; d < NV; ++d) o[rt][d] *= alpha[rt];
        }
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        sum[rt] += part[rt];
        down[rt] = -mx[rt];  // (infinite where a row has seen nothing)
      }
      // values: (m, y) in order, and before each m's a row of ones, with which the matrix unit adds up the
      // rounded weights (the vector instructions, which bound the step, have no room for that)
      constexpr uint32_t kOnes = 0x3F803F80u;
      const v8bf ones = __builtin_bit_cast(v8bf, v4u{kOnes, kOnes, kOnes, kOnes});
      auto out = [&](int from, int to) __attribute__((always_inline)) {
#pragma unroll
        for (int i = from; i < to; ++i) {
          const v8bf now = frag[i % kAhead];
          if (i + kAhead < NM * NV) frag[i % kAhead] = value(i + kAhead);
          if (i % NV == 0) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) kept[rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, pf[rt][i / NV], kept[rt], 0, 0, 0);
          }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            o[rt][i % NV] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(now, pf[rt][i / NV], o[rt][i % NV], 0, 0, 0);
        }
      };
      constexpr int kAll = NM * NV;
      static_assert(NT * NK % kAhead == 0, "scores end with the first values in frag");
      send(b);
      fetch(b + 1, none & 15u, slot);
      const int page = told(b + 4);
      __builtin_amdgcn_sched_barrier(0);
      out(0, kAll / 4);
      widen_keys(b + 1);
      out(kAll / 4, kAll / 2);
      widen_values(b + 1);
      out(kAll / 2, kAll);
#pragma unroll
      for (int i = 0; i < kAll; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // a read,
        __builtin_amdgcn_sched_group_barrier(0x008, RT, 0);  // matrix instructions,
        if (i % NV == 0) __builtin_amdgcn_sched_group_barrier(0x008, RT, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, I8 ? 6 : 3, 0);
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
      }
      next_page = checked(b + 4, page);
    }
    lds_barrier();  // the ring and the buffers may be filled again
  }
};

}  // namespace

}  // namespace wq
