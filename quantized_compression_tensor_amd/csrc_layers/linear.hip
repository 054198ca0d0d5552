// Matrix products of a linear layer, forward and backward, with their
// epilogues: z[M, N] = sum over k of a[m, k] b[n, k], and then
//   linear   out = act(z + bias) + residual
//   gated    out = act(z[:, :F]) * z[:, F:]
// in float32 on the bf16 matrix cores. An operand lies in memory with its k
// contiguous (x and W of the forward pass) or with its rows contiguous (W for
// dx = dz W, dz and x for dw = dz^T x).
//
// The backward pass first makes dz = dout act'(z) (gated: its two halves) in
// bf16, which is what the matrix cores take: one rounding of 2^-8 that both
// products share. The bias's gradient is summed from dz before that rounding.
// Working z out again inside both products would cost an activation for every
// tile that reads it, and rounding is needed there just the same.
#include <algorithm>
#include <type_traits>

#include "layers_device.h"
#include "layers_internal.h"

namespace taco {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
#define TACO_LDS __attribute__((address_space(3)))

// ------------------------------------------------------------ activations --

// Phi(z), the normal distribution's function, and e = exp(-z^2 / 2). For z < 0
// Phi = erfc(x) / 2 with x = |z| / sqrt(2), and erfc(x) = t Q(t) exp(-x^2),
// t = 1 / (1 + p x): Q is a polynomial of degree 8 fitted to
// exp(x^2) erfc(x) / t over x in [0, 9.5] by iteratively reweighted least
// squares, relative error below 1.3e-8; for z > 0 Phi = 1 - that. In float32
// Phi is within 2.1e-7, and within 2e-6 of its value for |z| < 6 (the rounding
// of exp's argument). About 20 instructions; erff takes two to three times as
// many, which showed in the epilogue and bound the backward pass.
TACO_DEV float normal_cdf(float z, float* e) {
  constexpr float kHalfLog2E = 0.72134752044448170f, kP = 0.26516504294495535f;   // kP = 0.375 / sqrt(2)
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(kP, __builtin_fabsf(z), 1.0f));
  float q = 0.0616967704f;
  q = __builtin_fmaf(q, t, -0.288076138f);
  q = __builtin_fmaf(q, t, 0.433895343f);
  q = __builtin_fmaf(q, t, -0.231078206f);
  q = __builtin_fmaf(q, t, 0.274845342f);
  q = __builtin_fmaf(q, t, 0.121038450f);
  q = __builtin_fmaf(q, t, 0.205430551f);
  q = __builtin_fmaf(q, t, 0.210633482f);
  q = __builtin_fmaf(q, t, 0.211614416f);
  *e = __builtin_amdgcn_exp2f(-(z * z) * kHalfLog2E);
  const float h = 0.5f * t * q * *e;
  return z < 0.0f ? h : 1.0f - h;
}
// 1 / (1 + exp(-z)), to a few units in the last place.
TACO_DEV float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

TACO_DEV float act_value(float t, int act) {
  float e;
  switch (act) {
    case kActGelu: return t * normal_cdf(t, &e);
    case kActSilu: return t * sigmoid(t);
    case kActRelu: return t < 0.0f ? 0.0f : t;   // NaN stays
    default: return t;
  }
}

// act'(t): Phi(t) + t phi(t); s (1 + t (1 - s)) with s = 1 / (1 + exp(-t)); t > 0.
TACO_DEV float act_slope(float t, int act) {
  switch (act) {
    case kActGelu: {
      float e;
      const float cdf = normal_cdf(t, &e);
      return __builtin_fmaf(t * e, 0.39894228040143268f, cdf);
    }
    case kActSilu: {
      const float s = sigmoid(t);
      return s * __builtin_fmaf(t, 1.0f - s, 1.0f);
    }
    case kActRelu: return t > 0.0f ? 1.0f : 0.0f;
    default: return 1.0f;
  }
}
// Both of the gated layer's, with what they share.
TACO_DEV void act_both(float t, int act, float* value, float* slope) {
  if (act == kActGelu) {
    float e;
    const float cdf = normal_cdf(t, &e);
    *value = t * cdf;
    *slope = __builtin_fmaf(t * e, 0.39894228040143268f, cdf);
  } else if (act == kActSilu) {
    const float s = sigmoid(t);
    *value = t * s;
    *slope = s * __builtin_fmaf(t, 1.0f - s, 1.0f);
  } else {
    *value = act_value(t, act);
    *slope = act_slope(t, act);
  }
}

// --------------------------------------------------------------- epilogue --

TACO_DEV void act_values(float* z, int act) {
  if (act == kActNone) return;
  if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_value(z[i], kActGelu);
  } else if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_value(z[i], kActSilu);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_value(z[i], kActRelu);
  }
}

// What an output reads besides its sum, where there is any (finish() uses it
// under the same condition).
TACO_DEV void load_bias(const Epilogue& e, int n, int count, float* b) {
  if (e.bias.p && count > 0) load8(e.bias.p, e.bias.dt, n, count, b);
}
TACO_DEV void load_residual(const Epilogue& e, int64_t m, int n, int count, float* r) {
  if (e.residual.p && count > 0) load8(e.residual.p, e.residual.dt, m * e.residual.ld + n, count, r);
}

// Whether an output is streamed past the caches: where a store instruction
// writes whole 128-byte lines, so bf16 whose rows start on one (4096 x 4096 x
// 512 23.2 us cached, 21.0 streamed). Otherwise the caches join the parts of a
// line, which two tiles write far apart in time (rows 4099 apart 22.2 us
// cached, 28.2 streamed; 8192 x 8192 x 64 with rows 8195 apart 45.2 and 62.4)
// or, in float32, two instructions, each half of a lane's eight (4096 x 4096 x
// 512 27.2 and 41.3). One loss: two outputs and a residual of rows 4099 apart,
// 78.6 and 75.3. (Few rows: no difference.)
TACO_DEV bool streamed(const Mat& t) {
  return t.dt == kBF16 && reinterpret_cast<uintptr_t>(t.p) % 128 == 0 && t.ld % 64 == 0;
}
TACO_DEV void store_out(const Mat& t, int64_t at, int count, const float* z) {
  if (streamed(t)) store8<true>(t.p, kBF16, at, count, z);
  else store8<false>(t.p, t.dt, at, count, z);
}

// Eight neighbouring columns n ... of row m, of which `count` exist, with
// their bias b and residual r.
TACO_DEV void finish(const Epilogue& e, int64_t m, int n, int count, float* z, const float* b, const float* r) {
  if (e.bias.p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += b[i];
  }
  if (e.preact.p) store_out(e.preact, m * e.preact.ld + n, count, z);
  act_values(z, e.act);
  if (e.residual.p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += r[i];
  }
  store_out(e.out, m * e.out.ld + n, count, z);
}
TACO_DEV void finish(const Epilogue& e, int64_t m, int n, int count, float* z) {
  float b[8], r[8];
  load_bias(e, n, count, b);
  load_residual(e, m, n, count, r);
  finish(e, m, n, count, z, b, r);
}
// The same of a gated layer with `width` output columns: z gate, u the other.
// A wave writes 64 bytes of a row, half a line: not streamed (4096 x 4096 x
// 5120 with preact 249.5 us, streamed 253.8).
TACO_DEV void finish_gated(const Epilogue& e, int width, int64_t m, int n, int count, float* z, const float* u) {
  if (e.preact.p) {
    store8<false>(e.preact.p, e.preact.dt, m * e.preact.ld + n, count, z);
    store8<false>(e.preact.p, e.preact.dt, m * e.preact.ld + width + n, count, u);
  }
  act_values(z, e.act);
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] *= u[i];
  store8<false>(e.out.p, e.out.dt, m * e.out.ld + n, count, z);
}

// Whole eights of Q rows, `apart` rows between two, in registers; the element
// type is looked at once.
template <int Q>
TACO_DEV void load_rows(const Mat& t, int64_t m, int apart, int n, float (&z)[Q][8]) {
  const int64_t at = m * t.ld + n;
  if (t.dt == kBF16) {
    Oct<kBF16> o[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) o[q].load(t.p, at + q * apart * t.ld);
#pragma unroll
    for (int q = 0; q < Q; ++q) o[q].get(z[q]);
  } else {
#pragma unroll
    for (int q = 0; q < Q; ++q) load8(t.p, kF32, at + q * apart * t.ld, z[q]);
  }
}
// `stream`: that of streamed(), or false.
template <int Q>
TACO_DEV void store_rows(const Mat& t, int64_t m, int apart, int n, const float (&z)[Q][8], bool stream) {
  const int64_t at = m * t.ld + n;
  if (stream) {
#pragma unroll
    for (int q = 0; q < Q; ++q) store8<true>(t.p, kBF16, at + q * apart * t.ld, 8, z[q]);
  } else if (t.dt == kBF16) {
#pragma unroll
    for (int q = 0; q < Q; ++q) store8<false>(t.p, kBF16, at + q * apart * t.ld, 8, z[q]);
  } else {
#pragma unroll
    for (int q = 0; q < Q; ++q) store8<false>(t.p, kF32, at + q * apart * t.ld, 8, z[q]);
  }
}
template <int Q>
TACO_DEV void act_rows(float (&z)[Q][8], int act) {
  if (act == kActNone) return;
  auto each = [&](int which) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[q][i] = act_value(z[q][i], which);
      __builtin_amdgcn_sched_barrier(0);   // one row's intermediate values at a time
    }
  };
  if (act == kActGelu) each(kActGelu);
  else if (act == kActSilu) each(kActSilu);
  else each(kActRelu);
}
// finish() and finish_gated() of such rows.
template <int Q>
TACO_DEV void finish_rows(const Epilogue& e, int64_t m, int apart, int n, float (&z)[Q][8], const float* b,
                          const float (&r)[Q][8]) {
  if (e.bias.p) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int i = 0; i < 8; ++i) z[q][i] += b[i];
  }
  if (e.preact.p) store_rows(e.preact, m, apart, n, z, streamed(e.preact));
  act_rows(z, e.act);
  if (e.residual.p) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int i = 0; i < 8; ++i) z[q][i] += r[q][i];
  }
  store_rows(e.out, m, apart, n, z, streamed(e.out));
}
template <int Q>
TACO_DEV void finish_gated_rows(const Epilogue& e, int width, int64_t m, int apart, int n, float (&z)[Q][8],
                                const float (&u)[Q][8]) {
  if (e.preact.p) {
    store_rows(e.preact, m, apart, n, z, false);
    store_rows(e.preact, m, apart, width + n, u, false);
  }
  act_rows(z, e.act);
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int i = 0; i < 8; ++i) z[q][i] *= u[q][i];
  store_rows(e.out, m, apart, n, z, false);
}

// ------------------------------------------------------------------ tiles --

template <int BM_, int BN_, int WGM_, int WGN_>
struct Tiles {
  static constexpr int BM = BM_, BN = BN_, BK = 64, WGM = WGM_, WGN = WGN_;
  static constexpr int kThreads = kWave * WGM * WGN;
  static constexpr int TM = BM / WGM / 16, TN = BN / WGN / 16;   // 16 x 16 MFMA tiles of a wave
  static constexpr int kA = BM * BK, kB = BN * BK;               // elements of an LDS stage
  static constexpr int kStagesA = 3, kStagesB = 2;
  // After how many of a slice's rows of MFMA tiles a stage is handed back: b's
  // in the first slice, a's in the second
  static constexpr int kFreeB = TM / 2, kFreeA = TM / 4;
  static constexpr int kTurnLd = TN * 16 + 4, kTurnMost = 32;    // the epilogue's turn: floats of a row, rows at most
  static constexpr int kLdsBytes = (kStagesA * kA + kStagesB * kB) * 2;
  static_assert(WGM * WGN * kTurnMost * kTurnLd * 4 <= kLdsBytes && kLdsBytes <= 160 * 1024, "LDS");
};
using TilesLarge = Tiles<256, 256, 2, 4>;
using TilesSmall = Tiles<128, 128, 2, 2>;
constexpr int kGroupM = 8;   // tile rows walked together (their b rows are shared through L2)

// An LDS read that transposes (see LdsTile::operand). The pointer is marked
// restrict because the compiler otherwise has each such read wait for every
// load into LDS that is under way; hand_over() waits for those that matter.
TACO_DEV s16x4 read_transposed(TACO_LDS s16x4* __restrict__ at) { return __builtin_amdgcn_ds_read_tr16_b64_v4i16(at); }

// A tile of R rows by 64 k in LDS, without padding, in chunks of 8 elements.
// A matrix product reads a chunk column (k contiguous) or blocks of 4 k by 16
// rows (rows contiguous, transposed by the LDS read itself); the chunks of a
// line are permuted by an xor of their number so that either read touches all
// LDS banks evenly.
//   k contiguous      line = row, 8 chunks of 8 k;  chunk c at c ^ ((row >> 1) & 7):
//                     16 neighbouring rows of one chunk column fill 256 bytes
//   rows contiguous   line = k, R / 8 chunks of 8 rows;  chunk c at
//                     c ^ (4 (k & 3) + 2 ((k >> 3) & 1)): the 8 k that half a
//                     wave reads, 32 bytes each, fill 256 bytes
template <bool BY_K, int R>
struct LdsTile {
  static constexpr int BK = 64;
  static constexpr int kPerLine = BY_K ? R / 8 : BK / 8;
  static constexpr int kChunks = R * BK / 8;
  static TACO_DEV int swizzle(int line) {
    return BY_K ? 4 * (line & 3) + 2 * ((line >> 3) & 1) : (line >> 1) & 7;
  }
  // Number in its line of the chunk at position q of the tile in LDS.
  static TACO_DEV int chunk_of(int q) { return (q % kPerLine) ^ swizzle(q / kPerLine); }
  // Operand of a 16 x 16 x 32 product: lane l holds row r0 + l % 16 and the
  // eight k of 32 kk + 8 (l / 16).
  static TACO_DEV bf16x8 operand(const uint16_t* t, int r0, int kk, int lane) {
    if constexpr (!BY_K) {
      const int r = r0 + (lane & 15), c = 4 * kk + (lane >> 4);
      return *reinterpret_cast<const bf16x8*>(t + r * BK + (c ^ swizzle(r)) * 8);
    } else {
      // a read takes, for each 16 lanes, 4 k of 16 rows from addresses of 4
      // rows each, and gives lane i of them the four k of row i
      const int k = 32 * kk + 8 * (lane >> 4) + ((lane >> 2) & 3);
      const int r = r0 + 4 * (lane & 3);
      union {
        s16x4 h[2];
        bf16x8 v;
      } u;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int kl = k + 4 * i;
        TACO_LDS uint16_t* at = (TACO_LDS uint16_t*)t + (kl * R + ((r >> 3) ^ swizzle(kl)) * 8 + (r & 7));
        u.h[i] = read_transposed((TACO_LDS s16x4*)at);
      }
      return u.v;
    }
  }
};

// How a thread's chunks of one operand's tile get from memory into LDS.
// GATED (k contiguous only): of each 64 lines the first 32 are rows of the
// gate's projection, from p, and the others rows of the other one, from p2.
template <bool BY_K, int R, int NT, bool GATED>
struct Chunks {
  using Tile = LdsTile<BY_K, R>;
  static constexpr int BK = Tile::BK;
  static constexpr int kPer = Tile::kChunks / NT;   // of a thread
  static constexpr int kLines = NT / Tile::kPerLine;   // between two of its chunks
  static_assert(Tile::kChunks % NT == 0, "whole chunks for every thread");
  static_assert(!GATED || (!BY_K && (NT == 256 || NT == 512)), "gated tiles");
  static TACO_DEV int line(int tid, int i) { return tid / Tile::kPerLine + i * kLines; }
  static TACO_DEV int chunk(int tid, int i) { return Tile::chunk_of(tid + i * NT); }
  // (k contiguous: the swizzle has a period of 16 lines, so all of a thread's
  // chunks have one number)
  static_assert(BY_K || kLines % 16 == 0, "one chunk number per thread");
  static TACO_DEV int row(int l) { return GATED ? l / 64 * 32 + l % 32 : l; }
  // Whether chunk i of this wave comes from p2 (wave-uniform: a wave's lines
  // lie within 32).
  static TACO_DEV bool second(int wave, int i) {
    return GATED && ((wave * (kWave / Tile::kPerLine) + i * kLines) / 32 & 1) != 0;
  }
};

// 16 bytes per lane from byte offset `off` of the resource to LDS: lane l's to
// t + 8 l.
TACO_DEV void load_to_lds(rsrc_t r, int off, uint16_t* t) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (TACO_LDS void*)t, 16, off, 0, 0, 0);
}

// Moves an operand's tiles straight into LDS, 16 bytes per lane without
// passing the registers. Wants rows on 16 bytes and eights along the
// contiguous axis (k_pack makes others so). What lies outside the operand
// reads as zeros: past its last row by the size of the buffer resource, past
// its last k (k contiguous) by an offset that is outside it.
template <bool BY_K, int R, int NT, bool GATED>
struct Loader : Chunks<BY_K, R, NT, GATED> {
  using C = Chunks<BY_K, R, NT, GATED>;
  static constexpr int BK = C::BK;
  static constexpr int kOutside = 0x7FFFFFF0;
  const char *p, *p2;
  int64_t bytes;    // of the operand from p on
  int64_t step;     // bytes from one K step to the next
  int off[C::kPer];
  int chunk_k;      // k of this thread's chunks in a step (k contiguous)
  TACO_DEV void init(const uint16_t* base, const uint16_t* base2, int64_t ld, int rows, int64_t K, int tid) {
    p = reinterpret_cast<const char*>(base);
    p2 = reinterpret_cast<const char*>(base2);
    // whole eights along the contiguous axis: what lies past it is readable
    bytes = 2 * (BY_K ? (K - 1) * ld + (rows + 7) / 8 * 8 : (rows - 1) * ld + (K + 7) / 8 * 8);
    step = 2 * (BY_K ? BK * ld : BK);
    chunk_k = BY_K ? 0 : 8 * C::chunk(tid, 0);
#pragma unroll
    for (int i = 0; i < C::kPer; ++i) off[i] = C::row(C::line(tid, i)) * (int)ld * 2 + 16 * C::chunk(tid, i);
  }
  // Starts load i of a step whose first k has `left` k after it; after the
  // last one, moves on to the next step.
  TACO_DEV void issue(uint16_t* t, int wave, int64_t left, int i) {
    const int64_t size = left > 0 ? bytes : 0;   // past the last step: no access
    const bool in = BY_K || chunk_k < left;
    load_to_lds(make_rsrc(C::second(wave, i) ? p2 : p, size), in ? off[i] : kOutside, t + (i * NT + wave * kWave) * 8);
    if (i == C::kPer - 1) {
      p += step;
      p2 += step;
      bytes -= step;
    }
  }
};

// Output tile of this workgroup: each XCD walks one contiguous range of tiles
// (xcd_ordered_block() for any index of any count), and inside it groups of
// kGroupM tile rows column by column, so the workgroups resident on an XCD share
// rows of a and of b through its L2.
TACO_DEV unsigned xcd_ordered(unsigned b, unsigned G) {
  const unsigned x = b % kXcds, l = b / kXcds, q = G / kXcds, r = G % kXcds;
  return x * q + (x < r ? x : r) + l;
}
TACO_DEV void tile_of(unsigned t, unsigned ntm, unsigned ntn, unsigned* tm, unsigned* tn) {
  const unsigned per_group = kGroupM * ntn, group = t / per_group, in_group = t % per_group;
  const unsigned first = group * kGroupM, rows = ntm - first < kGroupM ? ntm - first : kGroupM;
  *tm = first + in_group % rows;
  *tn = in_group / rows;
}

// A barrier before which a wave waits until at most LDS of its latest LDS
// accesses and LOADS of its latest loads into LDS are under way (LOADS < 0:
// any number; both complete in order). Written out because the compiler's own
// barrier would wait for all of them.
template <int LDS, int LOADS>
TACO_DEV void hand_over() {
  // s_waitcnt: vmcnt in bits 0-3 and 14-15, lgkmcnt in bits 8-11, expcnt (no wait) in bits 4-6
  constexpr int kVm = LOADS < 0 ? 63 : LOADS;
  static_assert(LDS < 16 && kVm < 64, "counters");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((kVm & 15) | (kVm >> 4) << 14 | LDS << 8 | 0x0070);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The kernel of every product: a workgroup sums one output tile over one part
// of K, in steps of 64 k, two slices of 32 each. What bounds it is how far
// ahead of their use loads can be under way (a step lasts about 1.4 us, a load
// about 1.3 us when every CU loads), so the LDS holds three steps of a and two
// of b, and a stage is handed back as soon as it has been read: b's operands
// are all in registers early in a step, a's follow one 16-row tile behind the
// products that used the registers before. Every load has then one and a half
// or two steps' time. The 16 x 16 x 32 products were faster than 32 x 32 x 16
// (8192^3: 750 against 815 us) although they leave more gaps: this size is
// bound by power, and they move half as many sums through the registers.
// Measured, random values, bf16 outputs, on one card 8192^3 forward 807 us
// (1360 TFLOP/s), dx 833, dw 879, where the library's product took 725, and
// 4096^3 104 (1320), 108 and 114 (112); on a faster one 737, 763, 798 and 96,
// 100, 104. In profiled launches (8192^3 900 us, 4096^3 108 and 114) the matrix
// cores are busy 0.73 of the time at 1.67 GHz, the gradients 0.68 and 0.62 at
// 2.1; the LDS serves reads in 0.25 to 0.29 of the cycles.
// A small tile takes 0.55 us a step on a CU of its own, and two together 1.1
// for both. The counters show no unit that it fills: matrix cores 0.42 to 0.45
// at 2.4 GHz, LDS 0.22 to 0.26, and L2 gives 14 to 19 TB/s where a loop of reads
// gets 31 to 33. Five stages of a and four of b instead of three and two, for one
// tile on a CU, were no faster, so a longer reach ahead is not what is missing.
// `block`: of the product's a.whole + a.rest * a.parts.
template <class TL, bool AK, bool BK_, bool GATED>
TACO_DEV void gemm(const GemmArgs& a, unsigned block) {
  constexpr int BM = TL::BM, BN = TL::BN, BK = TL::BK, TM = TL::TM, TN = TL::TN, NT = TL::kThreads;
  constexpr int kCols = GATED ? BN / 2 : BN;   // output columns of a tile
  static_assert(!GATED || TN == 4, "a wave holds the two projections of its columns");
  extern __shared__ __attribute__((aligned(1024))) uint16_t lds[];
  const int tid = (int)threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid) / kWave;
  const int wm = wave / TL::WGN, wn = wave % TL::WGN;
  const unsigned ntm = (unsigned)((a.M + BM - 1) / BM), ntn = (unsigned)(a.N + kCols - 1) / kCols;
  // the tiles with all of K, then the parts of the others, each in its own order
  const bool whole = block < a.whole;
  const unsigned index = whole ? xcd_ordered(block, a.whole) : xcd_ordered(block - a.whole, a.rest * a.parts);
  const unsigned part = whole ? 0 : index / a.rest;
  unsigned tm, tn;
  tile_of(whole ? index : a.whole + index % a.rest, ntm, ntn, &tm, &tn);
  const int64_t m0 = (int64_t)tm * BM, k0 = part * a.part;
  const int n0 = (int)tn * kCols;
  const int64_t K = whole || a.K - k0 < a.part ? a.K - k0 : a.part;   // of this part
  const int rows_a = (int)(a.M - m0 < BM ? a.M - m0 : BM), rows_b = a.N - n0 < kCols ? a.N - n0 : kCols;
  const uint16_t* pa = a.a.p + (AK ? m0 + k0 * a.a.ld : m0 * a.a.ld + k0);
  const uint16_t* pb = a.b.p + (BK_ ? n0 + k0 * a.b.ld : n0 * a.b.ld + k0);
  const uint16_t* pb2 = GATED ? pb + (int64_t)a.N * a.b.ld : pb;
  using LA = Loader<AK, BM, NT, false>;
  using LB = Loader<BK_, BN, NT, GATED>;
  LA la;
  LB lb;
  la.init(pa, pa, a.a.ld, rows_a, K, tid);
  lb.init(pb, pb2, a.b.ld, rows_b, K, tid);
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;

  const int steps = (int)((K + BK - 1) / BK);
  uint16_t *const lds_a = lds, *const lds_b = lds + TL::kStagesA * TL::kA;
  bf16x8 fa[TM], fb[2][TN];
  auto read_a = [&](const uint16_t* t, int kk, int i) { fa[i] = LdsTile<AK, BM>::operand(t, (wm * TM + i) * 16, kk, lane); };
  auto read_b = [&](const uint16_t* t, int kk) {
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[kk][j] = LdsTile<BK_, BN>::operand(t, (wn * TN + j) * 16, kk, lane);
  };
  auto multiply = [&](int kk, int i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[kk][j], acc[i][j], 0, 0, 0);
  };
  // Part `part` of `parts` of the loads of step ks into stage t.
  auto load = [&](auto& l, int ks, uint16_t* t, int part, int parts) {
    constexpr int kPer = std::remove_reference_t<decltype(l)>::kPer;
    const int each = (kPer + parts - 1) / parts;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i / each == part) l.issue(t, wave, K - (int64_t)ks * BK, i);
  };
  if (steps > 0) {
    uint16_t *a0 = lds_a, *a1 = lds_a + TL::kA, *a2 = lds_a + 2 * TL::kA;   // of this step and the next two
    uint16_t *b0 = lds_b, *b1 = lds_b + TL::kB;
    load(la, 0, a0, 0, 1);
    load(lb, 0, b0, 0, 1);
    load(la, 1, a1, 0, 1);
    load(lb, 1, b1, 0, 1);
    load(la, 2, a2, 0, 1);
    hand_over<0, 2 * LA::kPer + LB::kPer>();
#pragma unroll
    for (int i = 0; i < TM; ++i) read_a(a0, 0, i);
    read_b(b0, 0);
    constexpr int kFreeA = TL::kFreeA, kFreeB = TL::kFreeB;
#pragma unroll 1
    for (int ks = 0; ks < steps; ++ks) {
      read_b(b0, 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        // b0 has been read to its end: the reads since are those of kFreeB operands of a
        if (i == kFreeB) hand_over<kFreeB * (AK ? 2 : 1), -1>();
        if (i >= kFreeB) load(lb, ks + 2, b0, i - kFreeB, TM - kFreeB);
        multiply(0, i);
        read_a(a0, 1, i);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        if (i == kFreeA) {
          // a0 has been read to its end, a1 and b1 are there; past the last
          // step what is read from them is not used
          hand_over<0, LA::kPer + LB::kPer>();
#pragma unroll
          for (int q = 0; q < i; ++q) read_a(a1, 0, q);
        }
        if (i >= kFreeA) load(la, ks + 3, a0, i - kFreeA, TM - kFreeA);
        multiply(1, i);
        if (i >= kFreeA) read_a(a1, 0, i);
        if (i == kFreeA + 1) read_b(b1, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      uint16_t* t = a0;
      a0 = a1;
      a1 = a2;
      a2 = t;
      t = b0;
      b0 = b1;
      b1 = t;
    }
  }
  hand_over<0, 0>();

  // Accumulator e of lane l holds row 4 (l / 16) + e, column l % 16 of its
  // tile. Each wave turns kTurnRows rows at a time round through its own part
  // of LDS, so that a lane has eight neighbouring columns of a row, and has the
  // residuals of all of its rows under way together. A turn's code is there
  // once (the sums move down instead: its copies did not fit the instruction
  // cache), and tiles without an edge take a path of their own, whose branches
  // are all scalar: 2048 x 2048 x 64 7.4 to 6.3 us, 4096 x 4096 x 512 with
  // bias, gelu and a residual 38.6 to 32.3. A turn has 32 rows (gated 4096 x
  // 4096 x 512 43.4 us, with 16 rows 46.4), or 16 where there may be a residual,
  // whose registers there are not enough of.
  constexpr bool kPlain = BK_;   // a gradient: the sum itself is the output
  constexpr int kLd = TL::kTurnLd, kTurnRows = kPlain || GATED ? TL::kTurnMost : 16, kTurn = kTurnRows / 16;
  constexpr int kWaveCols = GATED ? TN * 8 : TN * 16, kLanes = kWaveCols / 8;
  constexpr int kPass = kWave / kLanes, kRound = kTurnRows / kPass;   // rows of a pass, passes
  float* turn = reinterpret_cast<float*>(lds) + wave * kTurnRows * kLd;
  const int c = (lane % kLanes) * 8, n = n0 + wn * kWaveCols + c, count = a.N - n;
  const bool full = rows_a == BM && rows_b == kCols;
  float bias[8];
  if (!GATED && !kPlain) load_bias(a.e, n, whole ? count : 0, bias);
#pragma unroll 1
  for (int i0 = 0; i0 < TM; i0 += kTurn) {
#pragma unroll
    for (int h = 0; h < kTurn; ++h)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          turn[(16 * h + 4 * (lane >> 4) + e) * kLd + j * 16 + (lane & 15)] = acc[h][j][e];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    int rows_done = i0 * 16;
    asm volatile("" : "+s"(rows_done));   // addresses are not carried from turn to turn: they would take 40 registers
    const int64_t m = m0 + wm * TM * 16 + rows_done + lane / kLanes;
    const float* row = turn + (lane / kLanes) * kLd + c;
    if (!whole || full) {
      float z[kRound][8], u[GATED ? kRound : 1][8], r[kPlain || GATED ? 1 : kRound][8];
      if constexpr (!GATED && !kPlain) {
        if (whole && a.e.residual.p) load_rows(a.e.residual, m, kPass, n, r);
      }
#pragma unroll
      for (int q = 0; q < kRound; ++q)
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
          *reinterpret_cast<f32x4*>(z[q] + h) = *reinterpret_cast<const f32x4*>(row + q * kPass * kLd + h);
          if constexpr (GATED)
            *reinterpret_cast<f32x4*>(u[q] + h) = *reinterpret_cast<const f32x4*>(row + q * kPass * kLd + kWaveCols + h);
        }
      if (!whole) {
        float* part_row = a.partials + ((int64_t)index * BM + (m - m0)) * BN + (n - n0);
#pragma unroll
        for (int q = 0; q < kRound; ++q) {
          if (m + q * kPass >= a.M || count <= 0) continue;
          keep8(part_row + q * kPass * BN, z[q]);   // eights past the last column too: the tile has room
          if constexpr (GATED) keep8(part_row + q * kPass * BN + kCols, u[q]);
        }
      } else if constexpr (GATED) {
        finish_gated_rows(a.e, a.N, m, kPass, n, z, u);
      } else if constexpr (kPlain) {
        store_rows(a.e.out, m, kPass, n, z, streamed(a.e.out));
      } else {
        finish_rows(a.e, m, kPass, n, z, bias, r);
      }
    } else {
#pragma unroll 1
      for (int q = 0; q < kRound; ++q) {
        if (m + q * kPass >= a.M || count <= 0) continue;
        float z[8], u[8], r[8];
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
          *reinterpret_cast<f32x4*>(z + h) = *reinterpret_cast<const f32x4*>(row + q * kPass * kLd + h);
          if (GATED) *reinterpret_cast<f32x4*>(u + h) = *reinterpret_cast<const f32x4*>(row + q * kPass * kLd + kWaveCols + h);
        }
        if constexpr (GATED) {
          finish_gated(a.e, a.N, m + q * kPass, n, count, z, u);
        } else if constexpr (kPlain) {
          store_out(a.e.out, (m + q * kPass) * a.e.out.ld + n, count, z);
        } else {
          load_residual(a.e, m + q * kPass, n, count, r);
          finish(a.e, m + q * kPass, n, count, z, bias, r);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i + kTurn < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = acc[i + kTurn][j];
  }
}

template <class TL, bool AK, bool BK_, bool GATED>
__global__ __launch_bounds__(TL::kThreads, 2) void k_gemm(GemmArgs a) {
  gemm<TL, AK, BK_, GATED>(a, blockIdx.x);
}
// All gradients at once, where the products do not fill the device: dx = dz W
// in the first `count_dx` workgroups, dw = dz^T x in the next `count_dw`, and
// the bias's, which reads what k_act_back left, in the others (1001 x 777 x
// 1285: 27.9 us with a launch of its own for the latter, 24.2).
template <class TL>
__global__ __launch_bounds__(TL::kThreads, 2) void k_gemm_pair(GemmArgs dx, GemmArgs dw, ColumnSumArgs sum,
                                                               unsigned count_dx, unsigned count_dw) {
  extern __shared__ __attribute__((aligned(1024))) uint16_t lds[];
  const unsigned b = blockIdx.x;
  if (b < count_dx) gemm<TL, false, true, false>(dx, b);
  else if (b < count_dx + count_dw) gemm<TL, true, true, false>(dw, b - count_dx);
  else column_sum<TL::kThreads / kWave>(sum, b - count_dx - count_dw, 0, reinterpret_cast<float*>(lds));
}

// Joins the parts of the tiles whose K is cut, in order, and finishes: a
// workgroup takes some rows of a tile (blockIdx.x), a lane eight columns. Bound
// by the parts' bytes, mostly out of the Infinity Cache: 15 us for 128 gated
// tiles in two parts with both projections kept (92 MB, 6 TB/s).
template <class TL, bool GATED>
__global__ __launch_bounds__(256) void k_join(GemmArgs a) {
  constexpr int BM = TL::BM, BN = TL::BN, kCols = GATED ? BN / 2 : BN, kOcts = kCols / 8, kRows = 256 / kOcts;
  const unsigned ntm = (unsigned)((a.M + BM - 1) / BM), ntn = (unsigned)(a.N + kCols - 1) / kCols;
  unsigned tm, tn;
  tile_of(a.whole + blockIdx.x, ntm, ntn, &tm, &tn);
  const int row = (int)blockIdx.y * kRows + (int)threadIdx.x / kOcts, col = (int)threadIdx.x % kOcts * 8;
  const int64_t m = (int64_t)tm * BM + row;
  const int n = (int)tn * kCols + col;
  if (m >= a.M || n >= a.N) return;
  float z[8], u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = 0.0f, u[e] = 0.0f;
  for (unsigned p = 0; p < a.parts; ++p) {
    const float* at = a.partials + (((int64_t)p * a.rest + blockIdx.x) * BM + row) * BN + col;
    float f[8];
    load8(at, kF32, 0, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] += f[e];
    if (GATED) {
      load8(at, kF32, kCols, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] += f[e];
    }
  }
  if (GATED) finish_gated(a.e, a.N, m, n, a.N - n, z, u);
  else finish(a.e, m, n, a.N - n, z);
}

// --------------------------------------------------------------- few rows --

// Up to 32 rows of x: the weight's bytes bound it, so every weight is read
// once, straight into the registers of a 16 x 16 x 32 product whose other
// operand is x (rows past the last one repeat it; their sums are not stored).
// A workgroup takes up to 16 weight rows (gated: eight of each projection; as
// many as give every CU the same number of workgroups), its sixteen waves units
// of 64 k in turn, so that a row's bytes are read 2 KiB at a time, two units of
// a wave together. The waves' sums are joined in LDS. Rows may start anywhere.
// One row, 8192 x 8192 weights: 27.6 us, 4.9 TB/s (eight waves with eight units
// each 31.8 us); 4096 x 4096: 7.6 us. With 24 rows the reads of x, which every
// workgroup makes, are more than those of the weights: 24 x 5120 into 2 x 1728
// gated 13.8 us (2.6 TB/s). Counters of that one: 37 MB from memory, 111 MB out
// of L2 (7 TB/s), neither near its rate, and waves that wait 0.96 of their time,
// for three rounds of loads one after the other. Loading further ahead was
// slower everywhere (that one 19.7 us and more), and x's lanes without a row
// left out no faster.
constexpr int kFewRows = 32, kFewWaves = 16;

template <int TM, bool GATED>
__global__ __launch_bounds__(kFewWaves * kWave) void k_few_rows(GemmArgs a) {
  constexpr int kUnits = 2;   // of a wave, loaded together
  __shared__ float parts[kFewWaves][TM][4 * kWave];
  __shared__ float sums[16 * TM][16];
  const int tid = (int)threadIdx.x, lane = tid & (kWave - 1), wave = wave_in_group();
  const int n0 = (int)blockIdx.x * a.cols, r = lane & 15;
  const int cols = a.N - n0 < a.cols ? a.N - n0 : a.cols;   // of this workgroup; lanes past them repeat the last
  int n = GATED ? r & 7 : r;
  n = n0 + (n < cols ? n : cols - 1);
  const uint16_t* pw = a.b.p + (GATED && r >= 8 ? n + (int64_t)a.N : n) * a.b.ld + 8 * (lane >> 4);
  const uint16_t* px[TM];
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    const int64_t m = 16 * t + r;
    px[t] = a.a.p + (m < a.M ? m : a.M - 1) * a.a.ld + 8 * (lane >> 4);
  }
  f32x4 acc[TM];
#pragma unroll
  for (int t = 0; t < TM; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto product = [&](const Oct<kBF16>& w, const Oct<kBF16>& x, int t) {
    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w.v), __builtin_bit_cast(bf16x8, x.v),
                                                     acc[t], 0, 0, 0);
  };
  const int units = (int)(a.K / 64);
  for (int first = wave; first < units; first += kFewWaves * kUnits) {
    Oct<kBF16> w[kUnits][2], x[kUnits][TM][2];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int unit = first + u * kFewWaves;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[u][h].clear();
        if (unit < units) w[u][h].load(pw, 64 * (int64_t)unit + 32 * h);
#pragma unroll
        for (int t = 0; t < TM; ++t) {
          x[u][t][h].clear();
          if (unit < units) x[u][t][h].load(px[t], 64 * (int64_t)unit + 32 * h);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < TM; ++t) product(w[u][h], x[u][t][h], t);
  }
  if (wave == units % kFewWaves) {
    // the last k, fewer than 64
    for (int64_t k = 64 * (int64_t)units; k < a.K; k += 32) {
      const int64_t left = a.K - k - 8 * (lane >> 4);
      const int count = left > 8 ? 8 : left > 0 ? (int)left : 0;
      Oct<kBF16> w, x;
      w.load(pw, k, count);
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        x.load(px[t], k, count);
        product(w, x, t);
      }
    }
  }
  // accumulator e of lane l holds weight row 4 (l / 16) + e, row l % 16 of x
#pragma unroll
  for (int t = 0; t < TM; ++t) *reinterpret_cast<f32x4*>(&parts[wave][t][4 * lane]) = acc[t];
  __syncthreads();
  for (int i = tid; i < TM * 4 * kWave; i += kFewWaves * kWave) {
    const int t = i / (4 * kWave), q = i % (4 * kWave), l = q / 4;
    float z = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) z += parts[w][t][q];
    sums[16 * t + l % 16][4 * (l / 16) + q % 4] = z;
  }
  __syncthreads();
  const int m = GATED ? tid : tid / 2, c = GATED ? 0 : tid % 2 * 8;
  if (m >= a.M || m >= 16 * TM || c >= cols) return;
  float z[8], u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    z[e] = sums[m][c + e];
    u[e] = sums[m][(c + 8 + e) % 16];
  }
  if (GATED) finish_gated(a.e, a.N, m, n0, cols, z, u);
  else finish(a.e, m, n0 + c, cols - c, z);
}

// ----------------------------------------------------------------- launch --

// Which tiles a product takes, and how many of them take all of K. Decided by
// the sizes alone, so that the workspace is known before the call.
struct Plan {
  bool large;
  unsigned whole, rest, parts;
  int64_t part;
};

constexpr int kCus = 256;   // of an MI355X; not asked of the device, so that sizes alone decide a workspace
static int64_t tiles_of(int64_t M, int64_t N, int bm, int cols) { return ((M + bm - 1) / bm) * ((N + cols - 1) / cols); }

// `other`: steps of the tiles of another product that run at the same time.
static Plan plan_of(int64_t M, int64_t N, int64_t K, bool gated, int64_t other = 0) {
  const int64_t large = tiles_of(M, N, 256, gated ? 128 : 256), steps = (K + 63) / 64;
  const bool is_large = large >= 192;
  const int64_t tiles = is_large ? large : tiles_of(M, N, 128, gated ? 64 : 128);
  // Tiles go to 256 CUs: one of 256 x 256 at a time, or two of 128 x 128, which
  // take twice as long together. The last round of tiles, if it is not full,
  // has its K cut where that shortens it by more than the parts' way through
  // memory and the launch that joins them take: 1100 x 4000 x 4000 47.8 us, cut
  // for two small tiles to a CU 64.1; gated 512 x 5120 x 5120 71.3 us, not cut
  // 91.7. Times in us: a step, a round of parts, the launch. A part keeps at
  // least eight steps (with four, 128 x 4096 x 4096 took 23.4 us, with eight
  // 18.8).
  const double step = is_large ? 1.45 : 0.56, round = is_large ? 30.0 : 6.0, launch = 3.0;
  const int64_t rest = tiles % kCus, most = std::min<int64_t>(steps / 8, 16);
  int64_t parts = 1;
  double least = 0.0;
  for (int64_t p = 1; rest > 0 && p <= std::max<int64_t>(most, 1); ++p) {
    const int64_t per = (steps + p - 1) / p;
    const double busy = other > 0 ? std::max((double)per, (double)(tiles * steps + other) / (double)kCus)
                                  : (double)((rest * p + kCus - 1) / kCus * per);
    const double t = busy * step + (p > 1 ? launch + round * (double)(rest * p) / (double)kCus : 0.0);
    if (p == 1 || t < least) parts = p, least = t;
  }
  if (parts <= 1) return Plan{is_large, (unsigned)tiles, 0, 1, 0};
  const int64_t per = (steps + parts - 1) / parts;
  return Plan{is_large, (unsigned)(tiles - rest), (unsigned)rest, (unsigned)((steps + per - 1) / per), per * 64};
}

static size_t partial_bytes(const Plan& p) {
  const size_t tile = p.large ? 256 * 256 : 128 * 128;
  return (size_t)p.rest * p.parts * tile * sizeof(float);
}
size_t gemm_partial_bytes(int64_t M, int64_t N, int64_t K, bool gated) {
  return M == 0 ? 0 : partial_bytes(plan_of(M, N, K, gated));
}

// Both gradients of a projection with `wide` weight rows: together where
// neither takes large tiles and both fit the slots.
struct PairPlan {
  bool together;
  Plan dx, dw;
};
static PairPlan pair_plan_of(int64_t M, int64_t wide, int64_t K) {
  const int64_t dx_tiles = tiles_of(M, K, 128, 128), dw_tiles = tiles_of(wide, K, 128, 128);
  PairPlan p = {false, plan_of(M, K, wide, false, dw_tiles * ((M + 63) / 64)),
                plan_of(wide, K, M, false, dx_tiles * ((wide + 63) / 64))};
  p.together = M > 0 && !p.dx.large && !p.dw.large && dx_tiles + dw_tiles <= 512;
  return p;
}
size_t gemm_pair_partial_bytes(int64_t M, int64_t wide, int64_t K) {
  const PairPlan p = pair_plan_of(M, wide, K);
  return p.together ? partial_bytes(p.dx) + partial_bytes(p.dw) : 0;
}

static void set_plan(GemmArgs* a, const Plan& p, void* partials) {
  a->whole = p.whole;
  a->rest = p.rest;
  a->parts = p.parts;
  a->part = p.part;
  a->partials = static_cast<float*>(partials);
}

template <class TL>
static void launch_join(const GemmArgs& a, hipStream_t s) {
  if (a.rest == 0) return;
  const int octs = (a.gated ? TL::BN / 2 : TL::BN) / 8, rows = 256 / octs;
  const dim3 join(a.rest, (unsigned)(TL::BM / rows));
  if (a.gated) hipLaunchKernelGGL((k_join<TL, true>), join, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_join<TL, false>), join, dim3(256), 0, s, a);
}

template <class TL>
static void launch_tiles(const GemmArgs& a, hipStream_t s) {
  const dim3 grid(a.whole + a.rest * a.parts), block(TL::kThreads);
  constexpr size_t lds = TL::kLdsBytes;
  if (a.gated) hipLaunchKernelGGL((k_gemm<TL, false, false, true>), grid, block, lds, s, a);
  else if (!a.a.by_k && !a.b.by_k) hipLaunchKernelGGL((k_gemm<TL, false, false, false>), grid, block, lds, s, a);
  else if (!a.a.by_k) hipLaunchKernelGGL((k_gemm<TL, false, true, false>), grid, block, lds, s, a);
  else hipLaunchKernelGGL((k_gemm<TL, true, true, false>), grid, block, lds, s, a);
  launch_join<TL>(a, s);
}

// Whether a forward product takes the kernel for few rows. Every workgroup
// reads all of x, so tiles are faster where rows times weights are many (16
// rows of 8192 x 8192: 33.2 against 39.5 us; 8 of 5120 x 20480: 46.5 against
// 53.7), and not where they are few (8 of 8192 x 8192: 30.8 against 32.7 us;
// 24 of 3456 x 5120: 15.6 against 19.9).
bool few_rows(int64_t M, int64_t N, int64_t K, bool gated) {
  const int64_t weights = (gated ? 2 : 1) * N * K;
  return M <= 4 || (M <= kFewRows && weights * M <= int64_t(1) << 29);
}

static void launch_few_rows(GemmArgs a, hipStream_t s) {
  // as many columns for a workgroup as give each CU the same number of them
  // (one row, 5120 x 20480: 41.9 us with 512 workgroups of 10 columns, 52.6
  // with 320 of 16); a few workgroups more than that run beside the others
  const int most = a.gated ? 8 : 16, cus = kCus;
  const int groups = (a.N + most - 1) / most, rounds = std::max(1, (groups - cus / 8 + cus - 1) / cus);
  a.cols = std::min(most, (a.N + rounds * cus - 1) / (rounds * cus));
  const dim3 grid((unsigned)((a.N + a.cols - 1) / a.cols)), block(kFewWaves * kWave);
  if (a.M <= 16) {
    if (a.gated) hipLaunchKernelGGL((k_few_rows<1, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_few_rows<1, false>), grid, block, 0, s, a);
  } else {
    if (a.gated) hipLaunchKernelGGL((k_few_rows<2, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_few_rows<2, false>), grid, block, 0, s, a);
  }
}

hipError_t launch_gemm(GemmArgs a, void* partials, hipStream_t s) {
  if (a.M == 0) return hipSuccess;
  if (!a.a.by_k && !a.b.by_k && few_rows(a.M, a.N, a.K, a.gated)) {
    launch_few_rows(a, s);
    return hipGetLastError();
  }
  const Plan p = plan_of(a.M, a.N, a.K, a.gated);
  set_plan(&a, p, partials);
  if (p.large) launch_tiles<TilesLarge>(a, s);
  else launch_tiles<TilesSmall>(a, s);
  return hipGetLastError();
}

hipError_t launch_gemm_pair(GemmArgs dx, GemmArgs dw, const ColumnSumArgs& sum, void* partials, hipStream_t s) {
  const PairPlan p = pair_plan_of(dx.M, dw.M, dx.N);
  if (!p.together) {
    launch_column_sum(sum, s);
    const hipError_t err = launch_gemm(dx, partials, s);
    return err == hipSuccess ? launch_gemm(dw, partials, s) : err;
  }
  set_plan(&dx, p.dx, partials);
  set_plan(&dw, p.dw, static_cast<char*>(partials) + partial_bytes(p.dx));
  const unsigned count_dx = dx.whole + dx.rest * dx.parts, count_dw = dw.whole + dw.rest * dw.parts;
  const unsigned count_sum = sum.out[0].p ? (unsigned)((sum.cols + kWave - 1) / kWave) : 0;
  const dim3 grid(count_dx + count_dw + count_sum), block(TilesSmall::kThreads);
  hipLaunchKernelGGL((k_gemm_pair<TilesSmall>), grid, block, TilesSmall::kLdsBytes, s, dx, dw, sum, count_dx, count_dw);
  launch_join<TilesSmall>(dx, s);
  launch_join<TilesSmall>(dw, s);
  return hipGetLastError();
}

// ----------------------------------------------------------------- packing --

// Copies bf16 matrices so that rows start on 16 bytes and hold a multiple of
// eight elements, zeros past the last: the tiles' loads into LDS want that,
// and a copy at memory's speed costs less than loads that do not (4096 x 4096
// x 4097 forward: 190 us with tiles staged through registers, 135 packed). A
// lane takes eight elements; `block` of `blocks` for matrix `which`.
TACO_DEV void pack(const PackArgs& a, unsigned block, unsigned blocks, unsigned which) {
  const PackArgs::One m = a.m[which];
  const int64_t octs = (m.cols + 7) / 8, total = m.rows * octs;
  for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < total; i += (int64_t)blocks * 256) {
    // (a division in 64 bits takes five times as long)
    const int64_t row = total <= UINT32_MAX ? (uint32_t)i / (uint32_t)octs : i / octs;
    const int64_t c = (i - row * octs) * 8, left = m.cols - c;
    Oct<kBF16> o;
    o.load(m.src.p, row * m.src.ld + c, left < 8 ? (int)left : 8);
    *reinterpret_cast<u32x4*>(m.dst + row * m.ld + c) = o.v;
  }
}
__global__ __launch_bounds__(256) void k_pack(PackArgs a) { pack(a, blockIdx.x, gridDim.x, blockIdx.y); }

// Workgroups for each matrix.
static unsigned pack_blocks(const PackArgs& a) {
  int64_t most = 0;
  for (int i = 0; i < a.count; ++i) most = std::max(most, a.m[i].rows * ((a.m[i].cols + 7) / 8));
  return (unsigned)std::min<int64_t>((most + 255) / 256, 4096);
}

hipError_t launch_pack(const PackArgs& a, hipStream_t s) {
  const unsigned blocks = pack_blocks(a);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(k_pack, dim3(blocks, (unsigned)a.count), dim3(256), 0, s, a);
  return hipGetLastError();
}

// ------------------------------------------------- backward of activations --

// Workgroup `group` of `groups` takes 512 columns (`slab`) of a range of rows,
// a wave every fourth row of them, two at a time, a lane eight neighbouring
// columns. Eight rows are a range; more where there would be over kActMaxGroups
// ranges. Memory bounds it: gated 8192 x 5120, silu, 80 us (5.2 TB/s). With
// gelu's slope the arithmetic takes about as long as the bytes, and the sums
// of dbias add a tenth of them: 4096 x 4096 26 us (4.2 TB/s).
constexpr int kActRows = 8, kActMaxGroups = 1024;
int act_back_groups(int64_t M) {
  const int64_t g = (M + kActRows - 1) / kActRows;
  return (int)(g < kActMaxGroups ? g : kActMaxGroups);
}

// d = d act'(z), and of the gated layer u = d u act'(z), d = d act(z).
TACO_DEV void times_slope(const float* z, float* d, int act) {
  auto each = [&](int which) {
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] *= act_slope(z[e], which);
  };
  if (act == kActGelu) each(kActGelu);
  else if (act == kActSilu) each(kActSilu);
  else each(kActRelu);
}
TACO_DEV void act_back_gated(const float* z, float* u, float* d, int act) {
  auto each = [&](int which) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float value, slope;
      act_both(z[e], which, &value, &slope);
      u[e] = d[e] * u[e] * slope;
      d[e] = d[e] * value;
    }
  };
  if (act == kActGelu) each(kActGelu);
  else if (act == kActSilu) each(kActSilu);
  else if (act == kActRelu) each(kActRelu);
  else each(kActNone);
}

template <bool GATED>
TACO_DEV void act_back(const ActBackArgs& a, unsigned group, unsigned groups, unsigned slab) {
  __shared__ float sums[4][512];
  const int lane = (int)threadIdx.x % kWave, wave = wave_in_group();
  const int c = ((int)slab * kWave + lane) * 8, n = a.N - c;
  const int64_t per = (a.M + groups - 1) / groups, first = group * per;
  const int64_t end = first + per < a.M ? first + per : a.M;
  float db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) db[e] = 0.0f;
  // dz's rows hold whole eights: zeros past the last column
  const int pad = n < 8 && n > 0 && !GATED ? 8 : n;
  // Z: z's type; WHOLE: each lane has eight columns
  auto rows = [&](auto z_type, auto whole) {
    constexpr int Z = z_type();
    constexpr bool WHOLE = whole();
    const int have = WHOLE ? 8 : n;
    for (int64_t m = first + wave; m < end; m += 8) {
      float d[2][8], z[2][8], u[2][8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t row = m + 4 * i;
        if (row >= end) break;
        load8(a.dout.p, kBF16, row * a.dout.ld + c, have, d[i]);
        if (GATED || a.act != kActNone) load8(a.z.p, Z, row * a.z.ld + c, have, z[i]);
        if (GATED) load8(a.z.p, Z, row * a.z.ld + a.N + c, have, u[i]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t row = m + 4 * i;
        if (row >= end) break;
        if constexpr (GATED) {
          act_back_gated(z[i], u[i], d[i], a.act);
          store8(a.dz, kBF16, row * a.ld_dz + c, have, u[i]);
          store8(a.dz, kBF16, row * a.ld_dz + a.N + c, have, d[i]);
        } else {
          if (a.act != kActNone) times_slope(z[i], d[i], a.act);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (!WHOLE && e >= n) d[i][e] = 0.0f;
            db[e] += d[i][e];
          }
          if (a.dz) store8(a.dz, kBF16, row * a.ld_dz + c, WHOLE ? 8 : pad, d[i]);
        }
      }
    }
  };
  const std::integral_constant<int, kBF16> bf16;
  const std::integral_constant<int, kF32> f32;
  // (wave-uniform, so that a wave runs one of them)
  const bool whole = a.N % 8 == 0 || ((int)slab + 1) * kWave * 8 <= a.N;
  if (n <= 0) {
  } else if (whole) {
    if (a.z.dt == kBF16) rows(bf16, std::true_type());
    else rows(f32, std::true_type());
  } else {
    if (a.z.dt == kBF16) rows(bf16, std::false_type());
    else rows(f32, std::false_type());
  }
  if constexpr (GATED) {
    // zeros past the last column of the second half
    const int64_t rest = -2 * (int64_t)a.N & 7;
    if (slab == 0 && threadIdx.x < rest)
      for (int64_t m = first; m < end; ++m) a.dz[m * a.ld_dz + 2 * (int64_t)a.N + threadIdx.x] = 0;
  } else {
    if (a.partials == nullptr) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[wave][lane * 8 + e] = db[e];
    __syncthreads();
    for (int i = (int)threadIdx.x; i < 512; i += 256) {
      const int col = (int)slab * 512 + i;
      if (col < a.N)
        a.partials[(int64_t)group * a.N + col] = (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
    }
  }
}

// dz, and in the workgroups after its `blocks` the copies that the products
// need beside it.
template <bool GATED>
__global__ __launch_bounds__(256) void k_act_back(ActBackArgs a, PackArgs p, unsigned groups, unsigned blocks,
                                                  unsigned packing) {
  if (blockIdx.x < blocks) act_back<GATED>(a, blockIdx.x % groups, groups, blockIdx.x / groups);
  else pack(p, (blockIdx.x - blocks) % packing, packing, (blockIdx.x - blocks) / packing);
}

hipError_t launch_act_back(const ActBackArgs& a, const PackArgs& p, hipStream_t s) {
  const unsigned groups = (unsigned)act_back_groups(a.M), packing = pack_blocks(p);
  const unsigned blocks = groups * (unsigned)((a.N + 511) / 512);
  const dim3 grid(blocks + packing * (unsigned)p.count);
  if (grid.x > 0) {
    if (a.gated) hipLaunchKernelGGL((k_act_back<true>), grid, dim3(256), 0, s, a, p, groups, blocks, packing);
    else hipLaunchKernelGGL((k_act_back<false>), grid, dim3(256), 0, s, a, p, groups, blocks, packing);
  }
  return hipGetLastError();
}

}  // namespace taco
