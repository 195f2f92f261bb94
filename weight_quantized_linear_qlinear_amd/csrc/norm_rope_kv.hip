// Norms of query and key heads, rotary positions with one axis or several, and writing K and V into
// the 8-bit or the 4-bit cache, in one pass; reading 4-bit cache slots back.
//
// For a head row x of D channels at token t (weight w: optional, per channel, q's and k's own):
//   y_c = x_c w_c / sqrt(mean_c x_c^2 + eps)
//   theta_i = positions[axes[i]][t] inv_freq[i],  i < R/2;  (a, b) -> factor (a cos - b sin, a sin + b cos)
//   for the pair (i, i + R/2), or (2 i, 2 i + 1) interleaved; channels from R on stay: without a weight as
//   they came, bit for bit, with one multiplied by it and the row's factor alone.
// Products with w and the rotation are one factor per channel and partner, and the row's factor goes to x (x w can leave
// fp32 where y does not); one rounding at the end.
// Angles, their reduction and the cosines are in 64 bits; q, and a K that goes to bf16 or to 8-bit
// codes, are computed in fp32 from there.  A K that goes to 4-bit codes is computed in fp64 altogether: next
// to a border a code's neighbour is up to half of its value away, so that an order of fp32 additions
// would show; the fp64 rate of a CU is the fp32 one, and K is a small share of the rows.  (In fp32, and in
// fp64 only the batches in which a code or a scale is within fp32's error of a border, one in 12: 8191
// tokens the same, 16 tokens 5.5 against 4.3 us.)
//
// One wave of a workgroup takes a token, or four do (or a share of its heads, while tokens are few), and
// compute its rotation once, channel by channel, into LDS.  A head row is D / 8 lanes, 8 channels each,
// so a lane's channels stay the same from row to row, and what their rotation multiplies them and
// their partners by (weights included: two operations per channel) stays in registers for all heads.
// Rows pass through the wave's LDS for the partners, 4-bit codes for the order of the cache.
//
// Bound by HBM for many tokens: 8192 tokens of 32 + 8 heads of 128, normed and turned, 33 us, 5.0 TB/s (32 heads turned
// alone, three axes, 24 us, 5.5 TB/s); by its one round of waves for fewer (4095 tokens of 16 + 16 heads of 64 11 us, 3.0
// TB/s; one token 3.6 us).  Into 4 bits by K's fp64 too: 8191 tokens of 32 + 8 + 8 heads of 128 40 us, 4.5 TB/s;
// 2048 tokens 18 us, two waves per SIMD.  Into 8 bits 333 tokens 6.7 us, 2048 16 us, 8191 40 us (4.6 TB/s).  K and V alone
// into 4 bits, 8191 tokens of 8 heads of 128 14 us (43 MB, 3.1 TB/s), of 16 of 64 15 us.
#include <type_traits>

#include "kv_rows.h"
#include "qlq_launch.h"

namespace qlq {

namespace {

constexpr int kWaves = 4;

// What a channel and its partner are multiplied by: x c + partner s.
template <class T>
struct alignas(2 * sizeof(T)) Turn {
  T c, s;
};

// Sine and cosine of r, |r| <= pi/4 (a little more does no harm), by their Taylor series: the first
// term left out is below 2^-58 of the result.
__device__ __forceinline__ void sincos_quarter(double r, double* s, double* c) {
  const double z = r * r;
  double p = 1.0 / 355687428096000.0;                        // 1 / 17!, and every second one down from there
  p = __builtin_fma(p, z, -1.0 / 1307674368000.0);
  p = __builtin_fma(p, z, 1.0 / 6227020800.0);
  p = __builtin_fma(p, z, -1.0 / 39916800.0);
  p = __builtin_fma(p, z, 1.0 / 362880.0);
  p = __builtin_fma(p, z, -1.0 / 5040.0);
  p = __builtin_fma(p, z, 1.0 / 120.0);
  p = __builtin_fma(p, z, -1.0 / 6.0);
  *s = __builtin_fma(p * z, r, r);
  double q = 1.0 / 20922789888000.0;                         // 1 / 16!
  q = __builtin_fma(q, z, -1.0 / 87178291200.0);
  q = __builtin_fma(q, z, 1.0 / 479001600.0);
  q = __builtin_fma(q, z, -1.0 / 3628800.0);
  q = __builtin_fma(q, z, 1.0 / 40320.0);
  q = __builtin_fma(q, z, -1.0 / 720.0);
  q = __builtin_fma(q, z, 1.0 / 24.0);
  q = __builtin_fma(q, z, -0.5);
  *c = __builtin_fma(q, z, 1.0);
}

// The rotation of token t, channel by channel, in fp32 and (where) in fp64: (factor cos, -+ factor sin); (1, 0)
// from channel R on.  Channel ch stands at [ch % 8][ch / 8], so that the lanes of a row read side by side.
__device__ __forceinline__ void token_turns(const NormRopeArgs& a, int64_t t, int first, int step, int tpr, Turn<double>* wide,
                                            Turn<float>* cs) {
  auto put = [&](int ch, double c, double s) {
    const int at = (ch & 7) * tpr + (ch >> 3);
    if (wide) wide[at] = {c, s};
    cs[at] = {(float)c, (float)s};
  };
  const int half = a.R / 2;
  for (int i = first; i < half; i += step) {
    const int64_t axis = a.axes ? min(max(a.axes[i], 0), a.A - 1) : 0;
    const int64_t pos = load_index(a.positions, a.pos64, axis * a.T + t);
    const double th = (double)pos * a.inv_freq[i];
    const double q = rint(th * 0x1.45f306dc9c883p-1);                    // 2 / pi
    double r = __builtin_fma(-q, 0x1.921fb54442d18p+0, th);             // pi / 2, high part
    r = __builtin_fma(-q, 0x1.1a62633145c07p-54, r);                    // and the rest of it
    double s, c;
    sincos_quarter(r, &s, &c);
    const int quarter = (int)((int64_t)q & 3);
    const double cc = (quarter & 1 ? s : c) * (quarter == 1 || quarter == 2 ? -a.factor : a.factor);
    const double ss = (quarter & 1 ? c : s) * (quarter >= 2 ? -a.factor : a.factor);
    put(a.interleaved ? 2 * i : i, cc, -ss);
    put(a.interleaved ? 2 * i + 1 : i + half, cc, ss);
  }
  for (int ch = a.R + first; ch < 8 * tpr; ch += step) put(ch, 1.0, 0.0);
}

// Another lane's value, for steps within 4, 8 and 16 lanes in the vector unit.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
template <int CTRL>
__device__ __forceinline__ int other(int v) { return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, true); }
template <int CTRL>
__device__ __forceinline__ uint32_t other(uint32_t v) { return (uint32_t)other<CTRL>((int)v); }
template <int CTRL>
__device__ __forceinline__ float other(float v) { return __builtin_bit_cast(float, other<CTRL>(__builtin_bit_cast(int, v))); }
template <int CTRL>
__device__ __forceinline__ double other(double v) {
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, (u32x2){other<CTRL>(w.x), other<CTRL>(w.y)});
}

struct Add {
  template <class T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
  __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};

// The four lanes of a group of 32 channels, to each of them.
template <class T, class OP>
__device__ __forceinline__ T quad(T v, OP op) {
  v = op(v, other<kXor1>(v));
  return op(v, other<kXor2>(v));
}

// Over the n lanes of a row (N where the compiler knows them, else 0); first: its first lane, c: this one's place.
template <int N, class T, class OP>
__device__ __forceinline__ T over_row(T v, int n, int first, int c, OP op) {
  if constexpr (N == 4 || N == 8 || N == 16 || N == 32 || N == 64) {
    v = quad(v, op);
    if constexpr (N >= 8) v = op(v, other<kHalfMirror>(v));
    if constexpr (N >= 16) v = op(v, other<kMirror>(v));
#pragma unroll
    for (int d = 16; d < N; d *= 2) v = op(v, __shfl_xor(v, d, 64));
    return v;
  }
  int step = 1;
  for (; n % (2 * step) == 0; step *= 2) v = op(v, __shfl_xor(v, step, 64));   // (rows begin at multiples of 2 step)
  T all = v;
  for (int d = step; d < n; d += step) {
    const int at = c + d >= n ? c + d - n : c + d;
    all = op(all, __shfl(v, (first + at) & 63, 64));
  }
  return all;
}

__device__ __forceinline__ void wave_sync() {                 // the wave's LDS writes before its reads
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The quotient y / s to 21 bits, the last of them set if anything is behind it: next to a border between
// codes (4 bits) the side stays, and a tie is one only where the quotient is.
__device__ __forceinline__ float quotient(double y, double s, double inv) {
  double q = y * inv;
  q = __builtin_fma(__builtin_fma(-q, s, y), inv, q);
  const u32x2 w = __builtin_bit_cast(u32x2, q);
  return (float)__builtin_bit_cast(double, (u32x2){0u, w.y | min(w.x, 1u)});
}

// Where a lane stands in the rows of its wave, and the wave's LDS.  KOUT: where K goes: 0 to bf16 (or
// there is none), 8 and 4 into a cache of that many bits, with V.  TPR: lanes per row, 0 for those that
// have no instance of their own.
template <int KOUT, int TPR>
struct Lane {
  int D, tpr, rpw, r, c;         // channels, lanes per row, rows per wave; this lane's row and place in it
  bool live;                     // (there are lanes left over where 64 / tpr is no whole number)
  int half, pc;                  // R / 2; the chunk that holds this one's partners (where R % 16 == 0)
  bool chunks;
  // LDS: the token's turns in fp64 (4 bits) and fp32, the wave's rows, codes (4 bits)
  Turn<double>* wide;
  Turn<float>* cs;
  uint16_t* mine;
  uint8_t* bytes;

  __device__ __forceinline__ Lane(const NormRopeArgs& a, int lane, uint8_t* token, uint8_t* own) {
    D = TPR ? TPR * 8 : a.D;
    tpr = TPR ? TPR : a.D / 8;
    rpw = 64 / tpr;
    r = lane / tpr;
    c = lane - r * tpr;
    live = r < rpw;
    half = a.R / 2;
    chunks = a.R % 16 == 0;
    pc = c * 8 >= a.R || a.interleaved || !chunks ? c : c * 8 < half ? c + half / 8 : c - half / 8;
    wide = KOUT == 4 ? reinterpret_cast<Turn<double>*>(token) : nullptr;
    cs = reinterpret_cast<Turn<float>*>(token + (KOUT == 4 ? 16 * D : 0));
    uint16_t* rows = reinterpret_cast<uint16_t*>(own);
    mine = rows + (live ? r : 0) * D;
    bytes = reinterpret_cast<uint8_t*>(rows + 512) + (live ? r : 0) * (D / 2);
  }

  // Over the lanes of a row, or of a group of 32 channels.
  template <class T, class OP>
  __device__ __forceinline__ T row(T v, OP op) const { return over_row<TPR>(v, tpr, r * tpr, c, op); }

  __device__ __forceinline__ u32x4 load(const uint16_t* p, int batch, int H, int vec) const {
    const int head = batch * rpw + r;
    u32x4 raw = {0u, 0u, 0u, 0u};
    if (live && head < H) raw = load8(p + head * D + c * 8, vec);
    return raw;
  }

  // Of channels 2 i and 2 i + 1 of this lane (i < 4), those that rotate: the others have no partner (their turn is
  // (1, 0), and 0 times an infinity is NaN).
  __device__ __forceinline__ bool turns(const NormRopeArgs& a, int i) const { return c * 8 + 2 * i < a.R; }
  __device__ __forceinline__ void drop_unturned(const NormRopeArgs& a, u32x4* part) const {
    if (a.R == D) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) (*part)[i] = turns(a, i) ? (*part)[i] : 0u;
  }

  // The channel that channel ch turns with.
  __device__ __forceinline__ int partner(const NormRopeArgs& a, int ch) const {
    return ch >= a.R ? ch : a.interleaved ? ch ^ 1 : ch < half ? ch + half : ch - half;
  }
  // This lane's weights, own and partners'.
  __device__ __forceinline__ void weights(const NormRopeArgs& a, const uint16_t* w, u32x4* own, u32x4* part) const {
    if (!live) return;
    *own = load8(w + c * 8, a.vec_w);
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) (*part)[i] = (*own)[i] >> 16 | (*own)[i] << 16;
    } else if (chunks) {
      *part = load8(w + pc * 8, a.vec_w);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) (*part)[i] = w[partner(a, c * 8 + 2 * i)] | (uint32_t)w[partner(a, c * 8 + 2 * i + 1)] << 16;
    }
    drop_unturned(a, part);
  }

  // What channel e of the lane at place c and its partner are multiplied by, weights (if any) included.
  template <class T>
  __device__ __forceinline__ Turn<T> turn(int e, const Turn<T>* turns, bool weighted, u32x4 own, u32x4 part, int c) const {
    auto at = [](u32x4 v, int i) { return (T)bf16_bits_to_f32(i & 1 ? v[i / 2] >> 16 : v[i / 2] & 0xFFFF); };
    Turn<T> v = turns[e * tpr + c];
    if (weighted) v.c *= at(own, e), v.s *= at(part, e);
    return v;
  }

  // The partners of this lane's channels.
  __device__ __forceinline__ u32x4 partners(const NormRopeArgs& a, u32x4 raw, bool there) const {
    u32x4 o;
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = raw[i] >> 16 | raw[i] << 16;
      drop_unturned(a, &o);
      return o;
    }
    if (there) st16(mine + c * 8, raw);
    wave_sync();
    if (chunks) {
      o = ld16(mine + pc * 8);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = mine[partner(a, c * 8 + 2 * i)] | (uint32_t)mine[partner(a, c * 8 + 2 * i + 1)] << 16;
    }
    __builtin_amdgcn_wave_barrier();                          // reads above before the next rows' writes
    drop_unturned(a, &o);
    return o;
  }

  // Rows of one batch of q or k in fp32, v their turns: f becomes the result.
  __device__ __forceinline__ void norm_turn(const NormRopeArgs& a, u32x4 raw, bool there, bool normed, const Turn<float>* v,
                                            float* f) const {
    float rho = 1.0f, o[8];
    bool big = false;
    if (normed) {
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(f[e], f[e], ss);
      ss = row(ss, Add());
      rho = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, 1.0f / (float)D, (float)a.eps));
      // squares beyond fp32, or (eps below 2^-64) lost under it: the sum again, in 64 bits
      big = !(ss < __builtin_inff());
      const bool lost = big || a.eps < 0x1p-64f;
      if (__ballot(lost)) {
        double s2 = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) s2 = __builtin_fma((double)f[e], (double)f[e], s2);
        s2 = row(s2, Add());
        if (lost) rho = (float)((big ? 0x1p64 : 1.0) / sqrt(s2 / D + a.eps));
      }
    }
    unpack8(partners(a, raw, there), o);
    if (__ballot(big)) {                                      // (rho is 2^64 of itself there)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (big) f[e] *= 0x1p-64f, o[e] *= 0x1p-64f;
    }
    if (normed) {                                             // x rho is at most sqrt(D): its products with weights leave
#pragma unroll                                                // fp32 only where the result does
      for (int e = 0; e < 8; ++e) f[e] *= rho, o[e] *= rho;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __builtin_fmaf(o[e], v[e].s, f[e] * v[e].c);
  }

  // The same in fp64, to 4-bit codes (byte j: channels 2 j and 2 j + 1) and the group's scale.
  __device__ __forceinline__ uint32_t norm_turn_codes(const NormRopeArgs& a, u32x4 raw, bool there, const float* f, u32x4 own,
                                                      u32x4 part, uint32_t* code) const {
    float o[8];
    unpack8(partners(a, raw, there), o);
    double y[8], rho = 1.0, am = 0.0, bad = 0.0;
    if (a.wk) {
      double ss = 0.0;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fma((double)f[e], (double)f[e], ss);
      rho = 1.0 / sqrt(row(ss, Add()) / D + a.eps);
    }
    int place = c;
    asm volatile("" : "+v"(place), "+v"(own), "+v"(part));    // (turns and weights kept in fp64 for all batches: 190 registers)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const Turn<double> v = turn(e, wide, a.wk != nullptr, own, part, place);
      y[e] = __builtin_fma((double)o[e], v.s, (double)f[e] * v.c) * rho;
      am = fmax(am, fabs(y[e]));
      bad = __builtin_fma(y[e], 0.0, bad);                    // NaN with a NaN or an infinity
    }
    am = quad(am, Max());
    bad = quad(bad, Add());
    const uint32_t sb = kv4_f16_scale((float)(am / 6.0), am == 0.0, bad != 0.0);
    const double s = (double)f16_value(sb), inv = 1.0 / s;
    *code = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *code |= f32x2_to_e2m1x2_sat(quotient(y[2 * j], s, inv), quotient(y[2 * j + 1], s, inv)) << (8 * j);
    return sb;
  }

  // bf16 as it came to 4-bit codes.  x has 8 bits and a border times s 14, so a quotient that is not on a
  // border is 2^-14 or more away from it: x times a reciprocal (2^-22), to 16 bits, is on the right side, and on it
  // where the quotient is.
  __device__ __forceinline__ uint32_t codes4(const float* f, uint32_t* code) const {
    uint32_t am = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) am = max(am, __builtin_bit_cast(uint32_t, f[e]) & 0x7FFFFFFFu);
    am = quad(am, Max());
    const uint32_t sb = kv4_f16_scale(__builtin_bit_cast(float, am) / 6.0f, am == 0, am >= 0x7F800000u);
    const float s = f16_value(sb), r0 = __builtin_amdgcn_rcpf(s);
    auto quotient = [&](float x) {
      return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x * r0) + 0x80u) & 0xFFFFFF00u);
    };
    *code = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) *code |= f32x2_to_e2m1x2_sat(quotient(f[2 * j]), quotient(f[2 * j + 1])) << (8 * j);
    return sb;
  }

  // A row in bf16; without a norm, channels that do not rotate are those of raw.
  __device__ __forceinline__ void store_bf16(const NormRopeArgs& a, uint16_t* out, const float* f, u32x4 raw, bool normed, int vec) const {
    u32x4 p = {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
    if (!normed && a.R < D) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = turns(a, i) ? p[i] : raw[i];
    }
    if (vec) {
      st16(out, p);
    } else {
      const uint32_t d[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = (uint16_t)(d[e / 2] >> (16 * (e & 1)));
    }
  }

  // A row of 4-bit codes and its scales to entry `at` (there: this lane has a row, stored: it has a slot).
  __device__ __forceinline__ void store4(Kv4Run run, uint32_t code, uint32_t sb, bool there, bool stored, uint8_t* codes,
                                         uint16_t* scales, int64_t at) const {
    if (there) {
#pragma unroll
      for (int j = 0; j < 4; ++j) bytes[run.first + (4 * (c & 3) + j) * run.step] = (uint8_t)(code >> (8 * j));
    }
    wave_sync();
    if (there && stored) {
      *reinterpret_cast<uint32_t*>(codes + at * (D / 2) + 4 * c) = *reinterpret_cast<const uint32_t*>(bytes + 4 * c);
      if ((c & 3) == 0) scales[at * (D / 32) + c / 4] = (uint16_t)sb;
    }
    __builtin_amdgcn_wave_barrier();                          // reads above before the next rows' writes
  }

  __device__ __forceinline__ void store8_k(const float* f, bool there, uint8_t* codes, uint16_t* scales, int64_t at) const {
    float am = 0.0f, d[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) am = fmaxf(am, fabsf(f[e]));
    const uint32_t sb = kv_f16_scale(quad(am, Max()), 127.0f);
    const RcpDiv dv(f16_value(sb));
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = dv(f[e]);
    if (!there) return;
    const u32x2 p = {f32_to_i8_sat(d[0]) | (f32_to_i8_sat(d[1]) << 8) | (f32_to_i8_sat(d[2]) << 16) | (f32_to_i8_sat(d[3]) << 24),
                     f32_to_i8_sat(d[4]) | (f32_to_i8_sat(d[5]) << 8) | (f32_to_i8_sat(d[6]) << 16) | (f32_to_i8_sat(d[7]) << 24)};
    *reinterpret_cast<u32x2*>(codes + at * D + c * 8) = p;
    if ((c & 3) == 0) scales[at * (D / 32) + c / 4] = (uint16_t)sb;
  }

  __device__ __forceinline__ void store8_v(const float* f, bool there, uint8_t* codes, uint16_t* scales, int64_t at) const {
    float am = 0.0f, d[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) am = fmaxf(am, fabsf(f[e]));
    const uint32_t sb = kv_f16_scale(row(am, Max()), 448.0f);
    const RcpDiv dv(f16_value(sb));
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = dv(f[e]);
    if (!there) return;
    const u32x2 p = {f32x4_to_e4m3x4_sat(d[0], d[1], d[2], d[3]), f32x4_to_e4m3x4_sat(d[4], d[5], d[6], d[7])};
    *reinterpret_cast<u32x2*>(codes + at * D + c * 8) = p;
    if (c == 0) scales[at] = (uint16_t)sb;
  }
};

// A batch of K rows in fp64 takes the time of about three of q (in units: what shares are cut by).
template <int KOUT>
constexpr int kUnitsK = KOUT == 4 ? 3 : 1;

// Waves per SIMD that the registers have to leave room for.  Into 4 bits, from 128 channels on, four: q's weights are
// then read behind K's rows, and spills of up to 12 bytes are worth it (us, three and four, heads of 128, 8191 tokens 61
// and 54, 3000 the same; of 256 54 and 48; of 160 50 and 46; of 64, 3000 tokens 20.1 and 21.6, 8192 the same).
template <int KOUT, int TPR>
constexpr int kRoom = KOUT == 4 && (TPR == 0 || TPR >= 16) ? 4 : 1;

template <int KOUT, int TPR>
__global__ __launch_bounds__(kWaves * 64, (kRoom<KOUT, TPR>)) void norm_rope_kernel(NormRopeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int D = TPR ? TPR * 8 : a.D;
  // waves per token and workgroup, the token's place in the workgroup, this wave's share of the token
  const int wpt = 1 << a.wpt_shift, tok = wave >> a.wpt_shift, shares = wpt * gridDim.y;
  const int share = blockIdx.y * wpt + (wave & (wpt - 1));
  const int t = blockIdx.x * (kWaves >> a.wpt_shift) + tok;
  const bool here = t < a.T;
  constexpr int kPerChannel = KOUT == 4 ? 24 : 8, kOwn = 1024 + (KOUT == 4 ? 256 : 0);
  const Lane<KOUT, TPR> l(a, lane, smem + tok * kPerChannel * D,
                          smem + (kWaves >> a.wpt_shift) * kPerChannel * D + wave * kOwn);
  // the token's batches of rows in a line: K's, q's, V's (V's last, so that their wave has something to do
  // while another one computes the rotation)
  constexpr int UK = kUnitsK<KOUT>;
  const int nk = (a.Hk + l.rpw - 1) / l.rpw, nv = KOUT ? nk : 0, nq = (a.Hq + l.rpw - 1) / l.rpw, n = UK * nk + nq + nv;
  const int u0 = here ? n * share / shares : n, u1 = here ? n * (share + 1) / shares : n;
  const int k0 = min((u0 + UK - 1) / UK, nk), k1 = min((u1 + UK - 1) / UK, nk);
  const int q0 = min(max(u0 - UK * nk, 0), nq), q1 = min(max(u1 - UK * nk, 0), nq);
  const int v0 = max(u0 - UK * nk - nq, 0), v1 = max(u1 - UK * nk - nq, 0);
  const uint16_t* qrow = a.q + (int64_t)t * a.q_stride;
  const uint16_t* krow = a.k + (int64_t)t * a.k_stride;
  const uint16_t* vrow = a.v + (int64_t)t * a.v_stride;
  // the first rows and the weights, in flight while the rotation is computed
  u32x4 kraw = {0u, 0u, 0u, 0u}, vraw = kraw, qraw = kraw, wk = kraw, wkp = kraw, wq = kraw, wqp = kraw;
  if (k0 < k1) kraw = l.load(krow, k0, a.Hk, a.vec_in);
  if (KOUT && v0 < v1) vraw = l.load(vrow, v0, a.Hk, a.vec_in);
  if (q0 < q1) qraw = l.load(qrow, q0, a.Hq, a.vec_in);
  if (a.wk && k0 < k1) l.weights(a, a.wk, &wk, &wkp);
  if (KOUT != 4 && a.wq && q0 < q1) l.weights(a, a.wq, &wq, &wqp);
  int64_t slot = -1;
  if (KOUT && (k0 < k1 || v0 < v1)) slot = load_index(a.slots, a.slot64, t);
  const bool stored = slot >= 0 && slot < a.pool;
  Kv4Run run{0, 1};
  if (KOUT == 4) run = kv4_run(D / 32, l.c / 4);

  if (here) token_turns(a, t, (wave & (wpt - 1)) * 64 + lane, wpt * 64, l.tpr, l.wide, l.cs);
  float f[8];
  uint32_t code, sb;
  if constexpr (KOUT != 0) {
    for (int b = v0; b < v1; ++b) {
      const u32x4 raw = vraw;
      if (b + 1 < v1) vraw = l.load(vrow, b + 1, a.Hk, a.vec_in);   // in flight meanwhile
      const int head = b * l.rpw + l.r;
      const bool there = l.live && head < a.Hk;
      const int64_t at = slot * a.Hk + head;
      unpack8(raw, f);
      if constexpr (KOUT == 4) {
        sb = l.codes4(f, &code);
        l.store4(run, code, sb, there, stored, a.v_codes, a.v_scales, at);
      } else {
        l.store8_v(f, there && stored, a.v_codes, a.v_scales, at);
      }
    }
  }
  if (wpt > 1) __syncthreads();
  else wave_sync();

  Turn<float> v[8];
  if (k0 < k1 && KOUT != 4) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = l.turn(e, l.cs, a.wk != nullptr, wk, wkp, l.c);
  }
  for (int b = k0; b < k1; ++b) {
    const u32x4 raw = kraw;
    if (b + 1 < k1) kraw = l.load(krow, b + 1, a.Hk, a.vec_in);
    const int head = b * l.rpw + l.r;
    const bool there = l.live && head < a.Hk;
    const int64_t at = slot * a.Hk + head;
    unpack8(raw, f);
    if constexpr (KOUT == 4) {
      sb = a.R || a.wk ? l.norm_turn_codes(a, raw, there, f, wk, wkp, &code) : l.codes4(f, &code);
      l.store4(run, code, sb, there, stored, a.k_codes, a.k_scales, at);
    } else {
      l.norm_turn(a, raw, there, a.wk != nullptr, v, f);
      if constexpr (KOUT == 8) l.store8_k(f, there && stored, a.k_codes, a.k_scales, at);
      else if (there) l.store_bf16(a, a.k_out + (int64_t)t * a.k_out_stride + head * D + l.c * 8, f, raw, a.wk != nullptr, a.vec_out);
    }
  }
  if (q0 >= q1) return;
  if (KOUT == 4 && a.wq) l.weights(a, a.wq, &wq, &wqp);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = l.turn(e, l.cs, a.wq != nullptr, wq, wqp, l.c);
  for (int b = q0; b < q1; ++b) {
    const u32x4 raw = qraw;
    if (b + 1 < q1) qraw = l.load(qrow, b + 1, a.Hq, a.vec_in);
    const int head = b * l.rpw + l.r;
    const bool there = l.live && head < a.Hq;
    unpack8(raw, f);
    l.norm_turn(a, raw, there, a.wq != nullptr, v, f);
    if (there) l.store_bf16(a, a.q_out + (int64_t)t * a.q_out_stride + head * D + l.c * 8, f, raw, a.wq != nullptr, a.vec_out);
  }
}

// Rows of chosen slots of a 4-bit cache back to bf16 (8 channels per thread); a slot outside the pool
// gives zeros.  For rows that kv4_gather_quads_kernel does not take; bound by its loads of single bytes: 8191 tokens of 16
// heads of 64 (43 MB) 11.0 us, 3.9 TB/s, of 8 of 96 and 4 of 192 (32 MB) 9.2 us, 3.5 TB/s.
__global__ __launch_bounds__(256) void kv4_gather_kernel(const uint8_t* __restrict__ kq, const uint16_t* __restrict__ ks,
                                                         const uint8_t* __restrict__ vq, const uint16_t* __restrict__ vs,
                                                         int64_t pool, int H, int D, const void* __restrict__ slots,
                                                         int slot64, int64_t n8, uint16_t* __restrict__ ko,
                                                         uint16_t* __restrict__ vo) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  const uint32_t row8 = (uint32_t)H * D / 8;                  // chunks per slot
  auto value8 = [](const uint8_t* p, int step, float s) {
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((uint32_t)p[j * step], 1.0f, 0);
      r[j] = pack_bf16x2(v.x * s, v.y * s);
    }
    return r;
  };
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n8; i += stride) {
    const int64_t n = i / row8;
    const uint32_t e = (uint32_t)(i - n * row8) * 8;          // channel within the slot's [H, D]
    const int64_t slot = load_index(slots, slot64, n);
    u32x4 k = {0u, 0u, 0u, 0u}, v = {0u, 0u, 0u, 0u};
    if (slot >= 0 && slot < pool) {
      const int64_t row = slot * H + e / D;
      const int ch = (int)(e % D), g = ch / 32;
      const Kv4Run run = kv4_run(D / 32, g);
      const int64_t at = row * (D / 2) + run.first + (int64_t)(ch % 32 / 2) * run.step;
      k = value8(kq + at, run.step, f16_value(ks[row * (D / 32) + g]));
      v = value8(vq + at, run.step, f16_value(vs[row * (D / 32) + g]));
    }
    st16(ko + i * 8, k);
    st16(vo + i * 8, v);
  }
}

// The same where a row's groups are a multiple of four: a thread takes channels 8 j .. 8 j + 7 of four groups, whose
// bytes 4 j .. 4 j + 3 of a run are dwords (in runs of four groups 16 bytes side by side).  Bound by HBM: 8191 tokens of 8
// heads of 128 (43 MB) 8.9 us, 4.8 TB/s; byte by byte 12.5 (with heads of 256, 8192 tokens and their append, 47.0 and 48.0).
__global__ __launch_bounds__(256) void kv4_gather_quads_kernel(const uint8_t* __restrict__ kq, const uint16_t* __restrict__ ks,
                                                               const uint8_t* __restrict__ vq, const uint16_t* __restrict__ vs,
                                                               int64_t pool, int H, int NG, const void* __restrict__ slots,
                                                               int slot64, int64_t total, uint16_t* __restrict__ ko,
                                                               uint16_t* __restrict__ vo) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  const uint32_t quads = NG / 4, each = (uint32_t)H * NG;     // threads per slot
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int64_t n = i / each;
    const uint32_t e = (uint32_t)(i - n * each), j = e & 3, hq = e >> 2, h = hq / quads, g0 = 4 * (hq - h * quads);
    const int64_t slot = load_index(slots, slot64, n);
    const bool there = slot >= 0 && slot < pool;
    const int64_t row = there ? slot * H + h : 0;
    const Kv4Run run = kv4_run(NG, g0);
    const int64_t at = row * (16 * NG) + run.first + 4 * j * run.step;
    uint32_t kd[4], vd[4];
    if (run.step == 4) {
      const u32x4 a = ld16(kq + at), b = ld16(vq + at);
#pragma unroll
      for (int c = 0; c < 4; ++c) kd[c] = a[c], vd[c] = b[c];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        kd[c] = *reinterpret_cast<const uint32_t*>(kq + at + c * run.step);
        vd[c] = *reinterpret_cast<const uint32_t*>(vq + at + c * run.step);
      }
    }
    uint16_t kss[4], vss[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) kss[g] = ks[row * NG + g0 + g], vss[g] = vs[row * NG + g0 + g];
    const int64_t out = ((n * H + h) * NG + g0) * 32 + 8 * j;
    auto put = [&](auto G) {
      constexpr int g = decltype(G)::value;
      auto value8 = [&](const uint32_t (&d)[4], float s) {
        u32x4 r;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d[c], 1.0f, g);
          r[c] = there ? pack_bf16x2(v.x * s, v.y * s) : 0u;
        }
        return r;
      };
      st16(ko + out + 32 * g, value8(kd, f16_value(kss[g])));
      st16(vo + out + 32 * g, value8(vd, f16_value(vss[g])));
    };
    put(std::integral_constant<int, 0>());
    put(std::integral_constant<int, 1>());
    put(std::integral_constant<int, 2>());
    put(std::integral_constant<int, 3>());
  }
}

template <int KOUT>
hipError_t launch_kout(const NormRopeArgs& in, hipStream_t st) {
  NormRopeArgs a = in;
  const int rpw = 64 / (a.D / 8), nk = (a.Hk + rpw - 1) / rpw;
  const int n = (a.Hq + rpw - 1) / rpw + (kUnitsK<KOUT> + (KOUT ? 1 : 0)) * nk;    // units of a token
  // A wave per token from 800 tokens on, four before that, and more workgroups per token while there are
  // fewer than 1024.  Kernel alone, us, four waves and one, 32 + 8 heads of 128 and 16 + 16 of 64: normed and turned 300 tokens
  // 5.7 and 10.1, 4.5 and 6.6; 700 8.6 and 11.0, 5.2 and 7.2; 1000 10.3 and 11.5, 6.0 and 7.3; 2000 12.6 and
  // 13.2, 9.0 and 8.1; 4095 19.8 and 17.2, 14.0 and 10.9.  Into 8 bits 700 10.7 and 12.6, 8.0 and 8.8; 1000 13.0 and 13.4,
  // 9.5 and 9.2; 2000 16.6 and 15.9, 13.9 and 11.0.  Into 4 bits 300 8.4 and 12.4, 7.8 and 8.9; 700 10.9 and 13.0,
  // 10.0 and 9.2; 1000 12.8 and 13.7, 12.8 and 9.6; 1500 14.5 and 16.7, 12.3 and 11.4; 4095 29.2 and 24.0, 27.4 and 19.4.
  // The sides cross between 500 tokens (64 channels, 4 bits) and 2500 (128, normed and turned): one border for all
  // forms, with up to 15 % lost around it.  Two waves, 4 bits with the gather: 2048 tokens 21.9 against 21.2, 8191 62 against 60.
  a.wpt_shift = 0;
  int gy = 1;
  if (a.T < 800) {
    a.wpt_shift = 2;
    gy = (1024 + a.T - 1) / a.T;
    if (gy > (n + kWaves - 1) / kWaves) gy = (n + kWaves - 1) / kWaves;
  }
  const int per = kWaves >> a.wpt_shift;
  const dim3 grid((unsigned)((a.T + per - 1) / per), (unsigned)gy);
  const size_t lds = (size_t)per * (KOUT == 4 ? 24 : 8) * a.D + kWaves * (1024 + (KOUT == 4 ? 256 : 0));   // at most 54 KB
  switch (a.D) {
    case 64: norm_rope_kernel<KOUT, 8><<<grid, kWaves * 64, lds, st>>>(a); break;
    case 96: norm_rope_kernel<KOUT, 12><<<grid, kWaves * 64, lds, st>>>(a); break;
    case 128: norm_rope_kernel<KOUT, 16><<<grid, kWaves * 64, lds, st>>>(a); break;
    case 192: norm_rope_kernel<KOUT, 24><<<grid, kWaves * 64, lds, st>>>(a); break;
    case 256: norm_rope_kernel<KOUT, 32><<<grid, kWaves * 64, lds, st>>>(a); break;
    default: norm_rope_kernel<KOUT, 0><<<grid, kWaves * 64, lds, st>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_rope(const NormRopeArgs& a, int kout, hipStream_t st) {
  return kout == 0 ? launch_kout<0>(a, st) : kout == 8 ? launch_kout<8>(a, st) : launch_kout<4>(a, st);
}

hipError_t launch_kv4_gather(const void* kq, const void* ks, const void* vq, const void* vs, int64_t pool, int H, int D,
                             const void* slots, int slot64, int64_t n, void* ko, void* vo, hipStream_t st) {
  const bool quads = D % 128 == 0;
  const int64_t n8 = n * H * D / 8, total = quads ? n8 / 4 : n8;
  int64_t g = (total + 255) / 256;
  if (g > 8192) g = 8192;
  if (quads) {
    kv4_gather_quads_kernel<<<(int)g, 256, 0, st>>>(static_cast<const uint8_t*>(kq), static_cast<const uint16_t*>(ks),
                                                   static_cast<const uint8_t*>(vq), static_cast<const uint16_t*>(vs), pool, H,
                                                   D / 32, slots, slot64, total, static_cast<uint16_t*>(ko),
                                                   static_cast<uint16_t*>(vo));
    return hipGetLastError();
  }
  kv4_gather_kernel<<<(int)g, 256, 0, st>>>(static_cast<const uint8_t*>(kq), static_cast<const uint16_t*>(ks),
                                           static_cast<const uint8_t*>(vq), static_cast<const uint16_t*>(vs), pool, H, D,
                                           slots, slot64, n8, static_cast<uint16_t*>(ko), static_cast<uint16_t*>(vo));
  return hipGetLastError();
}

}  // namespace qlq
