// Norms of query and key heads, rotary positions with one axis or several, and writing K and V into
// the 8-bit or the 4-bit cache, in one pass; reading 4-bit cache slots back.
//
// For a head row x of D channels at token t (weight w: optional, per channel, q's and k's own):
//   y_c = x_c w_c / sqrt(mean_c x_c^2 + eps)
//   theta_i = positions[axes[i]][t] inv_freq[i],  i < R/2;  (a, b) -> factor (a cos - b sin, a sin + b cos)
//   for the pair (i, i + R/2), or (2 i, 2 i + 1) interleaved; channels from R on stay.
// The rotation is linear, so x w is rotated and the row's factor comes last; one rounding at the end.
// Angles, their reduction and the cosines are in 64 bits; q, and a K that goes to bf16 or to 8-bit
// codes, are computed in fp32 from there.  A K that goes to 4-bit codes is computed in fp64 altogether: next
// to a border a code's neighbour is up to half of its value away, so that an order of fp32 additions
// would show; the fp64 rate of a CU is the fp32 one, and K is a small share of the rows.
//
// One workgroup takes TW tokens (or a share of one token's heads, while tokens are few): its threads
// compute the tokens' angles once for all heads into LDS.  A head row is D / 8 lanes of a wave, 8
// channels each; a wave's rows are all of one kind (K first, as the longest, then V, then q).  The row
// passes through the wave's LDS for the pair partners, and 4-bit codes pass through it into the order
// of the cache.
#include "kv_rows.h"
#include "qlq_launch.h"

namespace qlq {

namespace {

constexpr int kWaves = 4;

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

// Angles of tokens t0 .. t0 + n - 1: (factor cos, factor sin) at [k R/2 + i], in fp32 and (where) in fp64.
__device__ __forceinline__ void token_angles(const NormRopeArgs& a, int64_t t0, int n, Turn<double>* wide, Turn<float>* cs) {
  const int half = a.R / 2;
  for (int j = threadIdx.x; j < n * half; j += kWaves * 64) {
    const int k = j / half, i = j - k * half;
    const int64_t axis = a.axes ? min(max(a.axes[i], 0), a.A - 1) : 0;
    const int64_t pos = load_index(a.positions, a.pos64, axis * a.T + t0 + k);
    const double th = (double)pos * a.inv_freq[i];
    const double q = rint(th * 0x1.45f306dc9c883p-1);                    // 2 / pi
    double r = __builtin_fma(-q, 0x1.921fb54442d18p+0, th);             // pi / 2, high part
    r = __builtin_fma(-q, 0x1.1a62633145c07p-54, r);                    // and the rest of it
    double s, c;
    sincos_quarter(r, &s, &c);
    const int quarter = (int)((int64_t)q & 3);
    const double cc = (quarter & 1 ? s : c) * (quarter == 1 || quarter == 2 ? -a.factor : a.factor);
    const double ss = (quarter & 1 ? c : s) * (quarter >= 2 ? -a.factor : a.factor);
    if (wide) wide[j] = {cc, ss};
    cs[j] = {(float)cc, (float)ss};
  }
}

// Sum over the n lanes of a row that begins at lane `first` (c: this lane's place in it).
template <class T>
__device__ __forceinline__ T row_sum(T v, int n, int first, int c) {
  if ((n & (n - 1)) == 0) {
    for (int d = 1; d < n; d *= 2) v += __shfl_xor(v, d, 64);
    return v;
  }
  int step = 1;
  for (; n % (2 * step) == 0; step *= 2) v += __shfl_xor(v, step, 64);   // (rows begin at multiples of 2 step)
  T sum = v;
  for (int d = step; d < n; d += step) {
    const int at = c + d >= n ? c + d - n : c + d;
    sum += __shfl(v, (first + at) & 63, 64);
  }
  return sum;
}

// The four lanes of a group of 32 channels, to each of them.
template <class T, class OP>
__device__ __forceinline__ T quad(T v, OP op) {
  v = op(v, __shfl_xor(v, 1, 64));
  return op(v, __shfl_xor(v, 2, 64));
}

// A row's 8 channels (place c), times their weights in f, rotated.  mine: the wave's copy of the row
// (bf16); w: its weights, or null; wpart: those of the partner channels where they are a whole chunk.
template <class T>
__device__ __forceinline__ void rotate(const NormRopeArgs& a, const uint16_t* mine, const uint16_t* w, int c,
                                       const Turn<T>* cs, u32x4 wpart, T* f) {
  const int half = a.R / 2;
  if (a.interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = c * 4 + e;                                // pair (2 i, 2 i + 1)
      if (i < half) {
        const Turn<T> t = cs[i];
        const T x = f[2 * e], y = f[2 * e + 1];
        f[2 * e] = x * t.c - y * t.s;
        f[2 * e + 1] = x * t.s + y * t.c;
      }
    }
  } else if (a.R % 16 == 0) {
    const bool low = c * 8 < half;
    const int i0 = low ? c * 8 : c * 8 - half;
    float o[8], v[8];
    unpack8(ld16(mine + (low ? c * 8 + half : c * 8 - half)), o);
    unpack8(wpart, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const Turn<T> t = cs[i0 + e];
      const T y = w ? (T)o[e] * (T)v[e] : (T)o[e];
      f[e] = f[e] * t.c + (low ? -y : y) * t.s;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int ch = c * 8 + e;
      if (ch < a.R) {
        const bool low = ch < half;
        const int other = low ? ch + half : ch - half;
        const Turn<T> t = cs[low ? ch : other];
        T y = (T)bf16_bits_to_f32(mine[other]);
        if (w) y *= (T)bf16_bits_to_f32(w[other]);
        f[e] = f[e] * t.c + (low ? -y : y) * t.s;
      }
    }
  }
}

// Codes of 8 quotients x / s in 64 bits, rounded once; 2 per byte.
__device__ __forceinline__ void e2m1_from_f64(const double* x, double s, uint32_t* b) {
  const double inv = 1.0 / s;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    double q = x[e] * inv;
    q = __builtin_fma(__builtin_fma(-q, s, x[e]), inv, q);    // (exact where the quotient is: ties stay ties)
    const double m = fabs(q);
    const double step = m < 2.0 ? 0.5 : m < 4.0 ? 1.0 : 2.0, per = m < 2.0 ? 2.0 : m < 4.0 ? 1.0 : 0.5;
    v[e] = (float)copysign(fmin(rint(m * per) * step, 6.0), q);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = f32x2_to_e2m1x2_sat(v[2 * e], v[2 * e + 1]);
}

enum Kind { kK, kV, kQ };

// KOUT: where K goes: 0 to bf16 (or there is none), 8 and 4 into a cache of that many bits, with V.
template <int KOUT>
__global__ __launch_bounds__(kWaves * 64) void norm_rope_kernel(NormRopeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];            // angles: [TW][R / 2] in fp64 (4 bits), then fp32
  __shared__ __align__(16) uint16_t rows[kWaves][512];       // 64 lanes x 8 channels per wave
  __shared__ __align__(16) uint8_t bytes[kWaves][KOUT == 4 ? 256 : 16];
  Turn<double>* wide = KOUT == 4 ? reinterpret_cast<Turn<double>*>(smem) : nullptr;
  Turn<float>* cs_all = reinterpret_cast<Turn<float>*>(smem + (KOUT == 4 ? (size_t)a.TW * a.R * 8 : 0));
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = (int64_t)blockIdx.x * a.TW;
  const int ntok = (int)min((int64_t)a.TW, a.T - t0);
  const int tpr = a.D / 8, rpw = 64 / tpr;                    // lanes per row, rows per wave
  const int r = lane / tpr, c = lane - r * tpr, half = a.R / 2;
  const bool lane_live = r < rpw;
  const int nk = (ntok * a.Hk + rpw - 1) / rpw, nv = KOUT ? nk : 0, nq = (ntok * a.Hq + rpw - 1) / rpw;

  // Weights of this lane's channels and of their partners (a whole chunk where R % 16 == 0).
  const int pc = c * 8 < half ? c + half / 8 : c - half / 8;
  const bool whole = !a.interleaved && a.R % 16 == 0 && c * 8 < a.R && lane_live;
  u32x4 wk = {0u, 0u, 0u, 0u}, wkp = wk, wq = wk, wqp = wk;
  if (lane_live) {
    if (a.wk) wk = load8(a.wk + c * 8, a.vec_w);
    if (a.wq) wq = load8(a.wq + c * 8, a.vec_w);
    if (a.wk && whole) wkp = load8(a.wk + pc * 8, a.vec_w);
    if (a.wq && whole) wqp = load8(a.wq + pc * 8, a.vec_w);
  }
  Kv4Run run{0, 1};
  if (KOUT == 4) run = kv4_run(a.D / 32, c / 4);

  struct Row {
    u32x4 raw;
    int64_t slot;
    int tok, head, kind;
    bool live;
  };
  auto load = [&](int batch) -> Row {
    Row w;
    w.kind = batch < nk ? kK : batch < nk + nv ? kV : kQ;     // uniform for the wave
    const int H = w.kind == kQ ? a.Hq : a.Hk;
    const int at = (batch - (w.kind == kK ? 0 : w.kind == kV ? nk : nk + nv)) * rpw + r;
    w.live = lane_live && at < ntok * H;
    w.tok = w.live ? at / H : 0;
    w.head = w.live ? at - w.tok * H : 0;
    w.raw = (u32x4){0u, 0u, 0u, 0u};
    w.slot = -1;
    const int64_t t = t0 + w.tok;
    if (w.live) {
      const uint16_t* p = w.kind == kQ ? a.q + t * a.q_stride : w.kind == kK ? a.k + t * a.k_stride : a.v + t * a.v_stride;
      w.raw = load8(p + (int64_t)w.head * a.D + c * 8, a.vec_in);
      if (KOUT && w.kind != kQ) w.slot = load_index(a.slots, a.slot64, t);
    }
    return w;
  };
  const int step = gridDim.y * kWaves, all = nk + nv + nq;
  int batch = blockIdx.y * kWaves + wave;
  Row next = load(batch);
  if (a.R) token_angles(a, t0, ntok, wide, cs_all);
  __syncthreads();
  for (; batch < all; batch += step) {                        // uniform per wave
    const Row cur = next;
    next = load(batch + step);                                // the next batch's rows are in flight meanwhile
    const int64_t t = t0 + cur.tok;
    const uint16_t* w = cur.kind == kQ ? a.wq : cur.kind == kK ? a.wk : nullptr;
    const bool turns = a.R && cur.kind != kV;
    uint16_t* mine = rows[wave] + (lane_live ? r : 0) * a.D;
    if (turns && !a.interleaved) {
      // the wave's rows through its own LDS: written and read by this wave alone, in order
      if (cur.live) st16(mine + c * 8, cur.raw);
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
    float f[8];
    unpack8(cur.raw, f);
    const bool turning = turns && cur.live && c * 8 < a.R;
    const u32x4 wown = cur.kind == kQ ? wq : wk, wpart = cur.kind == kQ ? wqp : wkp;
    uint32_t b[4];                                            // 4 bits: the lane's codes, channels 2 j and 2 j + 1 in b[j]
    uint32_t sb = 0;
    const bool exact = KOUT == 4 && cur.kind == kK && (a.R || w);
    if (exact) {
      double x[8], rho = 1.0;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = f[e];
      if (w) {
        double ss = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __builtin_fma(x[e], x[e], ss);
        ss = row_sum(ss, tpr, r * tpr, c);
        rho = 1.0 / sqrt(ss / a.D + a.eps);
        float v[8];
        unpack8(wown, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= (double)v[e];
      }
      if (turning) rotate(a, mine, w, c, wide + cur.tok * half, wpart, x);
      double am = 0.0;
      int bad = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= rho;
        am = fmax(am, fabs(x[e]));
        bad |= !(fabs(x[e]) < __builtin_inf());
      }
      am = quad(am, [](double p, double q) { return fmax(p, q); });
      bad = quad(bad, [](int p, int q) { return p | q; });
      sb = kv4_f16_scale((float)(am / 6.0), am == 0.0, bad != 0);
      e2m1_from_f64(x, (double)f16_value(sb), b);
    } else {
      if (w) {
        float ss = 0.0f, v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(f[e], f[e], ss);
        ss = row_sum(ss, tpr, r * tpr, c);
        const float rho = 1.0f / sqrtf(ss / (float)a.D + (float)a.eps);
        unpack8(wown, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= v[e];
        if (turning) rotate(a, mine, w, c, cs_all + cur.tok * half, wpart, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= rho;
      } else if (turning) {
        rotate(a, mine, w, c, cs_all + cur.tok * half, wpart, f);
      }
    }
    __builtin_amdgcn_wave_barrier();                          // reads above before the next rows' writes

    if (cur.kind == kQ || KOUT == 0) {
      if (cur.live) {
        uint16_t* out = (cur.kind == kQ ? a.q_out + t * a.q_out_stride : a.k_out + t * a.k_out_stride) +
                        (int64_t)cur.head * a.D + c * 8;
        const u32x4 p = {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                         pack_bf16x2(f[6], f[7])};
        if (a.vec_out) {
          st16(out, p);
        } else {
          const uint32_t d[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) out[e] = (uint16_t)(d[e / 2] >> (16 * (e & 1)));
        }
      }
      continue;
    }
    const bool stored = cur.live && cur.slot >= 0 && cur.slot < a.pool;
    const int64_t at = cur.slot * a.Hk + cur.head;
    if constexpr (KOUT == 4) {
      if (!exact) {                                           // bf16 as it came: quotients in fp32 decide the same
        uint32_t am = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) am = max(am, __builtin_bit_cast(uint32_t, f[e]) & 0x7FFFFFFFu);
        am = quad(am, [](uint32_t p, uint32_t q) { return max(p, q); });
        sb = kv4_f16_scale(__builtin_bit_cast(float, am) / 6.0f, am == 0, am >= 0x7F800000u);
        const RcpDiv dv(f16_value(sb));
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = f32x2_to_e2m1x2_sat(dv(f[2 * e]), dv(f[2 * e + 1]));
      }
      uint8_t* code = bytes[wave] + (lane_live ? r : 0) * (a.D / 2);
      if (cur.live) {
#pragma unroll
        for (int j = 0; j < 4; ++j) code[run.first + (4 * (c & 3) + j) * run.step] = (uint8_t)b[j];
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      if (stored) {
        const uint32_t d = *reinterpret_cast<const uint32_t*>(code + 4 * c);
        uint8_t* codes = cur.kind == kK ? a.k_codes : a.v_codes;
        uint16_t* scales = cur.kind == kK ? a.k_scales : a.v_scales;
        *reinterpret_cast<uint32_t*>(codes + at * (a.D / 2) + 4 * c) = d;
        if ((c & 3) == 0) scales[at * (a.D / 32) + c / 4] = (uint16_t)sb;
      }
      __builtin_amdgcn_wave_barrier();                        // reads above before the next rows' writes
    } else if constexpr (KOUT == 8) {
      float am = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) am = fmaxf(am, fabsf(f[e]));
      am = quad(am, [](float p, float q) { return fmaxf(p, q); });
      if (cur.kind == kV) {                                   // one scale for the whole row
        float rm = am;
        for (int g = 4; g < tpr; g += 4) {
          const int src = c + g >= tpr ? c + g - tpr : c + g;
          rm = fmaxf(rm, __shfl(am, (r * tpr + src) & 63, 64));
        }
        am = rm;
      }
      if (stored) {
        sb = kv_f16_scale(am, cur.kind == kK ? 127.0f : 448.0f);
        const RcpDiv dv(f16_value(sb));
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = dv(f[e]);
        if (cur.kind == kK) {
          const u32x2 p = {f32_to_i8_sat(d[0]) | (f32_to_i8_sat(d[1]) << 8) | (f32_to_i8_sat(d[2]) << 16) |
                               (f32_to_i8_sat(d[3]) << 24),
                           f32_to_i8_sat(d[4]) | (f32_to_i8_sat(d[5]) << 8) | (f32_to_i8_sat(d[6]) << 16) |
                               (f32_to_i8_sat(d[7]) << 24)};
          *reinterpret_cast<u32x2*>(a.k_codes + at * a.D + c * 8) = p;
          if ((c & 3) == 0) a.k_scales[at * (a.D / 32) + c / 4] = (uint16_t)sb;
        } else {
          const u32x2 p = {f32x4_to_e4m3x4_sat(d[0], d[1], d[2], d[3]), f32x4_to_e4m3x4_sat(d[4], d[5], d[6], d[7])};
          *reinterpret_cast<u32x2*>(a.v_codes + at * a.D + c * 8) = p;
          if (c == 0) a.v_scales[at] = (uint16_t)sb;
        }
      }
    }
  }
}

// Rows of chosen slots of a 4-bit cache back to bf16 (8 channels per thread); a slot outside the pool
// gives zeros.
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

}  // namespace

hipError_t launch_norm_rope(const NormRopeArgs& a, int kout, hipStream_t st) {
  NormRopeArgs b = a;
  const int rpw = 64 / (a.D / 8);
  const int batches = (a.Hq + rpw - 1) / rpw + (kout ? 2 : 1) * ((a.Hk + rpw - 1) / rpw);
  b.TW = a.T >= 2048 ? 2 : 1;
  const int gy = a.T < 1024 ? (batches + kWaves - 1) / kWaves : 1;
  const dim3 grid((unsigned)((a.T + b.TW - 1) / b.TW), (unsigned)gy);
  const size_t lds = (size_t)b.TW * a.R * (kout == 4 ? 12 : 4);
  if (kout == 0) norm_rope_kernel<0><<<grid, kWaves * 64, lds, st>>>(b);
  else if (kout == 8) norm_rope_kernel<8><<<grid, kWaves * 64, lds, st>>>(b);
  else norm_rope_kernel<4><<<grid, kWaves * 64, lds, st>>>(b);
  return hipGetLastError();
}

hipError_t launch_kv4_gather(const void* kq, const void* ks, const void* vq, const void* vs, int64_t pool, int H, int D,
                             const void* slots, int slot64, int64_t n, void* ko, void* vo, hipStream_t st) {
  const int64_t n8 = n * H * D / 8;
  int64_t g = (n8 + 255) / 256;
  if (g > 8192) g = 8192;
  kv4_gather_kernel<<<(int)g, 256, 0, st>>>(static_cast<const uint8_t*>(kq), static_cast<const uint16_t*>(ks),
                                           static_cast<const uint8_t*>(vq), static_cast<const uint16_t*>(vs), pool, H, D,
                                           slots, slot64, n8, static_cast<uint16_t*>(ko), static_cast<uint16_t*>(vo));
  return hipGetLastError();
}

}  // namespace qlq
