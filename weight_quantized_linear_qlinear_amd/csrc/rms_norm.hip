// RMS norm with the residual's addition, to bf16 or straight to the next linear's 8-bit codes.
//
//   h = x + residual (fp32, not rounded; residual_out = bf16(h)),
//   rho = 1 / sqrt(mean_k h^2 + eps),   y = h * rho * w   (fp32),
//   out: bf16(y)  |  sat(rne(y / input_scale))  |  s = absmax_k |y| / qmax, sat(rne(y / s)).
//
// The codes are taken from the fp32 value: one rounding, where a norm to bf16 followed by the
// quantizer has two (and two more passes over the rows).  Sums of squares are fp64.
// y / s = (h w) g with one factor per row, g = rho / input_scale or, as s = absmax |h w| rho /
// qmax, g = qmax / absmax |h w|: the dynamic codes do not depend on rho, so a row needs one
// reduction (its sum of squares and its absmax together), and an element one product for its
// code instead of a division.  rho and g are formed in fp64, once per row, and g goes into the product
// as two fp32: what stands before a code's rounding is h w rounded once and the product rounded
// once.  (All of it in fp64, or fp64 only next to a rounding border, takes 56 instead of 43 us for
// 8192 rows of 4096 to FP8.)  A g below 2^-100, or so large that h w times its second part could
// overflow, divides element by element.
//
// Bound by HBM for many rows (2 K bytes of x, 2 K of the residual in and out, K of codes per
// row) and by latency for few: a row is read once, kept in registers as fp32 (8 elements per
// 16-byte chunk, NC chunks per thread) and written once.  Measured (MI355X, kernel alone): 8192
// rows of 4096 with a residual, bf16 out, 43.9 us (268 MB, 6.1 TB/s); 333 of 4096 to FP8 5.2 us;
// 1000 of 2048 to INT8 5.8 us; one of 2048 to FP8 2.7 us.  Rows that are no whole 16-byte chunks
// take the kernel below that reads elements, twice: 8192 of 4095 111 us (bf16) and 123 us (FP8, where
// 4096 columns take 44), 333 of 5001 15 and 17 us (5000 columns 6.6 and 7.1).
#include "qlq_device.h"
#include "qlq_launch.h"

namespace qlq {

namespace {

enum NormOut : int { kNormBf16 = 0, kNormStatic = 1, kNormDynamic = 2 };

struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;       // or null
  const uint16_t* w;
  void* y;                   // bf16 [M,K] or codes [M,K]; may be x or res (bf16)
  float* y_scale;            // [M], dynamic only
  uint16_t* res_out;         // or null; may be x or res
  int M, K;
  float eps, input_scale;
  int fp8;
};

__device__ __forceinline__ double wave_sum(double v) {
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// The larger one; NaN if either is (a row with a NaN keeps it in its scale).
__device__ __forceinline__ float most_of(float a, float b) { return __builtin_elementwise_maximum(a, b); }

__device__ __forceinline__ float wave_absmax(float v) {
  for (int off = 32; off > 0; off >>= 1) v = most_of(v, __shfl_xor(v, off, 64));
  return v;
}

// Code of v g, or of v / d g where g is not a normal number (d: what g would divide by).
struct Coder {
  float g, rest, num, den;       // g + rest = num / den
  int fp8;
  bool plain;
  // most: g up to which h w times `rest` is finite (2^100 where h w g is a code, 2^23 for any h w)
  __device__ __forceinline__ Coder(double n, double d, double most, int fp8_) : num((float)n), den((float)d), fp8(fp8_) {
    const double q = n / d;
    g = (float)q;
    rest = (float)(q - (double)g);
    plain = q >= 0x1p-100 && q <= most;
  }
  __device__ __forceinline__ float scaled(float v) const { return plain ? __builtin_fmaf(v, g, v * rest) : v / den * num; }
  __device__ __forceinline__ uint32_t one(float v) const {
    const float c = scaled(v);
    return fp8 ? f32_to_e4m3_sat(c) : f32_to_i8_sat(c);
  }
  __device__ __forceinline__ uint32_t four(const float* v) const {
    const float a = scaled(v[0]), b = scaled(v[1]), c = scaled(v[2]), d = scaled(v[3]);
    if (fp8) return f32x4_to_e4m3x4_sat(a, b, c, d);
    return f32_to_i8_sat(a) | (f32_to_i8_sat(b) << 8) | (f32_to_i8_sat(c) << 16) | (f32_to_i8_sat(d) << 24);
  }
};

// A row's 1 / sqrt(mean + eps) in fp64 from its sum of squares.
__device__ __forceinline__ double rho_of(double ss, int K, float eps) { return 1.0 / sqrt(ss / K + (double)eps); }

struct RowPart {
  double sum;
  float most;
};

// Sum of v and maximum of w over a row of T threads (T = 64: a wave; else through `red`).
template <int T, bool MAX>
__device__ __forceinline__ void row_reduce(double& v, float& w, RowPart* red) {
  v = wave_sum(v);
  if constexpr (MAX) w = wave_absmax(w);
  if constexpr (T > 64) {
    const int i = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[i] = RowPart{v, w};
    __syncthreads();
    v = red[0].sum, w = red[0].most;
#pragma unroll
    for (int k = 1; k < T / 64; ++k) v += red[k].sum, w = most_of(w, red[k].most);
  }
}

// T threads per row (64: four rows per workgroup of 256; 256 or 1024: one row per workgroup),
// up to NC chunks of 8 elements per thread: K <= 8 T NC, K % 8 == 0, aligned pointers.
template <int OUT, int T, int NC>
__global__ __launch_bounds__(T == 64 ? 256 : T) void rms_norm_kernel(NormArgs a) {
  constexpr int RPW = T == 64 ? 4 : 1;
  __shared__ RowPart red[T > 64 ? T / 64 : 1];
  const int t = T == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int m = blockIdx.x * RPW + (T == 64 ? (threadIdx.x >> 6) : 0);
  if (m >= a.M) return;                                       // whole waves; T > 64 has no idle row
  const int nv = a.K / 8;
  const int64_t base = (int64_t)m * a.K;
  u32x4 xr[NC], rr[NC], wr[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = t + c * T;
    const bool in = i < nv;
    xr[c] = in ? ld16_stream(a.x + base + i * 8) : (u32x4){0u, 0u, 0u, 0u};
    if (a.res) rr[c] = in ? ld16_stream(a.res + base + i * 8) : (u32x4){0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = t + c * T;
    wr[c] = i < nv ? ld16(a.w + i * 8) : (u32x4){0u, 0u, 0u, 0u};
  }
  float h[NC][8];
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const uint32_t xd[4] = {xr[c].x, xr[c].y, xr[c].z, xr[c].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[c][2 * e] = bf16_bits_to_f32(xd[e] & 0xFFFF);
      h[c][2 * e + 1] = bf16_bits_to_f32(xd[e] >> 16);
    }
    if (a.res) {
      const uint32_t rd[4] = {rr[c].x, rr[c].y, rr[c].z, rr[c].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[c][2 * e] += bf16_bits_to_f32(rd[e] & 0xFFFF);
        h[c][2 * e + 1] += bf16_bits_to_f32(rd[e] >> 16);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fma((double)h[c][e], (double)h[c][e], ss);
  }
  if (a.res_out) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = t + c * T;
      if (i < nv)
        st16(a.res_out + base + i * 8, (u32x4){pack_bf16x2(h[c][0], h[c][1]), pack_bf16x2(h[c][2], h[c][3]),
                                               pack_bf16x2(h[c][4], h[c][5]), pack_bf16x2(h[c][6], h[c][7])});
    }
  }
  float am = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {                              // h w
    const uint32_t wd[4] = {wr[c].x, wr[c].y, wr[c].z, wr[c].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[c][2 * e] *= bf16_bits_to_f32(wd[e] & 0xFFFF);
      h[c][2 * e + 1] *= bf16_bits_to_f32(wd[e] >> 16);
      if constexpr (OUT == kNormDynamic)
        am = most_of(am, most_of(fabsf(h[c][2 * e]), fabsf(h[c][2 * e + 1])));
    }
  }
  row_reduce<T, OUT == kNormDynamic>(ss, am, red);
  const double rho = rho_of(ss, a.K, a.eps);
  if constexpr (OUT == kNormBf16) {
    const float r = (float)rho;
    uint16_t* y = static_cast<uint16_t*>(a.y) + base;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = t + c * T;
      if (i < nv)
        st16(y + i * 8, (u32x4){pack_bf16x2(h[c][0] * r, h[c][1] * r), pack_bf16x2(h[c][2] * r, h[c][3] * r),
                                pack_bf16x2(h[c][4] * r, h[c][5] * r), pack_bf16x2(h[c][6] * r, h[c][7] * r)});
    }
  } else {
    const double qmax = a.fp8 ? 448.0 : 127.0;
    if (OUT == kNormDynamic && t == 0) a.y_scale[m] = am == 0.0f ? 1.0f : (float)((double)am * rho / qmax);
    const Coder code = OUT == kNormStatic ? Coder(rho, (double)a.input_scale, 0x1p23, a.fp8)
                                          : Coder(qmax, am == 0.0f ? 1.0 : (double)am, 0x1p100, a.fp8);
    uint8_t* y = static_cast<uint8_t*>(a.y) + base;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = t + c * T;
      if (i < nv) *reinterpret_cast<u32x2*>(y + i * 8) = (u32x2){code.four(h[c]), code.four(h[c] + 4)};
    }
  }
}

// Any K and alignment: element by element, x and the residual read again by each pass.  Only
// the last pass writes, each element by the thread that has just read it, so the outputs may
// be the inputs here too.
template <int OUT>
__global__ __launch_bounds__(256) void rms_norm_any_kernel(NormArgs a) {
  __shared__ RowPart red[4];
  const int t = threadIdx.x, m = blockIdx.x;
  const int64_t base = (int64_t)m * a.K;
  auto load = [&](int k) {
    const float v = bf16_bits_to_f32(a.x[base + k]);
    return a.res ? v + bf16_bits_to_f32(a.res[base + k]) : v;
  };
  double ss = 0.0;
  float am = 0.0f;
  for (int k = t; k < a.K; k += 256) {
    const float v = load(k);
    ss = __builtin_fma((double)v, (double)v, ss);
    if constexpr (OUT == kNormDynamic) am = most_of(am, fabsf(v * bf16_bits_to_f32(a.w[k])));
  }
  row_reduce<256, OUT == kNormDynamic>(ss, am, red);
  const double rho = rho_of(ss, a.K, a.eps), qmax = a.fp8 ? 448.0 : 127.0;
  const float r = (float)rho;
  if (OUT == kNormDynamic && t == 0) a.y_scale[m] = am == 0.0f ? 1.0f : (float)((double)am * rho / qmax);
  const Coder code = OUT == kNormStatic ? Coder(rho, (double)a.input_scale, 0x1p23, a.fp8)
                                        : Coder(qmax, am == 0.0f ? 1.0 : (double)am, 0x1p100, a.fp8);
  for (int k = t; k < a.K; k += 256) {
    const float v = load(k), hw = v * bf16_bits_to_f32(a.w[k]);
    if (a.res_out) a.res_out[base + k] = (uint16_t)(pack_bf16x2(v, v) & 0xFFFF);
    if constexpr (OUT == kNormBf16) static_cast<uint16_t*>(a.y)[base + k] = (uint16_t)(pack_bf16x2(hw * r, hw * r) & 0xFFFF);
    else static_cast<uint8_t*>(a.y)[base + k] = (uint8_t)code.one(hw);
  }
}

template <int OUT>
hipError_t launch_norm(const NormArgs& a, bool vec, hipStream_t st) {
  const int nv = a.K / 8;
  if (!vec || nv > 1024 * 8) {
    rms_norm_any_kernel<OUT><<<a.M, 256, 0, st>>>(a);
  } else if (a.M >= 1024 && nv <= 64 * 8) {
    // Many rows: a wave per row, no barrier.
    const int g = (a.M + 3) / 4;
    if (nv <= 64) rms_norm_kernel<OUT, 64, 1><<<g, 256, 0, st>>>(a);
    else if (nv <= 128) rms_norm_kernel<OUT, 64, 2><<<g, 256, 0, st>>>(a);
    else if (nv <= 256) rms_norm_kernel<OUT, 64, 4><<<g, 256, 0, st>>>(a);
    else rms_norm_kernel<OUT, 64, 8><<<g, 256, 0, st>>>(a);
  } else if (nv <= 256 * 8) {
    if (nv <= 256) rms_norm_kernel<OUT, 256, 1><<<a.M, 256, 0, st>>>(a);
    else if (nv <= 512) rms_norm_kernel<OUT, 256, 2><<<a.M, 256, 0, st>>>(a);
    else if (nv <= 1024) rms_norm_kernel<OUT, 256, 4><<<a.M, 256, 0, st>>>(a);
    else rms_norm_kernel<OUT, 256, 8><<<a.M, 256, 0, st>>>(a);
  } else {
    rms_norm_kernel<OUT, 1024, 8><<<a.M, 1024, 0, st>>>(a);
  }
  return hipGetLastError();
}

bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

hipError_t launch_rms_norm(const void* x, const void* residual, const void* w, int M, int K, float eps, int out,
                           int qtype, float input_scale, void* y, float* y_scale, void* residual_out, hipStream_t st) {
  NormArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(residual), static_cast<const uint16_t*>(w),
             y, y_scale, static_cast<uint16_t*>(residual_out), M, K, eps, input_scale, qtype == kFp8 ? 1 : 0};
  const bool vec = K % 8 == 0 && al(x, 16) && al(residual, 16) && al(w, 16) && al(residual_out, 16) &&
                   al(y, out == kNormBf16 ? 16 : 8);
  // A launch's threads are counted in 32 bits: at most 2^21 rows (of up to 1024 threads) at a time.
  constexpr int kRows = 1 << 21;
  for (int m = 0; m < M; m += kRows) {
    NormArgs b = a;
    const int64_t at = (int64_t)m * K;
    b.M = M - m < kRows ? M - m : kRows;
    b.x = a.x + at;
    if (a.res) b.res = a.res + at;
    if (a.res_out) b.res_out = a.res_out + at;
    b.y = static_cast<uint8_t*>(a.y) + (out == kNormBf16 ? 2 : 1) * at;
    if (a.y_scale) b.y_scale = a.y_scale + m;
    const hipError_t e = out == kNormBf16   ? launch_norm<kNormBf16>(b, vec, st)
                         : out == kNormStatic ? launch_norm<kNormStatic>(b, vec, st)
                                              : launch_norm<kNormDynamic>(b, vec, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qlq
