// Rotary positions, alone and in one pass with writing K and V into the 8-bit cache, and
// reading cache slots back.
//
// Rotation of the first R channels of a head row at position p (R even, the rest unchanged):
//   theta_i = p * inv_freq[i]  (i < R/2; product and reduction by 2 pi in 64 bits, so that
//   positions of millions keep their angle),  c = factor * cos, s = factor * sin  (fp32),
//   (a, b) -> (a c - b s, a s + b c)   for the pair (i, i + R/2), or (2i, 2i+1) interleaved.
// Cache entries are the codec's (kv_codec.hip): K int8 with an fp16 scale per 32 channels, V
// e4m3 with one per (token, head).  A rotated K is quantized from its fp32 value: one rounding
// fewer than rotating to bf16 first.
//
// One workgroup per TW tokens (or per token and a share of its heads, while tokens are few): its
// threads compute the tokens' R/2 angles once for all heads into LDS.  A head row is D/8 lanes
// of one wave, 8 channels each; the row passes through the wave's LDS so that a lane finds its
// pair partners, and every load of a row comes before its stores, so q may be rotated in
// place.  Bound by HBM for many tokens, by latency for few.  Measured (MI355X, kernel alone):
// 8191 tokens of 32 + 8 + 8 heads of 128 in 41.4 us (185 MB, 4.5 TB/s), 2048 in 13.9 us, 16 of
// 28 + 4 + 4 heads in 4.4 us; gathering 8191 slots of 8 heads 10.7 us (51 MB, 4.8 TB/s).
#include "qlq_device.h"
#include "qlq_launch.h"

namespace qlq {

namespace {

constexpr int kRopeWaves = 4;

__device__ __forceinline__ uint32_t kv_f16_scale(float absmax, float qmax) {   // the codec's rule
  if (absmax == 0.0f) return 0x3C00u;
  const float c = __builtin_amdgcn_fmed3f(absmax / qmax, 65504.0f, -65504.0f);
  const uint32_t s = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)c);
  return s == 0u ? 1u : s;
}

__device__ __forceinline__ float f16_value(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (uint16_t)b); }

__device__ __forceinline__ int64_t load_index(const void* p, int is64, int64_t i) {
  return is64 ? static_cast<const int64_t*>(p)[i] : (int64_t)static_cast<const int32_t*>(p)[i];
}

// Eight bf16 at p (any alignment unless vec).
__device__ __forceinline__ u32x4 load8(const uint16_t* p, bool vec) {
  if (vec) return ld16(p);
  u32x4 r;
  r.x = p[0] | ((uint32_t)p[1] << 16);
  r.y = p[2] | ((uint32_t)p[3] << 16);
  r.z = p[4] | ((uint32_t)p[5] << 16);
  r.w = p[6] | ((uint32_t)p[7] << 16);
  return r;
}

__device__ __forceinline__ void unpack8(u32x4 v, float* f) {
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = bf16_bits_to_f32(d[e] & 0xFFFF);
    f[2 * e + 1] = bf16_bits_to_f32(d[e] >> 16);
  }
}

// Angles of the positions of tokens t0 .. t0 + n - 1: cs[k R/2 + i] = (factor cos, factor sin).
__device__ __forceinline__ void token_angles(const RopeArgs& a, int64_t t0, int n, float2* cs) {
  const int half = a.R / 2;
  for (int j = threadIdx.x; j < n * half; j += kRopeWaves * 64) {
    const int k = j / half, i = j - k * half;
    const int64_t pos = load_index(a.positions, a.pos64, t0 + k);
    const double th = (double)pos * a.inv_freq[i];
    const double q = rint(th * 0x1.45f306dc9c883p-3);                    // 1 / (2 pi)
    double r = __builtin_fma(-q, 0x1.921fb54442d18p+2, th);             // 2 pi, high part
    r = __builtin_fma(-q, 0x1.1a62633145c07p-52, r);                    // and the rest of it
    float s, c;
    sincosf((float)r, &s, &c);
    cs[j] = make_float2(a.factor * c, a.factor * s);
  }
}

__global__ __launch_bounds__(kRopeWaves * 64) void rope_kv_kernel(RopeArgs a) {
  extern __shared__ __align__(16) float2 cs_all[];           // [TW][R / 2]
  __shared__ __align__(16) uint16_t rows[kRopeWaves][512];   // 64 lanes x 8 channels per wave
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * a.TW;
  const int ntok = (int)min((int64_t)a.TW, a.T - t0);
  const int tpr = a.D / 8, rpw = 64 / tpr;                    // lanes per row, rows per wave
  const int r = lane / tpr, c = lane % tpr;
  const int total = a.Hq + a.Hk + a.Hv, all = ntok * total;   // rows of a token: q, then k, then v
  const int step = gridDim.y * kRopeWaves * rpw;
  const int first = (blockIdx.y * kRopeWaves + wave) * rpw;
  const bool lane_live = r < rpw;
  // The row `at` of this lane: its token, its place in the token, its data and its cache slot.
  struct Row {
    u32x4 raw;
    int64_t slot;
    int tok, row;
    bool live;
  };
  auto load = [&](int at) -> Row {
    Row w;
    w.live = lane_live && at < all;
    w.tok = w.live ? at / total : 0;
    w.row = w.live ? at - w.tok * total : 0;
    w.raw = (u32x4){0u, 0u, 0u, 0u};
    w.slot = -1;
    const int64_t t = t0 + w.tok;
    if (w.live) {
      if (w.row < a.Hq) w.raw = load8(a.q + t * a.q_stride + (int64_t)w.row * a.D + c * 8, a.vec_in);
      else if (w.row < a.Hq + a.Hk) w.raw = load8(a.k + t * a.k_stride + (int64_t)(w.row - a.Hq) * a.D + c * 8, a.vec_in);
      else w.raw = load8(a.v + t * a.v_stride + (int64_t)(w.row - a.Hq - a.Hk) * a.D + c * 8, a.vec_in);
      if (a.Hk) w.slot = load_index(a.slots, a.slot64, t);
    }
    return w;
  };
  Row next = load(first + r);
  if (a.R) token_angles(a, t0, ntok, cs_all);
  __syncthreads();
  for (int base = first; base < all; base += step) {          // uniform per wave
    const Row cur = next;
    next = load(base + step + r);                             // the next batch's rows are in flight meanwhile
    const u32x4 raw = cur.raw;
    const int row = cur.row;
    const bool live = cur.live;
    const int64_t t = t0 + cur.tok, slot = cur.slot;
    const bool stored = slot >= 0 && slot < a.pool;
    const float2* cs = cs_all + cur.tok * (a.R / 2);
    float f[8];
    unpack8(raw, f);
    // the wave's rows through its own LDS: written and read by this wave alone, in order
    uint16_t* mine = rows[wave] + r * a.D;
    if (live) st16(mine + c * 8, raw);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const bool turns = live && row < a.Hq + a.Hk && c * 8 < a.R;
    if (turns) {
      const int half = a.R / 2;
      if (a.R % 16 == 0) {                                    // (also keeps the 16-byte reads aligned)
        // the chunk is whole: one run of cosines and sines, read as vectors
        const int i0 = a.interleaved ? c * 4 : c * 8 < half ? c * 8 : c * 8 - half;
        f32x4 w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!a.interleaved || e < 2) w[e] = *reinterpret_cast<const f32x4*>(&cs[i0 + 2 * e]);
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float co = w[e / 2][2 * (e & 1)], si = w[e / 2][2 * (e & 1) + 1];
            const float x = f[2 * e], y = f[2 * e + 1];
            f[2 * e] = x * co - y * si;
            f[2 * e + 1] = x * si + y * co;
          }
        } else {
          float o[8];
          unpack8(ld16(mine + (c * 8 < half ? c * 8 + half : c * 8 - half)), o);
          const float sign = c * 8 < half ? -1.0f : 1.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = f[e] * w[e / 2][2 * (e & 1)] + sign * o[e] * w[e / 2][2 * (e & 1) + 1];
        }
      } else if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = c * 4 + e;                            // pair (2 i, 2 i + 1)
          if (i < half) {
            const float2 w = cs[i];
            const float x = f[2 * e], y = f[2 * e + 1];
            f[2 * e] = x * w.x - y * w.y;
            f[2 * e + 1] = x * w.y + y * w.x;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int ch = c * 8 + e;
          if (ch < a.R) {
            const float2 w = cs[ch < half ? ch : ch - half];
            const float o = bf16_bits_to_f32(mine[ch < half ? ch + half : ch - half]);
            f[e] = ch < half ? f[e] * w.x - o * w.y : o * w.y + f[e] * w.x;
          }
        }
      }
    }
    __builtin_amdgcn_wave_barrier();                          // reads above before the next rows' writes
    if (row < a.Hq) {
      if (live) {
        uint16_t* out = a.q_out + t * a.q_out_stride + (int64_t)row * a.D + c * 8;
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
    }
    if (a.Hk && __ballot(live && row >= a.Hq)) {              // wave-uniform: some K or V rows
      float am = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) am = fmaxf(am, fabsf(f[e]));
      am = fmaxf(am, __shfl_xor(am, 1, 64));                  // 32 channels: 4 lanes (D % 32 == 0)
      am = fmaxf(am, __shfl_xor(am, 2, 64));
      float rm = am;                                          // the whole row, for V
      for (int g = 1; g < tpr / 4; ++g) {
        int src = lane + 4 * g;
        if (src >= (r + 1) * tpr) src -= tpr;
        rm = fmaxf(rm, __shfl(am, src & 63, 64));
      }
      if (live && row >= a.Hq && stored) {
        const bool is_k = row < a.Hq + a.Hk;
        const int h = is_k ? row - a.Hq : row - a.Hq - a.Hk;
        const int64_t at = slot * a.Hk + h;
        const uint32_t sb = is_k ? kv_f16_scale(am, 127.0f) : kv_f16_scale(rm, 448.0f);
        const RcpDiv dv(f16_value(sb));                       // (the codec's codes wherever the input is bf16)
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = dv(f[e]);
        if (is_k) {
          const u32x2 w = {f32_to_i8_sat(d[0]) | (f32_to_i8_sat(d[1]) << 8) | (f32_to_i8_sat(d[2]) << 16) |
                               (f32_to_i8_sat(d[3]) << 24),
                           f32_to_i8_sat(d[4]) | (f32_to_i8_sat(d[5]) << 8) | (f32_to_i8_sat(d[6]) << 16) |
                               (f32_to_i8_sat(d[7]) << 24)};
          *reinterpret_cast<u32x2*>(a.k_codes + at * a.D + c * 8) = w;
          if ((c & 3) == 0) a.k_scales[at * (a.D / 32) + c / 4] = (uint16_t)sb;
        } else {
          const u32x2 w = {f32x4_to_e4m3x4_sat(d[0], d[1], d[2], d[3]), f32x4_to_e4m3x4_sat(d[4], d[5], d[6], d[7])};
          *reinterpret_cast<u32x2*>(a.v_codes + at * a.D + c * 8) = w;
          if (c == 0) a.v_scales[at] = (uint16_t)sb;
        }
      }
    }
  }
}

// Rows of chosen slots back to bf16 (8 elements per thread, as the codec's dequantizer); a slot
// outside the pool gives zeros.
__global__ __launch_bounds__(256) void kv_gather_kernel(const uint8_t* __restrict__ kq, const uint16_t* __restrict__ ks,
                                                        const uint8_t* __restrict__ vq, const uint16_t* __restrict__ vs,
                                                        int64_t pool, int H, int D, const void* __restrict__ slots,
                                                        int slot64, int64_t n8, uint16_t* __restrict__ ko,
                                                        uint16_t* __restrict__ vo) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  const uint32_t row8 = (uint32_t)H * D / 8;                  // chunks per slot
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n8; i += stride) {
    const int64_t n = i / row8;
    const uint32_t e = (uint32_t)(i - n * row8) * 8;          // element within the slot's [H, D]
    const int64_t slot = load_index(slots, slot64, n);
    u32x4 k = {0u, 0u, 0u, 0u}, v = {0u, 0u, 0u, 0u};
    if (slot >= 0 && slot < pool) {
      const int64_t at = slot * H * D + e;
      const float sk = f16_value(ks[at / 32]), sv = f16_value(vs[slot * H + e / D]);
      const u32x2 kc = *reinterpret_cast<const u32x2*>(kq + at);
      const u32x2 vc = *reinterpret_cast<const u32x2*>(vq + at);
      k = __builtin_bit_cast(u32x4, dequant8<kInt8>(kc.x, kc.y, sk, -128.0f * sk));
      v = __builtin_bit_cast(u32x4, dequant8<kFp8>(vc.x, vc.y, sv, -128.0f * sv));
    }
    st16(ko + i * 8, k);
    st16(vo + i * 8, v);
  }
}

}  // namespace

hipError_t launch_rope_kv(const RopeArgs& a, hipStream_t st) {
  // A workgroup takes 4 waves x (64 / (D / 8)) head rows at a time.  Few tokens: one such batch
  // per workgroup (more, shorter workgroups); from 2048 on two tokens per workgroup share the
  // wait for positions and angles (2048 tokens, 32 + 2 x 8 heads of 128: 15.6 -> 13.8 us, 8191:
  // 46.1 -> 41.3 us; four tokens: 17.3 and 41.3 us; split by batches: 18.8 and 63 us).  Between, one
  // against two tokens, inputs in cache: 32 + 2 x 8 heads of 128, 1200 tokens 9.5 and 10.8 us, 1600
  // 11.9 and 12.3, 2047 12.9 and 12.6, 3000 17.6 and 18.0; 28 + 2 x 4, 8.2 and 8.9, 10.4 and 10.1,
  // 11.4 and 10.6, 15.5 and 14.6; 16 + 2 x 16 heads of 64 6.9 and 7.2, 8.5 and 8.2, 9.4 and 8.5, 12.7
  // and 11.6: they cross between 1400 and 2047 tokens, by the heads.
  RopeArgs b = a;
  const int rpw = 64 / (a.D / 8), rows = a.Hq + a.Hk + a.Hv;
  const int batches = (rows + kRopeWaves * rpw - 1) / (kRopeWaves * rpw);
  b.TW = a.T >= 2048 ? 2 : 1;
  const int gy = a.T < 1024 ? batches : 1;
  rope_kv_kernel<<<dim3((unsigned)((a.T + b.TW - 1) / b.TW), (unsigned)gy), kRopeWaves * 64,
                   (size_t)b.TW * (a.R / 2) * sizeof(float2), st>>>(b);
  return hipGetLastError();
}

hipError_t launch_kv_gather(const void* kq, const void* ks, const void* vq, const void* vs, int64_t pool, int H, int D,
                            const void* slots, int slot64, int64_t n, void* ko, void* vo, hipStream_t st) {
  const int64_t n8 = n * H * D / 8;
  int64_t g = (n8 + 255) / 256;
  if (g > 8192) g = 8192;
  kv_gather_kernel<<<(int)g, 256, 0, st>>>(static_cast<const uint8_t*>(kq), static_cast<const uint16_t*>(ks),
                                          static_cast<const uint8_t*>(vq), static_cast<const uint16_t*>(vs), pool, H, D,
                                          slots, slot64, n8, static_cast<uint16_t*>(ko), static_cast<uint16_t*>(vo));
  return hipGetLastError();
}

}  // namespace qlq
