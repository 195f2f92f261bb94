// Attention over the paged 8-bit KV cache for many query rows per KV head (a prompt chunk over
// its cached prefix).  The same definition, cache and cutting of the work as kv_attention.hip;
// what differs is where the time goes: with hundreds of rows per K and V load it is the matrix
// cores and the vector unit (exponentials, conversions), not HBM.
//
// A workgroup takes one KV head and 256 query rows (nq x G rows packed), 32 per wave; eight
// waves, so that each SIMD has two to fill one's vector work with the other's matrix work.  A
// tile of T tokens is converted once for all of them: K' = k_code k_scale and V' = v_code
// v_scale 2^-E in fp16 go to LDS (V' transposed), double buffered, one barrier per tile.  A
// wave's scores are S^T = K' Q^T and its values O^T += V'^T P^T on 32x32x16 products: lane l
// holds query l % 32, and its scores of a product are the operand that the values' products
// want, so the weights never cross lanes (V' is stored in the order of those tokens).
//
// Roundings to fp16's 11 bits: K', V' and the weights (kv_attention.hip has the weights' alone;
// there the products with the scales are fp32).  Range: K' overflows only for scales above 512,
// a tile with such a scale is computed in 2^-7 of it; E follows the largest V scale so far, so
// that V' of that scale keeps 2^6 .. 2^15 and smaller ones their 11 bits down to 2^-20 of it.
#include "kv_attention.h"

namespace qlq {

using namespace attn;

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileWaves = 8;
constexpr int kTileRows = 32 * kTileWaves;

__device__ __forceinline__ f32x16 mfma_f16_k16(f16x8 a, f16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float across32(float v, bool add) {   // over lanes l, l ^ 32
  const int i = __builtin_bit_cast(int, v);
  const auto r = __builtin_amdgcn_permlane32_swap(i, i, false, false);
  const int x = (int)r[0], y = (int)r[1];
  const float p = __builtin_bit_cast(float, x), q = __builtin_bit_cast(float, y);
  return add ? p + q : fmaxf(p, q);
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, f16x2 s) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, a) * s);
}

// A query tile's tokens: those that its rows can see.
struct Span {
  int i0, i1;                    // first and last query token
  int begin, end;                // tokens, begin a multiple of T
};

template <int T>
__device__ __forceinline__ Span span_of(const KvAttnArgs& a, const Extent& e, int qt) {
  Span s;
  s.i0 = qt * kTileRows / a.G;
  s.i1 = min(e.nq - 1, (qt * kTileRows + kTileRows - 1) / a.G);
  const int p0 = e.L - e.nq;
  s.end = min(max(a.causal ? p0 + s.i1 + 1 : e.L, 0), e.L);
  s.begin = a.window > 0 ? min(max(0, p0 + s.i0 - a.window + 1), s.end) & ~(T - 1) : 0;
  return s;
}

template <int T>
__device__ __forceinline__ int units_of(const Span& s) { return max(1, (s.end - s.begin + T - 1) / T); }

__device__ __forceinline__ int tiles_of(const KvAttnArgs& a, const Extent& e) {
  return (e.nq * a.G + kTileRows - 1) / kTileRows;
}

// Units (T tokens of one query tile) of sequence `b`, whole.
template <int T>
__device__ __forceinline__ int sequence_units(const KvAttnArgs& a, int b) {
  if (b >= a.B) return 0;
  const Extent e = extent_of(a, b);
  int n = 0;
  for (int qt = 0, k = tiles_of(a, e); qt < k; ++qt) n += units_of<T>(span_of<T>(a, e, qt));
  return n;
}

template <int NG>
struct TileShape {
  static constexpr int D = 32 * NG;
  static constexpr int T = NG <= 4 ? 64 : 32;    // tokens per tile
  static constexpr int KLD = D + 8;              // fp16 per token row of K' (16 bytes of padding: no bank conflicts)
};

template <int NG>
struct TileLds {
  typedef TileShape<NG> S;
  union {
    struct {
      _Float16 k[2][S::T][S::KLD];               // K' by token
      _Float16 v[2][S::D][S::T];                 // V' by channel, 16-byte pieces of 8 tokens swizzled
    };
    JoinLds join[kTileWaves];
  };
  // by tile % 4 (written two tiles ahead):
  float vs[4][S::T];                             // V scales, 2^-E each, 0 for a token that is not there
  float kmul[4], kback[4];                       // on K's scales, and what undoes it on the scores
  int e[4], gap[4];                              // E; whether a token is not there
};

// Where piece p (8 tokens) of channel d lies in its row: reads (16 channels, one piece) and
// writes (4 channels apart) then spread over the banks.
template <int T>
__device__ __forceinline__ int piece(int d, int p) {
  if constexpr (T == 64) return p ^ (((d >> 1) ^ (d >> 4)) & 7);
  return p ^ (((d >> 2) ^ (d >> 4)) & 3);
}

template <int NG>
__global__ __launch_bounds__(kTileWaves * 64) void kv_attention_tile_kernel(KvAttnArgs a) {
  typedef TileShape<NG> S;
  constexpr int D = S::D, T = S::T, TPW = T / kTileWaves, NB = T / 32, NL = TPW * D / 16;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  TileLds<NG>& sm = *reinterpret_cast<TileLds<NG>*>(smem_raw);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = a.Hk, h = blockIdx.x % hk, part = blockIdx.x / hk;    // a head's parts on one XCD where Hk is a multiple of 8
  const ConstInt* lens_table = (const ConstInt*)(uintptr_t)a.block_table;
  const int page_mask = (1 << a.page_shift) - 1;
  const uint32_t row_bytes = (uint32_t)hk * D;

  int total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) total += wave_sum(sequence_units<T>(a, b0 + lane));
  total = __builtin_amdgcn_readfirstlane(total);
  const int U = max(1, (total + a.parts - 1) / a.parts), u_end = min(total, (part + 1) * U);

  for (int u = part * U; u < u_end;) {                       // uniform for the workgroup
    // the sequence and the tile that unit u belongs to
    int b = 0, at = 0;
    for (int b0 = 0, before = 0; b0 < a.B; b0 += 64) {
      const int n = sequence_units<T>(a, b0 + lane), inc = before + wave_scan(n);
      const uint64_t hit = __ballot(u < inc && u >= inc - n);
      if (hit) {
        const int src = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
        b = b0 + src;
        at = __builtin_amdgcn_readlane(inc - n, src);
        break;
      }
      before = __builtin_amdgcn_readlane(inc, 63);
    }
    Extent e = extent_of(a, b);
    e.qs = __builtin_amdgcn_readfirstlane(e.qs);
    e.nq = __builtin_amdgcn_readfirstlane(e.nq);
    e.L = __builtin_amdgcn_readfirstlane(e.L);
    int qt = 0;
    Span sp = span_of<T>(a, e, 0);
    while (u >= at + units_of<T>(sp)) {
      at += units_of<T>(sp);
      sp = span_of<T>(a, e, ++qt);
    }
    const int units = units_of<T>(sp), u_next = min(u_end, at + units);
    const Chunks ck{at / U, (at + units - 1) / U - at / U + 1, part - at / U};
    const int c0 = sp.begin + T * (u - at), c1 = min(sp.end, sp.begin + T * (u_next - at));
    u = u_next;

    // this wave's rows
    const int r0 = qt * kTileRows + 32 * wave, rows = e.nq * a.G, live_rows = min(32, rows - r0);
    const int p0 = e.L - e.nq;
    const int first_p = p0 + r0 / a.G, last_p = p0 + (r0 + max(live_rows, 1) - 1) / a.G;   // positions
    int c32 = lane & 31, half = lane >> 5;
    asm volatile("" : "+v"(c32), "+v"(half));                // (nothing computed from them outlives a tile)
    const int myrow = r0 + c32;
    const bool live = c32 < live_rows;
    const int qi = live ? myrow / a.G : 0, qg = live ? myrow - qi * a.G : 0;
    const int qpos = live ? p0 + qi : -1;

    // q: channels 16 k + 8 half + 0..7 of the row, by a power of two into [-1, 1); the sign of the
    // scale goes with it, so that scores are multiplied by a positive number
    f16x8 qf[2 * NG];
    float cs;
    {
      const uint16_t* qp = a.q + (int64_t)(e.qs + qi) * a.q_stride + (int64_t)(h * a.G + qg) * D + 8 * half;
      u32x4 raw[2 * NG];
#pragma unroll
      for (int k = 0; k < 2 * NG; ++k) raw[k] = ld16(qp + 16 * k);
      float am = 0.0f;
#pragma unroll
      for (int k = 0; k < 2 * NG; ++k) {
        const uint32_t d[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          am = fmaxf(am, fmaxf(fabsf(bf16_bits_to_f32(d[i] & 0xFFFF)), fabsf(bf16_bits_to_f32(d[i] >> 16))));
      }
      am = across32(am, false);
      const int ex = am > 0.0f ? __builtin_amdgcn_frexp_expf(am) : 0;
      const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll
      for (int k = 0; k < 2 * NG; ++k) {
        const uint32_t d[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = live ? bf16_bits_to_f32(d[i] & 0xFFFF) * sign : 0.0f;
          const float y = live ? bf16_bits_to_f32(d[i] >> 16) * sign : 0.0f;
          qf[k][2 * i] = (_Float16)__builtin_ldexpf(x, -ex);
          qf[k][2 * i + 1] = (_Float16)__builtin_ldexpf(y, -ex);
        }
      }
      cs = fmaxf(__builtin_ldexpf(fabsf(a.scale) * kLog2e, ex), 0x1p-120f);   // (positive: -inf stays -inf)
    }

    // Loading: wave w brings tokens TPW w .. + TPW - 1 of a tile, which lie in one page (pages
    // hold 16 or more).  A lane converts 16 codes of one token's K and a 4 x 4 block of V.
    const ConstInt* table = lens_table + (int64_t)b * a.max_pages;
    auto page_of = [&](int t) { return table[min(t, a.max_tokens - 1) >> a.page_shift]; };
    auto entry_of = [&](int page, int t) {
      return page >= 0 && page < a.pages ? (page << a.page_shift) + (t & page_mask) : -1;
    };
    const int li = min(lane, NL - 1);
    const int krow = li / (D / 16), kchunk = li % (D / 16), vgrp = li / (D / 4), vcb = li % (D / 4);
    const uint32_t koff = krow * row_bytes + 16 * kchunk, voff = 4 * vgrp * row_bytes + 4 * vcb;
    const int first_t = TPW * wave;                          // this wave's first token of a tile
    u32x4 kraw;
    uint32_t vraw[4], ksraw;
    auto load = [&](int entry) {
      const int64_t at64 = (int64_t)max(entry, 0) * hk + h;
      kraw = ld16(a.k_codes + at64 * D + koff);
      ksraw = a.k_scales[(at64 + (int64_t)krow * hk) * NG + kchunk / 2];
      const uint8_t* vp = a.v_codes + at64 * D + voff;
#pragma unroll
      for (int i = 0; i < 4; ++i) vraw[i] = *reinterpret_cast<const uint32_t*>(vp + (size_t)i * row_bytes);
    };
    auto convert = [&](int n) {                              // the loaded tile, number n, into LDS buffer n % 2
      const int buf = n & 1;
      const float s = f16_lo(ksraw) * sm.kmul[n & 3];
      const f16x2 s2 = {(_Float16)s, (_Float16)s};
      const f32x4 vsc = *reinterpret_cast<const f32x4*>(&sm.vs[n & 3][first_t + 4 * vgrp]);
      if (lane < NL) {
        const uint32_t kd[4] = {kraw.x, kraw.y, kraw.z, kraw.w};
        u32x4 w[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t f = kd[i] ^ 0x80808080u;
          w[i / 2][2 * (i & 1)] = mul2(i8x2_to_f16<false>(f), s2);
          w[i / 2][2 * (i & 1) + 1] = mul2(i8x2_to_f16<true>(f), s2);
        }
        _Float16* kp = &sm.k[buf][first_t + krow][16 * kchunk];
        st16(kp, w[0]);
        st16(kp + 8, w[1]);
        // V: codes of a token that is not there may be NaN, so they go before the product
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = vsc[i] > 0.0f ? vraw[i] : 0u;
        const f16x2 v01 = {(_Float16)vsc[0], (_Float16)vsc[1]}, v23 = {(_Float16)vsc[2], (_Float16)vsc[3]};
        const uint32_t a01 = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u), b01 = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u);
        const uint32_t a23 = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u), b23 = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
        // tokens 4 g .. 4 g + 3 of the tile: piece 4 (g / 8) + 2 (g / 4 % 2) + g % 2, half g / 2 % 2 of it
        const int g = first_t / 4 + vgrp;
        const int p = 4 * (g >> 3) + 2 * ((g >> 2) & 1) + (g & 1), hf = (g >> 1) & 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t s01 = i < 2 ? a01 : b01, s23 = i < 2 ? a23 : b23;
          const uint32_t lo = i & 1 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s01, 1.0f, true))
                                    : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s01, 1.0f, false));
          const uint32_t hi = i & 1 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s23, 1.0f, true))
                                    : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s23, 1.0f, false));
          const int d = 4 * vcb + i;
          *reinterpret_cast<u32x2*>(&sm.v[buf][d][8 * piece<T>(d, p) + 4 * hf]) = (u32x2){mul2(lo, v01), mul2(hi, v23)};
        }
      }
    };
    // The scales of a whole tile, two tiles ahead (wave 0, a token per lane): E and K's multiplier.
    int run_e = -1000;
    float svr = 0.0f, kmax = 0.0f;
    int spage = 0;
    auto stat_page = [&](int t0) { return a.block_table[(int64_t)b * a.max_pages + (min(t0 + (lane & (T - 1)), a.max_tokens - 1) >> a.page_shift)]; };
    auto stat_load = [&](int t0, int page) {
      const int t = t0 + (lane & (T - 1)), en = entry_of(page, t);
      const bool there = en >= 0 && t < c1;
      const int64_t at64 = (int64_t)max(en, 0) * hk + h;
      svr = f16_lo(a.v_scales[at64]);
      kmax = 0.0f;
#pragma unroll
      for (int n = 0; n < NG; ++n) kmax = fmaxf(kmax, f16_lo(a.k_scales[at64 * NG + n]));
      svr = there ? fmaxf(svr, 0x1p-24f) : 0.0f;
      kmax = there ? kmax : 0.0f;
    };
    auto stat_write = [&](int n) {
      const float vm = max_across16(max_row16(svr)), km = max_across16(max_row16(kmax));
      if (vm > 0.0f) run_e = max(run_e, __builtin_amdgcn_frexp_expf(vm) - 6);
      const int gap = __ballot(svr == 0.0f) != 0;
      if (lane < T) sm.vs[n & 3][lane] = __builtin_ldexpf(svr, -run_e);
      if (lane == 0) {
        sm.kmul[n & 3] = km > 512.0f ? 0x1p-7f : 1.0f;
        sm.kback[n & 3] = km > 512.0f ? 0x1p7f : 1.0f;
        sm.e[n & 3] = run_e;
        sm.gap[n & 3] = gap;
      }
    };

    f32x16 o[NG];
    float m = kNegInf, l = 0.0f;
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[n][i] = 0.0f;

    __syncthreads();                                         // (LDS of the tile before is no longer read)
    const int wt = c0 + first_t;
    int page = page_of(wt + T);
    load(entry_of(page_of(wt), wt));
    if (wave == 0) {
      stat_load(c0, stat_page(c0));
      stat_write(0);
      stat_load(c0 + T, stat_page(c0 + T));
      stat_write(1);
      stat_load(c0 + 2 * T, stat_page(c0 + 2 * T));
      spage = stat_page(c0 + 3 * T);
    }
    __syncthreads();
    convert(0);
    load(entry_of(page, wt + T));
    page = page_of(wt + 2 * T);
    __syncthreads();
    int cur_e = sm.e[0];
    for (int base = c0, n = 0; base < c1; base += T, ++n) {
      const int buf = n & 1;
      const bool skip = live_rows <= 0 || (a.causal && base > last_p) || (a.window > 0 && base + T - 1 <= first_p - a.window);
      f32x16 s[NB];
      if (!skip) {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
#pragma unroll
          for (int i = 0; i < 16; ++i) s[k][i] = 0.0f;
#pragma unroll
          for (int c = 0; c < 2 * NG; ++c) {
            const f16x8 kf = *reinterpret_cast<const f16x8*>(&sm.k[buf][32 * k + c32][16 * c + 8 * half]);
            s[k] = mfma_f16_k16(kf, qf[c], s[k]);
          }
        }
      }
      if (base + T < c1) {                                   // the next tile: into the other buffer, and the one after that
        convert(n + 1);
        load(entry_of(page, wt + (n + 2) * T));
        page = page_of(wt + (n + 3) * T);
      }
      if (wave == 0) {
        stat_write(n + 2);
        stat_load(base + 3 * T, spage);
        spage = stat_page(base + 4 * T);
      }
      if (!skip) {
        const bool open = !__builtin_amdgcn_readfirstlane(sm.gap[n & 3]) && (!a.causal || base + T - 1 <= first_p) &&
                          (a.window <= 0 || base > last_p - a.window);
        const float cst = cs * sm.kback[n & 3];
        float mx = kNegInf;
        if (!open) {
#pragma unroll
          for (int k = 0; k < NB; ++k)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int tt = 32 * k + 8 * (i / 4) + 4 * half + (i & 3), t = base + tt;
              const bool see = sm.vs[n & 3][tt] > 0.0f && (!a.causal || t <= qpos) && (a.window <= 0 || t > qpos - a.window);
              s[k][i] = see ? s[k][i] : kNegInf;
            }
        }
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
          for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[k][i]);
        mx = across32(mx, false) * cst;
        const float mn = fmaxf(m, mx);
        const int e_new = sm.e[n & 3];
        const float ref = mn == kNegInf ? 0.0f : mn;
        if (__ballot(mn > m) || e_new != cur_e) {
          const float corr = __builtin_amdgcn_exp2f(m - ref);
          const float oc = __builtin_ldexpf(corr, cur_e - e_new);
          l *= corr;
#pragma unroll
          for (int d = 0; d < NG; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] *= oc;
          m = mn;
          cur_e = e_new;
        }
        f16x8 w[NB][2];
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k][i], cst, -ref));
            l += x;
            w[k][i / 8][i & 7] = (_Float16)x;
          }
#pragma unroll
        for (int d = 0; d < NG; ++d)
#pragma unroll
          for (int k = 0; k < NB; ++k)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const f16x8 vf = *reinterpret_cast<const f16x8*>(&sm.v[buf][32 * d + c32][8 * piece<T>(32 * d + c32, 4 * k + 2 * t + half)]);
              o[d] = mfma_f16_k16(vf, w[k][t], o[d]);
            }
      }
      __syncthreads();
    }

    // A lane has channels 32 d + 8 q + 4 half + 0..3 of its row.
    asm volatile("" : "+v"(c32), "+v"(half));
    const __amdgpu_buffer_rsrc_t rs = partial_rsrc(a.partials, a.partials_bytes);
    const bool split = ck.count > 1;
    auto part_row = [&](int c, int row) { return ((int64_t)(ck.slot(c) * hk + h) * kTileRows + 32 * wave + row) * (D + 4); };
    auto out_row = [&](int row) {                            // index of [token][query head]
      const int i = (r0 + row) / a.G;
      return (int64_t)(e.qs + i) * a.Hq + h * a.G + (r0 + row - i * a.G);
    };
    const float L = across32(l, true), back = __builtin_ldexpf(1.0f, cur_e);
    if (c32 < live_rows) {
      if (!split) {
        const float inv = L > 0.0f ? back / L : 0.0f;
        const int64_t row = out_row(c32);
#pragma unroll
        for (int d = 0; d < NG; ++d)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float v[4] = {o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
            store_out<4>(a.out + row * D + 32 * d + 8 * q + 4 * half, v, inv);
          }
        if (a.lse && half == 0) a.lse[row] = L > 0.0f ? (m + __builtin_amdgcn_logf(L)) * kLn2 : kNegInf;
      } else {
        const int64_t row = part_row(ck.mine, c32);
#pragma unroll
        for (int d = 0; d < NG; ++d)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float v[4] = {o[d][4 * q] * back, o[d][4 * q + 1] * back, o[d][4 * q + 2] * back, o[d][4 * q + 3] * back};
            store_run<4>(rs, row + 32 * d + 8 * q + 4 * half, v);
          }
        if (half == 0) {
          const float ml[2] = {m, L};
          store_run<2>(rs, row + D, ml);
        }
      }
    }
    if (split && live_rows > 0)
      join_chunks<D>(a, rs, sm.join[wave], lane, ck, live_rows, part_row, out_row, [&](int level, int c) {
        return level * a.level_counters + (ck.slot(c) * hk + h) * kTileWaves + wave;
      });
  }
}

template <int NG>
hipError_t launch_ng(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr int bytes = (int)sizeof(TileLds<NG>);
  static_assert(bytes <= 160 * 1024, "LDS");
  if (hipError_t e = set_lds_limit(reinterpret_cast<const void*>(kv_attention_tile_kernel<NG>), bytes, done); e != hipSuccess)
    return e;
  kv_attention_tile_kernel<NG><<<(int)p.grid, kTileWaves * 64, bytes, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_attention_tile(const KvAttnArgs& a, const KvAttnPlan& p, int D, hipStream_t st) {
  switch (D / 32) {
    case 1: return launch_ng<1>(a, p, st);
    case 2: return launch_ng<2>(a, p, st);
    case 3: return launch_ng<3>(a, p, st);
    case 4: return launch_ng<4>(a, p, st);
    case 6: return launch_ng<6>(a, p, st);
    default: return launch_ng<8>(a, p, st);
  }
}

}  // namespace qlq
