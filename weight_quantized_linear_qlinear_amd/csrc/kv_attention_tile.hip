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
// that this scale is at 2^5 .. 2^6 and V' below 2^15; fp16's smallest step is then 2^-29 of it.
//
// Bound by instruction issue: per 64 tokens a wave of 128-channel heads issues 32 products (32
// cycles each), 33 exponentials and about 280 other vector instructions (counted), and two waves
// share a SIMD; the matrix cores are busy 31 % of the time, LDS 25 %.  Measured (MI355X): two chunks of
// 1500 and 804 queries over 8192 and 4394 tokens, 32 heads over 8 of 128, 313 to 333 us (235 GFLOP,
// 730 TFLOP/s); a prompt of 512 tokens on its own 49 us, half of it storing and joining partial sums.
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

// Weights are 2^(x - m) of base-2 scores x, with m (the row's reference) kLift below the largest
// score when it is set and kept until a score passes it by kSlack: they stay below 2^15, fp16's 11
// bits reach down to 2^-21 of the largest, and o is hardly ever rescaled (following every new
// maximum of 32 rows takes 64 products per tile nearly every time).
constexpr float kLift = 7.0f, kSlack = 15.0f;

// A query tile's tokens: those that its rows can see.
struct Span {
  int i0, i1;                    // first and last query token
  int first;                     // the first token that a row sees
  int begin, end;                // tokens, begin a multiple of T
};

template <int T>
__device__ __forceinline__ Span span_of(const KvAttnArgs& a, const Extent& e, int qt) {
  Span s;
  s.i0 = qt * kTileRows / a.G;
  s.i1 = min(e.nq - 1, (qt * kTileRows + kTileRows - 1) / a.G);
  const int p0 = e.L - e.nq;
  s.end = min(max(a.causal ? p0 + s.i1 + 1 : e.L, 0), e.L);
  s.first = a.window > 0 ? min(max(0, p0 + s.i0 - a.window + 1), s.end) : 0;
  s.begin = s.first & ~(T - 1);
  return s;
}

template <int T>
__device__ __forceinline__ int units_of(const Span& s) { return max(1, (s.end - s.begin + T - 1) / T); }

__device__ __forceinline__ int tiles_of(const KvAttnArgs& a, const Extent& e) {
  return (e.nq * a.G + kTileRows - 1) / kTileRows;
}

// Calls visit(b, qt, units) for every query tile, 64 at a time in order (a tile per lane, units 0
// where there is none), until it returns false.
template <int T, class Visit>
__device__ __forceinline__ void walk_tiles(const KvAttnArgs& a, int lane, Visit visit) {
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int ends = wave_scan(b0 + lane < a.B ? tiles_of(a, extent_of(a, b0 + lane)) : 0);
    const int tiles = __builtin_amdgcn_readlane(ends, 63);
    int i = 0, start = 0;                                    // the sequence (b0 + i) that tile f0 belongs to, its first tile
    for (int f0 = 0; f0 < tiles; f0 += 64) {
      int mine = i, qt = f0 + lane - start;
      while (i < 63) {                                       // sequences that begin among these tiles
        const int next = __builtin_amdgcn_readlane(ends, i);
        if (next >= min(f0 + 64, tiles)) break;
        ++i;
        start = next;
        if (f0 + lane >= start) mine = i, qt = f0 + lane - start;
      }
      const bool valid = f0 + lane < tiles;
      const int b = valid ? b0 + mine : 0;
      const Extent e = extent_of(a, b);
      if (!visit(b, qt, valid ? units_of<T>(span_of<T>(a, e, qt)) : 0)) return;
    }
  }
}

constexpr int kAhead = 4;        // operands in flight from LDS before a product (2, 6 and 8 the same within 2 %)

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
  float vs[4][S::T];                             // V scales, 0 for a token that is not there
  uint32_t top[4][kTileWaves];                   // per wave's tokens: largest K scale (fp16 bits; bit 15: one is not there) and V scale
};

// Where piece p (8 tokens) of channel d lies in its row: p ^ swizzle(d), so that reads (16
// channels, one piece) spread over all banks and writes (4 channels apart) over half of them.
// It depends on d % 32 alone, so the reads of all 32-channel blocks share their addresses.
template <int T>
__device__ __forceinline__ int swizzle(int d) {
  if constexpr (T == 64) return ((d >> 1) & 7) ^ ((d >> 4) & 1);
  return ((d >> 2) & 3) ^ ((d >> 4) & 1);
}

// What a tile's values are scaled by, uniform for the workgroup.
struct TileScale {
  int e;                         // V' = V 2^-e
  bool big;                      // K' = K 2^-7
  bool gap;                      // a token is not there
};
constexpr int kNoScale = -1000;

// V's codes go to fp16 as 2^-8 of themselves (exact: 2^-17 is the smallest) and their scales as 2^(8 - E), so
// that a scale keeps its 11 bits down to 2^-27 of the largest.  (2^-19 with both as they are: beside a
// scale 2^24 times as large, which earlier rows of its query tile do not even see, 5 bits were left.)
constexpr int kCodeShift = 8;
constexpr float kCode = 0x1p-8f;

// N products that take one operand from LDS each, in exactly this order: AHEAD reads in front,
// then a product and the read of a later one in turn (left alone, the compiler reads each operand
// right before its product and waits for it).
template <int N, int AHEAD, class Read, class Product>
__device__ __forceinline__ void products(Read read, Product product) {
  f16x8 f[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) f[i] = read(i);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    product(i, f[i % AHEAD]);
    if (i + AHEAD < N) f[i % AHEAD] = read(i + AHEAD);
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <int NG>
__global__ __launch_bounds__(kTileWaves * 64) void kv_attention_tile_kernel(KvAttnArgs a) {
  typedef TileShape<NG> S;
  constexpr int D = S::D, T = S::T, TPW = T / kTileWaves, NB = T / 32, NL = TPW * D / 16;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  TileLds<NG>& sm = *reinterpret_cast<TileLds<NG>*>(smem_raw);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = a.Hk, h = blockIdx.x % hk, part = blockIdx.x / hk;    // a head's parts on one XCD where Hk is a multiple of 8
  const int page_mask = (1 << a.page_shift) - 1;
  const uint32_t row_bytes = (uint32_t)hk * D;

  int total = 0;
  walk_tiles<T>(a, lane, [&](int, int, int n) {
    total += wave_sum(n);
    return true;
  });
  total = __builtin_amdgcn_readfirstlane(total);
  const int U = max(1, (total + a.parts - 1) / a.parts), u_end = min(total, (part + 1) * U);

  for (int u = part * U; u < u_end;) {                       // uniform for the workgroup
    // the sequence and the tile that unit u belongs to, and the tile's first unit
    int b = -1, qt = 0, at = 0, before = 0;
    walk_tiles<T>(a, lane, [&](int tb, int tq, int n) {
      const int inc = before + wave_scan(n);
      const uint64_t hit = __ballot(u < inc && u >= inc - n);
      if (hit) {
        const int src = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
        b = __builtin_amdgcn_readlane(tb, src);
        qt = __builtin_amdgcn_readlane(tq, src);
        at = __builtin_amdgcn_readlane(inc - n, src);
      }
      before = __builtin_amdgcn_readlane(inc, 63);
      return hit == 0;
    });
    if (b < 0) break;                                        // (only if lengths change meanwhile or overflow the sum)
    Extent e = extent_of(a, b);
    e.qs = __builtin_amdgcn_readfirstlane(e.qs);
    e.nq = __builtin_amdgcn_readfirstlane(e.nq);
    e.L = __builtin_amdgcn_readfirstlane(e.L);
    const Span sp = span_of<T>(a, e, qt);
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
    const ConstInt* table = (const ConstInt*)(uintptr_t)(a.block_table + (int64_t)b * a.max_pages);
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
    TileScale next{kNoScale, false, false};
    auto load = [&](int entry) {
      const int64_t at64 = (int64_t)max(entry, 0) * hk + h;
      kraw = ld16(a.k_codes + at64 * D + koff);
      ksraw = a.k_scales[(at64 + (int64_t)krow * hk) * NG + kchunk / 2];
      const uint8_t* vp = a.v_codes + at64 * D + voff;
#pragma unroll
      for (int i = 0; i < 4; ++i) vraw[i] = *reinterpret_cast<const uint32_t*>(vp + (size_t)i * row_bytes);
    };
    // The loaded tile, number n, into LDS buffer n % 2.
    auto convert = [&](int n) {
      const int buf = n & 1;
      uint32_t top = sm.top[n & 3][lane & (kTileWaves - 1)];
      next.gap = __ballot((top & 0x8000u) != 0) != 0;
      top = row8(top & 0x7FFF7FFFu, MaxU16());
      top = __builtin_amdgcn_readfirstlane(top);
      next.big = (top & 0xFFFF) > 0x6000;
      const uint32_t vt = top >> 16;
      if (vt) next.e = max(next.e, (vt >= 0x400 ? (int)(vt >> 10) - 14 : 8 - __builtin_clz(vt)) - 6);
      const f16x2 s2 = __builtin_bit_cast(f16x2, (ksraw & 0xFFFF) | ksraw << 16);
      const uint32_t upper = next.big ? 0x48484848u : 0x64646464u;        // (the codes take the 2^-7: a small scale
      const float zero = next.big ? 9.0f : 1152.0f;                       // beside a big one keeps its bits)
      f32x4 vsc = *reinterpret_cast<const f32x4*>(&sm.vs[n & 3][first_t + 4 * vgrp]);
      if (lane < NL) {
        const uint32_t kd[4] = {kraw.x, kraw.y, kraw.z, kraw.w};
        u32x4 w[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t f = kd[i] ^ 0x80808080u;
          w[i / 2][2 * (i & 1)] = mul2(i8x2_to_f16<false>(f, upper, zero), s2);
          w[i / 2][2 * (i & 1) + 1] = mul2(i8x2_to_f16<true>(f, upper, zero), s2);
        }
        _Float16* kp = &sm.k[buf][first_t + krow][16 * kchunk];
        st16(kp, w[0]);
        st16(kp + 8, w[1]);
        // V: codes of a token that is not there may be NaN, so they go before the product
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = vsc[i] > 0.0f ? vraw[i] : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) vsc[i] = __builtin_ldexpf(vsc[i], kCodeShift - next.e);
        const f16x2 v01 = {(_Float16)vsc[0], (_Float16)vsc[1]}, v23 = {(_Float16)vsc[2], (_Float16)vsc[3]};
        const uint32_t a01 = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u), b01 = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u);
        const uint32_t a23 = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u), b23 = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
        // tokens 4 g .. 4 g + 3 of the tile: piece 4 (g / 8) + 2 (g / 4 % 2) + g % 2, half g / 2 % 2 of it
        const int g = first_t / 4 + vgrp;
        const int p = 4 * (g >> 3) + 2 * ((g >> 2) & 1) + (g & 1), hf = (g >> 1) & 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t s01 = i < 2 ? a01 : b01, s23 = i < 2 ? a23 : b23;
          const uint32_t lo = i & 1 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s01, kCode, true))
                                    : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s01, kCode, false));
          const uint32_t hi = i & 1 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s23, kCode, true))
                                    : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s23, kCode, false));
          const int d = 4 * vcb + i;
          *reinterpret_cast<u32x2*>(&sm.v[buf][d][8 * (p ^ swizzle<T>(d)) + 4 * hf]) = (u32x2){mul2(lo, v01), mul2(hi, v23)};
        }
      }
    };
    // The scales, two tiles ahead: lane l has token l % TPW of this wave's, K's block l / TPW.
    const int srow = lane & (TPW - 1), sblock = lane / TPW % NG;
    uint32_t svr, skr;
    int st_t, st_page;
    auto stat_load = [&](int t0, int page) {                 // t0: the wave's first token
      st_t = t0;
      st_page = page;
      const int64_t at64 = (int64_t)max(entry_of(page, t0), 0) * hk + (int64_t)srow * hk + h;
      svr = a.v_scales[at64];
      skr = a.k_scales[at64 * NG + sblock];
    };
    auto stat_write = [&](int n) {
      // (tokens before every row's window are left out like those of a bad page: their entries may hold anything)
      const bool there = entry_of(st_page, st_t) >= 0 && st_t + srow >= sp.first && st_t + srow < c1;
      const uint32_t kb = there ? skr & 0x7FFF : 0u, vb = there ? max(svr & 0x7FFF, 1u) : 0u;
      uint32_t top = across16(row16(kb | vb << 16, MaxU16()), MaxU16());
      if (__ballot(!there)) top |= 0x8000u;
      if (lane < TPW) sm.vs[n & 3][first_t + lane] = f16_lo(vb);
      if (lane == 0) sm.top[n & 3][wave] = top;
    };

    const int vswz = half ^ swizzle<T>(c32);                 // this lane's pieces: (4 k + 2 t) ^ vswz
    f32x16 o[NG];
    float m = kNegInf, l = 0.0f;
    int cur_e = kNoScale;                                    // E that o was computed with
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[n][i] = 0.0f;

    __syncthreads();                                         // (LDS of the tile before is no longer read)
    const int wt = c0 + first_t;
    int page = page_of(wt + T), page2 = page_of(wt + 2 * T);
    load(entry_of(page_of(wt), wt));
    stat_load(wt, page_of(wt));
    stat_write(0);
    stat_load(wt + T, page);
    stat_write(1);
    __syncthreads();
    convert(0);
    TileScale now = next;
    load(entry_of(page, wt + T));
    stat_load(wt + 2 * T, page2);
    page = page2;
    page2 = page_of(wt + 3 * T);
    __syncthreads();
    auto prepare = [&](int n) {                              // tile n's share of what tiles n + 1 .. n + 3 need
      if (c0 + (n + 1) * T < c1) {
        convert(n + 1);
        load(entry_of(page, wt + (n + 2) * T));
        stat_write(n + 2);
        stat_load(wt + (n + 3) * T, page2);
        page = page2;
        page2 = page_of(wt + (n + 4) * T);
      }
    };
    for (int base = c0, n = 0; base < c1; base += T, ++n) {
      const int buf = n & 1;
      const bool skip = live_rows <= 0 || (a.causal && base > last_p) || (a.window > 0 && base + T - 1 <= first_p - a.window);
      prepare(n);
      f32x16 s[NB];
      if (!skip) {
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[k][i] = 0.0f;
        const _Float16* kp = &sm.k[buf][c32][8 * half];
        products<2 * NG * NB, kAhead>(
            [&](int i) { return *reinterpret_cast<const f16x8*>(kp + 32 * S::KLD * (i % NB) + 16 * (i / NB)); },
            [&](int i, f16x8 kf) { s[i % NB] = mfma_f16_k16(kf, qf[i / NB], s[i % NB]); });
      }
      if (!skip) {
        const bool open = !now.gap && (!a.causal || base + T - 1 <= first_p) &&
                          (a.window <= 0 || base > last_p - a.window);
        const float cst = now.big ? cs * 0x1p7f : cs;
        const int t4 = base + 4 * half;
        if (!open) {
          if (now.gap) {
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
              for (int i = 0; i < 16; ++i)
                s[k][i] = sm.vs[n & 3][32 * k + 8 * (i / 4) + 4 * half + (i & 3)] > 0.0f ? s[k][i] : kNegInf;
          }
          const int64_t from = (int64_t)qpos - t4;             // (may be far below and above the tile)
          int hi = (int)max(min(from, (int64_t)T), (int64_t)-1), lo = (int)max(min(from - a.window, (int64_t)T), (int64_t)-1);
          asm volatile("" : "+v"(hi), "+v"(lo));             // (compared as 32 bits)
          if (a.causal) {
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
              for (int i = 0; i < 16; ++i) s[k][i] = 32 * k + 8 * (i / 4) + (i & 3) <= hi ? s[k][i] : kNegInf;
          }
          if (a.window > 0) {
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
              for (int i = 0; i < 16; ++i) s[k][i] = 32 * k + 8 * (i / 4) + (i & 3) > lo ? s[k][i] : kNegInf;
          }
        }
        float mx = kNegInf;
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
          for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[k][i]);
        mx = across32(mx, false) * cst;
        const int e_new = now.e;
        if (__ballot(mx > m + kSlack) || e_new != cur_e) {   // (m == -inf: mx > m)
          const float mn = fmaxf(m, mx - kLift);
          const float corr = mn == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
          const float oc = __builtin_ldexpf(corr, cur_e - e_new);
          l *= corr;
#pragma unroll
          for (int d = 0; d < NG; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] *= oc;
          m = mn;
          cur_e = e_new;
        }
        const float ref = m == kNegInf ? 0.0f : m;
        f16x8 w[NB][2];
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float x0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k][i], cst, -ref));
            const float x1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k][i + 1], cst, -ref));
            const f16x2 x = {(_Float16)x0, (_Float16)x1};
            l = __builtin_amdgcn_fdot2(x, (f16x2){(_Float16)1, (_Float16)1}, l, false);
            w[k][i / 8][i & 7] = x[0];
            w[k][i / 8][(i & 7) + 1] = x[1];
          }
        const _Float16* vrow = &sm.v[buf][c32][0];
        products<2 * NG * NB, kAhead>(
            [&](int i) {
              const int kt = i / NG, d = i % NG;              // 16 tokens, 32 channels
              return *reinterpret_cast<const f16x8*>(vrow + 32 * T * d + 8 * ((2 * kt) ^ vswz));
            },
            [&](int i, f16x8 vf) { o[i % NG] = mfma_f16_k16(vf, w[i / NG / 2][i / NG % 2], o[i % NG]); });
      }
      now = next;
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
        const float inv = L == 0.0f ? 0.0f : back / L;       // (NaN stays NaN)
        const int64_t row = out_row(c32);
#pragma unroll
        for (int d = 0; d < NG; ++d)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float v[4] = {o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
            store_out<4>(a.out + row * D + 32 * d + 8 * q + 4 * half, v, inv);
          }
        if (a.lse && half == 0) a.lse[row] = L == 0.0f ? kNegInf : (m + __builtin_amdgcn_logf(L)) * kLn2;
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
      join_chunks<D, true>(a, rs, sm.join[wave], lane, ck, live_rows, part_row, out_row, [&](int level, int c) {
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
