// Attention over the paged 4-bit KV cache (K and V e2m1 with an fp16 scale per 32 channels, rows in
// the order of kv_rows.h), for few query rows per KV head.  The definition, the cutting of the work
// and the joining are kv_attention.hip's; what differs is how a tile of 32 tokens is computed:
//   s_t = scale * sum_c k_scale[t,c] * (q_c . k_code[t,c])      (c: groups of 32 channels)
//   e_t = 2^(s_t log2e - m),  l = sum_t e_t,  o_c = sum_t fp16(e_t v_scale[t,c]) v_code[t,c],  out = o / l
// m is a running reference, 15 octaves below the largest s_t log2e + E_t seen, where 2^E_t bounds token
// t's V scales (the finite ones: a NaN stays in its own group): so every weight e_t v_scale fits fp16,
// has its 11 bits down to 2^-29 of the row's largest, and is rounded once.  Codes are exact in fp16, q is
// scaled per row by a power of two into [-1, 1) (as in kv_attention.hip); sums are fp32.
//
// Layout.  S^T = K Q^T: the lane of token l % 16 and channel group l / 16 has, in the cache's order, its
// eight channels of every group of 32 side by side: one load, and no byte moves before the conversion
// (two codes per instruction).  O^T = V^T P^T: lane column c has channels 2 c, 2 c + 1 of every group;
// nibbles of two tokens are put into one byte, which the conversion turns into the pair that the
// matrix unit wants.  Scales come one token per lane (K's in the lower, V's in the upper half of the
// wave) and reach the lanes of the scores through the wave's LDS, in the order of their tokens there.
//
// Bound by HBM and by instruction issue alike, two waves per SIMD: 64 tokens over up to 16384
// each, 32 heads over 8 of 128 (755 MB), 168 us, 4.5 TB/s; without the arithmetic about 155, with the arithmetic alone about
// as long.  A row is half a cache line at 128 channels, and the two heads that share one are read by two waves.
// Of the 239 registers (128 channels) the joining asks for the most, sixteen chunks' parts of two passes at a time:
// with one pass at a time the kernel has 145 (32 and 64 channels) to 160, and 237 and 275 of 192 and 256.
// One token over 131071, 28 heads over 4 of 128: 33 us, where the bytes take 15: four trips to memory to
// start, eight tiles one after another (1.3 us each) and three levels of joining.  A wave takes 16 rows; more rows are more tiles, which
// read K and V again, mostly from L2: with pairs of tiles per wave (32 rows, 252 registers) 16 sequences of
// 32 rows over 4000 tokens took 90 us, with single ones 54.
#include <type_traits>

#include "kv_attention.h"

namespace qlq {

using namespace attn;

namespace {

// The runs of groups of a 4-bit row: NG <= 8, no 5 or 7: at most two.
template <int NG>
struct Runs {
  static constexpr int P1 = NG >= 8 ? 8 : NG >= 4 ? 4 : NG >= 2 ? 2 : 1, P2 = NG - P1;
  static_assert(P2 == 0 || P2 == 1 || P2 == 2, "two runs of a power of two");
};

// Memory from p on, for loads at a lane's 32-bit offset plus a uniform one (no vector instructions for addresses).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t region(const uint8_t* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, -1, kBufferWord3);
}

// BYTES (1 .. 32, a power of two) there, aligned to 16 at the most, as dwords.
template <int BYTES>
struct Bytes {
  static constexpr int N = BYTES < 4 ? 1 : BYTES / 4;
  uint32_t d[N];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t lane, uint32_t at) {
    if constexpr (BYTES == 0) {
      d[0] = 0;
    } else if constexpr (BYTES == 1) {
      d[0] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rs, lane, at, 0);
    } else if constexpr (BYTES == 2) {
      d[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, lane, at, 0);
    } else if constexpr (BYTES == 4) {
      d[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, lane, at, 0);
    } else if constexpr (BYTES == 8) {
      const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, lane, at, 0));
      d[0] = v.x, d[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) {
        const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, lane + 16 * i, at, 0));
        d[4 * i] = v.x, d[4 * i + 1] = v.y, d[4 * i + 2] = v.z, d[4 * i + 3] = v.w;
      }
    }
  }
};

// Of two, neither a signalling NaN (fmaxf makes sure of that with an instruction each).
__device__ __forceinline__ float larger(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, __builtin_inff()); }

__device__ __forceinline__ float largest_across16(float v) {  // over lanes l, l ^ 16, l ^ 32, l ^ 48
  const int i = __builtin_bit_cast(int, v);
  const auto a = __builtin_amdgcn_permlane16_swap(i, i, false, false);
  const int x = (int)a[0], y = (int)a[1], j = __builtin_bit_cast(int, larger(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y)));
  const auto b = __builtin_amdgcn_permlane32_swap(j, j, false, false);
  const int z = (int)b[0], w = (int)b[1];
  return larger(__builtin_bit_cast(float, z), __builtin_bit_cast(float, w));
}

// fp16(v_i e_i) of eight, the products in fp32: one instruction each (the compiler's own choice takes three for
// two).  The wait states: the result of an exponential, which may be among e, and of a write of a high half are
// not there for the next instruction, and no vector instruction's for a matrix product within the next two (the
// compiler, which knows this rule, does not look into the block).
__device__ __forceinline__ f16x8 weigh(f16x8 v, const float (&e)[2][4]) {
  const u32x4 d = __builtin_bit_cast(u32x4, v);
  u32x4 w;
  uint32_t w0, w1, w2, w3;
  asm("s_nop 0\n\t"
      "v_fma_mixlo_f16 %0, %4, %8, 0 op_sel_hi:[1,0,0]\n\t"
      "v_fma_mixlo_f16 %1, %5, %10, 0 op_sel_hi:[1,0,0]\n\t"
      "v_fma_mixlo_f16 %2, %6, %12, 0 op_sel_hi:[1,0,0]\n\t"
      "v_fma_mixlo_f16 %3, %7, %14, 0 op_sel_hi:[1,0,0]\n\t"
      "v_fma_mixhi_f16 %0, %4, %9, 0 op_sel:[1,0,0] op_sel_hi:[1,0,0]\n\t"
      "v_fma_mixhi_f16 %1, %5, %11, 0 op_sel:[1,0,0] op_sel_hi:[1,0,0]\n\t"
      "v_fma_mixhi_f16 %2, %6, %13, 0 op_sel:[1,0,0] op_sel_hi:[1,0,0]\n\t"
      "v_fma_mixhi_f16 %3, %7, %15, 0 op_sel:[1,0,0] op_sel_hi:[1,0,0]\n\t"
      "s_nop 1"
      : "=&v"(w0), "=&v"(w1), "=&v"(w2), "=&v"(w3)
      : "v"(d.x), "v"(d.y), "v"(d.z), "v"(d.w), "v"(e[0][0]), "v"(e[0][1]), "v"(e[0][2]), "v"(e[0][3]), "v"(e[1][0]),
        "v"(e[1][1]), "v"(e[1][2]), "v"(e[1][3]));
  w = (u32x4){w0, w1, w2, w3};
  return __builtin_bit_cast(f16x8, w);
}

// Octaves from a row's reference up to its largest weight: 2^15 is the largest power of two in fp16.
constexpr float kLift = 15.0f;

// Waves per workgroup, one workgroup per CU.  Heads of 192 and 256 channels have 305 registers, the joining's among
// them, one wave per SIMD; held to 256 with eight waves, in us: 32 tokens over up to 9000 each 98 -> 89 and 126 -> 117, but 48 rows of
// 256 x 16 over 4000 55 -> 81, 24 rows over 20000 46 -> 61, 32 rows of 192 x 16 over 4000 56 -> 68.
constexpr int waves_of(int NG) { return NG <= 4 ? 8 : 4; }

// A wave's LDS: the token scales of its tile, in the order in which lanes hold the tokens (lane group
// g: 4 g .. 4 g + 3, then 16 more), or what joining needs.
template <int NG>
union WaveLds {
  struct {
    uint16_t s[2][NG][32];       // K, V scales (fp16) by group
    float ev[32];                // exponents that bound the V scales
  };
  JoinLds join;
};

template <int NG>
__global__ __launch_bounds__(waves_of(NG) * 64) void kv4_attention_kernel(KvAttnArgs a) {
  constexpr int D = 32 * NG, TR = 16, kWaves = waves_of(NG), P1 = Runs<NG>::P1, P2 = Runs<NG>::P2;
  constexpr bool kTwo = P2 > 0;
  __shared__ __align__(16) WaveLds<NG> lds[kWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  WaveLds<NG>& mine = lds[wave];
  // A head's units are cut over `waves` waves.  A workgroup's waves are on HW neighbouring KV heads, or all
  // on one; the workgroups on one stretch of the heads' lines sit on one XCD (workgroup b goes to XCD b % 8).
  const Extent mine_e = lane < a.B ? extent_of(a, lane) : Extent{};
  const int total = total_units<TR>(a, mine_e, lane), waves = a.parts * (kWaves >> a.hw_shift);
  const int U = max(1, (total + waves - 1) / waves);
  const int hw_shift = U > a.together ? a.hw_shift : 0, HW = 1 << hw_shift, HG = a.Hk >> hw_shift;
  const int parts = a.parts >> (a.hw_shift - hw_shift), TS = kWaves >> hw_shift;
  int part = blockIdx.x / HG, hg = blockIdx.x % HG;
  if (parts % 8 == 0) {
    const int li = blockIdx.x >> 3;
    part = (li / HG) * 8 + (blockIdx.x & 7);
    hg = li % HG;
  }
  const int h = hg * HW + (wave & (HW - 1)), me = part * TS + (wave >> hw_shift);     // head, place on its line
  const int u_end = min(total, (me + 1) * U);
  for (int u = me * U; u < u_end;) {
    const Tile it = tile_of<TR>(a, mine_e, u, lane);
    if (it.units == 0) break;                                  // (only if lengths change meanwhile or overflow the sum)
    const int u_next = min(u_end, it.begin + it.units);
    const int wf = it.begin / U;                               // this tile's chunks: one per wave that its units reach
    const Chunks ck{wf, (it.begin + it.units - 1) / U - wf + 1, me - wf};
    const int nq = it.e.nq, L = it.e.L, r0 = it.qt * TR, rows = nq * a.G;
    const int i0 = r0 / a.G, i1 = min(nq - 1, (r0 + TR - 1) / a.G);
    const int p0 = L - nq;                                     // position of query 0
    const int tend = min(max(a.causal ? p0 + i1 + 1 : L, 0), L);
    const int tmin = a.window > 0 ? min(max(0, p0 + i0 - a.window + 1), tend) : 0;      // the first token that a row sees
    const int tbeg = tmin & ~31;
    const int begin = begin_of(a, it.e);
    const int c0 = max(tbeg, begin + 32 * (u - it.begin));     // a multiple of 32
    const int c1 = min(tend, begin + 32 * (u_next - it.begin));
    u = u_next;

    int c16 = lane & 15, g4 = lane >> 4;
    asm volatile("" : "+v"(c16), "+v"(g4));                    // (nothing computed from them outlives a tile)

    // q's rows (packed: query token, then head of the group), channels 32 n + 8 g4 .. + 7.
    u32x4 qraw[NG];
    int qpos;
    {
      const int row = r0 + c16;
      const bool live = row < rows;
      const int i = live ? row / a.G : i0, g = live ? row - i * a.G : 0;
      qpos = live ? p0 + i : -1;
      const uint16_t* qp = a.q + (int64_t)(it.e.qs + i) * a.q_stride + (int64_t)(h * a.G + g) * D + 8 * g4;
#pragma unroll
      for (int n = 0; n < NG; ++n) qraw[n] = ld16(qp + 32 * n);
    }

    f32x4 o[NG][2];                                            // [group][channel of the pair]: channels 2 (4 g4 + j) + 0, 1 of it
    float m = kNegInf, l = 0.0f;
#pragma unroll
    for (int n = 0; n < NG; ++n) o[n][0] = o[n][1] = (f32x4){0.f, 0.f, 0.f, 0.f};

    // Tiles start at multiples of 32 tokens and pages hold 16 or more, so each half of a tile lies in
    // one page, whose first entry is uniform.  -1: the page is outside the pool (its tokens are left out).
    const int hk = a.Hk, page_mask = (1 << a.page_shift) - 1;
    const ConstInt* table = (const ConstInt*)(uintptr_t)(a.block_table + (int64_t)it.b * a.max_pages);
    auto page_of = [&](int t) { return table[min(t, a.max_tokens - 1) >> a.page_shift]; };
    auto entry_of = [&](int page, int t) {
      return page >= 0 && page < a.pages ? (page << a.page_shift) + (t & page_mask) : -1;
    };
    const uint32_t row_bytes = (uint32_t)hk * (D / 2);         // from one token to the next
    const uint32_t koff = c16 * row_bytes + 4 * P1 * g4, koff2 = c16 * row_bytes + 16 * P1 + 4 * P2 * g4;
    const uint32_t voff = 4 * g4 * row_bytes + P1 * c16, voff2 = 4 * g4 * row_bytes + 16 * P1 + P2 * c16;

    Bytes<4 * P1> k1[2];
    Bytes<4 * P2> k2[2];
    Bytes<P1> v1[8];
    Bytes<P2> v2[8];
    KScales<NG> sc;                                            // lanes 0 .. 31: K scales of token lane, 32 .. 63: V's
    const uint64_t sbase = (uint64_t)(uintptr_t)((lane < 32 ? a.k_scales : a.v_scales) + ((int64_t)c16 * hk + h) * NG);
    const uint32_t sstep = (uint32_t)hk * NG * 2;
    auto load_k = [&](int e0, int e1) {                        // and the scales
      const int f0 = max(e0, 0), f1 = max(e1, 0);
      sc.load(reinterpret_cast<const uint16_t*>(sbase + (uint64_t)(uint32_t)(lane & 16 ? f1 : f0) * sstep));
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const __amdgpu_buffer_rsrc_t rs = region(a.k_codes + ((int64_t)(u ? f1 : f0) * hk + h) * (D / 2));
        k1[u].load(rs, koff, 0);
        if constexpr (kTwo) k2[u].load(rs, koff2, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto load_v = [&](int e0, int e1) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const __amdgpu_buffer_rsrc_t rs = region(a.v_codes + ((int64_t)max(u ? e1 : e0, 0) * hk + h) * (D / 2));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v1[4 * u + j].load(rs, voff, j * row_bytes);
          if constexpr (kTwo) v2[4 * u + j].load(rs, voff2, j * row_bytes);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    int e0 = entry_of(page_of(c0), c0), e1 = entry_of(page_of(c0 + 16), c0 + 16);   // of the tile's halves
    int g0 = page_of(c0 + 32), g1 = page_of(c0 + 48);          // the next tile's pages
    load_k(e0, e1);
    load_v(e0, e1);

    // q: per query row a power of two into [-1, 1), fp16; rows past the last are zero.
    f16x8 qf[NG];
    float cs;
    {
      const bool live = r0 + c16 < rows;
      float f[NG][8], am = 0.0f;
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const uint32_t d[4] = {qraw[n].x, qraw[n].y, qraw[n].z, qraw[n].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[n][2 * e] = live ? bf16_bits_to_f32(d[e] & 0xFFFF) : 0.0f;
          f[n][2 * e + 1] = live ? bf16_bits_to_f32(d[e] >> 16) : 0.0f;
          am = fmaxf(am, fmaxf(fabsf(f[n][2 * e]), fabsf(f[n][2 * e + 1])));
        }
      }
      am = max_across16(am);
      const int ex = am > 0.0f ? __builtin_amdgcn_frexp_expf(am) : 0;   // am < 2^ex
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e) qf[n][e] = (_Float16)__builtin_ldexpf(f[n][e], -ex);
      cs = __builtin_ldexpf(a.scale * kLog2e, ex);
    }

    const int spos = ((lane >> 2) & 3) * 8 + ((lane >> 4) & 1) * 4 + (lane & 3);   // token lane % 32 in the order of the scores
    uint16_t* sput = &mine.s[lane >> 5][0][spos];
    for (int base = c0; base < c1; base += 32) {
      // (tokens before every row's window, behind the last and on pages outside the pool: scales 0)
      const bool all_valid = e0 >= 0 && e1 >= 0 && base + 32 <= c1 && base >= tmin;
      const int n0 = entry_of(g0, base + 32), n1 = entry_of(g1, base + 48);
      const int t0 = base + 4 * g4;                            // this lane's first token (u = j = 0)
      auto there = [&](int u, int j) {
        const int t = t0 + 16 * u + j;
        return (u ? e1 : e0) >= 0 && t < c1 && t >= tmin;
      };
      bool bad;                                                // a scale of the tile is NaN or infinite
      {
        const int t = base + (lane & 31);
        const bool in = all_valid || ((lane & 16 ? e1 : e0) >= 0 && t < c1 && t >= tmin);
        uint32_t top = 0;
#pragma unroll
        for (int n = 0; n < KScales<NG>::N; ++n) {
          const uint32_t d = in ? sc.d[n] & 0x7FFF7FFFu : 0u;
          top = max(top, max(d & 0xFFFFu, d >> 16));
          sput[64 * n] = (uint16_t)d;                          // (group 2 n)
          if (2 * n + 1 < NG) sput[64 * n + 32] = (uint16_t)(d >> 16);
        }
        bad = __ballot(top >= 0x7C00u) != 0;                   // a NaN or an infinity: it bounds nothing
        if (bad) {
          auto finite = [](uint32_t s) { return s < 0x7C00u ? s : 0u; };
          top = 0;
#pragma unroll
          for (int n = 0; n < KScales<NG>::N; ++n) {
            const uint32_t d = in ? sc.d[n] & 0x7FFF7FFFu : 0u;
            top = max(top, max(finite(d & 0xFFFFu), finite(d >> 16)));
          }
        }
        // 2^E >= the largest finite scale: its exponent + 1 (a zero counts as the smallest scale)
        const float f = fmaxf(f16_lo(top), 0x1p-24f);
        if (lane >= 32) mine.ev[spos] = (float)__builtin_amdgcn_frexp_expf(f);
      }
      wave_sync();

      // S^T: tokens 16 u + 4 g4 + j, query c16
      float s[2][4];
      f16x8 ks[NG];
#pragma unroll
      for (int n = 0; n < NG; ++n) ks[n] = __builtin_bit_cast(f16x8, ld16(&mine.s[0][n][8 * g4]));
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          u32x4 kw;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = n < P1 ? i * P1 + n : i * P2 + n - P1;
            kw[i] = n < P1 ? e2m1x2_to_f16(k1[u].d[(n < P1 ? at : 0) / 4], at % 4)
                           : e2m1x2_to_f16(k2[u].d[(n < P1 ? 0 : at) / 4], at % 4);
          }
          const f32x4 d = mfma_f16_k32(__builtin_bit_cast(f16x8, kw), qf[n], (f32x4){0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int j = 0; j < 4; ++j) s[u][j] = __builtin_fmaf((float)ks[n][4 * u + j], d[j], n == 0 ? 0.0f : s[u][j]);
        }
      }
      float ev[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) *reinterpret_cast<f32x4*>(ev[u]) = *reinterpret_cast<const f32x4*>(&mine.ev[8 * g4 + 4 * u]);
      load_k(n0, n1);
      g0 = page_of(base + 64);
      g1 = page_of(base + 80);

      // whole tile visible to every row?
      const bool open = all_valid && (!a.causal || base + 31 <= p0 + i0) && (a.window <= 0 || base > p0 + i1 - a.window);
      float e[2][4];
      float mx = kNegInf, f = cs;                              // scores are s f
      if (!open) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int t = t0 + 16 * u + j;
            const bool see = there(u, j) && (!a.causal || t <= qpos) && (a.window <= 0 || t > qpos - a.window);
            s[u][j] = see ? s[u][j] * f : kNegInf;
          }
        f = 1.0f;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) mx = larger(mx, __builtin_fmaf(s[u][j], f, ev[u][j]));
      mx = largest_across16(mx);
      const float mn = larger(m, mx - kLift);
      const float ref = mn == kNegInf ? 0.0f : mn;
      if (__ballot(mn > m)) {
        const float corr = __builtin_amdgcn_exp2f(m - ref);
        l *= corr;
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[n][0][j] *= corr, o[n][1][j] *= corr;
        m = mn;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e[u][j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][j], f, -ref));
          l += e[u][j];
        }

      // V scales that are NaN or infinite go to the rows that see their tokens and to no others (0 NaN is NaN): as NaN
      // into the sums of those rows' groups, and 0 takes their place.
      if (__builtin_expect(bad, 0)) {
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          u32x4 v = ld16(&mine.s[1][n][8 * g4]);
          int hit = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if ((v[i / 2] >> (16 * (i & 1)) & 0xFFFFu) < 0x7C00u) continue;
            v[i / 2] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
            hit |= s[i / 4][i & 3] != kNegInf;
          }
          wave_sync();                                         // (the 16 lanes of a lane group write the same)
          st16(&mine.s[1][n][8 * g4], v);
          if (across16(hit, OrI()) != 0)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][0][j] = o[n][1][j] = __builtin_nanf("");
        }
        wave_sync();
      }

      // O^T: per group, the weights times their V scales, and the channel pairs' two rows of V^T
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const f16x8 vs = __builtin_bit_cast(f16x8, ld16(&mine.s[1][n][8 * g4]));
        const f16x8 w = weigh(vs, e);
        const int b = n < P1 ? n : n - P1;                     // byte of the lane's run
        u32x4 lo, hi;                                          // channels 2 c16 and 2 c16 + 1: tokens 2 i, 2 i + 1
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = n < P1 ? v1[2 * i].d[b / 4] : v2[2 * i].d[0], y = n < P1 ? v1[2 * i + 1].d[b / 4] : v2[2 * i + 1].d[0];
          const uint32_t even = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), odd = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
          lo[i] = e2m1x2_to_f16(even, b % 4);
          hi[i] = e2m1x2_to_f16(odd, b % 4);
        }
        o[n][0] = mfma_f16_k32(__builtin_bit_cast(f16x8, lo), w, o[n][0]);
        o[n][1] = mfma_f16_k32(__builtin_bit_cast(f16x8, hi), w, o[n][1]);
      }
      load_v(n0, n1);
      e0 = n0;
      e1 = n1;
    }

    // A lane has channels 32 n + 8 g4 .. + 7 of its row.
    asm volatile("" : "+v"(c16), "+v"(g4));
    const bool split = ck.count > 1;
    const __amdgpu_buffer_rsrc_t rs = partial_rsrc(a.partials, a.partials_bytes);
    auto part_row = [&](int c, int row) { return (int64_t)((ck.slot(c) * hk + h) * a.tile_rows + row) * (D + 4); };
    auto out_row = [&](int grow) {                             // index of [token][query head]
      const int i = grow / a.G;
      return (int64_t)(it.e.qs + i) * a.Hq + h * a.G + (grow - i * a.G);
    };
    const float Lsum = sum_across16(l);                    // over the lane groups of a query
    if (r0 + c16 < rows) {
      const int64_t at = split ? part_row(ck.mine, c16) : out_row(r0 + c16);
      const float inv = Lsum == 0.0f ? 0.0f : 1.0f / Lsum;     // (NaN stays NaN)
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[2 * j] = o[n][0][j], v[2 * j + 1] = o[n][1][j];
        if (split) store_run<8>(rs, at + 32 * n + 8 * g4, v);
        else store_out<8>(a.out + at * D + 32 * n + 8 * g4, v, inv);
      }
      if (g4 == 0) {
        if (split) {
          const float ml[2] = {m, Lsum};
          store_run<2>(rs, at + D, ml);
        } else if (a.lse) {
          a.lse[at] = Lsum == 0.0f ? kNegInf : (m + __builtin_amdgcn_logf(Lsum)) * kLn2;
        }
      }
    }
    if (!split) continue;
    join_chunks<D, (NG >= 4)>(a, rs, mine.join, lane, ck, min(TR, rows - r0), part_row,
                              [&](int row) { return out_row(r0 + row); },
                              [&](int level, int c) { return level * a.level_counters + ck.slot(c) * hk + h; });
  }
}

template <int NG>
hipError_t launch_ng(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t st) {
  kv4_attention_kernel<NG><<<(int)p.grid, waves_of(NG) * 64, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

KvAttnPlan plan_kv4_attention(int64_t T, int64_t B, int64_t Hk, int64_t G, int64_t D, bool one_each) {
  KvAttnPlan p;
  const int64_t rows = one_each ? G : (T + B - 1) / B * G;   // query rows of an average sequence
  const int NG = (int)(D / 32);
  // From here on the many-row kernel.  16 sequences over 4000 tokens, then 64, kernel alone, in us, this one and that one:
  //   96 (16 heads over 4)   64 rows 44 and 64, 124 and 139; 80 rows 50 and 64, 148 and 140; 96 rows 56 and 65, 174 and 145
  //   128 (32 over 8)        64 rows 79 and 94, 211 and 294; 80 rows 87 and 97, 375 and 296; 96 rows 99 and 100, 370 and 299
  //   192 (32 over 8)        80 rows 161 and 174, 667 and 521; 96 rows 181 and 179, 654 and 528
  //   64 (32 over 8)         96 rows 72 and 81, 243 and 262; 128 rows 90 and 84, 299 and 264
  //   256 (16 over 2; that one spills)  256 rows 155 and 223, 526 and 538; 512 rows 261 and 288, 1013 and 853
  // The border of 96, 128 and 192 is the large calls'; small ones lose up to a third between 64 and 96 rows (8 heads over 2
  // of 192, 16 x 80 rows 56 and 81).
  if (rows > (NG <= 2 ? 96 : NG == 8 ? 256 : 64)) return plan_kv_attention(T, B, Hk, G, D, one_each);
  constexpr int64_t TR = 16;
  // Heads per workgroup.  Four that share cache lines, where every wave has more than ten tiles to take; else one, whose
  // chunks then sit close together.  Four and one, in us: 32 heads over 8 of 128, 64 tokens over 4000 each 82 and 96, over
  // 30000 x 4 46 and 53, over 131071 49 and 55, over 30000 23.0 and 21.6, over 8000 19.0 and 16.6; 16 of 64, 4 over
  // 30000 57 and 69, 1 over 8000 16.6 and 15.8; several tiles of rows, 24 rows over 20000 39 and 34 (32 over 8 of 128),
  // 25.7 and 22.1 (16 over 4 of 64).  A row of 256 channels is a line: one (1 over 8000 27 and 25).  Eight
  // heads instead of four: within 2 %, several rows 20 % slower.
  while ((2 << p.hw_shift) <= 4 && Hk % (2 << p.hw_shift) == 0) ++p.hw_shift;
  const int64_t HG = Hk >> p.hw_shift;
  const int64_t parts = 256 / HG;                              // one workgroup per CU
  p.parts = (int)(parts >= 8 ? parts / 8 * 8 : parts < 1 ? 1 : parts);
  p.together = NG == 8 || rows > TR ? 1 << 30 : 10;
  if (p.parts % (1 << p.hw_shift) != 0) p.together = 0;        // (many heads, few workgroups for each: no other cut)
  p.grid = p.parts * HG;
  p.waves = p.parts * (waves_of(NG) >> p.hw_shift);
  p.tile_rows = (int)(one_each && G < TR ? G : TR);
  p.counters = 2 * p.waves * Hk;
  p.tiles = one_each ? B * ((G + TR - 1) / TR) : T * G / TR + B;
  return p;
}

hipError_t launch_kv4_attention(const KvAttnArgs& a, const KvAttnPlan& p, int D, hipStream_t st) {
  if (p.R == 16) return launch_kv4_attention_tile(a, p, D, st);
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
