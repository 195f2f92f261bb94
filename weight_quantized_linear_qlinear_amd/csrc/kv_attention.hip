// Attention over the paged 8-bit KV cache (K int8 with an fp16 scale per 32 channels, V e4m3
// with one per (token, head)), for one query token per sequence or many.
//
// For a query row (token i of sequence b, head g of the KV head's group) at position
// p = L - nq + i, over the cached tokens t that the masks leave:
//   s_t = scale * sum_c k_scale[t,c] * (q_c . k_code[t,c])      (c: groups of 32 channels)
//   o   = sum_t 2^(s_t log2e) v_scale_t v_code_t / sum_t 2^(s_t log2e)
// in one pass with a running reference m and sum l.  v_scale_t is taken into the exponent:
//   x_t = s_t log2e + log2 v_scale_t,  m = max x_t - 15,  w_t = 2^(x_t - m) in [0, 2^15],
//   o = sum w_t v_code_t,  l = sum w_t / v_scale_t,
// so that the weights fit fp16 whatever the scales are.  Products run on the matrix cores in
// fp16 with fp32 accumulation: int8 and e4m3 codes are exact in fp16, q is scaled per row by a
// power of two into [-1, 1) (exact but for channels 2^-14 and more below the row's largest,
// whose absolute error stays under 2^-25 of it), and the weights' rounding to fp16 is the
// only other one: 2^-11 of a weight down to 2^-29 of the row's largest, below that 2^-40 of the
// largest (l adds the weights before it; the output's own rounding to bf16 is 2^-8).  With the
// largest weight 1 instead, many small ones beside a large one are lost: 31 of them 25 octaves down
// altogether, a long tail of 131071 to 0.3 % of the output.
//
// Layout.  A wave takes one KV head, 16 R query rows (nq x G rows packed, so that the heads of
// a group share every K and V load) and a run of tokens, 32 at a time, on its own; the waves of
// a workgroup take neighbouring heads, whose entries lie side by side.  S^T = K Q^T (tokens are
// the rows): lane l holds query l % 16 and tokens 4 (l / 16) + j, which is the operand that
// O^T = V^T P^T wants, so the weights never cross lanes.  V^T needs, per lane, one channel of
// eight tokens: each lane loads the same few channels of its eight tokens and transposes bytes
// pairwise while converting.
//
// Work is cut on the device, from the lengths it finds there (the host knows none of them and
// waits for nothing): every wave sums the sequences' tiles of 32 tokens and takes an equal run
// of them, so that ragged batches load the chip evenly.  Tiles that several waves share are
// joined by the last to finish, in the order of the chunks.
//
// Bound by HBM: a token is 266 bytes per KV head of 128, and 512 operations per query row that
// shares them.  Measured (MI355X): 64 sequences of 2048 to 8192 tokens, 8 KV heads
// of 128, 126 us (699 MB, 5.6 TB/s); one of 131071 over 4 KV heads 40 us (139 MB; 16 us of it
// join 256 chunks per head); 16 x 5 tokens, window 1024, 16 heads of 64 17.5 us (latency).
#include <type_traits>

#include "kv_attention.h"

namespace qlq {

using namespace attn;

namespace {

template <bool NT, class T>
__device__ __forceinline__ T ld(const T* p) {
  if constexpr (NT) return __builtin_nontemporal_load(p);
  return *p;
}

// BYTES (2, 4, 8 or 16) at p, aligned to BYTES, as dwords (2 bytes: the low half).
template <int BYTES, bool NT = false>
struct Raw {
  static constexpr int N = BYTES < 4 ? 1 : BYTES / 4;
  uint32_t d[N];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (BYTES == 2) {
      d[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (BYTES == 4) {
      d[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (BYTES == 8) {
      const u32x2 v = ld<NT>(reinterpret_cast<const u32x2*>(p));
      d[0] = v.x, d[1] = v.y;
    } else {
      const u32x4 v = ld<NT>(reinterpret_cast<const u32x4*>(p));
      d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = 0u;
  }
};

// A V piece covers 32 P channels (P a power of two): lane column c holds channels 2 P c ..
// 2 P c + 2 P - 1 of the piece.  NG groups of 32 channels are cut into the powers of two of NG.
template <int NG>
struct Pieces {
  static constexpr int P = NG >= 8 ? 8 : NG >= 4 ? 4 : NG >= 2 ? 2 : 1;   // the largest first
  static constexpr int Rest = NG - P;
};

// Products of one piece: o[n][r] += V^T[channel 2 P c + n][8 tokens] P^T[8 tokens][query].
template <int P, int R, bool NT>
__device__ __forceinline__ void pv_piece(const Raw<2 * P, NT> (&v)[8], const f16x8 (&w)[R], f32x4 (*o)[R]) {
  constexpr int DW = Raw<2 * P>::N;
#pragma unroll
  for (int d = 0; d < DW; ++d) {
    // byte pairs (token 2 i, token 2 i + 1) of channels 0, 1 and 2, 3 of this dword
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __builtin_amdgcn_perm(v[2 * i + 1].d[d], v[2 * i].d[d], 0x05010400u);
      if constexpr (P > 1) hi[i] = __builtin_amdgcn_perm(v[2 * i + 1].d[d], v[2 * i].d[d], 0x07030602u);
    }
#pragma unroll
    for (int n = 0; n < (P > 1 ? 4 : 2); ++n) {
      const uint32_t* s = n < 2 ? lo : hi;
      u32x4 a;
      if (n & 1) a = (u32x4){e4m3x2_to_f16<true>(s[0]), e4m3x2_to_f16<true>(s[1]), e4m3x2_to_f16<true>(s[2]), e4m3x2_to_f16<true>(s[3])};
      else a = (u32x4){e4m3x2_to_f16<false>(s[0]), e4m3x2_to_f16<false>(s[1]), e4m3x2_to_f16<false>(s[2]), e4m3x2_to_f16<false>(s[3])};
      const f16x8 av = __builtin_bit_cast(f16x8, a);
#pragma unroll
      for (int r = 0; r < R; ++r) o[4 * d + n][r] = mfma_f16_k32(av, w[r], o[4 * d + n][r]);
    }
  }
}

// Octaves from a row's reference up to its largest weight: 2^15 is the largest power of two in fp16.
constexpr float kLift = 15.0f;

// The first token that any query of the sequence can see (rounded down to a tile of 32), and
// the tiles of 32 from there.
__device__ __forceinline__ int begin_of(const KvAttnArgs& a, const Extent& e) {
  return a.window > 0 ? min(max(0, e.L - e.nq - a.window + 1), e.L) & ~31 : 0;
}
__device__ __forceinline__ int units_of(const KvAttnArgs& a, const Extent& e) {
  return max(1, (e.L - begin_of(a, e) + 31) >> 5);
}

// The work of one KV head is a line of units (32 tokens of one query tile), tile after tile;
// wave w of its waves takes units w U .. (w + 1) U - 1, whatever tiles they belong to.
// `mine` is the extent of sequence `lane` (nq 0 past the last), kept for the first 64.
template <int TR>
__device__ __forceinline__ int total_units(const KvAttnArgs& a, const Extent& mine, int lane) {
  int total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    Extent e = mine;
    if (b0) e = b0 + lane < a.B ? extent_of(a, b0 + lane) : Extent{};
    total += wave_sum((e.nq * a.G + TR - 1) / TR * units_of(a, e));
  }
  return __builtin_amdgcn_readfirstlane(total);
}

struct Tile {
  Extent e;
  int b, qt;                     // sequence, query tile
  int begin, units;              // its place on the line
};

// The tile that unit u belongs to (0 <= u < total): every wave on its own, 64 sequences at a time.
template <int TR>
__device__ __forceinline__ Tile tile_of(const KvAttnArgs& a, const Extent& mine, int u, int lane) {
  Tile t{};
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    Extent e = mine;
    if (b0) e = b0 + lane < a.B ? extent_of(a, b0 + lane) : Extent{};
    const int n = (e.nq * a.G + TR - 1) / TR * units_of(a, e);
    const int inc = before + wave_scan(n);
    const uint64_t hit = __ballot(u < inc && u >= inc - n);
    if (hit) {
      const int src = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
      auto of = [&](int v) { return __builtin_amdgcn_readlane(v, src); };
      t.e.qs = of(e.qs);
      t.e.nq = of(e.nq);
      t.e.L = of(e.L);
      t.b = b0 + src;
      t.units = units_of(a, t.e);
      const int begin = of(inc - n);
      t.qt = (u - begin) / t.units;
      t.begin = begin + t.qt * t.units;
      return t;
    }
    before = __builtin_amdgcn_readlane(inc, 63);
  }
  return t;
}

// Waves per workgroup (one workgroup per CU).  Heads of 32 and 64 leave registers for two waves per
// SIMD, which their short rows need: 32 sequences of 16000 tokens, 4 heads of 64, 62 us against 74,
// 16 x 5 tokens in a window of 1024, 16 heads of 64, 18.1 against 20.2; from 96 on eight waves are
// slower (8 heads of 96 67 against 64, 4 of 128 42 against 39).
constexpr int waves_of(int NG) { return NG <= 2 ? 8 : 4; }

// Whether 17 to 32 rows go as one tile of two subtiles or as two tiles that read K and V each: 16
// sequences of 24 rows over 4000 and 16000 tokens take 69 and 160 us against 74 and 199 for heads
// of 128, but 112 and 231 against 75 and 138 for heads of 256 (registers), 94 and 163 against 62
// and 149 of 192, 55 and 98 against 37 and 111 of 64 (twice the waves).
constexpr bool pairs_rows(int NG) { return NG == 3 || NG == 4; }

// A wave's LDS: the token scales of its tile, or what joining needs.
template <int NG>
union WaveLds {
  struct {
    float ks[NG][32];            // K scales by group and token
    float lv[32], rv[32];        // log2 and reciprocal of the V scales
  };
  JoinLds join;
};

template <int NG, int R>
__global__ __launch_bounds__(waves_of(NG) * 64) void kv_attention_kernel(KvAttnArgs a) {
  constexpr int D = 32 * NG, TR = 16 * R, kWaves = waves_of(NG);
  // Codes are read once per 16 R rows: streamed past the caches where a head's row fills whole
  // cache lines (128 bytes); shorter ones share lines between waves.
  constexpr bool NT = R == 1 && NG % 4 == 0;
  __shared__ __align__(16) WaveLds<NG> lds[kWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  WaveLds<NG>& mine = lds[wave];
  // HW neighbouring KV heads per workgroup, one per wave (a token's entries of all heads lie
  // side by side, and reading them together is what HBM rewards), and kWaves / HW waves on a
  // head's line.  The head groups of one part sit on one XCD (workgroup b goes to XCD b % 8),
  // whose L2 they share for the scales.
  const int HW = 1 << a.hw_shift, HG = a.Hk >> a.hw_shift, TS = kWaves >> a.hw_shift;
  int part = blockIdx.x / HG, hg = blockIdx.x % HG;
  if (a.parts % 8 == 0) {
    const int li = blockIdx.x >> 3;
    part = (li / HG) * 8 + (blockIdx.x & 7);
    hg = li % HG;
  }
  const int h = hg * HW + (wave & (HW - 1)), me = part * TS + (wave >> a.hw_shift);   // head, place on its line
  const Extent mine_e = lane < a.B ? extent_of(a, lane) : Extent{};
  const int total = total_units<TR>(a, mine_e, lane);
  const int U = max(1, (total + a.parts * TS - 1) / (a.parts * TS)), u_end = min(total, (me + 1) * U);
  for (int u = me * U; u < u_end;) {
    const Tile it = tile_of<TR>(a, mine_e, u, lane);
    if (it.units == 0) break;                                  // (only if lengths change meanwhile or overflow the sum)
    const int u_next = min(u_end, it.begin + it.units);
    // This tile's chunks: one per wave that its units reach
    const int wf = it.begin / U;
    const Chunks ck{wf, (it.begin + it.units - 1) / U - wf + 1, me - wf};
    const int nq = it.e.nq, L = it.e.L, r0 = it.qt * TR, rows = nq * a.G;
    const int i0 = r0 / a.G, i1 = min(nq - 1, (r0 + TR - 1) / a.G);
    const int p0 = L - nq;                                     // position of query 0
    const int tend = min(max(a.causal ? p0 + i1 + 1 : L, 0), L);
    const int tmin = a.window > 0 ? min(max(0, p0 + i0 - a.window + 1), tend) : 0;      // the first token that a row sees
    const int tbeg = tmin & ~31;
    const int begin = begin_of(a, it.e);
    const int c0 = max(tbeg, begin + 32 * (u - it.begin));              // a multiple of 32
    const int c1 = min(tend, begin + 32 * (u_next - it.begin));
    u = u_next;

    int c16 = lane & 15, g4 = lane >> 4;
    asm volatile("" : "+v"(c16), "+v"(g4));                    // (nothing computed from them outlives a tile)
    // Channels of a group that lane group g4 holds of K and q: 8 g4 on, or (two groups loaded at
    // once, 16 bytes per lane, and their halves swapped between the wave's halves) kq on.
    const int kq = ((g4 & 1) << 4) | ((g4 >> 1) << 3);

    // q's rows (packed: query token, then head of the group); their first use is further down.
    u32x4 qraw[R][NG];
    int qpos[R];
  #pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = r0 + 16 * r + c16;
      const bool live = row < rows;
      const int i = live ? row / a.G : i0, g = live ? row - i * a.G : 0;
      qpos[r] = live ? p0 + i : -1;
      const uint16_t* qp = a.q + (int64_t)(it.e.qs + i) * a.q_stride + (int64_t)(h * a.G + g) * D + (NG % 2 == 0 ? kq : 8 * g4);
  #pragma unroll
      for (int n = 0; n < NG; ++n) qraw[r][n] = ld16(qp + 32 * n);
    }

    f32x4 o[2 * NG][R];
    float m[R], l[R];
  #pragma unroll
    for (int n = 0; n < 2 * NG; ++n)
  #pragma unroll
      for (int r = 0; r < R; ++r) o[n][r] = (f32x4){0.f, 0.f, 0.f, 0.f};
  #pragma unroll
    for (int r = 0; r < R; ++r) m[r] = kNegInf, l[r] = 0.0f;

    const int hk = a.Hk, page_mask = (1 << a.page_shift) - 1;
    typedef Pieces<NG> P1;
    typedef Pieces<(P1::Rest > 0 ? P1::Rest : 1)> P2;          // NG <= 8, no 7: at most two pieces
    constexpr int RB1 = 2 * P1::P, RB2 = 2 * P2::P;
    constexpr bool kTwo = P1::Rest > 0;
    static_assert(!kTwo || P2::Rest == 0, "two pieces at most");

    // Tiles start at multiples of 32 tokens and pages hold 16 or more, so each half of a tile lies
    // in one page: its first entry is uniform, and all addresses are a uniform base plus an offset
    // that a lane keeps.  -1: the page is outside the pool (its tokens are left out).
    const ConstInt* table = (const ConstInt*)(uintptr_t)(a.block_table + (int64_t)it.b * a.max_pages);
    auto page_of = [&](int t) { return table[min(t, a.max_tokens - 1) >> a.page_shift]; };
    auto entry_of = [&](int page, int t) {
      return page >= 0 && page < a.pages ? (page << a.page_shift) + (t & page_mask) : -1;
    };
    const uint32_t row_bytes = (uint32_t)hk * D;               // from one token to the next
    const uint32_t koff = c16 * row_bytes + (NG % 2 == 0 ? 16 : 8) * g4;
    const uint32_t voff1 = 4 * g4 * row_bytes + RB1 * c16, voff2 = 4 * g4 * row_bytes + 32 * P1::P + RB2 * c16;

    // Pipeline: while a tile is computed, the next one's K, scales and V are in flight (K and the
    // scales from the moment the scores are done, V from the moment the values are), and the pages
    // of the one after that.  Loads come back in the order of their issue, so what is wanted first
    // is asked for first, and none of them is behind a branch (past the last tile they read the
    // pool's first entries).  A second buffer changed nothing (1 % slower): the loads are bound by
    // bandwidth, not by their latency.
    constexpr int KI = NG % 2 == 0 ? NG / 2 : NG;
    typedef typename std::conditional<NG % 2 == 0, u32x4, u32x2>::type KRaw;
    KRaw kr[2][KI];
    KScales<NG> ksr;
    uint32_t vsr;
    Raw<RB1, NT> v1[8];
    Raw<RB2, NT> v2[8];
    auto load_k = [&](int e0, int e1) {                        // and the scales: one token per lane
      const int64_t at = ((int64_t)(max(lane & 16 ? e1 : e0, 0) + c16)) * hk + h;
      ksr.load(a.k_scales + at * NG);
      vsr = a.v_scales[at];
  #pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t* p = a.k_codes + ((int64_t)max(u ? e1 : e0, 0) * hk + h) * D;
  #pragma unroll
        for (int n = 0; n < KI; ++n) {
          if constexpr (NG % 2 == 0) kr[u][n] = ld<NT>(reinterpret_cast<const u32x4*>(p + 64 * n + koff));
          else kr[u][n] = *reinterpret_cast<const u32x2*>(p + 32 * n + koff);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto load_v = [&](int e0, int e1) {
  #pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t* p = a.v_codes + ((int64_t)max(u ? e1 : e0, 0) * hk + h) * D;
  #pragma unroll
        for (int j = 0; j < 4; ++j) {
          v1[4 * u + j].load(p + (size_t)j * row_bytes + voff1);
          if constexpr (kTwo) v2[4 * u + j].load(p + (size_t)j * row_bytes + voff2);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    int e0 = entry_of(page_of(c0), c0), e1 = entry_of(page_of(c0 + 16), c0 + 16);   // of the tile's halves
    int g0 = page_of(c0 + 32), g1 = page_of(c0 + 48);          // the next tile's pages
    load_k(e0, e1);
    load_v(e0, e1);

    // q: per query row a power of two into [-1, 1), fp16; rows past the last are zero.
    f16x8 qf[R][NG];
    float cs[R];
  #pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool live = r0 + 16 * r + c16 < rows;
      float f[NG][8], am = 0.0f;
  #pragma unroll
      for (int n = 0; n < NG; ++n) {
        const uint32_t d[4] = {qraw[r][n].x, qraw[r][n].y, qraw[r][n].z, qraw[r][n].w};
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
        for (int e = 0; e < 8; ++e) qf[r][n][e] = (_Float16)__builtin_ldexpf(f[n][e], -ex);
      cs[r] = __builtin_ldexpf(a.scale * kLog2e, ex);
    }

    // Tokens before every row's window, in its first tile: no row sees them (so `open` is false there and
    // their scores are masked), and their values are cleared, for an entry that no query sees may hold
    // anything.  (17.5 against 17.2 us without it for 16 x 5 tokens in a window of 1024; as a condition of
    // each tile in the loop below 18.1, and 1 % where there is no window.)
    if (c0 < tmin) {
  #pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c0 + 4 * g4 + 16 * (i >> 2) + (i & 3) < tmin) {
          v1[i].clear();
          if constexpr (kTwo) v2[i].clear();
        }
    }

    for (int base = c0; base < c1; base += 32) {
      const bool all_valid = e0 >= 0 && e1 >= 0 && base + 32 <= c1;
      const int n0 = entry_of(g0, base + 32), n1 = entry_of(g1, base + 48);
      const int t0 = base + 4 * g4;                            // this lane's first token (u = j = 0)
      auto there = [&](int u, int j) { return (u ? e1 : e0) >= 0 && t0 + 16 * u + j < c1; };
      // V scales into the exponent.  A scale of zero (an entry never written) counts as the
      // smallest one: its codes are zero too.  Tokens that are not there count as scale 1.
      if (lane < 32) {
        const bool in = all_valid || ((lane & 16 ? e1 : e0) >= 0 && base + lane < c1);
        const float sv = in ? fmaxf(f16_lo(vsr), 0x1p-24f) : 1.0f;
        mine.lv[lane] = __builtin_amdgcn_logf(sv);
        mine.rv[lane] = __builtin_amdgcn_rcpf(sv);
  #pragma unroll
        for (int n = 0; n < NG; ++n) mine.ks[n][lane] = ksr.get(n);
      }
      wave_sync();

      // S^T: tokens 16 u + 4 g4 + j, query c16
      float s[R][2][4];
  #pragma unroll
      for (int u = 0; u < 2; ++u) {
  #pragma unroll
        for (int n = 0; n < NG; ++n) {
          u32x2 kw;
          if constexpr (NG % 2 == 0) {
            if (n % 2 == 0) {
              const auto lo = __builtin_amdgcn_permlane32_swap(kr[u][n / 2].x, kr[u][n / 2].z, false, false);
              const auto hi = __builtin_amdgcn_permlane32_swap(kr[u][n / 2].y, kr[u][n / 2].w, false, false);
              kr[u][n / 2] = (u32x4){lo[0], hi[0], lo[1], hi[1]};
              kw = (u32x2){lo[0], hi[0]};
            } else {
              kw = (u32x2){kr[u][n / 2].z, kr[u][n / 2].w};
            }
          } else {
            kw = (u32x2){kr[u][n].x, kr[u][n].y};
          }
          const f16x8 kf = i8x8_to_f16(kw);
          const f32x4 ks = *reinterpret_cast<const f32x4*>(&mine.ks[n][16 * u + 4 * g4]);
  #pragma unroll
          for (int r = 0; r < R; ++r) {
            const f32x4 d = mfma_f16_k32(kf, qf[r][n], (f32x4){0.f, 0.f, 0.f, 0.f});
  #pragma unroll
            for (int j = 0; j < 4; ++j) s[r][u][j] = n == 0 ? ks[j] * d[j] : __builtin_fmaf(ks[j], d[j], s[r][u][j]);
          }
        }
      }
      float lv[2][4], rv[2][4];
  #pragma unroll
      for (int u = 0; u < 2; ++u) {
        *reinterpret_cast<f32x4*>(lv[u]) = *reinterpret_cast<const f32x4*>(&mine.lv[16 * u + 4 * g4]);
        *reinterpret_cast<f32x4*>(rv[u]) = *reinterpret_cast<const f32x4*>(&mine.rv[16 * u + 4 * g4]);
      }
      load_k(n0, n1);
      g0 = page_of(base + 64);
      g1 = page_of(base + 80);

      // whole tile visible to every row of this workgroup?
      const int tmin_p = p0 + i0, tmax_p = p0 + i1;
      const bool open = all_valid && (!a.causal || base + 31 <= tmin_p) && (a.window <= 0 || base > tmax_p - a.window);
      if (!all_valid) {
  #pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!there(i >> 2, i & 3)) {
            v1[i].clear();
            if constexpr (kTwo) v2[i].clear();
          }
      }
      f16x8 w[R];
  #pragma unroll
      for (int r = 0; r < R; ++r) {
        float mx = kNegInf;
  #pragma unroll
        for (int u = 0; u < 2; ++u)
  #pragma unroll
          for (int j = 0; j < 4; ++j) {
            float v = __builtin_fmaf(s[r][u][j], cs[r], lv[u][j]);
            if (!open) {
              const int t = t0 + 16 * u + j;
              const bool see = there(u, j) && (!a.causal || t <= qpos[r]) && (a.window <= 0 || t > qpos[r] - a.window);
              v = see ? v : kNegInf;
            }
            s[r][u][j] = v;
            mx = fmaxf(mx, v);
          }
        mx = max_across16(mx);
        const float mn = fmaxf(m[r], mx - kLift);
        const float ref = mn == kNegInf ? 0.0f : mn;
        if (__ballot(mn > m[r])) {
          const float corr = __builtin_amdgcn_exp2f(m[r] - ref);
          l[r] *= corr;
  #pragma unroll
          for (int n = 0; n < 2 * NG; ++n)
  #pragma unroll
            for (int j = 0; j < 4; ++j) o[n][r][j] *= corr;
          m[r] = mn;
        }
  #pragma unroll
        for (int u = 0; u < 2; ++u)
  #pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float e = __builtin_amdgcn_exp2f(s[r][u][j] - ref);
            l[r] = __builtin_fmaf(e, rv[u][j], l[r]);
            w[r][4 * u + j] = (_Float16)e;
          }
      }
      pv_piece<P1::P, R, NT>(v1, w, o);
      if constexpr (kTwo) pv_piece<P2::P, R, NT>(v2, w, o + 2 * P1::P);
      load_v(n0, n1);
      e0 = n0;
      e1 = n1;
    }

    // A lane has, per 16-row subtile, channels 2 P (4 g4 + j) .. + 2 P - 1 of each piece of its row.
    // (The copies keep the compiler from computing addresses ahead of the tile loop.)
    constexpr int W1 = 2 * P1::P, W2 = 2 * P2::P;
    asm volatile("" : "+v"(c16), "+v"(g4));
    const bool split = ck.count > 1;
    const __amdgpu_buffer_rsrc_t rs = partial_rsrc(a.partials, a.partials_bytes);
    auto part_row = [&](int c, int row) { return (int64_t)((ck.slot(c) * hk + h) * a.tile_rows + row) * (D + 4); };
    auto out_row = [&](int grow) {                             // index of [token][query head]
      const int i = grow / a.G;
      return (int64_t)(it.e.qs + i) * a.Hq + h * a.G + (grow - i * a.G);
    };
  #pragma unroll
    for (int r = 0; r < R; ++r) {
      const float L = sum_across16(l[r]);                      // over the lane groups of a query
      const int row = 16 * r + c16;
      if (r0 + row < rows) {
        float v1r[4][W1], v2r[4][W2];
  #pragma unroll
        for (int j = 0; j < 4; ++j) {
  #pragma unroll
          for (int n = 0; n < W1; ++n) v1r[j][n] = o[n][r][j];
          if constexpr (kTwo)
  #pragma unroll
            for (int n = 0; n < W2; ++n) v2r[j][n] = o[W1 + n][r][j];
        }
        if (!split) {
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;          // (NaN stays NaN)
          const int64_t at = out_row(r0 + row);
          uint16_t* out = a.out + at * D;
  #pragma unroll
          for (int j = 0; j < 4; ++j) {
            store_out<W1>(out + (4 * g4 + j) * W1, v1r[j], inv);
            if constexpr (kTwo) store_out<W2>(out + 32 * P1::P + (4 * g4 + j) * W2, v2r[j], inv);
          }
          if (a.lse && g4 == 0) a.lse[at] = L == 0.0f ? kNegInf : (m[r] + __builtin_amdgcn_logf(L)) * kLn2;
        } else {
          const int64_t p = part_row(ck.mine, row);
  #pragma unroll
          for (int j = 0; j < 4; ++j) {
            store_run<W1>(rs, p + (4 * g4 + j) * W1, v1r[j]);
            if constexpr (kTwo) store_run<W2>(rs, p + 32 * P1::P + (4 * g4 + j) * W2, v2r[j]);
          }
          if (g4 == 0) {
            const float ml[2] = {m[r], L};
            store_run<2>(rs, p + D, ml);
          }
        }
      }
    }
    if (!split) continue;

    // (four chunks at a time from heads of 128 on: 72 -> 63 us for 32 x 8 rows of 256 over 8000 tokens;
    // heads of 64 lost 3 %)
    join_chunks<D, (NG >= 4)>(a, rs, mine.join, lane, ck, min(TR, rows - r0), part_row,
                              [&](int row) { return out_row(r0 + row); },
                              [&](int level, int c) { return level * a.level_counters + ck.slot(c) * hk + h; });
  }
}

template <int NG>
hipError_t launch_ng(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t st) {
  if constexpr (pairs_rows(NG))
    if (p.R == 2) {
      kv_attention_kernel<NG, 2><<<(int)p.grid, waves_of(NG) * 64, 0, st>>>(a);
      return hipGetLastError();
    }
  kv_attention_kernel<NG, 1><<<(int)p.grid, waves_of(NG) * 64, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

KvAttnPlan plan_kv_attention(int64_t T, int64_t B, int64_t Hk, int64_t G, int64_t D, bool one_each) {
  KvAttnPlan p;
  const int64_t rows = one_each ? G : (T + B - 1) / B * G;   // query rows of an average sequence
  // Many rows: kv_attention_tile.hip, one workgroup of eight waves per CU.  From where on, by 16
  // sequences of 4000 and 16000 tokens, there and here: 24 rows of 128 over 8 KV heads 93 and 262
  // against 69 and 159 us, 40 rows 94 and 269 against 100 and 261; 64 rows of 64 76 and 245 against
  // 62 and 199, of 192 107 and 265 against 88 and 241, of 256 125 and 352 against 97 and 214; 96
  // rows of 64 78 and 248 against 85 and 308, of 192 115 and 271 against 109 and 376.
  // One kernel takes the whole call, so a prompt beside single tokens is slow on either side of that
  // average (32 heads over 8 of 128, tokens over up to 4096): a prompt of 512 with 63 of them 289 us
  // where the two calls take 74 + 49, with 127 227 (133 + 49), with 255 298 (248 + 49); one of 2048 with
  // 255 of them 1400 (251 + 120).
  const bool pairs = pairs_rows((int)(D / 32));
  if (rows > (pairs ? 32 : 64)) {
    p.R = 16;
    p.parts = (int)(Hk >= 256 ? 1 : 256 / Hk);
    p.grid = p.parts * Hk;
    p.waves = p.parts;
    p.tile_rows = 256;
    p.counters = 2 * p.parts * Hk * 8;
    p.tiles = one_each ? B * ((G + 255) / 256) : T * G / 256 + B;
    return p;
  }
  p.R = rows <= 16 || !pairs ? 1 : 2;
  const int64_t TR = 16 * p.R;
  // Neighbouring KV heads per workgroup: a power of two that divides Hk, at most four (eight, where
  // there are eight waves: 70 against 75 us for 32 sequences of 4000 tokens and 16 heads of 64, but
  // 20.4 against 18.1 for 16 x 5 tokens in a window of 1024).
  while ((2 << p.hw_shift) <= 4 && Hk % (2 << p.hw_shift) == 0) ++p.hw_shift;
  const int waves = waves_of((int)(D / 32));
  // One workgroup per CU.  Half, one and a half, and two of them: 215, 165 and 141 us
  // against 126 for 64 sequences of up to 8192 tokens, and 27.0, 19.6 and 19.0 against 19.8 for
  // 16 x 5 tokens in a window of 1024 (four waves each): more waves are more chunks to join.
  const int64_t HG = Hk >> p.hw_shift;
  const int64_t parts = 256 / HG;
  p.parts = (int)(parts >= 8 ? parts / 8 * 8 : parts < 1 ? 1 : parts);
  p.grid = p.parts * HG;
  p.waves = p.parts * (waves >> p.hw_shift);
  p.tile_rows = (int)(one_each && G < TR ? G : TR);
  p.counters = 2 * p.waves * Hk;
  p.tiles = one_each ? B * ((G + TR - 1) / TR) : T * G / TR + B;
  return p;
}

hipError_t launch_kv_attention(const KvAttnArgs& a, const KvAttnPlan& p, int D, hipStream_t st) {
  if (p.R == 16) return launch_kv_attention_tile(a, p, D, st);
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
