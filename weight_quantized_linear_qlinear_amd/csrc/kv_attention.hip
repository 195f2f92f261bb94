// Attention over the paged 8-bit KV cache (K int8 with an fp16 scale per 32 channels, V e4m3
// with one per (token, head)), for one query token per sequence or many.
//
// For a query row (token i of sequence b, head g of the KV head's group) at position
// p = L - nq + i, over the cached tokens t that the masks leave:
//   s_t = scale * sum_c k_scale[t,c] * (q_c . k_code[t,c])      (c: groups of 32 channels)
//   o   = sum_t 2^(s_t log2e) v_scale_t v_code_t / sum_t 2^(s_t log2e)
// in one pass with a running reference m and sum l.  v_scale_t is taken into the exponent:
//   x_t = s_t log2e + log2 v_scale_t,  w_t = 2^(x_t - m) in [0, 1],  o = sum w_t v_code_t,
//   l = sum w_t / v_scale_t,
// so that the weights fit fp16 whatever the scales are.  Products run on the matrix cores in
// fp16 with fp32 accumulation: int8 and e4m3 codes are exact in fp16, q is scaled per row by a
// power of two into [-1, 1) (exact but for channels 2^-14 and more below the row's largest,
// whose absolute error stays under 2^-25 of it), and the weights' rounding to 11 bits is the
// only other one (2^-12 of a weight; the output's own rounding to bf16 is 2^-9).
//
// Layout.  A workgroup takes one KV head, 16 R query rows (nq x G rows packed, so that the
// heads of a group share every K and V load) and a run of tokens; its NW waves take 32 tokens
// each in turn, on their own, and are summed through LDS at the end.  S^T = K Q^T (tokens are
// the rows): lane l holds query l % 16 and tokens 4 (l / 16) + j, which is the operand that
// O^T = V^T P^T wants, so the weights never cross lanes.  V^T needs, per lane, one channel of
// eight tokens: each lane loads the same few channels of its eight tokens and transposes bytes
// pairwise while converting.
//
// Work is cut on the device, from the lengths it finds there (the host knows none of them and
// waits for nothing): every workgroup sums the sequences' tokens, derives one chunk length
// that gives about `target` workgroups, and finds its (sequence, query tile, chunk).  Chunks
// of one tile are joined by the last workgroup to finish, in the order of the chunks.
#include "qlq_device.h"
#include "qlq_launch.h"

namespace qlq {

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ f32x4 mfma_f16_k32(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float f16_lo(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (uint16_t)(b & 0xFFFF)); }
__device__ __forceinline__ float f16_hi(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (uint16_t)(b >> 16)); }

// Two int8 codes (bytes 0, 1 or 2, 3 of w ^ 0x80808080) as fp16: 1024 + (q + 128) by its bit
// pattern, minus 1152; exact.
template <bool HI>
__device__ __forceinline__ uint32_t i8x2_to_f16(uint32_t flipped) {
  const uint32_t b = __builtin_amdgcn_perm(0x64646464u, flipped, HI ? 0x04030402u : 0x04010400u);
  const f16x2 k = {(_Float16)1152.0f, (_Float16)1152.0f};
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, b) - k);
}

__device__ __forceinline__ f16x8 i8x8_to_f16(u32x2 w) {
  const uint32_t a = w.x ^ 0x80808080u, b = w.y ^ 0x80808080u;
  const u32x4 r = {i8x2_to_f16<false>(a), i8x2_to_f16<true>(a), i8x2_to_f16<false>(b), i8x2_to_f16<true>(b)};
  return __builtin_bit_cast(f16x8, r);
}

template <bool HI>
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
}

// BYTES (2, 4, 8 or 16) at p, aligned to BYTES, as dwords (2 bytes: the low half).
template <int BYTES>
struct Raw {
  static constexpr int N = BYTES < 4 ? 1 : BYTES / 4;
  uint32_t d[N];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (BYTES == 2) {
      d[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (BYTES == 4) {
      d[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (BYTES == 8) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(p);
      d[0] = v.x, d[1] = v.y;
    } else {
      const u32x4 v = ld16(p);
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
template <int P, int R>
__device__ __forceinline__ void pv_piece(const Raw<2 * P> (&v)[8], const f16x8 (&w)[R], f32x4 (*o)[R]) {
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

// One token's K scales (NG fp16).
template <int NG>
struct KScales {
  float s[NG];
  __device__ __forceinline__ void load(const uint16_t* p) {
    if constexpr (NG % 8 == 0) {
      const u32x4 v = ld16(p);
      s[0] = f16_lo(v.x), s[1] = f16_hi(v.x), s[2] = f16_lo(v.y), s[3] = f16_hi(v.y);
      s[4] = f16_lo(v.z), s[5] = f16_hi(v.z), s[6] = f16_lo(v.w), s[7] = f16_hi(v.w);
    } else if constexpr (NG == 4) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(p);
      s[0] = f16_lo(v.x), s[1] = f16_hi(v.x), s[2] = f16_lo(v.y), s[3] = f16_hi(v.y);
    } else if constexpr (NG % 2 == 0) {
#pragma unroll
      for (int i = 0; i < NG; i += 2) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(p + i);
        s[i] = f16_lo(v), s[i + 1] = f16_hi(v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NG; ++i) s[i] = f16_lo(p[i]);
    }
  }
};

// Sequence b: its query tokens, its cached tokens, and how many of those any query can see.
struct Extent {
  int qs, nq, L, begin;
  __device__ __forceinline__ int range() const { return L - begin; }
};

__device__ __forceinline__ Extent extent_of(const KvAttnArgs& a, int b) {
  Extent e;
  if (a.q_start) {
    const int lo = min(max(a.q_start[b], 0), a.T), hi = min(max(a.q_start[b + 1], lo), a.T);
    e.qs = lo;
    e.nq = hi - lo;
  } else {
    e.qs = b;
    e.nq = 1;
  }
  e.L = min(max(a.seq_lens[b], 0), a.max_tokens);
  e.begin = (a.window > 0 && e.nq > 0) ? max(0, e.L - e.nq - a.window + 1) : 0;
  e.begin = min(e.begin, e.L);
  return e;
}

__device__ __forceinline__ int64_t wave_sum64(int64_t v) {
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

__device__ __forceinline__ int wave_scan(int v, int lane) {   // inclusive
  for (int off = 1; off < 64; off <<= 1) {
    const int u = __shfl_up(v, off, 64);
    if (lane >= off) v += u;
  }
  return v;
}

struct Item {
  int b, qt, ch, nch, first;     // first: item index of chunk 0 of this (sequence, tile)
  Extent e;
  bool found;
};

// Finds item `item`: every wave on its own, 64 sequences at a time.
template <int TR>
__device__ __forceinline__ Item find_item(const KvAttnArgs& a, int item, int lane) {
  Item it;
  it.found = false;
  int64_t C = (int64_t)1 << 40;
  if (a.split) {
    int64_t total = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
      int64_t w = 0;
      if (b0 + lane < a.B) {
        const Extent e = extent_of(a, b0 + lane);
        w = (int64_t)((e.nq * a.G + TR - 1) / TR) * e.range();
      }
      total += wave_sum64(w);
    }
    C = (total + a.target - 1) / a.target;
    C = (C + a.chunk_step - 1) / a.chunk_step * a.chunk_step;
    if (C < a.chunk_step) C = a.chunk_step;
  }
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    int n = 0, nch = 1;
    Extent e{};
    if (b0 + lane < a.B) {
      e = extent_of(a, b0 + lane);
      const int nqt = (e.nq * a.G + TR - 1) / TR;
      nch = max(1, (int)((e.range() + C - 1) / C));
      n = nqt * nch;
    }
    const int inc = before + wave_scan(n, lane);
    const uint64_t hit = __ballot(n > 0 && item < inc && item >= inc - n);
    if (hit) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      it.b = b0 + src;
      it.nch = __shfl(nch, src, 64);
      const int begin = __shfl(inc - n, src, 64), tiles = __shfl(n, src, 64) / it.nch;
      const int rel = item - begin;
      it.qt = tiles - 1 - rel / it.nch;                    // the longest causal tiles first
      it.ch = rel % it.nch;
      it.first = item - it.ch;
      it.e.qs = __shfl(e.qs, src, 64);
      it.e.nq = __shfl(e.nq, src, 64);
      it.e.L = __shfl(e.L, src, 64);
      it.e.begin = __shfl(e.begin, src, 64);
      it.found = true;
      return it;
    }
    before = __shfl(inc, 63, 64);
  }
  return it;
}

// The row sums of the workgroup's waves, per 16-row subtile: acc[w][row][D + 4].
template <int NG, int NW>
struct Smem {
  static constexpr int D = 32 * NG, LD = D + 4;
  static constexpr int kMaxChunks = 256;
  union {
    float acc[NW][16][LD];
    float f[16][kMaxChunks];
    int slot[NW][2][32];
  };
  float m[NW][16], l[NW][16];
  float red[NW * 64 * 4];
  int last;
};

template <int NG, int R, int NW>
__global__ __launch_bounds__(NW * 64) void kv_attention_kernel(KvAttnArgs a) {
  constexpr int D = 32 * NG, TR = 16 * R;
  typedef Smem<NG, NW> S;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c16 = lane & 15, g4 = lane >> 4;
  // The heads of one item sit on one XCD (workgroup b goes to XCD b % 8): a token's scales of
  // all heads share cache lines.
  const int x = blockIdx.x & 7, li = blockIdx.x >> 3;
  const int item = (li / a.Hk) * 8 + x, h = li % a.Hk;
  const Item it = find_item<TR>(a, __builtin_amdgcn_readfirstlane(item), lane);
  if (!it.found) return;                                     // uniform for the workgroup
  const int nq = it.e.nq, L = it.e.L, r0 = it.qt * TR, rows = nq * a.G;
  const int i0 = r0 / a.G, i1 = min(nq - 1, (r0 + TR - 1) / a.G);
  const int p0 = L - nq;                                     // position of query 0
  const int tend = min(max(a.causal ? p0 + i1 + 1 : L, 0), L);
  const int tbeg = a.window > 0 ? min(max(0, p0 + i0 - a.window + 1), tend) : 0;
  const int per = ((tend - tbeg + it.nch - 1) / it.nch + 31) & ~31;
  const int c0 = min(tbeg + it.ch * per, tend), c1 = min(c0 + per, tend);

  // q: per query row a power of two into [-1, 1), fp16.
  f16x8 qf[R][NG];
  float cs[R];
  int qpos[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = r0 + 16 * r + c16;
    const bool live = row < rows;
    const int i = live ? row / a.G : 0, g = live ? row % a.G : 0;
    qpos[r] = live ? p0 + i : -1;
    const uint16_t* qp = a.q + (int64_t)(it.e.qs + i) * a.q_stride + (int64_t)(h * a.G + g) * D + 8 * g4;
    float f[NG][8], am = 0.0f;
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const u32x4 v = live ? ld16(qp + 32 * n) : (u32x4){0u, 0u, 0u, 0u};
      const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[n][2 * e] = bf16_bits_to_f32(d[e] & 0xFFFF);
        f[n][2 * e + 1] = bf16_bits_to_f32(d[e] >> 16);
        am = fmaxf(am, fmaxf(fabsf(f[n][2 * e]), fabsf(f[n][2 * e + 1])));
      }
    }
    am = fmaxf(am, __shfl_xor(am, 16, 64));
    am = fmaxf(am, __shfl_xor(am, 32, 64));
    const int ex = am > 0.0f ? __builtin_amdgcn_frexp_expf(am) : 0;   // am < 2^ex
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) qf[r][n][e] = (_Float16)__builtin_ldexpf(f[n][e], -ex);
    cs[r] = __builtin_ldexpf(a.scale * kLog2e, ex);
  }

  f32x4 o[2 * NG][R];
  float m[R], l[R];
#pragma unroll
  for (int n = 0; n < 2 * NG; ++n)
#pragma unroll
    for (int r = 0; r < R; ++r) o[n][r] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < R; ++r) m[r] = kNegInf, l[r] = 0.0f;

  const int32_t* table = a.block_table + (int64_t)it.b * a.max_pages;
  const int page_mask = (1 << a.page_shift) - 1;
  const int hk = a.Hk;
  typedef Pieces<NG> P1;
  typedef Pieces<(P1::Rest > 0 ? P1::Rest : 1)> P2;          // NG <= 8, no 7: at most two pieces
  constexpr int RB1 = 2 * P1::P, RB2 = 2 * P2::P;
  constexpr bool kTwo = P1::Rest > 0;
  static_assert(!kTwo || P2::Rest == 0, "two pieces at most");

  auto slot_of = [&](int base) {                             // lanes 0..31 (repeated above): token base + lane
    const int t = base + (lane & 31);
    int s = -1;
    if (t < c1) {
      const int page = table[t >> a.page_shift];
      if (page >= 0 && page < a.pages) s = (page << a.page_shift) | (t & page_mask);
    }
    return s;
  };

  int next_slot = slot_of(c0 + 32 * wave);
  int buf = 0;
  for (int base = c0 + 32 * wave; base < c1; base += 32 * NW) {
    const int my = next_slot;
    const bool all_valid = __ballot(my < 0) == 0;
    if (lane < 32) sm.slot[wave][buf][lane] = my;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    int kslot[2];
    int vslot[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      kslot[u] = max(sm.slot[wave][buf][16 * u + c16], 0);
      const i32x4 v = *reinterpret_cast<const i32x4*>(&sm.slot[wave][buf][16 * u + 4 * g4]);
#pragma unroll
      for (int j = 0; j < 4; ++j) vslot[u][j] = v[j];
    }
    buf ^= 1;
    // loads of the tile
    u32x2 kr[2][NG];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* p = a.k_codes + ((int64_t)kslot[u] * hk + h) * D + 8 * g4;
#pragma unroll
      for (int n = 0; n < NG; ++n) kr[u][n] = *reinterpret_cast<const u32x2*>(p + 32 * n);
    }
    KScales<NG> ks[2][4];
    uint32_t vsb[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t at = (int64_t)max(vslot[u][j], 0) * hk + h;
        ks[u][j].load(a.k_scales + at * NG);
        vsb[u][j] = a.v_scales[at];
      }
    Raw<RB1> v1[8];
    Raw<RB2> v2[8];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* p = a.v_codes + ((int64_t)max(vslot[u][j], 0) * hk + h) * D;
        v1[4 * u + j].load(p + RB1 * c16);
        if constexpr (kTwo) v2[4 * u + j].load(p + 32 * P1::P + RB2 * c16);
      }
    next_slot = slot_of(base + 32 * NW);

    // S^T: tokens 16 u + 4 g4 + j, query c16
    float s[R][2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[r][u][j] = 0.0f;
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const f16x8 kf = i8x8_to_f16(kr[u][n]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const f32x4 d = mfma_f16_k32(kf, qf[r][n], (f32x4){0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int j = 0; j < 4; ++j) s[r][u][j] = __builtin_fmaf(ks[u][j].s[n], d[j], s[r][u][j]);
        }
      }
    }
    // V scales into the exponent.  A scale of zero (an entry never written) counts as the
    // smallest one: its codes are zero too.
    float lv[2][4], rv[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float sv = fmaxf(f16_lo(vsb[u][j]), 0x1p-24f);
        if (!all_valid && vslot[u][j] < 0) sv = 1.0f;
        lv[u][j] = __builtin_amdgcn_logf(sv);
        rv[u][j] = __builtin_amdgcn_rcpf(sv);
      }
    // whole tile visible to every row of this workgroup?
    const int tmin_p = p0 + i0, tmax_p = p0 + i1;
    const bool open = all_valid && (!a.causal || base + 31 <= tmin_p) && (a.window <= 0 || base > tmax_p - a.window);
    if (!all_valid) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (vslot[i >> 2][i & 3] < 0) {
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
            const int t = base + 16 * u + 4 * g4 + j;
            const bool see = vslot[u][j] >= 0 && (!a.causal || t <= qpos[r]) && (a.window <= 0 || t > qpos[r] - a.window);
            v = see ? v : kNegInf;
          }
          s[r][u][j] = v;
          mx = fmaxf(mx, v);
        }
      mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
      mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
      const float mn = fmaxf(m[r], mx);
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
    pv_piece<P1::P, R>(v1, w, o);
    if constexpr (kTwo) pv_piece<P2::P, R>(v2, w, o + 2 * P1::P);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {                              // l over the lane groups of a query
    l[r] += __shfl_xor(l[r], 16, 64);
    l[r] += __shfl_xor(l[r], 32, 64);
  }

  // Sum over the waves, 16 rows at a time; thread (row, part) holds 2 NG channels of a row.
  constexpr int SEG = 16, CH = 2 * NG;
  const bool split = it.nch > 1;
  const int64_t tile_base = ((int64_t)item * hk + h) * a.tile_rows;       // this chunk's partial rows
  const __amdgpu_buffer_rsrc_t rs = partial_rsrc(a.partials, a.partials_bytes);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    __syncthreads();
    if (g4 == 0) {
      sm.m[wave][c16] = m[r];
      sm.l[wave][c16] = l[r];
    }
    __syncthreads();
    float M = kNegInf;
    for (int w2 = 0; w2 < NW; ++w2) M = fmaxf(M, sm.m[w2][c16]);
    const float f = M == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m[r] - M);
#pragma unroll
    for (int n = 0; n < 2 * NG; ++n) {
      // tile n, element j: channel of column c = 4 g4 + j
      constexpr int W1 = 2 * P1::P;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int ch = n < W1 ? (4 * g4 + j) * W1 + n : 32 * P1::P + (4 * g4 + j) * RB2 + (n - W1);
        sm.acc[wave][c16][ch] = o[n][r][j] * f;
      }
    }
    __syncthreads();
    for (int idx = tid; idx < 16 * SEG; idx += NW * 64) {
      const int row = idx / SEG, part = idx % SEG;
      const int grow = r0 + 16 * r + row;
      if (grow >= rows) continue;
      float Mr = kNegInf, Lr = 0.0f;
      for (int w2 = 0; w2 < NW; ++w2) Mr = fmaxf(Mr, sm.m[w2][row]);
      if (Mr != kNegInf)
        for (int w2 = 0; w2 < NW; ++w2) Lr += sm.l[w2][row] * __builtin_amdgcn_exp2f(sm.m[w2][row] - Mr);
      float v[CH];
#pragma unroll
      for (int e = 0; e < CH; ++e) v[e] = 0.0f;
      for (int w2 = 0; w2 < NW; ++w2)
#pragma unroll
        for (int e = 0; e < CH; ++e) v[e] += sm.acc[w2][row][part * CH + e];
      if (!split) {
        const float inv = Lr > 0.0f ? 1.0f / Lr : 0.0f;
        const int i = grow / a.G, g = grow % a.G;
        uint32_t* out = reinterpret_cast<uint32_t*>(a.out + ((int64_t)(it.e.qs + i) * a.Hq + h * a.G + g) * D + part * CH);
#pragma unroll
        for (int e = 0; e < CH; e += 2) out[e / 2] = pack_bf16x2(v[e] * inv, v[e + 1] * inv);
        if (a.lse && part == 0)
          a.lse[(int64_t)(it.e.qs + i) * a.Hq + h * a.G + g] = Lr > 0.0f ? (Mr + __builtin_amdgcn_logf(Lr)) * kLn2 : kNegInf;
      } else {
        const int64_t p = (tile_base + 16 * r + row) * (D + 4);          // [D sums][M, L, -, -]
#pragma unroll
        for (int e = 0; e < CH; e += 2)
          __builtin_amdgcn_raw_buffer_store_b64(
              (u32x2){__builtin_bit_cast(uint32_t, v[e]), __builtin_bit_cast(uint32_t, v[e + 1])}, rs,
              (int)((p + part * CH + e) * 4), 0, kCachePolicySc1);
        if (part == 0)
          __builtin_amdgcn_raw_buffer_store_b64(
              (u32x2){__builtin_bit_cast(uint32_t, Mr), __builtin_bit_cast(uint32_t, Lr)}, rs, (int)((p + D) * 4), 0,
              kCachePolicySc1);
      }
    }
  }
  if (!split) return;

  // Join the chunks: the last workgroup of this (tile, head) to arrive, in chunk order.
  wait_stores_performed();
  __syncthreads();
  uint32_t* counter = a.counters + (int64_t)it.first * hk + h;
  if (tid == 0) sm.last = arrive(counter) + 1u == (uint32_t)it.nch;
  __syncthreads();
  if (!sm.last) return;
  if (tid == 0) reset_counter(counter);
  constexpr int DP = D / 4;                                  // 16-byte parts of a row
  // One chunk's (M, L) of a row, and 16 bytes of its sums.
  auto load_ml = [&](int64_t row) {
    return __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, (int)((row + D) * 4), 0, kCachePolicySc1));
  };
  auto part_row = [&](int ch, int row) { return (((int64_t)(it.first + ch) * hk + h) * a.tile_rows + row) * (D + 4); };
  for (int r = 0; r < R; ++r) {
    const int live = min(16, rows - r0 - 16 * r);
    if (live <= 0) break;
    __syncthreads();
    // factors 2^(M_c - M) / L of every chunk, 16 threads per row
    const int frow = tid >> 4, fl = tid & 15;
    if (frow < 16) {
      float M = kNegInf;
      const bool on = frow < live;
      for (int c = fl; on && c < it.nch; c += 16) {
        const f32x2 ml = load_ml(part_row(c, 16 * r + frow));
        M = fmaxf(M, ml.x);
      }
      for (int off = 1; off < 16; off <<= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
      float Ls = 0.0f;
      for (int c = fl; on && c < it.nch; c += 16) {
        const f32x2 ml = load_ml(part_row(c, 16 * r + frow));
        const float f = M == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(ml.x - M);
        sm.f[frow][c] = f;
        Ls = __builtin_fmaf(ml.y, f, Ls);
      }
      for (int off = 1; off < 16; off <<= 1) Ls += __shfl_xor(Ls, off, 64);
      if (on && fl == 0) {
        sm.l[0][frow] = Ls > 0.0f ? 1.0f / Ls : 0.0f;
        if (a.lse) {
          const int grow = r0 + 16 * r + frow;
          a.lse[(int64_t)(it.e.qs + grow / a.G) * a.Hq + h * a.G + grow % a.G] =
              Ls > 0.0f ? (M + __builtin_amdgcn_logf(Ls)) * kLn2 : kNegInf;
        }
      }
    }
    __syncthreads();
    // `groups` threads share one 16-byte part of a row, each a share of the chunks
    const int parts = live * DP;
    const int groups = max(1, NW * 64 / parts);
    f32x4* red = reinterpret_cast<f32x4*>(sm.red);
    for (int p0i = 0; p0i < parts; p0i += NW * 64) {         // one pass unless parts > threads
      const int id = p0i + (groups > 1 ? tid % parts : tid);
      const int grp = groups > 1 ? tid / parts : 0;
      const bool on = id < parts && grp < groups;
      const int row = on ? id / DP : 0, dp = on ? id % DP : 0;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      if (on) {
        const int lo = it.nch * grp / groups, hi = it.nch * (grp + 1) / groups;
#pragma unroll 4
        for (int c = lo; c < hi; ++c) {
          const f32x4 v = load_partial(rs, part_row(c, 16 * r + row) / 4 + dp);
          acc += v * sm.f[row][c];
        }
      }
      if (groups > 1) {
        __syncthreads();
        red[tid] = acc;
        __syncthreads();
        if (on && grp == 0)
          for (int k = 1; k < groups; ++k) acc += red[k * parts + id];
      }
      if (on && grp == 0) {
        const float inv = sm.l[0][row];
        const int grow = r0 + 16 * r + row;
        uint32_t* out = reinterpret_cast<uint32_t*>(
            a.out + ((int64_t)(it.e.qs + grow / a.G) * a.Hq + h * a.G + grow % a.G) * D + dp * 4);
        out[0] = pack_bf16x2(acc.x * inv, acc.y * inv);
        out[1] = pack_bf16x2(acc.z * inv, acc.w * inv);
      }
    }
  }
}

template <int NG, int R, int NW>
hipError_t launch_one(const KvAttnArgs& a, int grid, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr int bytes = (int)sizeof(Smem<NG, NW>);
  static_assert(bytes <= 160 * 1024, "LDS");
  const void* k = reinterpret_cast<const void*>(kv_attention_kernel<NG, R, NW>);
  if (hipError_t e = set_lds_limit(k, bytes, done); e != hipSuccess) return e;
  kv_attention_kernel<NG, R, NW><<<grid, NW * 64, bytes, st>>>(a);
  return hipGetLastError();
}

template <int NG>
hipError_t launch_ng(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t st) {
  switch (p.R) {
    case 1: return launch_one<NG, 1, 8>(a, p.grid, st);
    default: return launch_one<NG, 2, 4>(a, p.grid, st);
  }
}

}  // namespace

KvAttnPlan plan_kv_attention(int64_t T, int64_t B, int64_t Hk, int64_t G, bool one_each) {
  KvAttnPlan p;
  const int64_t rows = one_each ? G : (T + B - 1) / B * G;   // query rows of an average sequence
  p.R = rows <= 16 ? 1 : 2;
  const int64_t TR = 16 * p.R;
  p.waves = p.R == 1 ? 8 : 4;
  // Query tiles: of every sequence together, at most
  const int64_t tiles = one_each ? B * ((G + TR - 1) / TR) : T * G / TR + B;
  // About two workgroups of eight waves per CU; at most 256 chunks of a tile are joined.
  int64_t target = (p.R == 1 ? 512 : 1024) / Hk;
  target = target < 1 ? 1 : target > 256 ? 256 : target;
  p.split = tiles < 4 * target;
  p.target = (int)target;
  p.chunk_step = 32 * p.waves;
  const int64_t items = tiles + (p.split ? target : 0);
  p.grid = (int64_t)((items + 7) / 8 * 8) * Hk;
  p.tile_rows = (int)(one_each && G < TR ? G : TR);
  p.items = items;
  return p;
}

hipError_t launch_kv_attention(const KvAttnArgs& a, const KvAttnPlan& p, int D, hipStream_t st) {
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
