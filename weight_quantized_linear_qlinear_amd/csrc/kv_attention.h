// Building blocks that the two attention kernels over the 8-bit cache share (kv_attention.hip:
// few query rows; kv_attention_tile.hip: many).
#pragma once

#include "qlq_device.h"
#include "qlq_launch.h"

namespace qlq {
namespace attn {


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
// pattern, minus 1152; exact.  With the upper byte of 8 and minus 9, 2^-7 of the codes.
template <bool HI>
__device__ __forceinline__ uint32_t i8x2_to_f16(uint32_t flipped, uint32_t upper = 0x64646464u, float zero = 1152.0f) {
  const uint32_t b = __builtin_amdgcn_perm(upper, flipped, HI ? 0x04030402u : 0x04010400u);
  const f16x2 k = {(_Float16)zero, (_Float16)zero};
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

// Memory that no kernel writes meanwhile, read through the scalar cache.
typedef __attribute__((address_space(4))) const int32_t ConstInt;

// One token's K scales, NG fp16 as raw dwords (aligned to their size's largest power of two).
template <int NG>
struct KScales {
  static constexpr int N = (NG + 1) / 2;
  uint32_t d[N];
  __device__ __forceinline__ void load(const uint16_t* p) {
    if constexpr (NG == 8) {
      const u32x4 v = ld16(p);
      d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
    } else if constexpr (NG == 4) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(p);
      d[0] = v.x, d[1] = v.y;
    } else if constexpr (NG % 2 == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = *reinterpret_cast<const uint32_t*>(p + 2 * i);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = p[2 * i] | (2 * i + 1 < NG ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    }
  }
  __device__ __forceinline__ float get(int i) const { return i & 1 ? f16_hi(d[i / 2]) : f16_lo(d[i / 2]); }
};

// Sequence b: its query tokens and its cached tokens.
struct Extent {
  int qs, nq, L;
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
  return e;
}

// Cross-lane steps in the vector unit (no trip through LDS).
template <int N>
__device__ __forceinline__ int row_ror(int v) {               // within 16 lanes
  return __builtin_amdgcn_mov_dpp(v, 0x120 + N, 0xf, 0xf, true);
}

template <class OP>
__device__ __forceinline__ int row16(int v, OP op) {          // over 16 lanes, to each of them
  v = op(v, row_ror<8>(v));
  v = op(v, row_ror<4>(v));
  v = op(v, row_ror<2>(v));
  return op(v, row_ror<1>(v));
}

template <class OP>
__device__ __forceinline__ int row8(int v, OP op) {           // over 8 lanes, where both halves of 16 hold the same
  v = op(v, row_ror<4>(v));
  v = op(v, row_ror<2>(v));
  return op(v, row_ror<1>(v));
}

template <class OP>
__device__ __forceinline__ int across16(int v, OP op) {       // over lanes l, l ^ 16, l ^ 32, l ^ 48
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = op((int)a[0], (int)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return op((int)b[0], (int)b[1]);
}

struct AddI {
  __device__ __forceinline__ int operator()(int a, int b) const { return a + b; }
};
struct AddF {
  __device__ __forceinline__ int operator()(int a, int b) const {
    return __builtin_bit_cast(int, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
  }
};
struct MaxF {
  __device__ __forceinline__ int operator()(int a, int b) const {
    return __builtin_bit_cast(int, fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
  }
};
struct MaxU16 {                                               // both halves on their own
  __device__ __forceinline__ int operator()(int a, int b) const {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(int, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
  }
};

__device__ __forceinline__ float max_across16(float v) {
  return __builtin_bit_cast(float, across16(__builtin_bit_cast(int, v), MaxF()));
}
__device__ __forceinline__ float sum_across16(float v) {
  return __builtin_bit_cast(float, across16(__builtin_bit_cast(int, v), AddF()));
}
__device__ __forceinline__ float max_row16(float v) {
  return __builtin_bit_cast(float, row16(__builtin_bit_cast(int, v), MaxF()));
}
__device__ __forceinline__ float sum_row16(float v) {
  return __builtin_bit_cast(float, row16(__builtin_bit_cast(int, v), AddF()));
}

__device__ __forceinline__ int wave_sum(int v) { return across16(row16(v, AddI()), AddI()); }
__device__ __forceinline__ int wave_scan(int v) {             // inclusive
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);    // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast 15 into rows 1, 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast 31 into rows 2, 3
  return v;
}

// W floats (2, or a multiple of 4) to a partial row at float offset `at`.
template <int W>
__device__ __forceinline__ void store_run(__amdgpu_buffer_rsrc_t rs, int64_t at, const float* v) {
  if constexpr (W == 2) {
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, (f32x2){v[0], v[1]}), rs, (int)(at * 4), 0, kCachePolicySc1);
  } else {
#pragma unroll
    for (int e = 0; e < W; e += 4) store_partial(rs, (at + e) / 4, (f32x4){v[e], v[e + 1], v[e + 2], v[e + 3]});
  }
}

// W values (even) times f to bf16 at p.
template <int W>
__device__ __forceinline__ void store_out(uint16_t* p, const float* v, float f) {
  uint32_t d[W / 2];
#pragma unroll
  for (int e = 0; e < W; e += 2) d[e / 2] = pack_bf16x2(v[e] * f, v[e + 1] * f);
  if constexpr (W == 2) {
    *reinterpret_cast<uint32_t*>(p) = d[0];
  } else if constexpr (W == 4) {
    *reinterpret_cast<u32x2*>(p) = (u32x2){d[0], d[1]};
  } else {
#pragma unroll
    for (int e = 0; e < W / 2; e += 4) st16(p + 2 * e, (u32x4){d[e], d[e + 1], d[e + 2], d[e + 3]});
  }
}

// Order within a wave: its LDS writes before its reads.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A line of work is cut into equal runs of units, one per part; a tile that parts share is cut
// into chunks, one per part.  A part has at most two chunks of shared tiles: the tile that began
// before it (slot 2 p) and the one that goes on after it (2 p + 1).
struct Chunks {
  int first, count, mine;        // part of chunk 0, chunks, this part's chunk
  __device__ __forceinline__ int slot(int c) const { return 2 * (first + c) + (c == 0 ? 1 : 0); }
};

constexpr int kJoin = 16;        // chunks joined at a time
struct JoinLds {
  float f[16][kJoin];            // factors by row and chunk
  float inv[16];                 // a row's reciprocal sum
};

// Joins n <= N chunks' partial rows, chunk_of(0) on, into the output (done) or the first one's.
template <int D, int N, int NP, class ChunkOf, class PartRow, class OutRow>
__device__ __forceinline__ void join_group(const KvAttnArgs& a, __amdgpu_buffer_rsrc_t rs, JoinLds& mine, int lane,
                                           int rows, int n, bool done, ChunkOf chunk_of, PartRow part_row,
                                           OutRow out_row) {
  const int c16 = lane & 15, g4 = lane >> 4;
  for (int r = 0; 16 * r < rows; ++r) {
    const int live = min(16, rows - 16 * r);
    wave_sync();
    // 64 lanes over (row, 16-byte part); NP passes' loads at a time, the first ahead of the factors
    constexpr int DP = D / 4;
    const int parts = live * DP;
    f32x4 v[NP][N];
    auto load_parts = [&](int b) {
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int id = min(b + 64 * k + lane, parts - 1), row = id / DP, dp = id % DP;
#pragma unroll
        for (int c = 0; c < N; ++c) v[k][c] = load_partial(rs, part_row(chunk_of(min(c, n - 1)), 16 * r + row) / 4 + dp);
      }
    };
    // factors 2^(M_c - M) of the chunks: four rows at a time, 16 lanes (chunks) per row
    f32x2 ml[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t p = part_row(chunk_of(min(c16, n - 1)), 16 * r + min(4 * q + g4, live - 1));
      ml[q] = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, (int)((p + D) * 4), 0, kCachePolicySc1));
    }
    load_parts(0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int row = 4 * q + g4;
      if (4 * q >= live) break;                              // uniform
      if (c16 >= n) ml[q] = (f32x2){kNegInf, 0.0f};
      const float M = max_row16(ml[q].x);
      const float f = M == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(ml[q].x - M);
      const float L = sum_row16(ml[q].y * f);
      mine.f[row][c16] = f;
      if (c16 == 0) {
        mine.inv[row] = L == 0.0f ? 0.0f : 1.0f / L;       // (NaN stays NaN)
        if (row < live) {
          if (!done) {
            const float out[2] = {M, L};
            store_run<2>(rs, part_row(chunk_of(0), 16 * r + row) + D, out);
          } else if (a.lse) {
            a.lse[out_row(16 * r + row)] = L == 0.0f ? kNegInf : (M + __builtin_amdgcn_logf(L)) * kLn2;
          }
        }
      }
    }
    wave_sync();
    for (int b = 0; b < parts; b += 64 * NP) {
      if (b) load_parts(b);
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int id = b + 64 * k + lane, row = min(id, parts - 1) / DP, dp = id % DP;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < N; ++c) sum += v[k][c] * mine.f[row][c];   // f is 0 past the last
        if (id < parts) {
          if (done) {
            const float inv = mine.inv[row];
            uint32_t* out = reinterpret_cast<uint32_t*>(a.out + out_row(16 * r + row) * D + dp * 4);
            out[0] = pack_bf16x2(sum.x * inv, sum.y * inv);
            out[1] = pack_bf16x2(sum.z * inv, sum.w * inv);
          } else {
            store_partial(rs, part_row(chunk_of(0), 16 * r + row) / 4 + dp, sum);
          }
        }
      }
    }
  }
}

// Joins the chunks of `rows` rows of a tile, kJoin at a time, then those groups, and so on: the
// last wave of a group to finish joins it (always in chunk order) into the group's first partial
// rows, the last group of all into the output.  A partial row is [D sums][M, L, -, -], row
// part_row(c, row) of the partial region; its stores were made by this wave before the call.
// counter_of(level, c): this wave's arrival counter of the group that chunk c leads.
template <int D, bool FEW, class PartRow, class OutRow, class CounterOf>
__device__ __forceinline__ void join_chunks(const KvAttnArgs& a, __amdgpu_buffer_rsrc_t rs, JoinLds& mine, int lane,
                                            const Chunks& ck, int rows, PartRow part_row, OutRow out_row,
                                            CounterOf counter_of) {
  for (int level = 0, stride = 1;; ++level, stride *= kJoin) {
    const int ch0 = ck.mine - ck.mine % (stride * kJoin);
    const int n = min(kJoin, (ck.count - ch0 + stride - 1) / stride);
    const bool done = stride * kJoin >= ck.count;                 // one group: joins into the output
    wait_stores_performed();
    uint32_t* counter = a.counters + counter_of(level, ch0);
    int last = 0;
    if (lane == 0) {
      last = arrive(counter) + 1u == (uint32_t)n;
      if (last) reset_counter(counter);
    }
    if (!__builtin_amdgcn_readfirstlane(last)) return;
    // Two to four chunks (a prompt's query tiles, mostly) are not read as kJoin: 62 -> 49 us for a
    // prompt of 512 tokens in 32 heads of 128.  Not for short rows (see the few-row kernel's call).
    if (FEW && n <= 4) join_group<D, 4, 3>(a, rs, mine, lane, rows, n, done, [&](int c) { return ch0 + c * stride; }, part_row, out_row);
    else join_group<D, kJoin, 2>(a, rs, mine, lane, rows, n, done, [&](int c) { return ch0 + c * stride; }, part_row, out_row);
    if (done) return;
  }
}

}  // namespace attn
}  // namespace qlq

