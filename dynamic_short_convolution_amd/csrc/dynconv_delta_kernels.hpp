// Chunked gated delta rule, gfx950. Per value head, with a_t = exp(g_t) and unit or raw q, k:
//
//   S_t = a_t S_{t-1} + k_t u_t^T,  u_t = beta_t (v_t - a_t S_{t-1}^T k_t),  o_t = scale S_t^T q_t.
//
// Over a chunk of 64 tokens with G_i the sum of g up to token i, Gam_ij = exp(G_i - G_j) for
// i >= j, E_i = exp(G_i), D_j = exp(G_63 - G_j), gamma = exp(G_63) and S0 the state before it:
//
//   A_ij = beta_i Gam_ij k_i.k_j (i > j),   T = (I + A)^-1,
//   Z = V - E (K S0),   U = T (beta Z),
//   O = scale (E (Q S0) + (Gam o Q K^T) U),   S1 = gamma S0 + K^T (D U).
//
// A document start (packed sequences), or a decay so small that exp(g) is 0 in float32, cuts
// every path across it: Gam_ij, E_i, D_j and gamma are 0 where one lies between.
//
// Work split. T, the only part with a serial inner dependence, does not involve the state: one
// workgroup per (sequence, head, chunk) forms it (k_delta_prep). The state is carried by
// k_delta_scan, one wave per 16 value columns: a matrix-core result holds rows 4q .. 4q+3 of
// column lane % 16, which is what the next product takes as its right operand once the
// contraction index is taken in the order (4q .. 4q+3 of one 16-row tile, then of the next);
// so S0, Z, U and S1 of a wave's columns stay in its registers from product to product, and
// only K, Q, T (left operands, shared by the workgroup's waves) pass through LDS.
//
// Precision. The matrix cores take bf16; a float32 operand enters as three terms of 8 bits
// (mantissa cut into pieces, exactly x = x0 + x1 + x2), a float16 one as two (exact), a bf16
// one as itself, and the products of terms whose orders add up to more than 2 (two, of at most
// 2^-22 of the factors' product each) are left out. That holds states and sums at float32
// accuracy at 2.7 times the rate of the float32 matrix instructions (6 products for two float32
// operands, 3 for a bf16 one). Operands formed here of products that only reach 16-bit results
// have two terms (P, U, Y, Yk rounded to nearest, at most 2^-17 off; S0 the first two of its three,
// 2^-15), and the product of two second terms (at most 2^-15) is left out: a third term would add
// half as many products again and LDS that the kernels do not have, to results that are themselves
// rounded to 2^-9 or 2^-12 (root mean square against 64 bits, relative to that of rounding the exact
// result: bf16 1.00001, float16 1.0004).
#pragma once

#include "dynconv_common.hpp"
#include "dynconv_delta_internal.hpp"

namespace dynconv {
namespace delta {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

constexpr int C = kDeltaChunk;
constexpr int kLdsBytes = 160 * 1024;

template <typename ET>
struct Store;  // terms of a stored element, and of an operand that only reaches stored results
template <>
struct Store<bf16_t> {
  static constexpr int NT = 1, NP = 2;
};
template <>
struct Store<f16_t> {
  static constexpr int NT = 2, NP = 2;
};
template <>
struct Store<float> {
  static constexpr int NT = 3, NP = 3;
};

// N terms of 8 values each: values 0..3 of the first 16-row tile, 4..7 of the second.
template <int N>
struct Frag {
  u32x4 t[N];
};

// The lane, as a value that the compiler cannot see through: addresses derived from it are
// formed anew where they are used. Left alone, it hoists every lane-dependent LDS and memory
// offset of a chunk's work out of the loop over chunks, and the registers that hold them over
// all of it push the work's own values out.
__device__ __forceinline__ int fresh_lane() {
  int l = int(threadIdx.x & 63);
  asm volatile("" : "+v"(l));
  return l;
}

// Keeps the scheduler from moving anything across: products are written with the next
// fragments' LDS reads ahead of the current ones' matrix instructions, and left alone the
// scheduler sinks every read to its use (read, wait 130 cycles, 3 matrix instructions, ...).
#define DELTA_FENCE() __builtin_amdgcn_sched_barrier(0)

// c += sum over terms (i, j) with i + j <= L of a_i b_j.
template <int L, int NA, int NB>
__device__ __forceinline__ void mma(f32x4_t& c, const Frag<NA>& a, const Frag<NB>& b) {
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j <= L)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.t[i]),
                                                    __builtin_bit_cast(bf16x8_t, b.t[j]), c, 0, 0, 0);
}

// The same for M tiles with one right operand, tiles innermost (independent accumulators).
template <int L, int M, int NA, int NB>
__device__ __forceinline__ void mma_tiles(f32x4_t* c, const Frag<NA>* a, const Frag<NB>& b) {
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j <= L) {
#pragma unroll
        for (int m = 0; m < M; ++m)
          c[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a[m].t[i]),
                                                         __builtin_bit_cast(bf16x8_t, b.t[j]), c[m], 0, 0, 0);
      }
}

__device__ __forceinline__ uint32_t top2(float lo, float hi) {  // upper halves of two floats
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ float below(float x) {  // x without its first 8 significant bits, exact
  return x - __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}

// The next of N terms of 4 values; x keeps what is left (exact). Three terms hold a float32 whole,
// so they are cut off, which is the shorter chain (rounding them too: prefill of 32768 tokens 693
// to 731 us). Two leave something out and are rounded to nearest, so that it has either sign (cut
// off, float16 outputs came out 2^-15 too small on average, and every workload took the same time
// within 1 %).
template <int N, bool LAST>
__device__ __forceinline__ u32x2 next_term(f32x4_t& x) {
  if constexpr (N < 3) {
    const u32x2 w = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
    if constexpr (!LAST) x -= f32x4_t{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
    return w;
  } else {
    const u32x2 w = {top2(x[0], x[1]), top2(x[2], x[3])};
    if constexpr (!LAST) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = below(x[e]);
    }
    return w;
  }
}

template <int N>
__device__ __forceinline__ Frag<N> split8(f32x4_t a, f32x4_t b) {
  Frag<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const u32x2 u = n + 1 < N ? next_term<N, false>(a) : next_term<N, true>(a);
    const u32x2 v = n + 1 < N ? next_term<N, false>(b) : next_term<N, true>(b);
    f.t[n] = u32x4{u[0], u[1], v[0], v[1]};
  }
  return f;
}

// Row-major LDS matrices keep each 32-column block in fragment order: columns 4q .. 4q+3 at
// place 8q, columns 16 + 4q .. at place 8q + 4, so a left operand's 8 values are one 16-byte
// read. Place of column c (the first of 4 when c is a multiple of 4).
__device__ __forceinline__ constexpr int place(int c) {
  return (c & ~31) + 2 * (c & 12) + ((c & 16) >> 2) + (c & 3);
}

// Left operand of tile row0 .. row0+15: contraction over columns col0 .. col0+31. Planes
// (terms) lie `plane` elements apart.
template <int N>
__device__ __forceinline__ Frag<N> rowfrag(const uint16_t* m, int ld, int plane, int row0, int col0, int ln) {
  const uint16_t* p = m + (row0 + (ln & 15)) * ld + col0 + 8 * (ln >> 4);
  Frag<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) f.t[n] = *reinterpret_cast<const u32x4*>(p + n * plane);
  return f;
}

// The transposed operand: index col0 + lane % 16 (col0 a multiple of 16), contraction over rows
// row0 .. row0+31. A 16-lane group's transposing read returns to lane i element i % 4 of what
// lanes i / 4 + 4e loaded, so lane j loads row 4q + j / 4, columns 4 (j % 4) .. + 3 of the
// tile. PLAIN: the matrix' columns are in their own order.
template <int N, bool PLAIN = false>
__device__ __forceinline__ Frag<N> colfrag(const uint16_t* m, int ld, int plane, int row0, int col0, int ln) {
  const int q = ln >> 4, j = ln & 15;
  const int c = PLAIN ? col0 + 4 * (j & 3) : place(col0) + 8 * (j & 3);
  const uint16_t* p = m + (row0 + 4 * q + (j >> 2)) * ld + c;
  Frag<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + n * plane));
    const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + n * plane + 16 * ld));
    const u32x2 ua = __builtin_bit_cast(u32x2, a), ub = __builtin_bit_cast(u32x2, b);
    f.t[n] = u32x4{ua[0], ua[1], ub[0], ub[1]};
  }
  return f;
}

// acc[m] += rows 16m .. 16m+15 of a [64][32 KB] matrix times b, m = 0..3. `f` holds the
// fragments of block 0; those of block kb + 1 are read while block kb's products run, and
// `next` issues the following product's reads before the last ones.
template <int L, int KB, int NA, int NB, typename Next>
__device__ __forceinline__ void row_product(f32x4_t* acc, Frag<NA>* f, const uint16_t* m, int ld, int plane,
                                            const Frag<NB>* b, Next next, int ln) {
  Frag<NA> g[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) g[0][i] = f[i];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    if (kb + 1 < KB) {
#pragma unroll
      for (int i = 0; i < 4; ++i) g[(kb + 1) & 1][i] = rowfrag<NA>(m, ld, plane, 16 * i, 32 * (kb + 1), ln);
    } else {
      next();
    }
    DELTA_FENCE();
    mma_tiles<L, 4>(acc, g[kb & 1], b[kb]);
    DELTA_FENCE();
  }
}
template <int NA>
__device__ __forceinline__ void row_load(Frag<NA>* f, const uint16_t* m, int ld, int plane, int ln) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = rowfrag<NA>(m, ld, plane, 16 * i, 0, ln);
}

// acc[i] += transposed rows of a [64][16 N] matrix times b: acc[i] takes columns 16i .. 16i+15,
// contraction over the 64 rows. Four column tiles (independent accumulators) of one 32-row
// block at a time, the next reads ahead.
template <int NA>
__device__ __forceinline__ void col_load(Frag<NA>* f, const uint16_t* m, int ld, int plane, int kb, int i0, int ln) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = colfrag<NA>(m, ld, plane, 32 * kb, 16 * (i0 + i), ln);
}
template <int L, int N, int NA, int NB, typename Next>
__device__ __forceinline__ void col_product(f32x4_t* acc, Frag<NA>* f, const uint16_t* m, int ld, int plane,
                                            const Frag<NB>* b, Next next, int ln) {
  Frag<NA> g[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) g[0][i] = f[i];
#pragma unroll
  for (int s = 0; s < N / 2; ++s) {  // step s: block s % 2 of tiles 4 (s / 2) ..
    if (s + 1 < N / 2) {
      col_load<NA>(g[(s + 1) & 1], m, ld, plane, (s + 1) & 1, (s + 1) / 2 * 4, ln);
    } else {
      next();
    }
    DELTA_FENCE();
    mma_tiles<L, 4>(acc + s / 2 * 4, g[s & 1], b[s & 1]);
    DELTA_FENCE();
  }
}

// A 16-byte read is served in passes of lanes 0-7 with 16-23, 8-15 with 24-31, ... over 256
// bytes: 8 rows at two neighbouring 16-byte places. Row pitches are therefore an odd multiple
// of 32 bytes (16 elements), which puts the 8 rows on the 8 even places.
constexpr int kPad = 16;

// LDS image of a lower-triangular matrix: rows 0..31 of 40 elements (32 used), rows 32..63 of
// 72 (the full padding would not let two workgroups of the backward scans share a CU's LDS).
constexpr int kLdA = 32 + 8, kLdB = 64 + 8, kTrapLo = 32 * kLdA, kTrapHi = 32 * kLdB;
constexpr int kTrapLds = kTrapLo + kTrapHi;
__device__ __forceinline__ constexpr int trap_off(int i) { return i < 32 ? i * kLdA : kTrapLo + (i - 32) * kLdB; }
template <int N>
__device__ __forceinline__ Frag<N> trap_row(const uint16_t* m, int tile, int kb, int ln) {  // kb <= tile / 2
  return tile < 2 ? rowfrag<N>(m, kLdA, kTrapLds, 16 * tile, 0, ln)
                  : rowfrag<N>(m + kTrapLo, kLdB, kTrapLds, 16 * tile - 32, 32 * kb, ln);
}
template <int N>
__device__ __forceinline__ Frag<N> trap_col(const uint16_t* m, int tile, int kb, int ln) {  // kb >= tile / 2
  return kb == 0 ? colfrag<N>(m, kLdA, kTrapLds, 0, 16 * tile, ln) : colfrag<N>(m + kTrapLo, kLdB, kTrapLds, 0, 16 * tile, ln);
}
// The same for an upper-triangular matrix: rows 0..31 of 72 (64 used), rows 32..63 of 40
// (columns 32..63).
__device__ __forceinline__ constexpr int utrap_off(int i, int j) {
  return i < 32 ? i * kLdB + j : kTrapHi + (i - 32) * kLdA + j - 32;
}
template <int N>
__device__ __forceinline__ Frag<N> utrap_row(const uint16_t* m, int tile, int kb, int ln) {  // kb >= tile / 2
  return tile < 2 ? rowfrag<N>(m, kLdB, kTrapLds, 16 * tile, 32 * kb, ln)
                  : rowfrag<N>(m + kTrapHi, kLdA, kTrapLds, 16 * tile - 32, 0, ln);
}

// Triangular products over the 64-row contraction, fragments of both blocks at once.
template <int N>
struct Trap {
  Frag<N> a[4], b[2];  // block 0 (or the block that all 4 tiles have), and the other two tiles'
};
// lower: tiles 0..3 of block 0, tiles 2, 3 of block 1
template <int N>
__device__ __forceinline__ void trap_load(Trap<N>& t, const uint16_t* m, int ln) {
#pragma unroll
  for (int i = 0; i < 4; ++i) t.a[i] = trap_row<N>(m, i, 0, ln);
  t.b[0] = trap_row<N>(m, 2, 1, ln);
  t.b[1] = trap_row<N>(m, 3, 1, ln);
}
template <int L, int N, int NB>
__device__ __forceinline__ void trap_product(f32x4_t* acc, const Trap<N>& t, const Frag<NB>* x) {
  mma_tiles<L, 4>(acc, t.a, x[0]);
  mma_tiles<L, 2>(acc + 2, t.b, x[1]);
}
// upper (a transposed lower one, or an upper image): tiles 0..3 of block 1, tiles 0, 1 of block 0
template <int N>
__device__ __forceinline__ void trap_load_t(Trap<N>& t, const uint16_t* m, int ln) {
#pragma unroll
  for (int i = 0; i < 4; ++i) t.a[i] = trap_col<N>(m, i, 1, ln);
  t.b[0] = trap_col<N>(m, 0, 0, ln);
  t.b[1] = trap_col<N>(m, 1, 0, ln);
}
template <int N>
__device__ __forceinline__ void utrap_load(Trap<N>& t, const uint16_t* m, int ln) {
#pragma unroll
  for (int i = 0; i < 4; ++i) t.a[i] = utrap_row<N>(m, i, 1, ln);
  t.b[0] = utrap_row<N>(m, 0, 0, ln);
  t.b[1] = utrap_row<N>(m, 1, 0, ln);
}
template <int L, int N, int NB>
__device__ __forceinline__ void utrap_product(f32x4_t* acc, const Trap<N>& t, const Frag<NB>* x) {
  mma_tiles<L, 4>(acc, t.a, x[1]);
  mma_tiles<L, 2>(acc, t.b, x[0]);
}

// Writes 4 consecutive elements' N terms.
template <int N>
__device__ __forceinline__ void put4(uint16_t* p, int plane, f32x4_t x) {
#pragma unroll
  for (int n = 0; n < N; ++n)
    *reinterpret_cast<u32x2*>(p + n * plane) = n + 1 < N ? next_term<N, false>(x) : next_term<N, true>(x);
}

template <typename ET>
__device__ __forceinline__ float ldf(const void* p, int64_t i) {
  if constexpr (sizeof(ET) == 2) {
    return Cvt<ET>::of_bits(static_cast<const uint16_t*>(p)[i]);
  } else {
    return static_cast<const float*>(p)[i];
  }
}
template <typename ET>
__device__ __forceinline__ void stf(void* p, int64_t i, float v) {
  if constexpr (sizeof(ET) == 2) {
    static_cast<uint16_t*>(p)[i] = Cvt<ET>::bits(v);
  } else {
    static_cast<float*>(p)[i] = v;
  }
}

// Global rows of a chunk go through buffer instructions: a uniform descriptor per chunk and
// 32-bit byte offsets (the ABI bounds token strides so that 64 rows stay below 2^31 bytes).
// Loads from outside the descriptor's range return 0 and stores to it are dropped, without a
// branch (a branch around a load makes each wait for the one before) and without a mask per
// row (16 of them held over a chunk spilled scalar registers): the range ends with the last
// row that exists, and lanes of columns that do not start at kNowhere. VEC is only set when
// rows do not overlap (token stride >= row length); the general form masks every element.
constexpr uint32_t kNowhere = 0x80000000u;
template <typename ET, bool VEC>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rsrc(const ET* p, int64_t s1, int rows, int cols) {
  const int range = VEC ? int((uint32_t(rows - 1) * uint32_t(s1) + uint32_t(cols)) * uint32_t(sizeof(ET))) : int(kNowhere);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<ET*>(p), 0, range, 0x00027000);
}
template <typename ET>
__device__ __forceinline__ float buf_ld(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  if constexpr (sizeof(ET) == 2) {
    return Cvt<ET>::of_bits(uint16_t(__builtin_amdgcn_raw_buffer_load_b16(r, int(off), 0, 0)));
  } else {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, int(off), 0, 0));
  }
}
template <typename ET>
__device__ __forceinline__ void buf_st(__amdgpu_buffer_rsrc_t r, uint32_t off, float v) {
  if constexpr (sizeof(ET) == 2) {
    __builtin_amdgcn_raw_buffer_store_b16(Cvt<ET>::bits(v), r, int(off), 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, int(off), 0, 0);
  }
}

// 8 consecutive stored elements of a row, as loaded; elements from `n` on read as zero (VEC:
// `off` alone decides).
template <typename ET>
struct Raw8 {
  u32x4 w[sizeof(ET) / 2];
};
template <typename ET, bool VEC>
__device__ __forceinline__ Raw8<ET> load8(__amdgpu_buffer_rsrc_t rs, uint32_t off, int n) {
  Raw8<ET> r;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < int(sizeof(ET) / 2); ++i)
      r.w[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, int(off) + 16 * i, 0, 0);
  } else {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t o = i < n ? off + i * uint32_t(sizeof(ET)) : kNowhere;
      if constexpr (sizeof(ET) == 2) {
        e[i] = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(rs, int(o), 0, 0));
      } else {
        e[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, int(o), 0, 0);
      }
    }
    if constexpr (sizeof(ET) == 2) {
      r.w[0] = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
    } else {
      r.w[0] = u32x4{e[0], e[1], e[2], e[3]};
      r.w[1] = u32x4{e[4], e[5], e[6], e[7]};
    }
  }
  return r;
}
template <typename ET>
__device__ __forceinline__ void floats8(const Raw8<ET>& r, f32x4_t& a, f32x4_t& b) {
  if constexpr (sizeof(ET) == 2) {
    a = f32x4_t{Cvt<ET>::lo(r.w[0][0]), Cvt<ET>::hi(r.w[0][0]), Cvt<ET>::lo(r.w[0][1]), Cvt<ET>::hi(r.w[0][1])};
    b = f32x4_t{Cvt<ET>::lo(r.w[0][2]), Cvt<ET>::hi(r.w[0][2]), Cvt<ET>::lo(r.w[0][3]), Cvt<ET>::hi(r.w[0][3])};
  } else {
    a = __builtin_bit_cast(f32x4_t, r.w[0]);
    b = __builtin_bit_cast(f32x4_t, r.w[1]);
  }
}
// Its terms, 16 bytes each.
template <typename ET>
__device__ __forceinline__ Frag<Store<ET>::NT> terms8(const Raw8<ET>& r) {
  if constexpr (Store<ET>::NT == 1) {
    Frag<1> f;
    f.t[0] = r.w[0];
    return f;
  } else {
    f32x4_t a, b;
    floats8<ET>(r, a, b);
    return split8<Store<ET>::NT>(a, b);
  }
}

// A [64][DK] tile of q or k rows: loads into registers, then stores its terms to LDS.
template <typename ET, int DK, int NTHR, bool VEC>
struct Tile {
  // (three planes of q and of k with the full padding would not leave room in LDS)
  static constexpr int LD = DK + (Store<ET>::NT < 3 ? kPad : 8), PLANE = C * LD, N = C * DK / 8 / NTHR;
  static_assert(C * DK / 8 % NTHR == 0, "whole passes");
  Raw8<ET> r[N];
  // `base`: the chunk's first element; rows s1 apart; `rows` valid rows, `cols` valid columns
  // (a multiple of 8 with VEC).
  __device__ __forceinline__ void load(const ET* base, int64_t s1, int rows, int cols, int tid) {
    const __amdgpu_buffer_rsrc_t rs = chunk_rsrc<ET, VEC>(base, s1, rows, cols);
    constexpr int STEP = NTHR / (DK / 8);
    const int row = tid / (DK / 8), col = tid % (DK / 8) * 8;
    const uint32_t pitch = uint32_t(s1) * uint32_t(sizeof(ET));
    const int n = cols - col;
    const uint32_t off = n > 0 ? uint32_t(row) * pitch + uint32_t(col) * uint32_t(sizeof(ET)) : kNowhere;
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = load8<ET, VEC>(rs, off + i * STEP * pitch, row + i * STEP < rows ? n : 0);
  }
  __device__ __forceinline__ void store(uint16_t* m, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int idx = tid + i * NTHR;
      const int row = idx / (DK / 8), col = idx % (DK / 8) * 8;
      const Frag<Store<ET>::NT> f = terms8<ET>(r[i]);
      uint16_t* p = m + row * LD + place(col);  // columns col + 4 .. are 8 places on
#pragma unroll
      for (int n = 0; n < Store<ET>::NT; ++n) {
        *reinterpret_cast<u32x2*>(p + n * PLANE) = u32x2{f.t[n][0], f.t[n][1]};
        *reinterpret_cast<u32x2*>(p + n * PLANE + 8) = u32x2{f.t[n][2], f.t[n][3]};
      }
    }
  }
};

// Pointers that come out of the parameter block as generic ones, said to be global: a generic
// ("flat") load also counts as an LDS access, and every LDS wait would wait for it.
template <typename T>
using global_t = __attribute__((address_space(1))) T;
template <typename T>
__device__ __forceinline__ const global_t<T>* in_global(const void* p) {
  return (const global_t<T>*)p;
}
template <typename T>
__device__ __forceinline__ global_t<T>* in_global(void* p) {
  return (global_t<T>*)p;
}

// T's three planes of a chunk, through registers into the padded LDS image.
template <int NTHR>
struct TrapTile {
  static constexpr int TOTAL = 3 * kTrapElems / 8, N = (TOTAL + NTHR - 1) / NTHR;
  u32x4 r[N];
  __device__ __forceinline__ void load(const uint16_t* src, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int idx = tid + i * NTHR;
      r[i] = in_global<u32x4>(src)[min(idx, TOTAL - 1)];
    }
  }
  __device__ __forceinline__ void store(uint16_t* m, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int idx = tid + i * NTHR;
      if (idx >= TOTAL) continue;
      const int plane = idx / (kTrapElems / 8), e = idx % (kTrapElems / 8);
      const int off = e < 128 ? (e >> 2) * kLdA + (e & 3) * 8 : kTrapLo + ((e - 128) >> 3) * kLdB + (e & 7) * 8;
      *reinterpret_cast<u32x4*>(m + plane * kTrapLds + off) = r[i];
    }
  }
};

__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }

// exp(G_i - G_j), 0 across a document start. The cumulated logarithms are pairs of floats, so
// the difference keeps float32 accuracy relative to itself, not to the sums.
__device__ __forceinline__ float gam(float ghi_i, float glo_i, int n_i, float ghi_j, float glo_j, int n_j) {
  const float d = (ghi_i - ghi_j) + (glo_i - glo_j);
  return n_i == n_j ? fast_exp(d) : 0.f;
}

__device__ __forceinline__ f32x4_t ld4(const float* p) { return *reinterpret_cast<const f32x4_t*>(p); }
// A per-token array's values at this lane's rows 16 mt + 4 q .. + 3.
__device__ __forceinline__ void tok_load(f32x4_t* x, const float* arr, int ln) {
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) x[mt] = ld4(arr + 16 * mt + 4 * (ln >> 4));
}
__device__ __forceinline__ f32x4_t zero4() { return f32x4_t{0.f, 0.f, 0.f, 0.f}; }

// The 10 tiles on and below the diagonal, in rows.
__device__ __forceinline__ void tile_of(int t, int& ti, int& tj) {
  ti = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
  tj = t - ti * (ti + 1) / 2;
}

// ---------------------------------------------------------------------------------
// T = (I + A)^-1 and the per-token factors of one chunk
// ---------------------------------------------------------------------------------

constexpr int kInvLd = 68;

// T takes the place of the staged K, which A no longer needs: 38 KiB in all for bf16, four
// workgroups per CU (with a place of its own two, and 166 us instead of 106 for 8192 chunks of
// 128-wide heads).
template <typename ET, int DK>
struct PrepLds {
  static constexpr int K = 0, KBYTES = Store<ET>::NT * Tile<ET, DK, 64, true>::PLANE * 2;
  static constexpr int T = 0, TBYTES = C * kInvLd * 4;
  static constexpr int A = KBYTES > TBYTES ? KBYTES : TBYTES;
  static constexpr int TOK = A + C * kInvLd * 4;
  static constexpr int BYTES = TOK + kTokArrays * C * 4;
};

// The inverse in float32: each wave inverts one 16 x 16 diagonal block by forward substitution
// (one column per lane), then block diagonal d = 1, 2, 3 follows as
// T_ij = -T_ii sum_{j <= k < i} A_ik T_kj on the float32 matrix instructions, whose result
// layout is again their right operand's. Bound by the latency of its short serial phases, which
// the CU's other workgroups hide in part: 102 us for 8192 chunks, of which the 0.3 GB it moves
// would take 61 at the rate of a copy.
template <typename ET, int DK, bool VEC>
__global__ __launch_bounds__(256) void k_delta_prep(const DeltaParams p) {
  using L = PrepLds<ET, DK>;
  using TK = Tile<ET, DK, 256, VEC>;
  static_assert(L::BYTES <= kLdsBytes, "LDS of a CU");
  extern __shared__ __align__(16) char lds[];
  uint16_t* sK = reinterpret_cast<uint16_t*>(lds + L::K);
  float* sA = reinterpret_cast<float*>(lds + L::A);
  float* sT = reinterpret_cast<float*>(lds + L::T);
  float* tok = reinterpret_cast<float*>(lds + L::TOK);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, n16 = lane & 15, ln = lane;
  const int64_t ci = blockIdx.x;
  const int c = int(ci % p.nC);
  const int hv = int(ci / p.nC % p.Hv);
  const int b = int(ci / p.nC / p.Hv);
  const int hk = hv / p.group;
  const int t0 = c * C, rows = min(C, p.T - t0);

  // every load that the first phase needs, before it waits for one
  TK tk, tq;
  tk.load(static_cast<const ET*>(p.k) + b * p.ks0 + hk * p.ks2 + t0 * p.ks1, p.ks1, rows, p.dkn, tid);
  if (p.eps >= 0.f)
    tq.load(static_cast<const ET*>(p.q) + b * p.qs0 + hk * p.qs2 + t0 * p.qs1, p.qs1, rows, p.dkn, tid);
  float g = 0.f, bt = 0.f;
  bool cut = false;
  if (wave == 0 && lane < rows) {
    const int t = t0 + lane;
    g = p.g[b * p.gs0 + t * p.gs1 + hv * p.gs2];
    bt = ldf<ET>(p.beta, b * p.bs0 + t * p.bs1 + hv * p.bs2);
    if (p.seg != nullptr && t > 0) {
      const int32_t* sg = p.seg + b * p.ss0;
      cut = sg[t * p.ss1] != sg[(t - 1) * p.ss1];
    }
  }
  // (rows behind the last token are zeros: no length to divide by)
  auto norms = [&](const TK& t, float* out) {
#pragma unroll
    for (int i = 0; i < TK::N; ++i) {
      f32x4_t x, y;
      floats8<ET>(t.r[i], x, y);
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) s += x[e] * x[e] + y[e] * y[e];
#pragma unroll
      for (int m = 1; m < DK / 8; m <<= 1) s += __shfl_xor(s, m);
      const int idx = tid + i * 256, row = idx / (DK / 8);
      if (idx % (DK / 8) == 0) out[row] = p.eps < 0.f || row >= rows ? 1.f : 1.f / sqrtf(s + p.eps);
    }
  };
  norms(tk, tok + kTokRk * C);
  tk.store(sK, tid);
  if (p.eps < 0.f) {
    if (tid < C) tok[kTokRq * C + tid] = 1.f;
  } else {
    norms(tq, tok + kTokRq * C);
  }
  if (wave == 0) {
    // exp is 0 in float32 below 2^-150: such a token keeps nothing of what came before it
    if (g <= -103.972084f) cut = true;
    if (cut) g = 0.f;
    const unsigned long long mask = __ballot(cut);
    const int cnt = __popcll(mask & ((2ull << lane) - 1ull));
    double G = g;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double o = __shfl_up(G, m);
      if (lane >= m) G += o;
    }
    const double GC = __shfl(G, 63);
    const int cntC = __popcll(mask);
    const float hi = float(G);
    tok[kTokGhi * C + lane] = hi;
    tok[kTokGlo * C + lane] = float(G - double(hi));
    tok[kTokE * C + lane] = cnt == 0 ? expf(hi) : 0.f;
    tok[kTokD * C + lane] = cnt == cntC ? expf(float(GC - G)) : 0.f;
    tok[kTokN * C + lane] = __int_as_float(cnt);
    tok[kTokBeta * C + lane] = bt;
  }
  __syncthreads();

  // A, tile by tile: rows i = 4q .. 4q+3, column j = lane % 16
  for (int t = wave; t < 10; t += 4) {
    int ti, tj;
    tile_of(t, ti, tj);
    f32x4_t acc = zero4();
#pragma unroll
    for (int kb = 0; kb < DK / 32; ++kb) {
      const auto fa = rowfrag<Store<ET>::NT>(sK, TK::LD, TK::PLANE, 16 * ti, 32 * kb, ln);
      const auto fb = rowfrag<Store<ET>::NT>(sK, TK::LD, TK::PLANE, 16 * tj, 32 * kb, ln);
      mma<2>(acc, fa, fb);
    }
    const int j = 16 * tj + n16;
    const float gh = tok[kTokGhi * C + j], gl = tok[kTokGlo * C + j], rkj = tok[kTokRk * C + j];
    const int nj = __float_as_int(tok[kTokN * C + j]);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * ti + 4 * q + r;
      float a = 0.f;
      if (i > j) {
        a = acc[r] * rkj * tok[kTokRk * C + i] * tok[kTokBeta * C + i] *
            gam(tok[kTokGhi * C + i], tok[kTokGlo * C + i], __float_as_int(tok[kTokN * C + i]), gh, gl, nj);
      }
      sA[i * kInvLd + j] = a;
    }
  }
  __syncthreads();
  {
    const float* a = sA + 16 * wave * kInvLd + 16 * wave;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == n16 ? 1.f : 0.f;
#pragma unroll
      for (int k = 0; k < i; ++k) s -= a[i * kInvLd + k] * x[k];
      x[i] = s;
    }
    if (q == 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sT[(16 * wave + i) * kInvLd + 16 * wave + n16] = x[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int d = 1; d < 4; ++d) {
    if (wave < 4 - d) {
      const int tj = wave, ti = wave + d;
      f32x4_t acc = zero4();
      for (int k = tj; k < ti; ++k) {
        const f32x4_t a = ld4(sA + (16 * ti + n16) * kInvLd + 16 * k + 4 * q);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], sT[(16 * k + 4 * q + r) * kInvLd + 16 * tj + n16], acc, 0, 0, 0);
      }
      const f32x4_t a = ld4(sT + (16 * ti + n16) * kInvLd + 16 * ti + 4 * q);
      f32x4_t res = zero4();
#pragma unroll
      for (int r = 0; r < 4; ++r) res = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], acc[r], res, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) sT[(16 * ti + 4 * q + r) * kInvLd + 16 * tj + n16] = -res[r];
    }
    __syncthreads();
  }
  uint16_t* wT = p.wT + ci * (3 * kTrapElems);
  for (int e = tid; e < kTrapElems / 8; e += 256) {
    const int row = e < 128 ? e >> 2 : 32 + ((e - 128) >> 3);
    // the 8 values at places 8 k .. of the row, in fragment order; zeros above the diagonal tiles
    const int k = e < 128 ? e & 3 : (e - 128) & 7, col = 32 * (k >> 2) + 4 * (k & 3);
    f32x4_t x = zero4(), y = zero4();
    if ((col >> 4) <= (row >> 4)) x = ld4(sT + row * kInvLd + col);
    if ((col >> 4) + 1 <= (row >> 4)) y = ld4(sT + row * kInvLd + col + 16);
    const Frag<3> f = split8<3>(x, y);
#pragma unroll
    for (int n = 0; n < 3; ++n) reinterpret_cast<u32x4*>(wT + n * kTrapElems)[e] = f.t[n];
  }
  float* wTok = p.wTok + ci * (kTokArrays * C);
  for (int e = tid; e < kTokArrays * C / 4; e += 256)
    reinterpret_cast<f32x4_t*>(wTok)[e] = reinterpret_cast<const f32x4_t*>(tok)[e];
}

// ---------------------------------------------------------------------------------
// Forward scan over the chunks of one (sequence, value head), 16 columns per wave
// ---------------------------------------------------------------------------------

constexpr int kScanWaves = 4;  // 16-column groups of a scan's workgroup

template <typename ET, int DK, bool STATES>
struct ScanLds {
  static constexpr int NT = Store<ET>::NT, NP = Store<ET>::NP;
  static constexpr int K = 0;
  static constexpr int Q = K + NT * Tile<ET, DK, 64, true>::PLANE * 2;
  static constexpr int T = Q + (STATES ? 0 : NT * Tile<ET, DK, 64, true>::PLANE * 2);
  static constexpr int P = T + 3 * kTrapLds * 2;
  static constexpr int TOK = P + (STATES ? 0 : NP * kTrapLds * 2);
  // Two waves per 16 columns (see delta_scan) and what one hands the other: S0's and U's terms
  static constexpr bool PAIR = !STATES && NT < 3;
  static constexpr int HS = TOK + kTokArrays * C * 4, HSW = DK / 32 * NP * 1024;  // per wave
  static constexpr int HU = HS + (PAIR ? kScanWaves * HSW : 0), HUW = 2 * NP * 1024;
  static constexpr int BYTES = HU + (PAIR ? kScanWaves * HUW : 0);
  static constexpr int THREADS = 64 * kScanWaves * (PAIR ? 2 : 1);
};

__device__ __forceinline__ int delta_cols(const DeltaParams& p, int nw) { return (p.nCG + nw - 1) / nw; }

// The 16 values of a wave's column in a chunk: token 16 mt + 4 q + r in v[4 mt + r].
// `base`: the chunk's first element, `rows` its tokens, `cols` the head's width.
template <typename ET, bool VEC>
__device__ __forceinline__ void load_cols(float* v, const ET* base, int64_t s1, int rows, int col, int cols, int ln) {
  const int q = ln >> 4;
  const __amdgpu_buffer_rsrc_t rs = chunk_rsrc<ET, VEC>(base, s1, rows, cols);
  const uint32_t pitch = uint32_t(s1) * uint32_t(sizeof(ET));
  const uint32_t o0 = col < cols ? 4u * q * pitch + uint32_t(col) * uint32_t(sizeof(ET)) : kNowhere;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int t = 16 * (e >> 2) + (e & 3);
    const uint32_t o = o0 + uint32_t(t) * pitch;
    v[e] = buf_ld<ET>(rs, VEC || (col < cols && t + 4 * q < rows) ? o : kNowhere);
  }
}
template <typename ET, bool VEC>
__device__ __forceinline__ void store_cols(const f32x4_t* v, ET* base, int64_t s1, int rows, int col, int cols, int ln) {
  const int q = ln >> 4;
  const __amdgpu_buffer_rsrc_t rs = chunk_rsrc<ET, VEC>(base, s1, rows, cols);
  const uint32_t pitch = uint32_t(s1) * uint32_t(sizeof(ET));
  const uint32_t o0 = col < cols ? 4u * q * pitch + uint32_t(col) * uint32_t(sizeof(ET)) : kNowhere;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int t = 16 * (e >> 2) + (e & 3);
    const uint32_t o = o0 + uint32_t(t) * pitch;
    buf_st<ET>(rs, VEC || (col < cols && t + 4 * q < rows) ? o : kNowhere, v[e >> 2][e & 3]);
  }
}

// State rows 16 i + 4 q + r of a column, from and to [dk][dv] float32.
template <int DK>
__device__ __forceinline__ void load_state(f32x4_t* S, const float* src, int64_t s2, int dkn, int col, bool ok, int ln) {
  const int q = ln >> 4;
#pragma unroll
  for (int i = 0; i < DK / 16; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * i + 4 * q + r;
      S[i][r] = (src != nullptr && ok && row < dkn) ? in_global<float>(src)[row * s2 + col] : 0.f;
    }
}
template <int DK>
__device__ __forceinline__ void store_state(const f32x4_t* S, float* dst, int64_t s2, int dkn, int col, bool ok, int ln) {
  const int q = ln >> 4;
  if (dst == nullptr || !ok) return;
#pragma unroll
  for (int i = 0; i < DK / 16; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * i + 4 * q + r;
      if (row < dkn) in_global<float>(static_cast<void*>(dst))[row * s2 + col] = S[i][r];
    }
}

// Images of a wave's [rows x 16] matrix: 16 bytes per lane and 16 rows, per 32 rows 128 such
// pieces. Piece (column n, row group q, half h of the 32 rows) is at 32 (n / 4) + 16 h +
// 4 (n % 4) + q: 16 neighbouring ones, taken by 16 lanes into an LDS matrix whose rows are
// columns, 32 bytes modulo 128 apart, fall on all its banks.
// Written once and read once (each is as large as many heads' q, k and v): neither keeps them in
// the caches (training step of packed documents 718 us, 697 with such stores, 684 with such loads
// in the chunk gradients too).
__device__ __forceinline__ int image_piece(int ln) { return 8 * (ln & 12) + 4 * (ln & 3) + (ln >> 4); }
template <int N>
__device__ __forceinline__ void store_image(const f32x4_t* x, float* dst, int ln) {
  auto* d = in_global<f32x4_t>(static_cast<void*>(dst)) + image_piece(ln);
#pragma unroll
  for (int i = 0; i < N; ++i) __builtin_nontemporal_store(x[i], &d[128 * (i >> 1) + 16 * (i & 1)]);
}
template <int N>
__device__ __forceinline__ void load_image(f32x4_t* x, const float* src, int ln) {
  const auto* d = in_global<f32x4_t>(src) + image_piece(ln);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = d[128 * (i >> 1) + 16 * (i & 1)];
}

// Where a workgroup of a scan stands: its column block, segment of chunks, sequence and head.
struct ScanAt {
  int cb, seg;
  int64_t bh;
};
__device__ __forceinline__ ScanAt scan_at(const DeltaParams& p, uint32_t bid, int ncb) {
  ScanAt a;
  a.cb = int(bid % ncb);
  a.seg = int(bid / ncb % p.nSeg);
  a.bh = bid / ncb / p.nSeg;
  return a;
}

// What a scan leaves behind: outputs (kOutputs), the state before each chunk and u for the
// backward (kStates), or the end state of its segment alone (kEnds).
//
// Segments. With few sequences and heads the chunks of one are cut into p.nSeg segments that
// run at the same time. A segment's end state is M S + N in terms of its start state S: a first
// pass (kEnds) carries the value columns from zero (N) and the columns of the unit matrix with
// no values (M, dk more columns), k_delta_join adds the segments up one behind the other, and
// the second pass starts every segment from its own state. The gradient's scan does the same
// in reverse with the transposed M.
// Roles. One wave carries 16 columns of S through K S0, T Z and K^T D U. A sequence and head of
// 128 x 128 has 8 such waves, so a batch that fills the chip has one per SIMD, and a lone wave
// issues an instruction about every 5 cycles. The outputs do not feed the recurrence: where LDS
// allows (16-bit storage), a second wave on the same SIMD forms P, Q S0 and P U from the terms of
// S0 and U that the first leaves in LDS (B8 T4096, 16 heads, bf16: 368 us with one wave, 323 with
// two; 0.7 GB would take 146 at the rate of a copy). What bounds it now is the chain of a chunk
// (barriers, the terms' splits between products): the vector units are busy for 46 % of the
// time, LDS for 45 %, the matrix units for 31 %.
enum { kOutputs = 0, kStates = 1, kEnds = 2 };

// Fragments handed from wave to wave through LDS, 16 bytes per lane and term.
template <int N, int COUNT>
__device__ __forceinline__ void hand_over(char* m, const Frag<N>* f, int ln) {
#pragma unroll
  for (int i = 0; i < COUNT; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) *reinterpret_cast<u32x4*>(m + (i * N + n) * 1024 + ln * 16) = f[i].t[n];
}
template <int N, int COUNT>
__device__ __forceinline__ void take_over(Frag<N>* f, const char* m, int ln) {
#pragma unroll
  for (int i = 0; i < COUNT; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) f[i].t[n] = *reinterpret_cast<const u32x4*>(m + (i * N + n) * 1024 + ln * 16);
}

template <typename ET, int DK, int NW, int MODE, bool VEC>
__device__ __forceinline__ void delta_scan(const DeltaParams p, char* lds, uint32_t bid) {
  constexpr bool STATES = MODE != kOutputs;
  using L = ScanLds<ET, DK, STATES>;
  constexpr bool PAIR = L::PAIR;
  constexpr int NT = L::NT, NP = L::NP, NTHR = L::THREADS, KB = DK / 32;
  static_assert(NW == kScanWaves, "waves of the LDS layout");
  using TK = Tile<ET, DK, NTHR, VEC>;
  static_assert(L::BYTES <= kLdsBytes, "LDS of a CU");
  uint16_t* sK = reinterpret_cast<uint16_t*>(lds + L::K);
  uint16_t* sQ = reinterpret_cast<uint16_t*>(lds + L::Q);
  uint16_t* sT = reinterpret_cast<uint16_t*>(lds + L::T);
  uint16_t* sP = reinterpret_cast<uint16_t*>(lds + L::P);
  float* tok = reinterpret_cast<float*>(lds + L::TOK);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15;
  const int q = lane >> 4;
  int ln = lane;
  const int ncb = delta_cols(p, NW);
  const ScanAt at = scan_at(p, bid, MODE == kEnds ? ncb + DK / kDeltaCols / NW : ncb);
  const bool unit = at.cb >= ncb;  // columns of the unit matrix
  if (MODE == kEnds && (at.seg + 1 == p.nSeg || (unit && at.seg == 0))) return;  // nothing starts from there
  const int cw = PAIR ? wave % NW : wave;
  const int cg = (unit ? at.cb - ncb : at.cb) * NW + cw;
  const int64_t bh = at.bh;
  const int c0 = at.seg * p.segLen, c1 = min(p.nC, c0 + p.segLen);
  const int hv = int(bh % p.Hv), b = int(bh / p.Hv), hk = hv / p.group;
  const int col = unit ? p.dvn : cg * kDeltaCols + n16;  // no value column: values read as zero
  const bool ok = col < p.dvn;
  const ET* kbase = static_cast<const ET*>(p.k) + b * p.ks0 + hk * p.ks2;
  const ET* qbase = static_cast<const ET*>(p.q) + b * p.qs0 + hk * p.qs2;
  const ET* vbase = static_cast<const ET*>(p.v) + b * p.vs0 + hv * p.vs2;
  ET* obase = STATES ? nullptr : static_cast<ET*>(p.out) + b * p.os0 + hv * p.os2;

  if constexpr (!STATES) {
    // the tiles above the diagonal that a 32-wide contraction block still reads
    for (int e = tid; e < NP * 128; e += NTHR) {
      const int n = e >> 7, row = (e >> 2) & 31, part = e & 3;
      const int i = row < 16 ? row : row + 16, j = (row < 16 ? 16 : 48) + 4 * part;
      *reinterpret_cast<u32x2*>(sP + n * kTrapLds + trap_off(i) + place(j)) = u32x2{0u, 0u};
    }
  }

  TK tk, tq;
  TrapTile<NTHR> tt;
  f32x4_t ttok[(kTokArrays * C / 4 + NTHR - 1) / NTHR];
  auto fetch = [&](int c, int tid) {
    const int64_t t0 = int64_t(c) * C;
    const int rows = min(C, p.T - int(t0));
    tk.load(kbase + t0 * p.ks1, p.ks1, rows, p.dkn, tid);
    if constexpr (!STATES) tq.load(qbase + t0 * p.qs1, p.qs1, rows, p.dkn, tid);
    tt.load(p.wT + (bh * p.nC + c) * (3 * kTrapElems), tid);
    const auto* w = in_global<f32x4_t>(p.wTok + (bh * p.nC + c) * (kTokArrays * C));
#pragma unroll
    for (int i = 0; i * NTHR < kTokArrays * C / 4; ++i) ttok[i] = w[min(tid + i * NTHR, kTokArrays * C / 4 - 1)];
  };
  auto stage = [&](int tid) {
    tk.store(sK, tid);
    if constexpr (!STATES) tq.store(sQ, tid);
    tt.store(sT, tid);
#pragma unroll
    for (int i = 0; i * NTHR < kTokArrays * C / 4; ++i)
      if (tid + i * NTHR < kTokArrays * C / 4) reinterpret_cast<f32x4_t*>(tok)[tid + i * NTHR] = ttok[i];
  };
  // P = scale Gam o Q K^T: tiles transposed (rows j, column i), so a lane holds four neighbours
  // of one row of P
  auto pairs = [&] {
    const int q = ln >> 4, n16 = ln & 15;
#pragma unroll
    for (int s = 0; s < (10 + NW - 1) / NW; ++s) {
      const int t = cw + s * NW;
      if (t < 10) {
        int ti, tj;
        tile_of(t, ti, tj);
        Frag<NT> fj[KB], fi[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          fj[kb] = rowfrag<NT>(sK, TK::LD, TK::PLANE, 16 * tj, 32 * kb, ln);
          fi[kb] = rowfrag<NT>(sQ, TK::LD, TK::PLANE, 16 * ti, 32 * kb, ln);
        }
        const int i = 16 * ti + n16, j0 = 16 * tj + 4 * q;
        const float gh = tok[kTokGhi * C + i], gl = tok[kTokGlo * C + i], rqi = tok[kTokRq * C + i] * p.scale;
        const int ni = __float_as_int(tok[kTokN * C + i]);
        const f32x4_t ghj = ld4(tok + kTokGhi * C + j0), glj = ld4(tok + kTokGlo * C + j0);
        const f32x4_t nj = ld4(tok + kTokN * C + j0), rkj = ld4(tok + kTokRk * C + j0);
        DELTA_FENCE();
        f32x4_t acc[2] = {zero4(), zero4()};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) mma<NP - 1>(acc[kb & 1], fj[kb], fi[kb]);
        f32x4_t x;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          x[r] = j0 + r <= i ? (acc[0][r] + acc[1][r]) * rqi * rkj[r] *
                                   gam(gh, gl, ni, ghj[r], glj[r], __float_as_int(nj[r]))
                             : 0.f;
        put4<NP>(sP + trap_off(i) + place(j0), kTrapLds, x);
      }
    }
  };
  // o = scale E (Q S0), s0: its terms
  auto from_state = [&](f32x4_t* o, Frag<NT>* fq, const Frag<NP>* s0) {
    f32x4_t te[4], tr[4];
    row_product<NP - 1, KB>(o, fq, sQ, TK::LD, TK::PLANE, s0, [&] {
      tok_load(te, tok + kTokE * C, ln);
      tok_load(tr, tok + kTokRq * C, ln);
    }, ln);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) o[mt] *= te[mt] * tr[mt] * p.scale;
  };
  // o += P U, and out
  auto finish = [&](f32x4_t* o, const Frag<NP>* uf, int c) {
    Trap<NP> fp;
    trap_load(fp, sP, ln);
    DELTA_FENCE();
    trap_product<NP - 1>(o, fp, uf);
    const int64_t t0 = int64_t(c) * C;
    store_cols<ET, VEC>(o, obase + t0 * p.os1, p.os1, min(C, p.T - int(t0)), col, p.dvn, ln);
  };

  if (c1 > c0) fetch(c0, tid);
  if constexpr (PAIR) {
    if (wave >= NW) {
      const char* hs = lds + L::HS + cw * L::HSW;
      const char* hu = lds + L::HU + cw * L::HUW;
      for (int c = c0; c < c1; ++c) {
        ln = fresh_lane();
        __syncthreads();  // every wave is done with the previous chunk's tiles
        stage(wave * 64 + ln);
        __syncthreads();
        pairs();
        if (c + 1 < c1) fetch(c + 1, wave * 64 + ln);
        __syncthreads();  // P is complete, S0 and U are handed over
        f32x4_t o[4] = {zero4(), zero4(), zero4(), zero4()};
        Frag<NT> fq[4];
        Frag<NP> s0[KB], uf[2];
        row_load<NT>(fq, sQ, TK::LD, TK::PLANE, ln);
        take_over<NP, KB>(s0, hs, ln);
        from_state(o, fq, s0);
        take_over<NP, 2>(uf, hu, ln);
        finish(o, uf, c);
      }
      return;
    }
  }

  if constexpr (PAIR) __builtin_amdgcn_s_setprio(1);  // the chain that sets the time (2 % of it)
  f32x4_t S[DK / 16];
  if (at.seg == 0 && (MODE == kEnds || p.nSeg == 1)) {
    load_state<DK>(S, p.state_in == nullptr ? nullptr : p.state_in + b * p.sis0 + hv * p.sis1, p.sis2, p.dkn, col, ok, ln);
  } else if (MODE == kEnds) {
#pragma unroll
    for (int i = 0; i < DK / 16; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = unit && 16 * i + 4 * q + r == cg * kDeltaCols + n16 ? 1.f : 0.f;
  } else {
    // what the segment before ends in; for the first one the initial state, from where the first
    // pass put it (no segment ends in the last place): another workgroup of this launch writes
    // the final state, which may be in the initial one's memory
    const int from = at.seg == 0 ? p.nSeg - 1 : at.seg - 1;
    load_image<DK / 16>(S, p.wEnd + ((bh * p.nSeg + from) * p.nCG + min(cg, p.nCG - 1)) * (DK * 16), ln);
  }
  if (MODE == kEnds && at.seg == 0 && cg < p.nCG)
    store_image<DK / 16>(S, p.wEnd + ((bh * p.nSeg + p.nSeg - 1) * p.nCG + cg) * (DK * 16), ln);

  for (int c = c0; c < c1; ++c) {
    ln = fresh_lane();
    __syncthreads();  // every wave is done with the previous chunk's tiles
    stage(wave * 64 + ln);
    float v[16];
    {
      const int64_t t0 = int64_t(c) * C;
      load_cols<ET, VEC>(v, vbase + t0 * p.vs1, p.vs1, min(C, p.T - int(t0)), col, p.dvn, ln);
    }
    __syncthreads();

    if constexpr (!STATES && !PAIR) pairs();
    if (MODE == kStates && cg < p.nCG) {
      store_image<DK / 16>(S, p.wS + ((bh * p.nC + c) * p.nCG + cg) * (DK * 16), ln);
    }

    f32x4_t z[4] = {zero4(), zero4(), zero4(), zero4()};  // beta (v - E K S0)
    f32x4_t o[4] = {zero4(), zero4(), zero4(), zero4()};  // the output, where no other wave forms it
    {
      Frag<NT> fk[4];
      f32x4_t te[4], tr[4], tb[4];
      row_load<NT>(fk, sK, TK::LD, TK::PLANE, ln);
      Frag<3> sf[KB];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) sf[kb] = split8<3>(S[2 * kb], S[2 * kb + 1]);
      // for the outputs the first NP of them (a second term rounded for itself: 347 us instead of 337
      // at B8 T4096, and the same errors against 64 bits)
      Frag<NP> so[KB];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int n = 0; n < NP; ++n) so[kb].t[n] = sf[kb].t[n];
      if constexpr (PAIR) hand_over<NP, KB>(lds + L::HS + cw * L::HSW, so, ln);
      row_product<2, KB>(z, fk, sK, TK::LD, TK::PLANE, sf, [&] {
        if constexpr (!STATES && !PAIR) row_load<NT>(fk, sQ, TK::LD, TK::PLANE, ln);
        tok_load(te, tok + kTokE * C, ln);
        tok_load(tr, tok + kTokRk * C, ln);
        tok_load(tb, tok + kTokBeta * C, ln);
      }, ln);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r) z[mt][r] = tb[mt][r] * (v[4 * mt + r] - te[mt][r] * tr[mt][r] * z[mt][r]);
      if constexpr (!STATES && !PAIR) from_state(o, fk, so);
    }
    f32x4_t u[4] = {zero4(), zero4(), zero4(), zero4()};
    const float gamma = tok[kTokE * C + C - 1];
    f32x4_t td[4], trk[4];
    {
      Trap<3> ft;
      trap_load(ft, sT, ln);
      const Frag<3> zf[2] = {split8<3>(z[0], z[1]), split8<3>(z[2], z[3])};
      tok_load(td, tok + kTokD * C, ln);
      tok_load(trk, tok + kTokRk * C, ln);
      DELTA_FENCE();
      trap_product<2>(u, ft, zf);
      DELTA_FENCE();
    }
    if constexpr (MODE == kStates) {
      if (cg < p.nCG) store_image<4>(u, p.wU + ((bh * p.nC + c) * p.nCG + cg) * (C * kDeltaCols), ln);
    }
    const Frag<NP> uf[2] = {split8<NP>(u[0], u[1]), split8<NP>(u[2], u[3])};
    if constexpr (PAIR) {
      hand_over<NP, 2>(lds + L::HU + cw * L::HUW, uf, ln);
      __syncthreads();
    }
    ln = fresh_lane();
    if (c + 1 < c1) fetch(c + 1, wave * 64 + ln);
    {
      Frag<NT> fc[4];
      col_load<NT>(fc, sK, TK::LD, TK::PLANE, 0, 0, ln);
      f32x4_t d[4];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) d[mt] = u[mt] * td[mt] * trk[mt];
      const Frag<3> df[2] = {split8<3>(d[0], d[1]), split8<3>(d[2], d[3])};
#pragma unroll
      for (int i = 0; i < DK / 16; ++i) S[i] *= gamma;
      col_product<2, DK / 16>(S, fc, sK, TK::LD, TK::PLANE, df, [] {}, ln);
    }
    if constexpr (!STATES && !PAIR) {
      __syncthreads();  // P is complete
      finish(o, uf, c);
    }
  }
  if constexpr (MODE == kOutputs) {
    if (at.seg + 1 == p.nSeg)
      store_state<DK>(S, p.state_out == nullptr ? nullptr : p.state_out + b * p.sos0 + hv * p.sos1, p.sos2, p.dkn, col, ok, ln);
  }
  if constexpr (MODE == kEnds) {
    const int64_t seg = bh * p.nSeg + at.seg;
    if (unit) {
      store_state<DK>(S, p.wM + seg * (DK * DK), DK, DK, cg * kDeltaCols + n16, true, ln);
    } else if (cg < p.nCG) {
      store_image<DK / 16>(S, p.wEnd + (seg * p.nCG + cg) * (DK * 16), ln);
    }
  }
}

template <typename ET, int DK, int NW, bool VEC>
__global__ __launch_bounds__((ScanLds<ET, DK, false>::THREADS), 1) void k_delta_scan(const DeltaParams p) {
  extern __shared__ __align__(16) char lds[];
  delta_scan<ET, DK, NW, kOutputs, VEC>(p, lds, xcd_logical_block(blockIdx.x, gridDim.x));
}

// ---------------------------------------------------------------------------------
// Backward: reverse scan of the state's gradient, 16 columns per wave
// ---------------------------------------------------------------------------------
//
// With dS1 the gradient of the state after the chunk and dO that of the outputs:
//   dU  = P^T dO + D (K dS1),   dR = T^T dU,   dV = dZ = beta dR,
//   dS0 = gamma dS1 + scale Q^T (E dO) - K^T (beta E dR),
// all of them column by column, like the forward, and without the states: so this scan and the
// one that carries the states run side by side in one launch, two waves on a SIMD (a lone wave
// issues an instruction about every 5 cycles, two share the SIMD's issue at half that).
// Everything that needs both is left to k_delta_grad, which gets U and S0 from the state scan,
// dR, dS1 and the sums of dR o V over a wave's columns from here.

template <typename ET, int DK>
struct BackLds {
  static constexpr int NT = Store<ET>::NT;
  static constexpr int K = 0;
  static constexpr int Q = K + NT * Tile<ET, DK, 64, true>::PLANE * 2;
  static constexpr int T = Q + NT * Tile<ET, DK, 64, true>::PLANE * 2;
  static constexpr int P = T + 3 * kTrapLds * 2;
  static constexpr int TOK = P + 3 * kTrapLds * 2;
  static constexpr int BYTES = TOK + kTokArrays * C * 4;
};

// Sum over the 16 lanes of a group (DPP operand modifiers), in every lane.
__device__ __forceinline__ float sum16(float x) {
  auto add = [](float v, float o) { return v + o; };
  x = add(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0xB1, 0xf, 0xf, true)));   // lane ^ 1
  x = add(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x4E, 0xf, 0xf, true)));   // lane ^ 2
  x = add(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x141, 0xf, 0xf, true)));  // mirror of 8
  x = add(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x140, 0xf, 0xf, true)));  // mirror of 16
  return x;
}

// ENDS: only the gradient at its segment's start, from zero at the segment's end.
template <typename ET, int DK, int NW, bool ENDS, bool VEC>
__device__ __forceinline__ void delta_back(const DeltaParams p, char* lds, uint32_t bid) {
  using L = BackLds<ET, DK>;
  constexpr int NT = L::NT, NTHR = 64 * NW, KB = DK / 32;
  using TK = Tile<ET, DK, NTHR, VEC>;
  static_assert(L::BYTES <= kLdsBytes, "LDS of a CU");
  uint16_t* sK = reinterpret_cast<uint16_t*>(lds + L::K);
  uint16_t* sQ = reinterpret_cast<uint16_t*>(lds + L::Q);
  uint16_t* sT = reinterpret_cast<uint16_t*>(lds + L::T);
  uint16_t* sP = reinterpret_cast<uint16_t*>(lds + L::P);
  float* tok = reinterpret_cast<float*>(lds + L::TOK);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int ln = lane;
  const int ncb = delta_cols(p, NW);
  const ScanAt at = scan_at(p, bid, ncb);
  if (ENDS && at.seg == 0) return;  // nothing ends there
  const int cg = at.cb * NW + wave;
  const bool live = cg < p.nCG;  // a wave past the last column group still stages tiles
  const int64_t bh = at.bh;
  const int c0 = at.seg * p.segLen, c1 = min(p.nC, c0 + p.segLen);
  const int hv = int(bh % p.Hv), b = int(bh / p.Hv), hk = hv / p.group;
  const ET* kbase = static_cast<const ET*>(p.k) + b * p.ks0 + hk * p.ks2;
  const ET* qbase = static_cast<const ET*>(p.q) + b * p.qs0 + hk * p.qs2;
  const ET* vbase = static_cast<const ET*>(p.v) + b * p.vs0 + hv * p.vs2;
  const ET* dobase = static_cast<const ET*>(p.dO) + b * p.dos0 + hv * p.dos2;
  ET* dvbase = static_cast<ET*>(p.dv) + b * p.dvs0 + hv * p.dvs2;

  f32x4_t dS[DK / 16];
  {
    const int col = cg * kDeltaCols + (lane & 15);
    if (at.seg + 1 == p.nSeg) {
      load_state<DK>(dS, p.dstate_out == nullptr ? nullptr : p.dstate_out + b * p.dsos0 + hv * p.dsos1, p.dsos2, p.dkn,
                     col, col < p.dvn, ln);
    } else if (ENDS) {
#pragma unroll
      for (int i = 0; i < DK / 16; ++i) dS[i] = zero4();
    } else {
      load_image<DK / 16>(dS, p.wBegin + ((bh * p.nSeg + at.seg + 1) * p.nCG + min(cg, p.nCG - 1)) * (DK * 16), ln);
    }
  }
  // the tiles below the diagonal of P^T that a 32-wide contraction block still reads
  for (int e = tid; e < 3 * 128; e += NTHR) {
    const int n = e >> 7, row = (e >> 2) & 31, part = e & 3;
    const int i = row < 16 ? row + 16 : row + 32, j = (row < 16 ? 0 : 32) + 4 * part;
    *reinterpret_cast<u32x2*>(sP + n * kTrapLds + utrap_off(i, place(j))) = u32x2{0u, 0u};
  }

  TK tk, tq;
  TrapTile<NTHR> tt;
  f32x4_t ttok[(kTokArrays * C / 4 + NTHR - 1) / NTHR];
  auto fetch = [&](int c, int tid) {
    const int64_t t0 = int64_t(c) * C;
    const int rows = min(C, p.T - int(t0));
    tk.load(kbase + t0 * p.ks1, p.ks1, rows, p.dkn, tid);
    tq.load(qbase + t0 * p.qs1, p.qs1, rows, p.dkn, tid);
    tt.load(p.wT + (bh * p.nC + c) * (3 * kTrapElems), tid);
    const auto* w = in_global<f32x4_t>(p.wTok + (bh * p.nC + c) * (kTokArrays * C));
#pragma unroll
    for (int i = 0; i * NTHR < kTokArrays * C / 4; ++i) ttok[i] = w[min(tid + i * NTHR, kTokArrays * C / 4 - 1)];
  };
  fetch(c1 - 1, tid);
  for (int c = c1 - 1; c >= c0; --c) {
    ln = fresh_lane();
    const int tid = wave * 64 + ln, q = ln >> 4, n16 = ln & 15;
    const int col = cg * kDeltaCols + n16;
    const int64_t cim = (bh * p.nC + c) * p.nCG + (live ? cg : 0);
    __syncthreads();  // every wave is done with the previous chunk's tiles
    tk.store(sK, tid);
    tq.store(sQ, tid);
    tt.store(sT, tid);
#pragma unroll
    for (int i = 0; i * NTHR < kTokArrays * C / 4; ++i)
      if (tid + i * NTHR < kTokArrays * C / 4) reinterpret_cast<f32x4_t*>(tok)[tid + i * NTHR] = ttok[i];
    float v[16], dO[16];
    const int64_t t0 = int64_t(c) * C;
    const int rows = min(C, p.T - int(t0));
    load_cols<ET, VEC>(dO, dobase + t0 * p.dos1, p.dos1, rows, col, p.dvn, ln);
    if (!ENDS) load_cols<ET, VEC>(v, vbase + t0 * p.vs1, p.vs1, rows, col, p.dvn, ln);
    __syncthreads();

    // P^T: tiles of P = scale Gam o Q K^T (rows i, column j), four neighbours of a row of P^T
#pragma unroll
    for (int s = 0; s < (10 + NW - 1) / NW; ++s) {
      const int t = wave + s * NW;
      if (t < 10) {
        int ti, tj;
        tile_of(t, ti, tj);
        Frag<NT> fj[KB], fi[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          fi[kb] = rowfrag<NT>(sQ, TK::LD, TK::PLANE, 16 * ti, 32 * kb, ln);
          fj[kb] = rowfrag<NT>(sK, TK::LD, TK::PLANE, 16 * tj, 32 * kb, ln);
        }
        const int j = 16 * tj + n16, i0 = 16 * ti + 4 * q;
        const float gh = tok[kTokGhi * C + j], gl = tok[kTokGlo * C + j], rkj = tok[kTokRk * C + j] * p.scale;
        const int nj = __float_as_int(tok[kTokN * C + j]);
        const f32x4_t ghi = ld4(tok + kTokGhi * C + i0), gli = ld4(tok + kTokGlo * C + i0);
        const f32x4_t ni = ld4(tok + kTokN * C + i0), rqi = ld4(tok + kTokRq * C + i0);
        DELTA_FENCE();
        f32x4_t acc[2] = {zero4(), zero4()};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) mma<2>(acc[kb & 1], fi[kb], fj[kb]);
        f32x4_t x;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          x[r] = j <= i0 + r ? (acc[0][r] + acc[1][r]) * rkj * rqi[r] *
                                   gam(ghi[r], gli[r], __float_as_int(ni[r]), gh, gl, nj)
                             : 0.f;
        put4<3>(sP + utrap_off(j, place(i0)), kTrapLds, x);
      }
    }

    ln = fresh_lane();
    const float gamma = tok[kTokE * C + C - 1];
    f32x4_t dU[4] = {zero4(), zero4(), zero4(), zero4()};  // D (K dS1), then dU
    f32x4_t ta[4], tb[4];  // token factors, read anew where they are used: registers are scarce here
    {
      Frag<NT> fk[4];
      row_load<NT>(fk, sK, TK::LD, TK::PLANE, ln);
      if (!ENDS && live) store_image<DK / 16>(dS, p.wdS + cim * (DK * 16), ln);
      Frag<3> sf[KB];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) sf[kb] = split8<3>(dS[2 * kb], dS[2 * kb + 1]);
      row_product<2, KB>(dU, fk, sK, TK::LD, TK::PLANE, sf, [&] {
        tok_load(ta, tok + kTokD * C, ln);
        tok_load(tb, tok + kTokRk * C, ln);
      }, ln);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) dU[mt] *= ta[mt] * tb[mt];
    }
    __syncthreads();  // P^T is complete
    ln = fresh_lane();
    f32x4_t dR[4] = {zero4(), zero4(), zero4(), zero4()};
    {
      Trap<3> ft;
      utrap_load(ft, sP, ln);
      const Frag<NT> of[2] = {split8<NT>(f32x4_t{dO[0], dO[1], dO[2], dO[3]}, f32x4_t{dO[4], dO[5], dO[6], dO[7]}),
                              split8<NT>(f32x4_t{dO[8], dO[9], dO[10], dO[11]}, f32x4_t{dO[12], dO[13], dO[14], dO[15]})};
      DELTA_FENCE();
      utrap_product<2>(dU, ft, of);
      DELTA_FENCE();
      trap_load_t(ft, sT, ln);
      const Frag<3> uf[2] = {split8<3>(dU[0], dU[1]), split8<3>(dU[2], dU[3])};
      DELTA_FENCE();
      utrap_product<2>(dR, ft, uf);
      tok_load(ta, tok + kTokE * C, ln);
      tok_load(tb, tok + kTokBeta * C, ln);
      DELTA_FENCE();
    }
    ln = fresh_lane();
    if (!ENDS && live) store_image<4>(dR, p.wR + cim * (C * kDeltaCols), ln);
    if (c > c0) fetch(c - 1, wave * 64 + ln);
    {
      Frag<NT> fc[4];
      col_load<NT>(fc, sK, TK::LD, TK::PLANE, 0, 0, ln);
      f32x4_t dz[4], tc[4];
      tok_load(tc, tok + kTokRk * C, ln);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        if constexpr (!ENDS) {
          f32x4_t x;
#pragma unroll
          for (int r = 0; r < 4; ++r) x[r] = sum16(dR[mt][r] * v[4 * mt + r]);
          if (live && (ln & 15) == 0) *in_global<f32x4_t>(static_cast<void*>(p.wDot + cim * C + 16 * mt + 4 * (ln >> 4))) = x;
        }
        dz[mt] = dR[mt] * tb[mt];
      }
      if (!ENDS) store_cols<ET, VEC>(dz, dvbase + t0 * p.dvs1, p.dvs1, rows, cg * kDeltaCols + (ln & 15), p.dvn, ln);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) dz[mt] = -(dz[mt] * ta[mt] * tc[mt]);
      const Frag<3> rf[2] = {split8<3>(dz[0], dz[1]), split8<3>(dz[2], dz[3])};
#pragma unroll
      for (int i = 0; i < DK / 16; ++i) dS[i] *= gamma;
      col_product<2, DK / 16>(dS, fc, sK, TK::LD, TK::PLANE, rf, [&] {
        col_load<NT>(fc, sQ, TK::LD, TK::PLANE, 0, 0, ln);
        tok_load(tc, tok + kTokRq * C, ln);
      }, ln);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r) dz[mt][r] = dO[4 * mt + r] * (ta[mt][r] * tc[mt][r] * p.scale);
      const Frag<3> of[2] = {split8<3>(dz[0], dz[1]), split8<3>(dz[2], dz[3])};
      col_product<2, DK / 16>(dS, fc, sQ, TK::LD, TK::PLANE, of, [] {}, ln);
    }
  }
  if (ENDS) {
    if (live) store_image<DK / 16>(dS, p.wBegin + ((bh * p.nSeg + at.seg) * p.nCG + cg) * (DK * 16), ln);
  } else if (at.seg == 0) {
    const int col = cg * kDeltaCols + (ln & 15);
    store_state<DK>(dS, p.dstate == nullptr ? nullptr : p.dstate + b * p.dsis0 + hv * p.dsis1, p.dsis2, p.dkn, col,
                    col < p.dvn, ln);
  }
}

// Both scans of the backward: the first `back` workgroups carry dS, the others S. At B8 T4096, 16
// heads, bf16 707 us; they write 1.7 GB of images and read 0.6 GB, 480 us at the rate of a copy,
// and the CU's vector units are busy for 40 % of the time, LDS for 32 %, the matrix units for 25 %.
template <typename ET, int DK, int NW, bool ENDS, bool VEC>
__global__ __launch_bounds__(64 * NW, Store<ET>::NT == 1 ? 2 : 1) void k_delta_scans(const DeltaParams p, uint32_t back) {
  extern __shared__ __align__(16) char lds[];
  if (blockIdx.x < back) {
    delta_back<ET, DK, NW, ENDS, VEC>(p, lds, xcd_logical_block(blockIdx.x, back));
  } else {
    delta_scan<ET, DK, NW, ENDS ? kEnds : kStates, VEC>(p, lds, xcd_logical_block(blockIdx.x - back, gridDim.x - back));
  }
}

// The forward's first pass over segments (T 32768, 16 heads: 322 us in 8 segments).
template <typename ET, int DK, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW, 2) void k_delta_ends(const DeltaParams p) {
  extern __shared__ __align__(16) char lds[];
  delta_scan<ET, DK, NW, kEnds, VEC>(p, lds, xcd_logical_block(blockIdx.x, gridDim.x));
}

// Joins the segments of one (sequence, head) for 16 columns: wEnd[g] = M_g wEnd[g-1] + wEnd[g]
// for g = 1 .. nSeg-2, in place, so that wEnd[g] is what segment g + 1 starts from. The
// workgroups from `fwd` on do the same backwards with the transposed M on wBegin. A wave owns 32
// rows of the result and splits only their part of M into terms, which is most of a step's work
// (one wave for all rows: 57 us for 8 segments of 16 heads of 128 x 128, in four 23).
template <int DK>
__global__ __launch_bounds__(2 * DK) void k_delta_join(const DeltaParams p, uint32_t fwd) {
  constexpr int KB = DK / 32;
  __shared__ __align__(16) char terms[2][KB * 3 * 1024];
  const int ln = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = ln >> 4, n16 = ln & 15;
  const bool rev = blockIdx.x >= fwd;
  const uint32_t bid = rev ? blockIdx.x - fwd : blockIdx.x;
  const int cg = int(bid % p.nCG);
  const int64_t bh = bid / p.nCG;
  float* w = rev ? p.wBegin : p.wEnd;
  auto segment = [&](int s) { return rev ? p.nSeg - 1 - s : s; };
  auto image = [&](int s) { return w + ((bh * p.nSeg + segment(s)) * p.nCG + cg) * (DK * 16) + wave * 512; };
  // rows (columns, in reverse) 16 i .. of M, as left operands
  struct Rows {
    f32x4_t a[KB], b[KB];
  };
  auto load = [&](Rows& m, int s, int i) {
    const auto* M = in_global<float>(p.wM + (bh * p.nSeg + segment(s)) * (DK * DK));
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      if (!rev) {
        const auto* row = M + (16 * i + n16) * DK + 32 * kb + 4 * q;
        m.a[kb] = *(const global_t<f32x4_t>*)row;
        m.b[kb] = *(const global_t<f32x4_t>*)(row + 16);
      } else {
        const auto* column = M + (32 * kb + 4 * q) * DK + 16 * i + n16;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          m.a[kb][r] = column[r * DK];
          m.b[kb][r] = column[(16 + r) * DK];
        }
      }
    }
  };
  Rows m[2];
  f32x4_t S[2], next[2];
  load_image<2>(S, image(0), ln);
  load_image<2>(next, image(1), ln);
#pragma unroll
  for (int i = 0; i < 2; ++i) load(m[i], 1, 2 * wave + i);
  for (int s = 1; s + 1 < p.nSeg; ++s) {
    const Frag<3> own = split8<3>(S[0], S[1]);
    hand_over<3, 1>(terms[s & 1] + wave * 3 * 1024, &own, ln);
    const int after = min(s + 1, p.nSeg - 2);
#pragma unroll
    for (int i = 0; i < 2; ++i) S[i] = next[i];
    load_image<2>(next, image(after), ln);
    __syncthreads();  // of the two buffers the other is free: its readers have come here
    Frag<3> sf[KB];
    take_over<3, KB>(sf, terms[s & 1], ln);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) mma<2>(S[i], split8<3>(m[i].a[kb], m[i].b[kb]), sf[kb]);
      load(m[i], after, 2 * wave + i);
    }
    store_image<2>(S, image(s), ln);
  }
}

// ---------------------------------------------------------------------------------
// Backward: dq, dk, dg, dbeta of one chunk and key head
// ---------------------------------------------------------------------------------
//
// Over the value columns (32 at a time, staged from the scans' images):
//   dP = scale dO U^T,  F = dR U^T  (dA = -F),  os = dO S0^T,  rs = dR S0^T,  ug = U dS1^T,
// then with Y = rq rk Gam o dP (i >= j), Yk = -beta rk rk Gam o F (i > j) and raw q, k:
//   dq' = rq scale E os + Y K
//   dk' = rk (D ug - beta E rs) + Y^T Q + (Yk + Yk^T) K
// are rq dq and rk dk in terms of the normalised rows; the norm's own gradient takes their
// part along q (k) away: dq = dq' - rq q (rq q.dq'). The decay's gradient adds up all paths
// that cross a token, dg_t = sum_{i >= t > j} X_ij + sum_{i >= t} into_i + sum_{j < t} out_j
// + gamma <S0, dS1> with X = Y o Q K^T + Yk o K K^T, from row and column sums of the same
// products, so that pairs on one side of t cancel but for the float32 rounding of the tiles'
// sums, and only over t's own document, so that no rounding of another one's is left in it; into =
// rq scale E (q.os) - beta E rk (k.rs) and out = D rk (k.ug); the cumulative sums are in 64 bits.
// dbeta_i = dR_i.V_i - E rk (k.rs)_i + sum_j dA_ij Gam k.k. What reaches dg keeps all terms
// (float32).

template <typename ET, int DK, bool ONE>
struct GradLds {
  static constexpr int NT = Store<ET>::NT, NP = Store<ET>::NP;
  // Waves, each with DK / NW key columns. Four, and two workgroups per CU, where registers (no
  // sums over heads) and LDS (bf16) allow it, or 64 columns leave no more; else one workgroup of
  // eight (2016 chunks and heads of 128, pairs of them on one key head, bf16: 245 us with four,
  // 225 with eight).
  static constexpr int NW = DK == 128 && !(NT == 1 && ONE) ? 8 : 4;
  static constexpr int ULD = C + kPad, OLD = 32 + kPad, SLD = DK + kPad;
  static constexpr int UPL = 32 * ULD, OPL = C * OLD, SPL = 32 * SLD;
  // first part: staged operands of 32 value columns
  static constexpr int U = 0;
  static constexpr int R = U + 3 * UPL * 2;
  static constexpr int O = R + 3 * UPL * 2;
  static constexpr int S = O + NT * OPL * 2;
  static constexpr int END1 = S + 3 * SPL * 2;
  // second part, in the same place
  static constexpr int K = 0;
  static constexpr int Q = K + NT * Tile<ET, DK, 64, true>::PLANE * 2;
  static constexpr int Y = Q + NT * Tile<ET, DK, 64, true>::PLANE * 2;
  static constexpr int YK = Y + NP * kTrapLds * 2;
  static constexpr int END2 = YK + NP * kTrapLds * 2;
  static constexpr int TOK = END1 > END2 ? END1 : END2;
  static constexpr int SUM = TOK + kTokArrays * C * 4;  // per-wave sums [3][NW][64] and <S0, dS1> [NW]
  static constexpr int BYTES = SUM + 3 * NW * C * 4 + NW * 4;
};

// Images of two 16-column groups (NB blocks of 32 indices each) through registers into the 32
// rows of a [columns][index] LDS matrix of N terms.
template <int NB, int NTHR>
struct ImageTile {
  static constexpr int P = NB * 128, N = 2 * P / NTHR;  // pieces of a group, and of a thread
  static_assert(2 * P % NTHR == 0 && (P % NTHR == 0 || NTHR == 2 * P), "whole passes");
  f32x4_t r[N];
  static __device__ __forceinline__ bool first(int i, int tid) { return i * NTHR + (NTHR > P ? tid : 0) < P; }
  // `second`: whether the second group exists (it follows the first); if not, zeros.
  __device__ __forceinline__ void load(const float* src, bool second, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const auto* base = in_global<char>(src) + (i * NTHR - (first(i, tid) || second ? 0 : P)) * 16;
      r[i] = __builtin_nontemporal_load((const global_t<f32x4_t>*)(base + uint32_t(tid) * 16u));
    }
  }
  template <int NTERM>
  __device__ __forceinline__ void store(uint16_t* m, int ld, int plane, bool second, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int g = first(i, tid) ? 0 : 1, f = tid + NTHR * i - P * g;
      const int kb = f >> 7, h = (f >> 4) & 1, n = (f >> 3 & 12) + (f >> 2 & 3), q = f & 3;
      put4<NTERM>(m + (16 * g + n) * ld + 32 * kb + 16 * h + 4 * q, plane, g == 0 || second ? r[i] : zero4());
    }
  }
};

// ONE: a single value head per key head (no sums to carry from head to head). 611 to 667 us at B8
// T4096, 16 heads, bf16, for 1.3 GB (270 us at the rate of a copy): the images are read once, and what
// bounds the kernel is the latency of its phases between barriers, five per 32 value columns
// because S0 and dS1 take turns in LDS (69 KiB, so that two workgroups share a CU), with two waves
// per SIMD: vector units 44 % busy, LDS 34 %, matrix units 29 %. Of the 244 registers the three
// sums of the column loop take 96 and the images under way 52 (all of them a block ahead: 50 spilled).
template <typename ET, int DK, bool VEC, bool ONE>
__global__ __launch_bounds__((64 * GradLds<ET, DK, ONE>::NW), (Store<ET>::NT == 1 && ONE ? 2 : 1)) void k_delta_grad(
    const DeltaParams p) {
  using L = GradLds<ET, DK, ONE>;
  constexpr int NT = L::NT, NP = L::NP, LV = NP - 1, KB = DK / 32, NW = L::NW, NN = DK / 16 / NW, NTHR = 64 * NW;
  constexpr int SLOTS = (10 + NW - 1) / NW;  // tiles of a triangle per wave
  using TK = Tile<ET, DK, NTHR, VEC>;
  static_assert(L::BYTES <= kLdsBytes, "LDS of a CU");
  extern __shared__ __align__(16) char lds[];
  uint16_t* sU = reinterpret_cast<uint16_t*>(lds + L::U);
  uint16_t* sR = reinterpret_cast<uint16_t*>(lds + L::R);
  uint16_t* sO = reinterpret_cast<uint16_t*>(lds + L::O);
  uint16_t* sS = reinterpret_cast<uint16_t*>(lds + L::S);
  uint16_t* sK = reinterpret_cast<uint16_t*>(lds + L::K);
  uint16_t* sQ = reinterpret_cast<uint16_t*>(lds + L::Q);
  uint16_t* sY = reinterpret_cast<uint16_t*>(lds + L::Y);
  uint16_t* sYk = reinterpret_cast<uint16_t*>(lds + L::YK);
  float* tok = reinterpret_cast<float*>(lds + L::TOK);
  float* sum = reinterpret_cast<float*>(lds + L::SUM);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int ln = lane;
  const int64_t id = blockIdx.x;
  const int c = int(id % p.nC);
  const int hk = int(id / p.nC % p.Hk);
  const int b = int(id / p.nC / p.Hk);
  const int t0 = c * C, rows = min(C, p.T - t0);
  const int dc = 16 * NN * wave;  // first of this wave's key columns

  f32x4_t aq[4][NN], ak[4][NN];
#pragma unroll
  for (int mt = 0; mt < 4; ++mt)
#pragma unroll
    for (int n = 0; n < NN; ++n) aq[mt][n] = ak[mt][n] = zero4();

  // Element 16 mt + 4 q + r of a column that `f` holds the rows 32 (mt / 2) .. of.
  auto element = [&](const Frag<NT>& f, int mt, int r) {
    float x = 0.f;
#pragma unroll
    for (int i = NT - 1; i >= 0; --i) {
      const uint32_t w = f.t[i][2 * (mt & 1) + (r >> 1)];
      x += __uint_as_float(r & 1 ? w & 0xffff0000u : w << 16);
    }
    return x;
  };
  auto columns = [&](Frag<NT>* f, const uint16_t* m, int kb) {
#pragma unroll
    for (int n = 0; n < NN; ++n) f[n] = colfrag<NT>(m, TK::LD, TK::PLANE, 32 * kb, dc + 16 * n, ln);
  };
  for (int gh = 0; gh < (ONE ? 1 : p.group); ++gh) {
    ln = fresh_lane();
    const int tid = wave * 64 + ln, lane = ln, q = ln >> 4, n16 = ln & 15;
    const int hv = hk * p.group + gh;
    const int64_t ci = (int64_t(b) * p.Hv + hv) * p.nC + c;
    const ET* dobase = static_cast<const ET*>(p.dO) + b * p.dos0 + hv * p.dos2 + t0 * p.dos1;
    f32x4_t dP[SLOTS], F[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) dP[s] = F[s] = zero4();
    if (gh > 0) __syncthreads();  // the previous head's factors are read
    static_assert(kTokArrays * C / 4 % 64 == 0, "whole waves: no divergent branch while the sums over heads are held");
    if (wave < kTokArrays * C / 4 / 64)
      reinterpret_cast<f32x4_t*>(tok)[tid] = reinterpret_cast<const f32x4_t*>(p.wTok + ci * (kTokArrays * C))[tid];
    f32x4_t os[4][NN], rs[4][NN], ug[4][NN];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int n = 0; n < NN; ++n) os[mt][n] = rs[mt][n] = ug[mt][n] = zero4();
    float through = 0.f;  // <S0, dS1>
    {
      ImageTile<2, NTHR> iu, ir;
      ImageTile<KB, NTHR> is, ig;
      Raw8<ET> io;
      auto fetch = [&](int cb, int tid) {
        const int64_t cim = ci * p.nCG + cb;
        const bool second = cb + 1 < p.nCG;
        iu.load(p.wU + cim * (C * kDeltaCols), second, tid);
        ir.load(p.wR + cim * (C * kDeltaCols), second, tid);
        const int row = tid >> 2, c0 = cb * kDeltaCols + (tid & 3) * 8;
        const int n = row < rows ? p.dvn - c0 : 0;  // (row 64 and on, of a workgroup of 512: none)
        const uint32_t off = (uint32_t(row) * uint32_t(p.dos1) + uint32_t(c0)) * uint32_t(sizeof(ET));
        io = load8<ET, VEC>(chunk_rsrc<ET, VEC>(dobase, p.dos1, rows, p.dvn), n > 0 ? off : kNowhere, n);
      };
      auto fetch_states = [&](int cb, int tid) {
        const int64_t cim = ci * p.nCG + cb;
        const bool second = cb + 1 < p.nCG;
        is.load(p.wS + cim * (DK * 16), second, tid);
        ig.load(p.wdS + cim * (DK * 16), second, tid);
      };
      fetch(0, tid);
      for (int cb = 0; cb < p.nCG; cb += 2) {
        ln = fresh_lane();
        const int tid = wave * 64 + ln;
        const bool second = cb + 1 < p.nCG;
        fetch_states(cb, tid);  // under way during the products of U, dR and dO
        __syncthreads();  // the previous contents are read
        iu.template store<3>(sU, L::ULD, L::UPL, second, tid);
        ir.template store<3>(sR, L::ULD, L::UPL, second, tid);
        if (NTHR == 4 * C || tid < 4 * C) {  // 64 rows of 4 pieces
          const Frag<NT> f = terms8<ET>(io);
          uint16_t* o = sO + (tid >> 2) * L::OLD + place((tid & 3) * 8);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            *reinterpret_cast<u32x2*>(o + i * L::OPL) = u32x2{f.t[i][0], f.t[i][1]};
            *reinterpret_cast<u32x2*>(o + i * L::OPL + 8) = u32x2{f.t[i][2], f.t[i][3]};
          }
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
          const int t = wave + NW * s;
          if (t < 10) {
            int ti, tj;
            tile_of(t, ti, tj);
            const auto fu = colfrag<3, true>(sU, L::ULD, L::UPL, 0, 16 * tj, ln);
            const auto fo1 = rowfrag<NT>(sO, L::OLD, L::OPL, 16 * ti, 0, ln);
            const auto fr1 = colfrag<3, true>(sR, L::ULD, L::UPL, 0, 16 * ti, ln);
            DELTA_FENCE();
            mma<2>(dP[s], fu, fo1);
            mma<2>(F[s], fu, fr1);
          }
        }
        is.template store<3>(sS, L::SLD, L::SPL, second, tid);
#pragma unroll
        for (int i = 0; i < ImageTile<KB, NTHR>::N; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (is.first(i, tid) || second) through += is.r[i][e] * ig.r[i][e];
        __syncthreads();
        {
          Frag<3> fs[NN], fr[2];
          Frag<NT> fo[2];
          auto read = [&](int mt) {
            fo[mt & 1] = rowfrag<NT>(sO, L::OLD, L::OPL, 16 * mt, 0, ln);
            fr[mt & 1] = colfrag<3, true>(sR, L::ULD, L::UPL, 0, 16 * mt, ln);
          };
#pragma unroll
          for (int n = 0; n < NN; ++n) fs[n] = colfrag<3, true>(sS, L::SLD, L::SPL, 0, dc + 16 * n, ln);
          read(0);
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            if (mt < 3) read(mt + 1);
            DELTA_FENCE();
#pragma unroll
            for (int n = 0; n < NN; ++n) {
              mma<2>(os[mt][n], fo[mt & 1], fs[n]);
              mma<2>(rs[mt][n], fr[mt & 1], fs[n]);
            }
            DELTA_FENCE();
          }
        }
        __syncthreads();  // S0 is read: dS1 takes its place
        ig.template store<3>(sS, L::SLD, L::SPL, second, tid);
        __syncthreads();
        if (cb + 2 < p.nCG) fetch(cb + 2, wave * 64 + fresh_lane());
        {
          Frag<3> fg[NN], fu[2];
#pragma unroll
          for (int n = 0; n < NN; ++n) fg[n] = colfrag<3, true>(sS, L::SLD, L::SPL, 0, dc + 16 * n, ln);
          fu[0] = colfrag<3, true>(sU, L::ULD, L::UPL, 0, 0, ln);
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            if (mt < 3) fu[(mt + 1) & 1] = colfrag<3, true>(sU, L::ULD, L::UPL, 0, 16 * (mt + 1), ln);
            DELTA_FENCE();
#pragma unroll
            for (int n = 0; n < NN; ++n) mma<2>(ug[mt][n], fu[mt & 1], fg[n]);
            DELTA_FENCE();
          }
        }
      }
    }
    through = sum16(through);
    through += __shfl_xor(through, 16);
    through += __shfl_xor(through, 32);
    __syncthreads();
    {
      TK tk, tq;
      tk.load(static_cast<const ET*>(p.k) + b * p.ks0 + hk * p.ks2 + t0 * p.ks1, p.ks1, rows, p.dkn, tid);
      tq.load(static_cast<const ET*>(p.q) + b * p.qs0 + hk * p.qs2 + t0 * p.qs1, p.qs1, rows, p.dkn, tid);
      // tiles above the diagonal that a 32-wide block reads, and sums of tiles that do not exist
      for (int e = tid; e < 2 * NP * 128; e += NTHR) {
        const int n = e >> 7, row = (e >> 2) & 31, part = e & 3;
        const int i = row < 16 ? row : row + 16, j = (row < 16 ? 16 : 48) + 4 * part;
        *reinterpret_cast<u32x2*>((n < NP ? sY + n * kTrapLds : sYk + (n - NP) * kTrapLds) + trap_off(i) + place(j)) = u32x2{0u, 0u};
      }
      tk.store(sK, tid);
      tq.store(sQ, tid);
    }
    __syncthreads();
    // q.os, k.rs and k.ug of every token over this wave's key columns, and os, rs, ug into dq', dk'
    ln = fresh_lane();
    Frag<NT> cq[NN], ck[NN];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      if (mt % 2 == 0) {
        columns(cq, sQ, mt / 2);
        columns(ck, sK, mt / 2);
      }
      const int t = 16 * mt + 4 * (ln >> 4);
      const f32x4_t e = ld4(tok + kTokE * C + t), be = ld4(tok + kTokBeta * C + t), d = ld4(tok + kTokD * C + t);
      const f32x4_t rk = ld4(tok + kTokRk * C + t), rq = ld4(tok + kTokRq * C + t);
      f32x4_t a = zero4(), k1 = zero4(), k2 = zero4();
#pragma unroll
      for (int n = 0; n < NN; ++n) {
        os[mt][n] *= rq * p.scale * e;
        rs[mt][n] *= rk * e;
        ug[mt][n] *= rk * d;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float qe = element(cq[n], mt, r), ke = element(ck[n], mt, r);
          a[r] += qe * os[mt][n][r];
          k1[r] += ke * rs[mt][n][r];
          k2[r] += ke * ug[mt][n][r];
        }
        aq[mt][n] += os[mt][n];
        ak[mt][n] += ug[mt][n] - be * rs[mt][n];
        // added here: left to itself the compiler adds at the next use, and spills up to 33 of the
        // terms that it holds until then
        asm volatile("" : "+v"(aq[mt][n]), "+v"(ak[mt][n]));
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        a[r] = sum16(a[r]);
        k1[r] = sum16(k1[r]);
        k2[r] = sum16(k2[r]);
      }
      if ((ln & 15) == 0) {
        *reinterpret_cast<f32x4_t*>(sum + wave * C + t) = a;
        *reinterpret_cast<f32x4_t*>(sum + (NW + wave) * C + t) = k1;
        *reinterpret_cast<f32x4_t*>(sum + (2 * NW + wave) * C + t) = k2;
      }
    }
    if (ln == 0) sum[3 * NW * C + wave] = through;
    __syncthreads();
    float into = 0.f, out = 0.f, kr = 0.f;  // this lane's token, in wave 0
    if (wave == 0) {
      through = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) through += sum[3 * NW * C + w];
      through *= tok[kTokE * C + C - 1];
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        into += sum[w * C + ln];
        kr += sum[(NW + w) * C + ln];
        out += sum[(2 * NW + w) * C + ln];
      }
      into -= tok[kTokBeta * C + ln] * kr;
    }
    __syncthreads();
    for (int e = wave * 64 + ln; e < 3 * 4 * C; e += NTHR) sum[e] = 0.f;  // sums of tiles that do not exist
    __syncthreads();
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int t = wave + NW * s;
      if (t < 10) {
        int ti, tj;
        tile_of(t, ti, tj);
        f32x4_t qk = zero4(), kk = zero4();
        {
          Frag<NT> fj[KB], fq[KB], fk[KB];
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            fj[kb] = rowfrag<NT>(sK, TK::LD, TK::PLANE, 16 * tj, 32 * kb, ln);
            fq[kb] = rowfrag<NT>(sQ, TK::LD, TK::PLANE, 16 * ti, 32 * kb, ln);
            fk[kb] = rowfrag<NT>(sK, TK::LD, TK::PLANE, 16 * ti, 32 * kb, ln);
          }
          DELTA_FENCE();
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            mma<2>(qk, fj[kb], fq[kb]);
            mma<2>(kk, fj[kb], fk[kb]);
          }
        }
        const int i = 16 * ti + n16, j0 = 16 * tj + 4 * q;
        const float ghi = tok[kTokGhi * C + i], glo = tok[kTokGlo * C + i], rki = tok[kTokRk * C + i];
        const float rqi = tok[kTokRq * C + i], be = tok[kTokBeta * C + i];
        const int ni = __float_as_int(tok[kTokN * C + i]);
        const f32x4_t ghj = ld4(tok + kTokGhi * C + j0), glj = ld4(tok + kTokGlo * C + j0);
        const f32x4_t nj = ld4(tok + kTokN * C + j0), rkj = ld4(tok + kTokRk * C + j0);
        f32x4_t y, yk;
        float xi = 0.f, bi = 0.f, xj[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = j0 + r;
          const float gm = j <= i ? gam(ghi, glo, ni, ghj[r], glj[r], __float_as_int(nj[r])) * rkj[r] : 0.f;
          y[r] = p.scale * rqi * gm * dP[s][r];
          const float f = j < i ? -(rki * gm * F[s][r]) : 0.f;
          yk[r] = be * f;
          const float x = j < i ? y[r] * qk[r] + yk[r] * kk[r] : 0.f;
          xi += x;
          xj[r] = x;
          bi += f * kk[r];
        }
        put4<NP>(sY + trap_off(i) + place(j0), kTrapLds, y);
        put4<NP>(sYk + trap_off(i) + place(j0), kTrapLds, yk);
        xi += __shfl_xor(xi, 16);
        bi += __shfl_xor(bi, 16);
        xi += __shfl_xor(xi, 32);
        bi += __shfl_xor(bi, 32);
        if (q == 0) {
          sum[tj * C + i] = xi;
          sum[8 * C + tj * C + i] = bi;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) xj[r] = sum16(xj[r]);
        if (n16 == 0) *reinterpret_cast<f32x4_t*>(sum + 4 * C + ti * C + j0) = f32x4_t{xj[0], xj[1], xj[2], xj[3]};
      }
    }
    __syncthreads();
    if (wave == 0) {  // dg and dbeta, one token per lane
      float rz = -kr;
      for (int g = 0; g < p.nCG; ++g) rz += p.wDot[(ci * p.nCG + g) * C + lane];
      double ahead = out, behind = into;
      float db = rz;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        ahead += double(sum[4 * C + s * C + lane]) - double(sum[s * C + lane]);
        db += sum[8 * C + s * C + lane];
      }
      const double own = ahead;
      const int n = __float_as_int(tok[kTokN * C + lane]);
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        const double a = __shfl_up(ahead, m), h = __shfl_down(behind, m);
        if (__shfl_up(n, m) == n && lane >= m) ahead += a;
        if (lane + m < 64) behind += h;
      }
      const int before = lane == 0 ? 0 : __float_as_int(tok[kTokN * C + lane - 1]);
      const float dg = n != before ? 0.f : float(ahead - own + behind + double(through));
      if (lane < rows) {
        p.dg[b * p.dgs0 + (t0 + lane) * p.dgs1 + hv * p.dgs2] = dg;
        stf<ET>(p.dbeta, b * p.dbs0 + (t0 + lane) * p.dbs1 + hv * p.dbs2, db);
      }
    }
    ln = fresh_lane();
    Frag<NT> fk[2][NN], fq[2][NN];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      columns(fk[kb], sK, kb);
      columns(fq[kb], sQ, kb);
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      Frag<NP> yr[2], kr[2], yc[2], kc[2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        if (kb <= mt / 2) {
          yr[kb] = trap_row<NP>(sY, mt, kb, ln);
          kr[kb] = trap_row<NP>(sYk, mt, kb, ln);
        }
        if (kb >= mt / 2) {
          yc[kb] = trap_col<NP>(sY, mt, kb, ln);
          kc[kb] = trap_col<NP>(sYk, mt, kb, ln);
        }
      }
      DELTA_FENCE();
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int n = 0; n < NN; ++n) {
          if (kb <= mt / 2) {
            mma<LV>(aq[mt][n], yr[kb], fk[kb][n]);
            mma<LV>(ak[mt][n], kr[kb], fk[kb][n]);
          }
          if (kb >= mt / 2) {
            mma<LV>(ak[mt][n], yc[kb], fq[kb][n]);
            mma<LV>(ak[mt][n], kc[kb], fk[kb][n]);
          }
        }
    }
  }

  // the norms' own gradients, then out; q and k of the last head are still in LDS
  ln = fresh_lane();
  const int q = ln >> 4, n16 = ln & 15;
  const bool unit = p.eps >= 0.f;
  Frag<NT> cq[NN], ck[NN];
  if (unit) {
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      if (mt % 2 == 0) {
        columns(cq, sQ, mt / 2);
        columns(ck, sK, mt / 2);
      }
      f32x4_t a = zero4(), k = zero4();
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int n = 0; n < NN; ++n) {
          a[r] += aq[mt][n][r] * element(cq[n], mt, r);
          k[r] += ak[mt][n][r] * element(ck[n], mt, r);
        }
        a[r] = sum16(a[r]);
        k[r] = sum16(k[r]);
      }
      if (n16 == 0) {
        *reinterpret_cast<f32x4_t*>(sum + wave * C + 16 * mt + 4 * q) = a;
        *reinterpret_cast<f32x4_t*>(sum + (NW + wave) * C + 16 * mt + 4 * q) = k;
      }
    }
    __syncthreads();
  }
  const __amdgpu_buffer_rsrc_t outq = chunk_rsrc<ET, VEC>(
      static_cast<ET*>(p.dq) + b * p.dqs0 + hk * p.dqs2 + t0 * p.dqs1, p.dqs1, rows, p.dkn);
  const __amdgpu_buffer_rsrc_t outk = chunk_rsrc<ET, VEC>(
      static_cast<ET*>(p.dk) + b * p.dks0 + hk * p.dks2 + t0 * p.dks1, p.dks1, rows, p.dkn);
  const uint32_t pitchq = uint32_t(p.dqs1) * uint32_t(sizeof(ET)), pitchk = uint32_t(p.dks1) * uint32_t(sizeof(ET));
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    f32x4_t pq = zero4(), pk = zero4();
    if (unit) {
      if (mt % 2 == 0) {
        columns(cq, sQ, mt / 2);
        columns(ck, sK, mt / 2);
      }
      const int t = 16 * mt + 4 * q;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        pq += ld4(sum + w * C + t);
        pk += ld4(sum + (NW + w) * C + t);
      }
      const f32x4_t rq = ld4(tok + kTokRq * C + t), rk = ld4(tok + kTokRk * C + t);
      pq *= rq * rq;
      pk *= rk * rk;
    }
#pragma unroll
    for (int n = 0; n < NN; ++n) {
      const int d = dc + 16 * n + n16;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float a = aq[mt][n][r], k = ak[mt][n][r];
        if (unit) {
          a -= pq[r] * element(cq[n], mt, r);
          k -= pk[r] * element(ck[n], mt, r);
        }
        const int t = 16 * mt + r;  // + 4 q
        const bool in = d < p.dkn && (VEC || t + 4 * q < rows);
        buf_st<ET>(outq, in ? (4 * q + t) * pitchq + uint32_t(d) * uint32_t(sizeof(ET)) : kNowhere, a);
        buf_st<ET>(outk, in ? (4 * q + t) * pitchk + uint32_t(d) * uint32_t(sizeof(ET)) : kNowhere, k);
      }
    }
  }
}

template <typename KernelT, typename... Args>
hipError_t launch_delta(KernelT kernel, int64_t blocks, int threads, int lds_bytes, hipStream_t s, const Args&... args) {
  if (lds_bytes > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds_bytes);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3(unsigned(blocks)), dim3(unsigned(threads)), unsigned(lds_bytes), s, args...);
  return hipGetLastError();
}

template <typename ET, int DK, bool VEC>
hipError_t delta_prep_launch(const DeltaParams& p, hipStream_t s) {
  if (p.nC == 0) return hipSuccess;
  return launch_delta(k_delta_prep<ET, DK, VEC>, int64_t(p.B) * p.Hv * p.nC, 256, PrepLds<ET, DK>::BYTES, s, p);
}

template <typename ET, int DK, bool VEC>
hipError_t delta_fwd_dk(const DeltaParams& p, hipStream_t s) {
  constexpr int NW = kScanWaves;
  hipError_t e = delta_prep_launch<ET, DK, VEC>(p, s);
  if (e != hipSuccess) return e;
  const int64_t bh = int64_t(p.B) * p.Hv, ncb = (p.nCG + NW - 1) / NW;
  if (p.nSeg > 1) {
    e = launch_delta(k_delta_ends<ET, DK, NW, VEC>, bh * p.nSeg * (ncb + DK / kDeltaCols / NW), 64 * NW,
                     ScanLds<ET, DK, true>::BYTES, s, p);
    if (e == hipSuccess && p.nSeg > 2) e = launch_delta(k_delta_join<DK>, bh * p.nCG, 2 * DK, 0, s, p, uint32_t(bh * p.nCG));
    if (e != hipSuccess) return e;
  }
  return launch_delta(k_delta_scan<ET, DK, NW, VEC>, bh * p.nSeg * ncb, ScanLds<ET, DK, false>::THREADS,
                      ScanLds<ET, DK, false>::BYTES, s, p);
}

template <typename ET>
hipError_t delta_fwd_et(const DeltaParams& p, hipStream_t s) {
  if (p.vec) return delta_dk_pad(p.dkn) == 64 ? delta_fwd_dk<ET, 64, true>(p, s) : delta_fwd_dk<ET, 128, true>(p, s);
  return delta_dk_pad(p.dkn) == 64 ? delta_fwd_dk<ET, 64, false>(p, s) : delta_fwd_dk<ET, 128, false>(p, s);
}

template <typename ET, int DK, bool VEC>
hipError_t delta_bwd_dk(const DeltaParams& p, hipStream_t s) {
  constexpr int NW = kScanWaves;
  constexpr int scan_lds = ScanLds<ET, DK, true>::BYTES, back_lds = BackLds<ET, DK>::BYTES;
  constexpr int scans_lds = scan_lds > back_lds ? scan_lds : back_lds;
  hipError_t e = delta_prep_launch<ET, DK, VEC>(p, s);
  if (e != hipSuccess) return e;
  const int64_t bh = int64_t(p.B) * p.Hv, ncb = (p.nCG + NW - 1) / NW, blocks = bh * p.nSeg * ncb;
  if (p.nSeg > 1) {
    e = launch_delta(k_delta_scans<ET, DK, NW, true, VEC>, 2 * blocks + bh * p.nSeg * (DK / kDeltaCols / NW), 64 * NW,
                     scans_lds, s, p, uint32_t(blocks));
    if (e == hipSuccess && p.nSeg > 2) e = launch_delta(k_delta_join<DK>, 2 * bh * p.nCG, 2 * DK, 0, s, p, uint32_t(bh * p.nCG));
    if (e != hipSuccess) return e;
  }
  e = launch_delta(k_delta_scans<ET, DK, NW, false, VEC>, 2 * blocks, 64 * NW, scans_lds, s, p, uint32_t(blocks));
  if (e != hipSuccess) return e;
  const int64_t chunks = int64_t(p.B) * p.Hk * p.nC;
  using One = GradLds<ET, DK, true>;
  using Group = GradLds<ET, DK, false>;
  if (p.group == 1) return launch_delta(k_delta_grad<ET, DK, VEC, true>, chunks, 64 * One::NW, One::BYTES, s, p);
  return launch_delta(k_delta_grad<ET, DK, VEC, false>, chunks, 64 * Group::NW, Group::BYTES, s, p);
}

template <typename ET>
hipError_t delta_bwd_et(const DeltaParams& p, hipStream_t s) {
  if (p.vec) return delta_dk_pad(p.dkn) == 64 ? delta_bwd_dk<ET, 64, true>(p, s) : delta_bwd_dk<ET, 128, true>(p, s);
  return delta_dk_pad(p.dkn) == 64 ? delta_bwd_dk<ET, 64, false>(p, s) : delta_bwd_dk<ET, 128, false>(p, s);
}

}  // namespace delta
}  // namespace dynconv
