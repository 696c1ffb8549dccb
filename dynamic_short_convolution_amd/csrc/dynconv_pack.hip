// Activations in 8 bits (checkpoints for a backward pass) and back, gfx950.
//
// Per row, every 64 channels share a step 2^e, e = floor(log2 max|x|) - 6 (at least -126): the largest
// value is 64 to 127.99 steps, so codes round(x / step), to nearest even and cut at 127, are off by at
// most half a step below 127.5 of them and by less than one above: 1/128 of the largest value. Multiplying
// by a power of two is exact, so the codes do not depend on the arithmetic, and code times step fits
// the type that was packed. A group that holds an infinity or NaN gets the scale 255 and codes 0: it reads as
// NaN (0 times infinity), as the scale's bits 255 << 23 say without a test.
// Memory bound: 16 bytes of the row per lane (at any alignment of its elements), the maximum by a butterfly
// over the group's lanes, four rows' loads of a lane under way at a time. 32768 x 2048 bf16: 38 to 40 us (5.1
// TB/s); 5003 x 1537 float32: 11.8 us and back 9.3.
#include <type_traits>

#include "dynconv_common.hpp"
#include "dynconv_internal.hpp"

namespace dynconv {

namespace {

constexpr int kThreads = 256, kGroup = 64;  // kGroup: channels that share a step

struct PackTensor {
  const void* p;
  int64_t s0, s1, s2;
};
struct PackParams {
  PackTensor x, codes, scales;
  uint32_t rows, n1, n2, D;
  uint32_t lanes, perBlock, rowBlocks;  // lanes of a row (whole groups); of a workgroup's; rows' workgroups
  bool flat;                            // the rows of every tensor are n2 apart by one stride
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xf, 0xf, true));
}
// The largest of N (8 or 16) neighbouring lanes, in each of them: lanes 1 and 2 apart within a quad, 4 and 8
// apart by mirrors.
template <int N>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  v = max(v, dpp<0xB1>(v));
  v = max(v, dpp<0x4E>(v));
  v = max(v, dpp<0x141>(v));
  if constexpr (N >= 16) v = max(v, dpp<0x140>(v));
  return v;
}

// Words of a piece at the alignment of its elements (global memory takes 16 bytes at any).
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(1))) u32x2_any;
typedef uint32_t __attribute__((aligned(1))) u32_any;
template <int E, bool WHOLE>
struct Codes {
  typedef uint32_t T;
  typedef std::conditional_t<WHOLE, uint32_t, u32_any> At;
};
template <bool WHOLE>
struct Codes<8, WHOLE> {
  typedef u32x2 T;
  typedef std::conditional_t<WHOLE, u32x2, u32x2_any> At;
};

__device__ __forceinline__ int64_t offset(const PackParams& p, const PackTensor& t, uint32_t row) {
  if (p.flat) return int64_t(row) * t.s2;
  const uint32_t q = row / p.n2, i0 = q / p.n1;
  return int64_t(i0) * t.s0 + int64_t(q - i0 * p.n1) * t.s1 + int64_t(row - q * p.n2) * t.s2;
}

// A lane's place: its columns, and the rows that it goes through. Where pieces are not WHOLE, a row's last one
// begins early enough to end with it, so that it is read and written with 16 bytes as well: its first `skip`
// columns are the piece's before it too (40 million bf16 elements in rows of 100: 28 us, with the last piece element by
// element 90; rows of 515 36 and 77). Only rows shorter than a piece go element by element (n < E).
template <int E, bool WHOLE>
struct Walk {
  uint32_t c, row, step;  // c: its own first column
  uint32_t from, skip;    // where its piece begins
  int n;                  // elements of a piece, the same for all lanes
  bool on;
  __device__ __forceinline__ explicit Walk(const PackParams& p) {
    const uint32_t cb = blockIdx.x / p.rowBlocks, rb = blockIdx.x - cb * p.rowBlocks;
    const uint32_t side = kThreads / p.perBlock, sub = threadIdx.x / p.perBlock;  // rows side by side
    const uint32_t l = cb * p.perBlock + threadIdx.x - sub * p.perBlock;
    c = l * E;
    on = sub < side && l < p.lanes;
    n = WHOLE || p.D >= E ? E : int(p.D);
    from = WHOLE || c >= p.D || p.D < E ? c : min(c, p.D - E);
    skip = c - from;
    row = rb * side + sub;
    step = p.rowBlocks * side;
  }
};
constexpr int kAhead = 4;  // rows whose loads a lane has under way

// A piece: E consecutive elements (WHOLE: aligned), or the n of a shorter row.
template <typename ET, int E, bool WHOLE>
__device__ __forceinline__ void read(float (&v)[E], const PackTensor& t, int64_t off, int n) {
  typedef typename std::conditional<sizeof(ET) == 2, uint16_t, uint32_t>::type Bits;
  const Bits* p = static_cast<const Bits*>(t.p) + off;
  u32x4 w;
  if (WHOLE || n == E) {
    w = WHOLE ? *reinterpret_cast<const u32x4*>(p) : *reinterpret_cast<const u32x4_any*>(p);
  } else {  // into the words by shifts: registers have no index
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int e = 0; e < n; ++e) {
      const uint64_t b = uint64_t(p[e]) << (e % (E / 2) * int(8 * sizeof(ET)));
      lo |= e < E / 2 ? b : 0;
      hi |= e < E / 2 ? 0 : b;
    }
    w = u32x4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(ET) == 2) {
      v[2 * i] = Cvt<ET>::lo(w[i]), v[2 * i + 1] = Cvt<ET>::hi(w[i]);
    } else {
      v[i] = __uint_as_float(w[i]);
    }
  }
}

template <typename ET, int E, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_pack8(const PackParams p) {
  const Walk<E, WHOLE> me(p);
  if (!me.on) return;  // whole groups of lanes
  // A last piece that is alone in its group of channels shares columns with another group's, whose codes
  // have another step: it leaves them to that one and stores its own byte by byte.
  const bool lone = !WHOLE && p.D % kGroup < E;
  const bool wide = WHOLE || (me.n == E && !(lone && me.skip > 0));
  int8_t* out = const_cast<int8_t*>(static_cast<const int8_t*>(p.codes.p)) + me.from;
  uint8_t* sc = const_cast<uint8_t*>(static_cast<const uint8_t*>(p.scales.p)) + me.c / kGroup;
  for (uint32_t row = me.row; row < p.rows; row += kAhead * me.step) {
    float v[kAhead][E];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[u][e] = 0.f;
      const uint32_t r = row + u * me.step;  // below 2^31 + 4 * 2^20
      if (me.c < p.D) read<ET, E, WHOLE>(v[u], p.x, offset(p, p.x, r < p.rows ? r : row) + me.from, me.n);
    }
    uint32_t q[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint32_t r = row + u * me.step;
      if (r >= p.rows) break;
      uint32_t top = 0;  // as integers the magnitudes keep their order, and infinities and NaN come last
#pragma unroll
      for (int e = 0; e < E; ++e) top = max(top, lone && uint32_t(e) < me.skip ? 0u : __float_as_uint(v[u][e]) & 0x7fffffffu);
      top = group_max<kGroup / E>(top);
      const int biased = int(top >> 23);
      const bool lost = biased == 255;
      const uint32_t scale = lost ? 255u : uint32_t(max(biased - 6, 1));
      const float inverse = lost ? 0.f : __uint_as_float((254u - scale) << 23);
      uint32_t code[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float c = fminf(fmaxf(rintf(v[u][e] * inverse), -127.f), 127.f);
        code[e] = lost ? 0u : uint32_t(int(c)) & 0xffu;
      }
#pragma unroll
      for (int i = 0; i < E / 4; ++i)
        q[u][i] = code[4 * i] | code[4 * i + 1] << 8 | code[4 * i + 2] << 16 | code[4 * i + 3] << 24;
      if (me.c >= p.D) continue;
      if (me.c % kGroup == 0) sc[offset(p, p.scales, r)] = uint8_t(scale);
      typename Codes<E, WHOLE>::T w;
      if constexpr (E == 8) {
        w = u32x2{q[u][0], q[u][1]};
      } else {
        w = q[u][0];
      }
      if (wide) *reinterpret_cast<typename Codes<E, WHOLE>::At*>(out + offset(p, p.codes, r)) = w;
    }
    if constexpr (!WHOLE)
      if (!wide && me.c < p.D)
#pragma unroll 1
        for (int e = int(me.skip); e < me.n; ++e)
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const uint32_t r = row + u * me.step;
            if (r >= p.rows) break;
            const uint64_t bytes = E == 8 ? uint64_t(q[u][1]) << 32 | q[u][0] : q[u][0];
            out[offset(p, p.codes, r) + e] = int8_t(uint8_t(bytes >> (8 * e)));
          }
  }
}

template <typename ET, int E, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_unpack8(const PackParams p) {
  typedef typename Codes<E, WHOLE>::T Word;
  typedef typename Codes<E, WHOLE>::At WordAt;
  const Walk<E, WHOLE> me(p);
  if (!me.on || me.c >= p.D) return;
  for (uint32_t row = me.row; row < p.rows; row += kAhead * me.step) {
    Word w[kAhead];
    uint32_t scale[kAhead], next[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint32_t r = row + u * me.step, s = r < p.rows ? r : row;
      const int8_t* in = static_cast<const int8_t*>(p.codes.p) + offset(p, p.codes, s) + me.from;
      if (WHOLE || me.n == E) {
        w[u] = *reinterpret_cast<const WordAt*>(in);
      } else {
        uint32_t q[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (e < me.n) q[e / 4] |= uint32_t(uint8_t(in[e])) << (8 * (e % 4));
        if constexpr (E == 8) {
          w[u] = u32x2{q[0], q[1]};
        } else {
          w[u] = q[0];
        }
      }
      const uint8_t* sc = static_cast<const uint8_t*>(p.scales.p) + offset(p, p.scales, s);
      scale[u] = sc[me.from / kGroup];
      if constexpr (!WHOLE) next[u] = sc[me.c / kGroup];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint32_t r = row + u * me.step;
      if (r >= p.rows) break;
      const float step = __uint_as_float(scale[u] << 23), own = WHOLE ? step : __uint_as_float(next[u] << 23);
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        uint32_t word;
        if constexpr (E == 8) {
          word = w[u][e / 4];
        } else {
          word = w[u];
        }
        v[e] = float(int8_t(word >> (8 * (e % 4)) & 0xff)) * (WHOLE || uint32_t(e) < me.skip ? step : own);
      }
      ET* out = const_cast<ET*>(static_cast<const ET*>(p.x.p)) + offset(p, p.x, r) + me.from;
      if (WHOLE || me.n == E) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (sizeof(ET) == 2) {
            o[i] = Cvt<ET>::pack2(v[2 * i], v[2 * i + 1]);
          } else {
            o[i] = __float_as_uint(v[i]);
          }
        }
        if constexpr (WHOLE) {
          *reinterpret_cast<u32x4*>(out) = o;
        } else {
          *reinterpret_cast<u32x4_any*>(out) = o;
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (e < me.n) {
            if constexpr (sizeof(ET) == 2) {
              *reinterpret_cast<uint16_t*>(out + e) = Cvt<ET>::bits(v[e]);
            } else {
              out[e] = v[e];
            }
          }
      }
    }
  }
}

template <typename ET, bool WHOLE>
hipError_t launch(PackParams p, bool unpack, hipStream_t s) {
  constexpr int E = 16 / int(sizeof(ET));
  p.lanes = (p.D + kGroup - 1) / kGroup * (kGroup / E);
  p.perBlock = p.lanes < kThreads ? p.lanes : kThreads;
  const uint32_t colBlocks = (p.lanes + p.perBlock - 1) / p.perBlock, side = kThreads / p.perBlock;
  // eight workgroups per CU, each with at least its first rows
  const uint32_t need = uint32_t((uint64_t(p.rows) + side - 1) / side), most = colBlocks < 2048 ? 2048 / colBlocks : 1;
  p.rowBlocks = need < most ? need : most;
  const dim3 grid(colBlocks * p.rowBlocks);
  if (unpack) {
    hipLaunchKernelGGL((k_unpack8<ET, E, WHOLE>), grid, dim3(kThreads), 0, s, p);
  } else {
    hipLaunchKernelGGL((k_pack8<ET, E, WHOLE>), grid, dim3(kThreads), 0, s, p);
  }
  return hipGetLastError();
}

template <typename ET>
hipError_t dispatch(const PackParams& p, bool whole, bool unpack, hipStream_t s) {
  return whole ? launch<ET, true>(p, unpack, s) : launch<ET, false>(p, unpack, s);
}

bool aligned(const void* p, int64_t a) { return (reinterpret_cast<uintptr_t>(p) % uint64_t(a)) == 0; }

// A tensor [n0,n1,n2,last] of eb-byte elements, read or written in pieces of `piece` bytes where *whole.
dynconv_status take(PackTensor* t, const void* p, const int64_t* s, const int64_t* n, int64_t last, int eb, int piece,
                    bool output, bool* whole) {
  if (p == nullptr || s == nullptr) return DYNCONV_ERR_INVALID_ARG;
  if (!aligned(p, eb) || (last > 1 && s[3] != 1)) return DYNCONV_ERR_UNSUPPORTED;
  if (!aligned(p, piece)) *whole = false;
  for (int i = 0; i < 3; ++i) {
    if (s[i] < 0) return DYNCONV_ERR_UNSUPPORTED;
    if (n[i] <= 1) continue;
    if (output && s[i] == 0) return DYNCONV_ERR_INVALID_ARG;
    if (s[i] * eb % piece != 0) *whole = false;
  }
  t->p = p;
  t->s0 = s[0], t->s1 = s[1], t->s2 = s[2];
  return DYNCONV_OK;
}

// Whether t's rows follow each other by the stride of the last dimension of more than one, which becomes s2.
bool flat(PackTensor* t, const int64_t* n) {
  const int64_t s[3] = {t->s0, t->s1, t->s2};
  int64_t step = 0, count = 1;
  for (int i = 2; i >= 0; --i) {
    if (n[i] <= 1) continue;
    if (count == 1) {
      step = s[i];
    } else if (s[i] != step * count) {
      return false;
    }
    count *= n[i];
  }
  t->s2 = step;
  return true;
}

dynconv_status run(const void* x, const int64_t* xs, const int8_t* codes, const int64_t* cs, const uint8_t* scales,
                   const int64_t* ss, int64_t n0, int64_t n1, int64_t n2, int64_t D, dynconv_dtype dtype, bool unpack,
                   void* stream) {
  if (dtype != DYNCONV_F32 && dtype != DYNCONV_BF16 && dtype != DYNCONV_F16) return DYNCONV_ERR_INVALID_ARG;
  const int64_t n[3] = {n0, n1, n2};
  for (int64_t i : n)
    if (i < 0) return DYNCONV_ERR_INVALID_ARG;
  if (D < 0) return DYNCONV_ERR_INVALID_ARG;
  for (int64_t i : n)
    if (i > INT32_MAX) return DYNCONV_ERR_UNSUPPORTED;
  if (D > (int64_t(1) << 24)) return DYNCONV_ERR_UNSUPPORTED;
  if (n0 == 0 || n1 == 0 || n2 == 0 || D == 0) return DYNCONV_OK;
  if (n0 > INT32_MAX / n1 || n0 * n1 > INT32_MAX / n2) return DYNCONV_ERR_UNSUPPORTED;
  const int eb = dtype == DYNCONV_F32 ? 4 : 2;
  bool whole = D * eb % 16 == 0, any = true;
  PackParams p{};
  dynconv_status st;
  if ((st = take(&p.x, x, xs, n, D, eb, 16, unpack, &whole)) != DYNCONV_OK) return st;
  if ((st = take(&p.codes, codes, cs, n, D, 1, 16 / eb, !unpack, &whole)) != DYNCONV_OK) return st;
  if ((st = take(&p.scales, scales, ss, n, (D + kGroup - 1) / kGroup, 1, 1, !unpack, &any)) != DYNCONV_OK) return st;
  if (x == static_cast<const void*>(codes) || x == static_cast<const void*>(scales) ||
      static_cast<const void*>(codes) == static_cast<const void*>(scales))
    return DYNCONV_ERR_INVALID_ARG;
  p.n1 = uint32_t(n1), p.n2 = uint32_t(n2), p.D = uint32_t(D);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  p.rows = uint32_t(n0 * n1 * n2);
  p.flat = flat(&p.x, n) && flat(&p.codes, n) && flat(&p.scales, n);
  const hipError_t e = dtype == DYNCONV_BF16  ? dispatch<bf16_t>(p, whole, unpack, s)
                       : dtype == DYNCONV_F16 ? dispatch<f16_t>(p, whole, unpack, s)
                                              : dispatch<float>(p, whole, unpack, s);
  return e == hipSuccess ? DYNCONV_OK : record_hip_error(e);
}

}  // namespace

}  // namespace dynconv

extern "C" {

dynconv_status dynconv_pack(const void* x, const int64_t* xs, int8_t* codes, const int64_t* cs, uint8_t* scales,
                             const int64_t* ss, int64_t n0, int64_t n1, int64_t n2, int64_t D, dynconv_dtype dtype,
                             void* stream) {
  return dynconv::run(x, xs, codes, cs, scales, ss, n0, n1, n2, D, dtype, false, stream);
}

dynconv_status dynconv_unpack(const int8_t* codes, const int64_t* cs, const uint8_t* scales, const int64_t* ss, void* y,
                               const int64_t* ys, int64_t n0, int64_t n1, int64_t n2, int64_t D, dynconv_dtype dtype,
                               void* stream) {
  return dynconv::run(y, ys, codes, cs, scales, ss, n0, n1, n2, D, dtype, true, stream);
}

}  // extern "C"
