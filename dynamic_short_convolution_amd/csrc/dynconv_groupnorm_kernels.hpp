// Group norm, channels last, with weight, bias, SiLU and a SiLU gate, gfx950: kernels, compiled once per
// storage type.
//
//   n = (x - mean) / sqrt(var + eps),  z = n w + b,  y = act(z) silu(gate),  act = SiLU or none
//   dz = dy silu(gate) act'(z),  dn = dz w,  dx = (dn - mean(dn) - n mean(dn n)) / sqrt(var + eps),
//   dw = sum dz n,  db = sum dz,  dgate = dy act(z) silu'(gate)
// The means run over the Cg channels of a group, of one token or of all tokens of a sequence.
#pragma once

#include <type_traits>

#include "dynconv_common.hpp"
#include "dynconv_groupnorm_internal.hpp"

namespace dynconv {

namespace group {

constexpr int kThreads = 256;
constexpr int kScaleGroup = 64;

struct i8_t {
  int8_t bits;
};

// Words of a piece at the alignment of its elements (global memory takes 16 bytes at any).
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(1))) u32x2_any;
typedef uint32_t __attribute__((aligned(1))) u32_any;

// A piece: E consecutive elements, 16 bytes of the storage type (codes of 8 bits as integers). WHOLE:
// aligned, all of them a group's. Else a group's last piece begins early enough to end with it, so that all
// pieces are read and written with 16 bytes and no lane goes another way: its first `skip` elements are the
// piece's before it too, which count there and are written twice, the same bits. Only groups of fewer than
// E channels are read and written element by element (n, the same for all lanes); what is not theirs
// reads as zero. Last pieces element by element took 1.2 to 3 times as long (8 sequences of 1515 tokens, 3 groups
// of 1100 bf16 channels, forward and backward per token: 723 us, now 277; 27 groups of 57: 238, now 196).
template <int E, bool WHOLE>
struct Piece {
  int c, skip;  // its first channel in the group
  __device__ __forceinline__ Piece(int at, int Cg) {
    c = WHOLE ? at : max(0, min(at, Cg - E));
    skip = at - c;
  }
  static __device__ __forceinline__ int size(int Cg) { return WHOLE ? E : min(E, Cg); }
  static __device__ __forceinline__ bool counts(int e, int skip, int n) { return WHOLE || (e >= skip && e < n); }
};
template <typename ET, int E, bool WHOLE>
__device__ __forceinline__ void load(float (&v)[E], const void* base, int64_t off, int n) {
  const ET* p = static_cast<const ET*>(base) + off;
  if (WHOLE || n >= E) {
    if constexpr (sizeof(ET) == 1) {
      uint32_t w[E / 4];
      if constexpr (E == 8) {
        const u32x2 q = WHOLE ? *reinterpret_cast<const u32x2*>(p) : *reinterpret_cast<const u32x2_any*>(p);
        w[0] = q[0], w[1] = q[1];
      } else {
        w[0] = WHOLE ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const u32_any*>(p);
      }
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = float(int8_t(w[i / 4] >> (8 * (i % 4)) & 0xff));
    } else {
      const u32x4 w = WHOLE ? *reinterpret_cast<const u32x4*>(p) : *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(ET) == 2) {
          v[2 * i] = Cvt<ET>::lo(w[i]), v[2 * i + 1] = Cvt<ET>::hi(w[i]);
        } else {
          v[i] = __uint_as_float(w[i]);
        }
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      v[e] = 0.f;
      if (e < n) {
        if constexpr (sizeof(ET) == 1) {
          v[e] = float(*reinterpret_cast<const int8_t*>(p + e));
        } else if constexpr (sizeof(ET) == 2) {
          v[e] = Cvt<ET>::of_bits(*reinterpret_cast<const uint16_t*>(p + e));
        } else {
          v[e] = p[e];
        }
      }
    }
  }
}
template <typename ET, int E, bool WHOLE>
__device__ __forceinline__ void store(const float (&v)[E], const void* base, int64_t off, int n) {
  ET* p = const_cast<ET*>(static_cast<const ET*>(base)) + off;
  if (WHOLE || n >= E) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(ET) == 2) {
        w[i] = Cvt<ET>::pack2(v[2 * i], v[2 * i + 1]);
      } else {
        w[i] = __float_as_uint(v[i]);
      }
    }
    if constexpr (WHOLE) {
      *reinterpret_cast<u32x4*>(p) = w;
    } else {
      *reinterpret_cast<u32x4_any*>(p) = w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e < n) {
        if constexpr (sizeof(ET) == 2) {
          *reinterpret_cast<uint16_t*>(p + e) = Cvt<ET>::bits(v[e]);
        } else {
          p[e] = v[e];
        }
      }
  }
}

// A token's piece of x from channel c on; in 8 bits with its scale (of WHOLE pieces one, else up to two).
template <typename IT, int E, bool WHOLE>
__device__ __forceinline__ void load_x(float (&v)[E], const GroupTensor& t, int64_t b, int64_t tok, int c, int n) {
  load<IT, E, WHOLE>(v, t.p, b * t.s0 + tok * t.s1 + c, n);
  if constexpr (sizeof(IT) == 1) {
    const uint8_t* sc = t.sc + (b * t.c0 + tok * t.c1);
    const uint32_t at = uint32_t(c) / kScaleGroup, left = kScaleGroup - uint32_t(c) % kScaleGroup;
    const float step = __uint_as_float(uint32_t(sc[at]) << 23);
    if constexpr (WHOLE) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] *= step;
    } else {
      const float next = __uint_as_float(uint32_t(sc[left < uint32_t(n) ? at + 1 : at]) << 23);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] *= uint32_t(e) < left ? step : next;
    }
  }
}

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504088896340736f));
}

// y of one element.
__device__ __forceinline__ float value(float n, float w, float b, bool silu, bool gated, float g) {
  float z = __builtin_fmaf(n, w, b);
  if (silu) z *= sigmoid(z);
  if (gated) z *= g * sigmoid(g);
  return z;
}
// dz of one element, and the gate's gradient.
__device__ __forceinline__ float slope(float n, float w, float b, bool silu, bool gated, float g, float dy, float& dgate) {
  const float z = __builtin_fmaf(n, w, b);
  float act = z, d = 1.f;
  if (silu) {
    const float s = sigmoid(z);
    act = z * s;
    d = s * (1.f + z * (1.f - s));
  }
  if (gated) {
    const float s = sigmoid(g);
    dgate = dy * act * (s * (1.f + g * (1.f - s)));
    dy *= g * s;
  }
  return dy * d;
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
// Sums over the LPR lanes of a row, in every one of them, without LDS up to a wave: lanes 1 and 2 apart
// within a quad, 4 and 8 apart by mirrors (whose quads and halves are equal by then), 16 and 32
// apart by swaps. `red`: one array per call site.
template <int LPR>
__device__ __forceinline__ float wave_sum(float x) {
  if constexpr (LPR >= 2) x += dpp<0xB1>(x);
  if constexpr (LPR >= 4) x += dpp<0x4E>(x);
  if constexpr (LPR >= 8) x += dpp<0x141>(x);
  if constexpr (LPR >= 16) x += dpp<0x140>(x);
  if constexpr (LPR >= 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  if constexpr (LPR >= 64) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  return x;
}
template <int LPR, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float (&red)[N][4]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = wave_sum<LPR>(x[i]);
  if constexpr (LPR == 256) {
    __syncthreads();  // the previous sums are read
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[i][threadIdx.x >> 6] = x[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = (red[i][0] + red[i][1]) + (red[i][2] + red[i][3]);
  }
}
template <int LPR>
__device__ __forceinline__ double row_sum(double x, double* red) {
#pragma unroll
  for (int m = 1; m < (LPR < 64 ? LPR : 64); m <<= 1) x += __shfl_xor(x, m);
  if constexpr (LPR == 256) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = (red[0] + red[1]) + (red[2] + red[3]);
  }
  return x;
}

// ---------------------------------------------------------------------------------
// Per token. A row (one group of one token) belongs to the fewest lanes that hold it in one 16-byte
// piece each, up to a wave, then several pieces or a workgroup: each input is read once, the mean and the
// squares around it are two sums over registers. Longer rows are read again. A workgroup takes gpw
// neighbouring groups of tpw tokens at a time, a lane the same channels every time, the next tokens' loads under
// way meanwhile (those after them too: 230 us against 232, and 50 against 45 for ragged float32 groups).
// Bound by memory: 32768 tokens of 16 groups of 128 with gate, bf16, forward 94 to 109 us (3.7 to 4.3 TB/s),
// backward 132 to 155 (4.3 to 5.1), from 8-bit x 130 to 152; 5003 tokens of 27 groups of 57, float32, 17 and 25 us (3.6
// and 3.7).
// ---------------------------------------------------------------------------------
struct Token {
  int64_t b, t;
};
__device__ __forceinline__ Token token_at(const GroupParams& p, int64_t token) {
  if (p.B == 1) return {0, token};
  const uint32_t b = uint32_t(token) / uint32_t(p.T);  // below 2^31 tokens
  return {b, int64_t(uint32_t(token) - b * uint32_t(p.T))};
}

// A row's deviations from its mean, in place of x, and what turns them into n = d rstd + shift. A first mean
// is off by some roundings of itself, which is much beside a small deviation (1100 channels of 1000.1 made n 0.02 instead of
// 0); the mean of the deviations from it is off by as many roundings of that.
struct Norm {
  float rstd, shift;
};
template <int E, bool WHOLE, int LPR, int NV>
__device__ __forceinline__ Norm normalise(float (&x)[NV][E], const int (&skip)[NV], int n, float inv, float eps, float (&red1)[1][4],
                                          float (&red2)[2][4]) {
  typedef Piece<E, WHOLE> P;
  float sum[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (skip[i] < E) {
#pragma unroll
      for (int e = 0; e < E; ++e) sum[0] += P::counts(e, skip[i], n) ? x[i][e] : 0.f;
    }
  row_sums<LPR>(sum, red1);
  const float mean = sum[0] * inv;
  float of[2] = {0.f, 0.f};  // the deviations, their squares
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (skip[i] < E) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[i][e] -= mean;
        const float d = P::counts(e, skip[i], n) ? x[i][e] : 0.f;
        of[0] += d, of[1] += d * d;
      }
    }
  row_sums<LPR>(of, red2);
  // one rounding: where the squares are past float32, the variance is infinite (n is 0) and not the difference of two
  const float off = of[0] * inv, var = __builtin_fmaf(-off, off, of[1] * inv);
  const float rstd = 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);
  return {rstd, -off * rstd};
}

template <typename ET, int E, bool WHOLE, int LPR, int NV>
__global__ __launch_bounds__(kThreads) void k_group_fwd(const GroupParams p) {
  constexpr int NA = NV > 0 ? NV : 1;
  __shared__ float red1[1][4], red2[2][4];
  __shared__ double dred[2][4];
  const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  const int tsub = slot / p.gpw, gsub = slot - tsub * p.gpw;
  const int gi = blockIdx.y * p.gpw + gsub;
  const bool mine = tsub < p.tpw && gi < p.G;
  const int c0 = (mine ? gi : 0) * p.Cg;
  typedef Piece<E, WHOLE> P;
  const int n = P::size(p.Cg);
  const bool gated = p.gate.p != nullptr, silu = p.silu != 0;
  const float inv = 1.f / float(p.Cg);
  const int64_t tokens = int64_t(p.B) * p.T, step = int64_t(gridDim.x) * p.tpw;
  auto finish = [&](const float (&d)[E], const float (&g)[E], const float (&w)[E], const float (&bi)[E], Norm at, int64_t off) {
    float y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = value(__builtin_fmaf(d[e], at.rstd, at.shift), w[e], bi[e], silu, gated, g[e]);
    store<ET, E, WHOLE>(y, p.y.p, off, n);
  };
  if constexpr (NV > 0) {
    float w[NA][E], bi[NA][E], nx[NA][E], ng[NA][E];
    int cc[NA], skip[NA];  // lanes past the row read its start and drop it (skip E)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * LPR) * E;
      const P at(c < p.Cg ? c : 0, p.Cg);
      skip[i] = c < p.Cg ? at.skip : E;
      cc[i] = c0 + at.c;
#pragma unroll
      for (int e = 0; e < E; ++e) w[i][e] = 1.f, bi[i][e] = 0.f;
      if (p.weight != nullptr) load<ET, E, WHOLE>(w[i], p.weight, cc[i], n);
      if (p.bias != nullptr) load<ET, E, WHOLE>(bi[i], p.bias, cc[i], n);
    }
    auto fetch = [&](int64_t tok) {
      const Token q = token_at(p, tok < tokens ? tok : tokens - 1);
#pragma unroll
      for (int i = 0; i < NV; ++i) load<ET, E, WHOLE>(nx[i], p.x.p, q.b * p.x.s0 + q.t * p.x.s1 + cc[i], n);
      if (gated) {
#pragma unroll
        for (int i = 0; i < NV; ++i) load<ET, E, WHOLE>(ng[i], p.gate.p, q.b * p.gate.s0 + q.t * p.gate.s1 + cc[i], n);
      }
    };
    int64_t tok0 = int64_t(blockIdx.x) * p.tpw;
    fetch(tok0 + tsub);
    for (; tok0 < tokens; tok0 += step) {
      float x[NV][E], g[NV][E];
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) x[i][e] = nx[i][e], g[i][e] = ng[i][e];
      if (tok0 + step < tokens) fetch(tok0 + step + tsub);
      const Norm norm = normalise<E, WHOLE, LPR, NV>(x, skip, n, inv, p.eps, red1, red2);
      if (mine && tok0 + tsub < tokens) {
        const Token q = token_at(p, tok0 + tsub);
        const int64_t oy = q.b * p.y.s0 + q.t * p.y.s1;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (skip[i] < E) finish(x[i], g[i], w[i], bi[i], norm, oy + cc[i]);
      }
    }
  } else {
    for (int64_t token = blockIdx.x; token < tokens; token += step) {  // one group of one token at a time
      const Token q = token_at(p, token);
      const int64_t ox = q.b * p.x.s0 + q.t * p.x.s1 + c0, og = q.b * p.gate.s0 + q.t * p.gate.s1 + c0;
      double sum = 0.0, sq = 0.0;  // 64 bits: of any number of channels, and no difference of two of them loses the variance
      for (int c = lane * E; c < p.Cg; c += LPR * E) {
        const P at(c, p.Cg);
        float x[E];
        load<ET, E, WHOLE>(x, p.x.p, ox + at.c, n);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const double v = P::counts(e, at.skip, n) ? x[e] : 0.f;
          sum += v, sq += v * v;
        }
      }
      const double mean = row_sum<LPR>(sum, dred[0]) / p.Cg;
      const double var = row_sum<LPR>(sq, dred[1]) / p.Cg - mean * mean;
      const float rstd = 1.f / sqrtf((var < 0.0 ? 0.f : float(var)) + p.eps);
      for (int at = lane * E; at < p.Cg; at += LPR * E) {
        const int c = P(at, p.Cg).c;
        float x[E], g[E], w[E], bi[E];
        load<ET, E, WHOLE>(x, p.x.p, ox + c, n);
        if (gated) load<ET, E, WHOLE>(g, p.gate.p, og + c, n);
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = 1.f, bi[e] = 0.f;
        if (p.weight != nullptr) load<ET, E, WHOLE>(w, p.weight, c0 + c, n);
        if (p.bias != nullptr) load<ET, E, WHOLE>(bi, p.bias, c0 + c, n);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] -= float(mean);
        finish(x, g, w, bi, Norm{rstd, 0.f}, q.b * p.y.s0 + q.t * p.y.s1 + c0 + c);
      }
    }
  }
}

// The sums of the weight's and the bias's gradient stay in a lane's registers and leave as one partial row per
// workgroup.
template <typename ET, int E, bool WHOLE, int LPR, int NV, bool PACKED>
__global__ __launch_bounds__(kThreads) void k_group_bwd(const GroupParams p) {
  using IT = std::conditional_t<PACKED, i8_t, ET>;
  constexpr int NA = NV > 0 ? NV : 1;
  __shared__ float red1[1][4], red2[2][2][4];
  __shared__ double dred[4][4];
  extern __shared__ float fold[];  // NV > 0: [tpw][gpw Cg]
  const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  const int tsub = slot / p.gpw, gsub = slot - tsub * p.gpw;
  const int gi = blockIdx.y * p.gpw + gsub;
  const bool mine = tsub < p.tpw && gi < p.G;
  const int c0 = (mine ? gi : 0) * p.Cg;
  typedef Piece<E, WHOLE> P;
  const int n = P::size(p.Cg);
  const bool gated = p.gate.p != nullptr, silu = p.silu != 0;
  const float inv = 1.f / float(p.Cg);
  const int64_t tokens = int64_t(p.B) * p.T;
  float dw[NA][E], db[NA][E], w[NA][E], bi[NA][E];
  int cc[NA], skip[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int c = (lane + i * LPR) * E;
    const P at(c < p.Cg ? c : 0, p.Cg);
    skip[i] = c < p.Cg ? at.skip : E;
    cc[i] = at.c;
#pragma unroll
    for (int e = 0; e < E; ++e) dw[i][e] = 0.f, db[i][e] = 0.f, w[i][e] = 1.f, bi[i][e] = 0.f;
    if constexpr (NV > 0) {
      if (p.weight != nullptr) load<ET, E, WHOLE>(w[i], p.weight, c0 + cc[i], n);
      if (p.bias != nullptr) load<ET, E, WHOLE>(bi[i], p.bias, c0 + cc[i], n);
    }
  }
  bool first = true;
  const int64_t step = int64_t(gridDim.x) * p.tpw;
  float nx[NA][E], ndy[NA][E], ng[NA][E];
  auto fetch = [&](int64_t tok) {
    const Token q = token_at(p, tok < tokens ? tok : tokens - 1);
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      load_x<IT, E, WHOLE>(nx[i], p.x, q.b, q.t, c0 + cc[i], n);
      load<ET, E, WHOLE>(ndy[i], p.dy.p, q.b * p.dy.s0 + q.t * p.dy.s1 + c0 + cc[i], n);
    }
    if (gated) {
#pragma unroll
      for (int i = 0; i < NA; ++i) load<ET, E, WHOLE>(ng[i], p.gate.p, q.b * p.gate.s0 + q.t * p.gate.s1 + c0 + cc[i], n);
    }
  };
  if constexpr (NV > 0) fetch(int64_t(blockIdx.x) * p.tpw + tsub);
  for (int64_t tok0 = int64_t(blockIdx.x) * p.tpw; tok0 < tokens; tok0 += step) {
    const bool have = mine && tok0 + tsub < tokens;
    const Token here = token_at(p, have ? tok0 + tsub : tokens - 1);
    const int64_t b = here.b, t = here.t;
    const int64_t og = b * p.gate.s0 + t * p.gate.s1 + c0, ody = b * p.dy.s0 + t * p.dy.s1 + c0;
    const int64_t odx = b * p.dx.s0 + t * p.dx.s1 + c0, odg = b * p.dgate.s0 + t * p.dgate.s1 + c0;
    if constexpr (NV > 0) {
      float x[NV][E], dy[NV][E], g[NV][E];
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) x[i][e] = nx[i][e], dy[i][e] = ndy[i][e], g[i][e] = ng[i][e];
      if (tok0 + step < tokens) fetch(tok0 + step + tsub);
      const Norm at = normalise<E, WHOLE, LPR, NV>(x, skip, n, inv, p.eps, red1, red2[0]);
      float m[2] = {0.f, 0.f};  // of dn, of dn n
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (skip[i] < E) {
          float dz[E], dg[E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            x[i][e] = __builtin_fmaf(x[i][e], at.rstd, at.shift);
            dg[e] = 0.f;
            dz[e] = slope(x[i][e], w[i][e], bi[i][e], silu, gated, g[i][e], dy[i][e], dg[e]);
            dy[i][e] = dz[e] * w[i][e];
            const bool counts = P::counts(e, skip[i], n);
            m[0] += counts ? dy[i][e] : 0.f;
            m[1] += counts ? dy[i][e] * x[i][e] : 0.f;
          }
          if (have) {
            if (gated) store<ET, E, WHOLE>(dg, p.dgate.p, odg + cc[i], n);
#pragma unroll
            for (int e = 0; e < E; ++e) dw[i][e] += dz[e] * x[i][e], db[i][e] += dz[e];
          }
        }
      row_sums<LPR>(m, red2[1]);
      m[0] *= inv, m[1] *= inv;
      if (have) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (skip[i] < E) {
            float dx[E];
#pragma unroll
            for (int e = 0; e < E; ++e) dx[e] = at.rstd * (dy[i][e] - m[0] - x[i][e] * m[1]);
            store<ET, E, WHOLE>(dx, p.dx.p, odx + cc[i], n);
          }
      }
    } else {
      double sum = 0.0, sq = 0.0;
      for (int c = lane * E; c < p.Cg; c += LPR * E) {
        const P at(c, p.Cg);
        float x[E];
        load_x<IT, E, WHOLE>(x, p.x, b, t, c0 + at.c, n);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const double v = P::counts(e, at.skip, n) ? x[e] : 0.f;
          sum += v, sq += v * v;
        }
      }
      const double dmean = row_sum<LPR>(sum, dred[0]) / p.Cg;
      const double var = row_sum<LPR>(sq, dred[1]) / p.Cg - dmean * dmean;
      const float mean = float(dmean), rstd = 1.f / sqrtf((var < 0.0 ? 0.f : float(var)) + p.eps);
      auto point = [&](int c, float (&norm)[E], float (&dn)[E], float (&dz)[E], float (&dg)[E]) {
        float wv[E], bv[E], g[E];
        load_x<IT, E, WHOLE>(norm, p.x, b, t, c0 + c, n);
        load<ET, E, WHOLE>(dn, p.dy.p, ody + c, n);
        if (gated) load<ET, E, WHOLE>(g, p.gate.p, og + c, n);
#pragma unroll
        for (int e = 0; e < E; ++e) wv[e] = 1.f, bv[e] = 0.f;
        if (p.weight != nullptr) load<ET, E, WHOLE>(wv, p.weight, c0 + c, n);
        if (p.bias != nullptr) load<ET, E, WHOLE>(bv, p.bias, c0 + c, n);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          norm[e] = (norm[e] - mean) * rstd;
          dg[e] = 0.f;
          dz[e] = slope(norm[e], wv[e], bv[e], silu, gated, g[e], dn[e], dg[e]);
          dn[e] = dz[e] * wv[e];
        }
      };
      double s1 = 0.0, s2 = 0.0;
      for (int c = lane * E; c < p.Cg; c += LPR * E) {
        const P at(c, p.Cg);
        float norm[E], dn[E], dz[E], dg[E];
        point(at.c, norm, dn, dz, dg);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const double v = P::counts(e, at.skip, n) ? dn[e] : 0.f;
          s1 += v, s2 += P::counts(e, at.skip, n) ? v * double(norm[e]) : 0.0;
        }
      }
      const float m1 = float(row_sum<LPR>(s1, dred[2]) / p.Cg), m2 = float(row_sum<LPR>(s2, dred[3]) / p.Cg);
      // the partial sums of a lane's columns stay in the workgroup's own rows of memory
      float* part = p.colpart != nullptr ? p.colpart + int64_t(blockIdx.x) * 2 * p.C + c0 : nullptr;
      for (int c = lane * E; c < p.Cg && have; c += LPR * E) {
        const P at(c, p.Cg);
        float norm[E], dn[E], dz[E], dg[E], dx[E];
        point(at.c, norm, dn, dz, dg);
#pragma unroll
        for (int e = 0; e < E; ++e) dx[e] = rstd * (dn[e] - m1 - norm[e] * m2);
        store<ET, E, WHOLE>(dx, p.dx.p, odx + at.c, n);
        if (gated) store<ET, E, WHOLE>(dg, p.dgate.p, odg + at.c, n);
        if (part != nullptr) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (!P::counts(e, at.skip, n)) continue;
            float* to = part + at.c + e;
            to[0] = first ? dz[e] * norm[e] : to[0] + dz[e] * norm[e];
            to[p.C] = first ? dz[e] : to[p.C] + dz[e];
          }
        }
      }
    }
    first = false;
  }
  if constexpr (NV > 0) {
    if (p.colpart == nullptr) return;
    float* part = p.colpart + int64_t(blockIdx.x) * 2 * p.C;
    if (p.tpw == 1) {
      if (!mine) return;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (skip[i] < E) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (!P::counts(e, skip[i], n)) continue;
            part[c0 + cc[i] + e] = dw[i][e];
            part[p.C + c0 + cc[i] + e] = db[i][e];
          }
        }
      return;
    }
    const int width = p.gpw * p.Cg;
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
      if (mine) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (skip[i] < E) {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (P::counts(e, skip[i], n)) fold[tsub * width + gsub * p.Cg + cc[i] + e] = which ? db[i][e] : dw[i][e];
          }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < width; c += kThreads) {
        if (int(blockIdx.y) * width + c >= p.C) break;
        float s = 0.f;
        for (int q = 0; q < p.tpw; ++q) s += fold[q * width + c];
        part[which * p.C + blockIdx.y * width + c] = s;
      }
    }
  }
}

// ---------------------------------------------------------------------------------
// Over the tokens of a sequence. A workgroup owns gpb whole groups (or part of the columns of a
// wide one at a time) of a run of tokens; a lane keeps its channels and goes along the tokens, tps
// of them side by side. x is read twice: once for the sums, once for the result; the backward reads x and dy for
// the column sums, from which the groups' means follow, and again for the result. Bound by memory: 8
// sequences of 0 to 4096 tokens (half of them in all), 32 groups of 64, bf16: sums 25 to 28 us, result 36 to 38, column
// sums 43 to 45, gradient 50 to 54 (2.4 to 5 TB/s), three small sums 17; from 8-bit x sums 19, column sums 47, gradient
// 52 to 54. With float32 in place of float64 sums the
// first pass takes as long.
// ---------------------------------------------------------------------------------
struct Place {
  int b, g0, t0, t1, n, tsub, l;  // t0..t1: its tokens, of n that exist; l: lane of the token
  int g, c;                       // the lane's group, and its first channel there
  bool on;
};
template <int E>
__device__ __forceinline__ Place place(const GroupParams& p) {
  Place q;
  q.b = int(blockIdx.x) / p.nChunk;
  const int k = int(blockIdx.x) - q.b * p.nChunk;
  q.g0 = blockIdx.y * p.gpb;
  q.n = p.lengths != nullptr ? min(max(p.lengths[q.b], 0), p.T) : p.T;
  q.t0 = k * p.chunk;
  q.t1 = min(p.T, q.t0 + p.chunk);
  q.tsub = threadIdx.x / p.lpt;
  q.l = threadIdx.x - q.tsub * p.lpt;
  const int gl = q.l / p.lpg;  // 0 where a group has all lanes
  q.g = q.g0 + (p.gpb > 1 ? gl : 0);
  q.c = (p.gpb > 1 ? q.l - gl * p.lpg : q.l) * E;
  q.on = q.tsub < p.tps && q.g < p.G;
  return q;
}
constexpr int kAhead = 4, kAheadGrad = 2;  // tokens whose loads a lane has under way

// Zeros for the lane's tokens from `end` on (those behind the sequence; nothing of theirs is read).
template <typename ET, int E, bool WHOLE>
__device__ __forceinline__ void zero_tokens(const GroupTensor& out, const GroupParams& p, const Place& q, int end, int c, int n) {
  float zero[E];
#pragma unroll
  for (int e = 0; e < E; ++e) zero[e] = 0.f;
  int t = q.t0 + q.tsub;
  if (t < end) t += (end - t + p.tps - 1) / p.tps * p.tps;
  for (; t < q.t1; t += p.tps) store<ET, E, WHOLE>(zero, out.p, q.b * out.s0 + t * out.s1 + c, n);
}

// Sums over the lanes of each of a workgroup's groups: v[i] of thread (tsub, l). The result of group g is in
// out[g][i] for every thread after the call. red: N values per thread. As many neighbouring threads as there
// are (a power of two) add up a group, in a wave without LDS.
template <int N>
__device__ __forceinline__ void group_sums(const GroupParams& p, const Place& q, const double (&v)[N], double* red,
                                           double* out) {
  const int lanes = p.gpb > 1 ? p.lpg : p.lpt;  // lanes of a group and token
  int per = 1;
  while (per * 2 * p.gpb <= kThreads) per *= 2;
  const int g = threadIdx.x / per, j = threadIdx.x - g * per;
#pragma unroll
  for (int i = 0; i < N; ++i) red[i * kThreads + threadIdx.x] = q.on ? v[i] : 0.0;
  __syncthreads();
  double s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = 0.0;
  if (g < p.gpb)
    for (int e = j; e < lanes * p.tps; e += per) {
      const int at = (e / lanes) * p.lpt + g * lanes + e % lanes;
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] += red[i * kThreads + at];
    }
  for (int m = 1; m < per && m < 64; m *= 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor(s[i], m);
  }
  if (per > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[i * kThreads + (threadIdx.x >> 6)] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = 0.0;
      for (int w = 0; w < per / 64; ++w) s[i] += red[i * kThreads + g * (per / 64) + w];
    }
  }
  if (g < p.gpb && j == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) out[g * N + i] = s[i];
  }
  __syncthreads();
}

template <typename ET, int E, bool WHOLE, bool PACKED>
__global__ __launch_bounds__(kThreads) void k_group_stats(const GroupParams p) {
  using IT = std::conditional_t<PACKED, i8_t, ET>;
  __shared__ double red[kThreads * 2], out[kThreads * 2];
  const Place q = place<E>(p);
  const int end = min(q.t1, q.n);
  typedef Piece<E, WHOLE> P;
  const int n = P::size(p.Cg);
  double v[2] = {0.0, 0.0};  // 64 bits: the squares' sum is good for the variance of any offset that float32 holds
  for (int cl = q.c; q.on && cl < p.Cg; cl += p.lpt * E) {
    const P at(cl, p.Cg);
    const int c = q.g * p.Cg + at.c;
    for (int t = q.t0 + q.tsub; t < end; t += kAhead * p.tps) {
      float x[kAhead][E];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) load_x<IT, E, WHOLE>(x[u], p.x, q.b, min(t + u * p.tps, end - 1), c, n);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (t + u * p.tps < end) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const double one = P::counts(e, at.skip, n) ? x[u][e] : 0.f;
            v[0] += one, v[1] += one * one;
          }
        }
    }
  }
  group_sums<2>(p, q, v, red, out);
  double* part = p.part + int64_t(blockIdx.x) * p.G * 2;
  for (int i = threadIdx.x; i < p.gpb * 2; i += kThreads)
    if (q.g0 + i / 2 < p.G) part[q.g0 * 2 + i] = out[i];
}

template <typename ET, int E, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_group_apply(const GroupParams p) {
  const Place q = place<E>(p);
  if (!q.on) return;
  const int end = min(q.t1, q.n);
  const bool gated = p.gate.p != nullptr, silu = p.silu != 0;
  typedef Piece<E, WHOLE> P;
  const int n = P::size(p.Cg);
  for (int cl = q.c; cl < p.Cg; cl += p.lpt * E) {
    const int c = q.g * p.Cg + P(cl, p.Cg).c;
    float w[E], bi[E];
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = 1.f, bi[e] = 0.f;
    if (p.weight != nullptr) load<ET, E, WHOLE>(w, p.weight, c, n);
    if (p.bias != nullptr) load<ET, E, WHOLE>(bi, p.bias, c, n);
    const float* st = p.stats + (int64_t(q.b) * p.G + q.g) * 2;
    const float mean = st[0], rstd = st[1];
    int t = q.t0 + q.tsub;
    for (; t < end; t += kAhead * p.tps) {
      float x[kAhead][E], g[kAhead][E];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) load_x<ET, E, WHOLE>(x[u], p.x, q.b, min(t + u * p.tps, end - 1), c, n);
      if (gated) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          load<ET, E, WHOLE>(g[u], p.gate.p, q.b * p.gate.s0 + min(t + u * p.tps, end - 1) * p.gate.s1 + c, n);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int tok = t + u * p.tps;
        if (tok >= end) break;
        float y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = value((x[u][e] - mean) * rstd, w[e], bi[e], silu, gated, g[u][e]);
        store<ET, E, WHOLE>(y, p.y.p, q.b * p.y.s0 + tok * p.y.s1 + c, n);
      }
    }
    zero_tokens<ET, E, WHOLE>(p.y, p, q, end, c, n);
  }
}

// Column sums of dz n and dz over a workgroup's tokens.
template <typename ET, int E, bool WHOLE, bool PACKED>
__global__ __launch_bounds__(kThreads) void k_group_columns(const GroupParams p) {
  using IT = std::conditional_t<PACKED, i8_t, ET>;
  __shared__ float fold[kThreads][E + 1];
  const Place q = place<E>(p);
  const int end = min(q.t1, q.n);
  const bool gated = p.gate.p != nullptr, silu = p.silu != 0;
  typedef Piece<E, WHOLE> P;
  const int n = P::size(p.Cg);
  float* part = p.colpart + int64_t(blockIdx.x) * 2 * p.C;
  for (int cb = 0; cb < p.Cg; cb += p.lpt * E) {  // once, but for groups wider than the workgroup
    const P at(q.c + cb, p.Cg);
    const int c = q.g * p.Cg + at.c;
    const bool on = q.on && q.c + cb < p.Cg;
    float dw[E], db[E], w[E], bi[E];
#pragma unroll
    for (int e = 0; e < E; ++e) dw[e] = 0.f, db[e] = 0.f, w[e] = 1.f, bi[e] = 0.f;
    if (on) {
      if (p.weight != nullptr) load<ET, E, WHOLE>(w, p.weight, c, n);
      if (p.bias != nullptr) load<ET, E, WHOLE>(bi, p.bias, c, n);
      const float* st = p.stats + (int64_t(q.b) * p.G + q.g) * 2;
      const float mean = st[0], rstd = st[1];
      for (int t = q.t0 + q.tsub; t < end; t += kAheadGrad * p.tps) {
        float x[kAheadGrad][E], dy[kAheadGrad][E], g[kAheadGrad][E];
#pragma unroll
        for (int u = 0; u < kAheadGrad; ++u) {
          const int64_t tok = min(t + u * p.tps, end - 1);
          load_x<IT, E, WHOLE>(x[u], p.x, q.b, tok, c, n);
          load<ET, E, WHOLE>(dy[u], p.dy.p, q.b * p.dy.s0 + tok * p.dy.s1 + c, n);
        }
        if (gated) {
#pragma unroll
          for (int u = 0; u < kAheadGrad; ++u)
            load<ET, E, WHOLE>(g[u], p.gate.p, q.b * p.gate.s0 + min(t + u * p.tps, end - 1) * p.gate.s1 + c, n);
        }
#pragma unroll
        for (int u = 0; u < kAheadGrad; ++u)
          if (t + u * p.tps < end) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const float norm = (x[u][e] - mean) * rstd;
              float dg;
              const float dz = slope(norm, w[e], bi[e], silu, gated, g[u][e], dy[u][e], dg);
              dw[e] += dz * norm;
              db[e] += dz;
            }
          }
      }
    }
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e) fold[threadIdx.x][e] = which ? db[e] : dw[e];
      __syncthreads();
      if (q.tsub == 0 && on) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (!P::counts(e, at.skip, n)) continue;
          float s = 0.f;
          for (int r = 0; r < p.tps; ++r) s += fold[r * p.lpt + q.l][e];
          part[which * p.C + c + e] = s;
        }
      }
    }
  }
}

// dx (and dgate) of a workgroup's tokens from the sequence's column sums.
template <typename ET, int E, bool WHOLE, bool PACKED>
__global__ __launch_bounds__(kThreads) void k_group_gradient(const GroupParams p) {
  using IT = std::conditional_t<PACKED, i8_t, ET>;
  __shared__ double red[kThreads * 2], out[kThreads * 2];
  const Place q = place<E>(p);
  const int end = min(q.t1, q.n);
  const bool gated = p.gate.p != nullptr, silu = p.silu != 0;
  typedef Piece<E, WHOLE> P;
  const int n = P::size(p.Cg);
  // mean(dn n) and mean(dn) of each group: the column sums with the weight on them
  double v[2] = {0.0, 0.0};
  if (q.on && q.tsub == 0)
    for (int cl = q.c; cl < p.Cg; cl += p.lpt * E) {
      const P at(cl, p.Cg);
      const int c = q.g * p.Cg + at.c;
      float w[E];
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] = 1.f;
      if (p.weight != nullptr) load<ET, E, WHOLE>(w, p.weight, c, n);
      const float* cs = p.colsum + int64_t(q.b) * 2 * p.C + c;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (P::counts(e, at.skip, n)) v[0] += double(w[e]) * double(cs[e]), v[1] += double(w[e]) * double(cs[p.C + e]);
    }
  group_sums<2>(p, q, v, red, out);
  if (!q.on) return;
  const double inv = q.n > 0 ? 1.0 / (double(q.n) * p.Cg) : 0.0;
  for (int cl = q.c; cl < p.Cg; cl += p.lpt * E) {
    const int c = q.g * p.Cg + P(cl, p.Cg).c;
    float w[E], bi[E];
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = 1.f, bi[e] = 0.f;
    if (p.weight != nullptr) load<ET, E, WHOLE>(w, p.weight, c, n);
    if (p.bias != nullptr) load<ET, E, WHOLE>(bi, p.bias, c, n);
    const float* st = p.stats + (int64_t(q.b) * p.G + q.g) * 2;
    const float mean = st[0], rstd = st[1];
    const float m2 = float(out[(q.g - q.g0) * 2] * inv), m1 = float(out[(q.g - q.g0) * 2 + 1] * inv);
    for (int t = q.t0 + q.tsub; t < end; t += kAheadGrad * p.tps) {
      float x[kAheadGrad][E], dy[kAheadGrad][E], gt[kAheadGrad][E];
#pragma unroll
      for (int u = 0; u < kAheadGrad; ++u) {
        const int64_t tok = min(t + u * p.tps, end - 1);
        load_x<IT, E, WHOLE>(x[u], p.x, q.b, tok, c, n);
        load<ET, E, WHOLE>(dy[u], p.dy.p, q.b * p.dy.s0 + tok * p.dy.s1 + c, n);
      }
      if (gated) {
#pragma unroll
        for (int u = 0; u < kAheadGrad; ++u)
          load<ET, E, WHOLE>(gt[u], p.gate.p, q.b * p.gate.s0 + min(t + u * p.tps, end - 1) * p.gate.s1 + c, n);
      }
#pragma unroll
      for (int u = 0; u < kAheadGrad; ++u) {
        const int tok = t + u * p.tps;
        if (tok >= end) break;
        float dx[E], dg[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float norm = (x[u][e] - mean) * rstd;
          dg[e] = 0.f;
          const float dz = slope(norm, w[e], bi[e], silu, gated, gt[u][e], dy[u][e], dg[e]);
          dx[e] = rstd * (dz * w[e] - m1 - norm * m2);
        }
        store<ET, E, WHOLE>(dx, p.dx.p, q.b * p.dx.s0 + tok * p.dx.s1 + c, n);
        if (gated) store<ET, E, WHOLE>(dg, p.dgate.p, q.b * p.dgate.s0 + tok * p.dgate.s1 + c, n);
      }
    }
    zero_tokens<ET, E, WHOLE>(p.dx, p, q, end, c, n);
    if (gated) zero_tokens<ET, E, WHOLE>(p.dgate, p, q, end, c, n);
  }
}

// ---------------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------------
template <typename ET, int E, bool WHOLE, int LPR, int NV>
hipError_t tokens_nv(const GroupParams& p, bool packed, bool bwd, hipStream_t s) {
  GroupParams q = p;
  const int64_t blocks = group_token_blocks(int64_t(p.B) * p.T, p.G, p.Cg, E, bwd, &q.gpw, &q.tpw);
  const dim3 grid(unsigned(blocks), unsigned((p.G + q.gpw - 1) / q.gpw));
  if (!bwd) {
    hipLaunchKernelGGL((k_group_fwd<ET, E, WHOLE, LPR, NV>), grid, dim3(kThreads), 0, s, q);
    return hipGetLastError();
  }
  const size_t lds = NV > 0 && q.tpw > 1 ? size_t(q.tpw) * size_t(q.gpw) * size_t(p.Cg) * sizeof(float) : 0;
  if (packed) {
    hipLaunchKernelGGL((k_group_bwd<ET, E, WHOLE, LPR, NV, true>), grid, dim3(kThreads), lds, s, q);
  } else {
    hipLaunchKernelGGL((k_group_bwd<ET, E, WHOLE, LPR, NV, false>), grid, dim3(kThreads), lds, s, q);
  }
  return hipGetLastError();
}

template <typename ET, bool WHOLE>
hipError_t tokens_e(const GroupParams& p, bool packed, bool bwd, hipStream_t s) {
  constexpr int E = 16 / int(sizeof(ET));
  const GroupPlan pl = group_plan(p.Cg, E);
  if (pl.lpr == 1) return tokens_nv<ET, E, WHOLE, 1, 1>(p, packed, bwd, s);
  if (pl.lpr == 2) return tokens_nv<ET, E, WHOLE, 2, 1>(p, packed, bwd, s);
  if (pl.lpr == 4) return tokens_nv<ET, E, WHOLE, 4, 1>(p, packed, bwd, s);
  if (pl.lpr == 8) return tokens_nv<ET, E, WHOLE, 8, 1>(p, packed, bwd, s);
  if (pl.lpr == 16) return tokens_nv<ET, E, WHOLE, 16, 1>(p, packed, bwd, s);
  if (pl.lpr == 32) return tokens_nv<ET, E, WHOLE, 32, 1>(p, packed, bwd, s);
  if (pl.lpr == 64) {
    if (pl.nv == 1) return tokens_nv<ET, E, WHOLE, 64, 1>(p, packed, bwd, s);
    if (E == 8 || pl.nv == 2) return tokens_nv<ET, E, WHOLE, 64, 2>(p, packed, bwd, s);
    if constexpr (E == 4) return tokens_nv<ET, E, WHOLE, 64, 4>(p, packed, bwd, s);
  }
  if constexpr (E == 8)
    if (pl.nv == 1) return tokens_nv<ET, E, WHOLE, 256, 1>(p, packed, bwd, s);
  if (pl.nv == 2) return tokens_nv<ET, E, WHOLE, 256, 2>(p, packed, bwd, s);
  if (pl.nv == 4) return tokens_nv<ET, E, WHOLE, 256, 4>(p, packed, bwd, s);
  return tokens_nv<ET, E, WHOLE, 256, 0>(p, packed, bwd, s);
}

template <typename ET>
hipError_t tokens(const GroupParams& p, bool whole, bool packed, bool bwd, hipStream_t s) {
  return whole ? tokens_e<ET, true>(p, packed, bwd, s) : tokens_e<ET, false>(p, packed, bwd, s);
}

template <typename ET, bool WHOLE>
hipError_t sequences_e(GroupParams p, bool packed, GroupStage stage, hipStream_t s) {
  constexpr int E = 16 / int(sizeof(ET));
  if (stage == kGroupColumns || stage == kGroupGradient) p.chunk = p.gradChunk, p.nChunk = p.nGradChunk;
  const dim3 grid(unsigned(p.B) * unsigned(p.nChunk), unsigned((p.G + p.gpb - 1) / p.gpb)), block(kThreads);
  if (stage == kGroupStats) {
    if (packed) {
      hipLaunchKernelGGL((k_group_stats<ET, E, WHOLE, true>), grid, block, 0, s, p);
    } else {
      hipLaunchKernelGGL((k_group_stats<ET, E, WHOLE, false>), grid, block, 0, s, p);
    }
  } else if (stage == kGroupApply) {
    hipLaunchKernelGGL((k_group_apply<ET, E, WHOLE>), grid, block, 0, s, p);
  } else if (stage == kGroupColumns) {
    if (packed) {
      hipLaunchKernelGGL((k_group_columns<ET, E, WHOLE, true>), grid, block, 0, s, p);
    } else {
      hipLaunchKernelGGL((k_group_columns<ET, E, WHOLE, false>), grid, block, 0, s, p);
    }
  } else if (packed) {
    hipLaunchKernelGGL((k_group_gradient<ET, E, WHOLE, true>), grid, block, 0, s, p);
  } else {
    hipLaunchKernelGGL((k_group_gradient<ET, E, WHOLE, false>), grid, block, 0, s, p);
  }
  return hipGetLastError();
}

template <typename ET>
hipError_t sequences(const GroupParams& p, bool whole, bool packed, GroupStage stage, hipStream_t s) {
  return whole ? sequences_e<ET, true>(p, packed, stage, s) : sequences_e<ET, false>(p, packed, stage, s);
}

}  // namespace group

}  // namespace dynconv
