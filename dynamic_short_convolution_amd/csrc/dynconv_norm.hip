// RMS norm with weight, SiLU gate and residual scale, gfx950, forward and backward.
//
//   n = x / sqrt(mean(x^2) + eps),  y = n w silu(z)
//   residual before: h = residual + alpha x (rounded to the storage type, also an output) takes
//   x's place; residual after: y = residual + alpha n w silu(z)
//
// Memory bound: each input is read once and each output written once. A row belongs to 16, 64
// or 256 lanes, the fewest whose registers hold it whole in at most 4 loads of 16 bytes per
// tensor and lane (8 of one element for rows that allow no wide loads), so the mean and the
// result take one pass; longer rows are read again. The weight's gradient is kept per lane
// over all rows of a workgroup, written as one partial row per workgroup and summed in a
// fixed order. Sums are float32; those of many terms, whose roundings can all fall the same way,
// 64-bit: the partial rows', and a lane's over a longer row (up to 65536 terms; costs under 1 %).
// A lane's part of the weight's gradient has at most 512 rows.
// Times, forward / backward: 524288 rows of 128 with a gate, bf16, 85 / 142 us (4.7 TB/s); 32768
// rows of 2048 with the residual before, bf16, 93 / 146 us (5.8 / 4.6 TB/s); 5003 rows of 1537 with
// gate and residual, float32, element by element, 23 / 31 us (5.3 / 4.9 TB/s); longer rows, 4096 of
// 16384, bf16, 60 / 313 us (4.4 / 1.3 TB/s: the backward reads its rows twice and adds to its
// partial row in memory once per row). A large copy reaches 4.8 TB/s.
#include "dynconv_common.hpp"
#include "dynconv_internal.hpp"
#include "dynconv_norm_internal.hpp"

namespace dynconv {

namespace {

constexpr int kThreads = 256;

// E consecutive elements (16 bytes, or one).
template <typename ET, int E>
__device__ __forceinline__ void load(float (&v)[E], const void* base, int64_t off) {
  if constexpr (E == 1) {
    if constexpr (sizeof(ET) == 2) {
      v[0] = Cvt<ET>::of_bits(static_cast<const uint16_t*>(base)[off]);
    } else {
      v[0] = static_cast<const float*>(base)[off];
    }
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const ET*>(base) + off);
    if constexpr (sizeof(ET) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = Cvt<ET>::lo(w[i]);
        v[2 * i + 1] = Cvt<ET>::hi(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    }
  }
}
template <typename ET, int E>
__device__ __forceinline__ void store(const float (&v)[E], const void* base, int64_t off) {
  void* out = const_cast<void*>(base);
  if constexpr (E == 1) {
    if constexpr (sizeof(ET) == 2) {
      static_cast<uint16_t*>(out)[off] = Cvt<ET>::bits(v[0]);
    } else {
      static_cast<float*>(out)[off] = v[0];
    }
  } else {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(ET) == 2) {
        w[i] = Cvt<ET>::pack2(v[2 * i], v[2 * i + 1]);
      } else {
        w[i] = __float_as_uint(v[i]);
      }
    }
    *reinterpret_cast<u32x4*>(static_cast<ET*>(out) + off) = w;
  }
}
template <typename ET>
__device__ __forceinline__ float rounded(float x) {
  if constexpr (sizeof(ET) == 2) {
    return Cvt<ET>::of_bits(Cvt<ET>::bits(x));
  } else {
    return x;
  }
}

// residual + alpha x as float32 arithmetic has it (product and sum rounded separately), then
// the storage type. A fused product would decide ties of the sum by the rounding error of
// alpha: with alpha = 0.22 one in a thousand float16 sums is such a tie.
template <typename ET>
__device__ __forceinline__ float stream_sum(float residual, float alpha, float x) {
#pragma clang fp contract(off)
  const float ax = alpha * x;
  const float h = residual + ax;
  return rounded<ET>(h);
}

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504088896340736f));
}

// Sum over the LPR lanes of a row, in every one of them. `red`: 4 floats per call site.
template <int LPR>
__device__ __forceinline__ float row_sum(float x, float* red) {
#pragma unroll
  for (int m = 1; m < (LPR < 64 ? LPR : 64); m <<= 1) x += __shfl_xor(x, m);
  if constexpr (LPR == 256) {
    __syncthreads();  // the previous sum is read
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = (red[0] + red[1]) + (red[2] + red[3]);
  }
  return x;
}

struct RowAt {
  int64_t i0;
  int32_t i1, i2;
};
__device__ __forceinline__ RowAt row_at(const NormParams& p, int64_t row) {
  RowAt r;
  const int64_t a = row / p.n2;
  r.i2 = int32_t(row - a * p.n2);
  r.i0 = a / p.n1;
  r.i1 = int32_t(a - r.i0 * p.n1);
  return r;
}
__device__ __forceinline__ int64_t at(const NormTensor& t, const RowAt& r) {
  return r.i0 * t.s0 + r.i1 * t.s1 + r.i2 * t.s2;
}

// NV > 0: the row lives in registers (NV vectors of E elements per lane). NV == 0: any length,
// the row is read twice.
template <typename ET, int E, int LPR, int NV>
__global__ __launch_bounds__(kThreads) void k_norm_fwd(const NormParams p) {
  __shared__ float red[4];
  const int lane = threadIdx.x % LPR;
  const int64_t row = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR;
  if (row >= p.rows) return;  // whole rows; with 256 lanes a whole workgroup
  const RowAt r = row_at(p, row);
  const int64_t ox = at(p.x, r), og = at(p.gate, r), orr = at(p.res, r), oy = at(p.y, r), oh = at(p.h, r);
  auto value = [&](float (&v)[E], int c) {  // what is normalised
    load<ET>(v, p.x.p, ox + c);
    if (p.before) {
      float s[E];
      load<ET>(s, p.res.p, orr + c);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = stream_sum<ET>(s[e], p.alpha, v[e]);
    }
  };
  auto finish = [&](const float (&v)[E], const float (&g)[E], const float (&s)[E], float rstd, int c) {
    float w[E], y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = 1.f;
    if (p.weight != nullptr) load<ET>(w, p.weight, c);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      y[e] = v[e] * rstd * w[e];
      if (p.gate.p != nullptr) y[e] *= g[e] * sigmoid(g[e]);
      if (p.after) y[e] = s[e] + p.alpha * y[e];
    }
    store<ET>(y, p.y.p, oy + c);
    if (p.before) store<ET>(v, p.h.p, oh + c);
  };
  const float inv = 1.f / float(p.D);
  if constexpr (NV > 0) {
    float v[NV][E], g[NV][E], s[NV][E];
    float ss = 0.f;
    // every load before the first use, one branch per tensor (a branch between loads makes
    // each wait for the one before); lanes past the row read its start and drop it
    int cc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * LPR) * E;
      cc[i] = c < p.D ? c : 0;
      load<ET>(v[i], p.x.p, ox + cc[i]);
    }
    if (p.res.p != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) load<ET>(s[i], p.res.p, orr + cc[i]);
    }
    if (p.gate.p != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) load<ET>(g[i], p.gate.p, og + cc[i]);
    }
    if (p.before) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) v[i][e] = stream_sum<ET>(s[i][e], p.alpha, v[i][e]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((lane + i * LPR) * E < p.D) {
#pragma unroll
        for (int e = 0; e < E; ++e) ss += v[i][e] * v[i][e];
      }
    const float rstd = 1.f / sqrtf(row_sum<LPR>(ss, red) * inv + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * LPR) * E;
      if (c < p.D) finish(v[i], g[i], s[i], rstd, c);
    }
  } else {
    double ss = 0.0;
    for (int c = lane * E; c < p.D; c += LPR * E) {
      float v[E];
      value(v, c);
#pragma unroll
      for (int e = 0; e < E; ++e) ss += double(v[e]) * double(v[e]);
    }
    const float rstd = 1.f / sqrtf(row_sum<LPR>(float(ss), red) * inv + p.eps);
    for (int c = lane * E; c < p.D; c += LPR * E) {
      float v[E], g[E], s[E];
      value(v, c);
      if (p.gate.p != nullptr) load<ET>(g, p.gate.p, og + c);
      if (p.after) load<ET>(s, p.res.p, orr + c);
      finish(v, g, s, rstd, c);
    }
  }
}

// dn = dy' w silu(z) with dy' = dy (alpha dy with the residual after), c = mean(dn n):
//   dx = (dn - n c) / sqrt(mean(x^2) + eps),  dw += dy' silu(z) n,  dz = dy' n w silu'(z);
// residual before: dresidual = dx + dh, dx = alpha dresidual.
template <typename ET, int E, int LPR, int NV>
__global__ __launch_bounds__(kThreads) void k_norm_bwd(const NormParams p) {
  constexpr int RPB = kThreads / LPR, NA = NV > 0 ? NV : 1;
  __shared__ float red[2][4];
  extern __shared__ float fold[];  // NV > 0 and several rows per pass: [RPB][D]
  const int lane = threadIdx.x % LPR, rg = threadIdx.x / LPR;
  const float inv = 1.f / float(p.D), up = p.after ? p.alpha : 1.f;
  const bool gated = p.gate.p != nullptr;
  float dw[NA][E];
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) dw[i][e] = 0.f;

  // one vector's terms: dn, silu(z) dy' n (weight gradient per unit), and the gate's gradient
  auto terms = [&](const float (&x)[E], const float (&dy)[E], const float (&z)[E], const float (&w)[E], int e, float& dn,
                   float& act, float& dact) {
    act = 1.f;
    dact = 0.f;
    if (gated) {
      const float sg = sigmoid(z[e]);
      act = z[e] * sg;
      dact = sg * (1.f + z[e] * (1.f - sg));
    }
    dn = up * dy[e] * w[e] * act;
  };

  bool first = true;
  for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < p.rows; row0 += int64_t(gridDim.x) * RPB) {
    const int64_t row = row0 + rg;
    const bool have = row < p.rows;
    const RowAt r = row_at(p, have ? row : p.rows - 1);
    const int64_t ox = at(p.x, r), og = at(p.gate, r), ody = at(p.dy, r), odh = at(p.dh, r);
    const int64_t odx = at(p.dx, r), odr = at(p.dres, r), odg = at(p.dgate, r);
    auto finish = [&](const float (&x)[E], const float (&dy)[E], const float (&z)[E], const float (&dh)[E],
                      const float (&w)[E], float rstd, float cm, int c, float (&acc)[E]) {
      float dx[E], dz[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float dn, act, dact;
        terms(x, dy, z, w, e, dn, act, dact);
        const float n = x[e] * rstd;
        dx[e] = rstd * (dn - n * cm);
        dz[e] = up * dy[e] * n * w[e] * dact;
        acc[e] += up * dy[e] * act * n;
      }
      if (gated) store<ET>(dz, p.dgate.p, odg + c);
      if (p.before) {
#pragma unroll
        for (int e = 0; e < E; ++e) dx[e] += dh[e];
        if (p.dres.p != nullptr) store<ET>(dx, p.dres.p, odr + c);
#pragma unroll
        for (int e = 0; e < E; ++e) dx[e] *= p.alpha;
      }
      store<ET>(dx, p.dx.p, odx + c);
    };
    if constexpr (NV > 0) {
      float x[NV][E], dy[NV][E], z[NV][E], dh[NV][E], w[NV][E];
      int cc[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * LPR) * E;
        cc[i] = c < p.D ? c : 0;
        load<ET>(x[i], p.x.p, ox + cc[i]);
        load<ET>(dy[i], p.dy.p, ody + cc[i]);
#pragma unroll
        for (int e = 0; e < E; ++e) w[i][e] = 1.f, dh[i][e] = 0.f;
      }
      if (gated) {
#pragma unroll
        for (int i = 0; i < NV; ++i) load<ET>(z[i], p.gate.p, og + cc[i]);
      }
      if (p.dh.p != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i) load<ET>(dh[i], p.dh.p, odh + cc[i]);
      }
      if (p.weight != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i) load<ET>(w[i], p.weight, cc[i]);
      }
      float ss = 0.f, sd = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((lane + i * LPR) * E < p.D) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            float dn, act, dact;
            terms(x[i], dy[i], z[i], w[i], e, dn, act, dact);
            ss += x[i][e] * x[i][e];
            sd += dn * x[i][e];
          }
        }
      const float rstd = 1.f / sqrtf(row_sum<LPR>(ss, red[0]) * inv + p.eps);
      const float cm = row_sum<LPR>(sd, red[1]) * inv * rstd;
      if (have) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (lane + i * LPR) * E;
          if (c < p.D) finish(x[i], dy[i], z[i], dh[i], w[i], rstd, cm, c, dw[i]);
        }
      }
    } else {
      auto fetch = [&](float (&x)[E], float (&dy)[E], float (&z)[E], float (&w)[E], int c) {
        load<ET>(x, p.x.p, ox + c);
        load<ET>(dy, p.dy.p, ody + c);
        if (gated) load<ET>(z, p.gate.p, og + c);
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = 1.f;
        if (p.weight != nullptr) load<ET>(w, p.weight, c);
      };
      double ss = 0.0, sd = 0.0;
      for (int c = lane * E; c < p.D; c += LPR * E) {
        float x[E], dy[E], z[E], w[E];
        fetch(x, dy, z, w, c);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float dn, act, dact;
          terms(x, dy, z, w, e, dn, act, dact);
          ss += double(x[e]) * double(x[e]);
          sd += double(dn) * double(x[e]);
        }
      }
      const float rstd = 1.f / sqrtf(row_sum<LPR>(float(ss), red[0]) * inv + p.eps);
      const float cm = row_sum<LPR>(float(sd), red[1]) * inv * rstd;
      // the partial sums of a lane's columns stay in the workgroup's own row of memory
      float* part = p.dw_part + int64_t(blockIdx.x) * p.D;
      for (int c = lane * E; c < p.D; c += LPR * E) {
        float x[E], dy[E], z[E], w[E], dh[E], acc[E];
        fetch(x, dy, z, w, c);
#pragma unroll
        for (int e = 0; e < E; ++e) dh[e] = 0.f, acc[e] = 0.f;
        if (p.dh.p != nullptr) load<ET>(dh, p.dh.p, odh + c);
        finish(x, dy, z, dh, w, rstd, cm, c, acc);
        if (p.dw_part != nullptr) {
#pragma unroll
          for (int e = 0; e < E; ++e) part[c + e] = first ? acc[e] : part[c + e] + acc[e];
        }
      }
    }
    first = false;
  }
  if constexpr (NV > 0) {
    if (p.dw_part == nullptr) return;
    float* part = p.dw_part + int64_t(blockIdx.x) * p.D;
    if constexpr (RPB == 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * LPR) * E;
        if (c < p.D) {
#pragma unroll
          for (int e = 0; e < E; ++e) part[c + e] = dw[i][e];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * LPR) * E;
        if (c < p.D) {
#pragma unroll
          for (int e = 0; e < E; ++e) fold[rg * p.D + c + e] = dw[i][e];
        }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < p.D; c += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int g = 0; g < RPB; ++g) s += fold[g * p.D + c];
        part[c] = s;
      }
    }
  }
}

// dweight: the column sums of the partial rows, in 64 bits and a fixed order. A workgroup takes
// 32 columns, its 32 thread groups every 32nd row, eight loads under way at a time; the group
// sums are added by a butterfly (the workgroups are few, so what counts is the length of a
// thread's chain: 1024 rows of 1537 columns 5.8 us, with 8 groups of one load each 48 us).
constexpr int kSumCols = 32, kSumGroups = 32;
__global__ __launch_bounds__(kSumCols * kSumGroups) void k_norm_dweight(const float* __restrict__ part, int64_t n,
                                                                        int32_t D, float* __restrict__ out) {
  __shared__ double red[kSumGroups][kSumCols + 1];
  const int col = threadIdx.x % kSumCols, grp = threadIdx.x / kSumCols;
  const int64_t i = int64_t(blockIdx.x) * kSumCols + col;
  double s = 0.0;
  if (i < D) {
    for (int64_t c = grp; c < n; c += 8 * kSumGroups) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = part[min(c + u * kSumGroups, n - 1) * D + i];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += c + u * kSumGroups < n ? double(v[u]) : 0.0;
    }
  }
  red[grp][col] = s;
  __syncthreads();
  s = red[col][grp];  // group `col`'s sum of column `grp`
#pragma unroll
  for (int m = 1; m < kSumGroups; m <<= 1) s += __shfl_xor(s, m);
  const int64_t o = int64_t(blockIdx.x) * kSumCols + grp;
  if (col == 0 && o < D) out[o] = float(s);
}

// Lanes per row and vectors per lane (0: the looping form) for rows of D elements.
struct NormPlan {
  int lpr, nv;
};
NormPlan norm_plan(int64_t D, int E) {
  const int most = E == 1 ? 8 : 4;
  for (int lpr : {16, 64, 256}) {
    const int64_t per = (D + int64_t(lpr) * E - 1) / (int64_t(lpr) * E);
    if (per > most) continue;
    int nv = 1;
    while (nv < per) nv *= 2;
    return {lpr, nv};
  }
  return {256, 0};
}

int vec_elems(dynconv_dtype dt, bool vec) { return vec ? (dt == DYNCONV_F32 ? 4 : 8) : 1; }

template <typename ET, int E, int LPR, int NV>
hipError_t launch(const NormParams& p, bool bwd, int64_t blocks, hipStream_t s) {
  if (!bwd) {
    constexpr int64_t most = int64_t(1) << 23;  // a dimension of a launch has fewer than 2^32 threads
    const dim3 grid(unsigned(blocks < most ? blocks : most), unsigned((blocks + most - 1) / most));
    hipLaunchKernelGGL((k_norm_fwd<ET, E, LPR, NV>), grid, dim3(kThreads), 0, s, p);
  } else {
    const size_t lds = NV > 0 && LPR < kThreads ? size_t(kThreads / LPR) * size_t(p.D) * sizeof(float) : 0;
    hipLaunchKernelGGL((k_norm_bwd<ET, E, LPR, NV>), dim3(unsigned(blocks)), dim3(kThreads), lds, s, p);
  }
  return hipGetLastError();
}

template <typename ET, int E, int LPR>
hipError_t launch_nv(const NormParams& p, int nv, bool bwd, int64_t blocks, hipStream_t s) {
  if (nv == 1) return launch<ET, E, LPR, 1>(p, bwd, blocks, s);
  if (nv == 2) return launch<ET, E, LPR, 2>(p, bwd, blocks, s);
  if (nv == 4) return launch<ET, E, LPR, 4>(p, bwd, blocks, s);
  if constexpr (E == 1) {
    if (nv == 8) return launch<ET, E, LPR, 8>(p, bwd, blocks, s);
  }
  if constexpr (LPR == 256) return launch<ET, E, LPR, 0>(p, bwd, blocks, s);
  return hipErrorInvalidValue;
}

template <typename ET, int E>
hipError_t launch_lpr(const NormParams& p, bool bwd, int64_t blocks, hipStream_t s) {
  const NormPlan pl = norm_plan(p.D, E);
  if (pl.lpr == 16) return launch_nv<ET, E, 16>(p, pl.nv, bwd, blocks, s);
  if (pl.lpr == 64) return launch_nv<ET, E, 64>(p, pl.nv, bwd, blocks, s);
  return launch_nv<ET, E, 256>(p, pl.nv, bwd, blocks, s);
}

template <typename ET>
hipError_t launch_et(const NormParams& p, bool vec, bool bwd, int64_t blocks, hipStream_t s) {
  return vec ? launch_lpr<ET, 16 / int(sizeof(ET))>(p, bwd, blocks, s) : launch_lpr<ET, 1>(p, bwd, blocks, s);
}

hipError_t dispatch(const NormParams& p, dynconv_dtype dt, bool vec, bool bwd, int64_t blocks, hipStream_t s) {
  if (dt == DYNCONV_BF16) return launch_et<bf16_t>(p, vec, bwd, blocks, s);
  if (dt == DYNCONV_F16) return launch_et<f16_t>(p, vec, bwd, blocks, s);
  return launch_et<float>(p, vec, bwd, blocks, s);
}

}  // namespace

int64_t norm_bwd_blocks(int64_t rows, int64_t D, dynconv_dtype dt, bool vec) {
  const int rpb = kThreads / norm_plan(D, vec_elems(dt, vec)).lpr;
  const int64_t need = (rows + rpb - 1) / rpb;
  // four workgroups per CU, and more where a lane would add over 512 rows to its float32 sums
  const int64_t most = need > 512 * 1024 ? (need + 511) / 512 : 1024;
  return need < most ? need : most;
}

int64_t norm_bwd_blocks_max(int64_t rows, int64_t D, dynconv_dtype dt) {
  const int64_t a = norm_bwd_blocks(rows, D, dt, true), b = norm_bwd_blocks(rows, D, dt, false);
  return a > b ? a : b;
}

hipError_t norm_dweight(const float* part, int64_t n, int32_t D, float* out, hipStream_t s) {
  hipLaunchKernelGGL(k_norm_dweight, dim3(unsigned((D + kSumCols - 1) / kSumCols)), dim3(kSumCols * kSumGroups), 0, s,
                     part, n, D, out);
  return hipGetLastError();
}

hipError_t norm_fwd(const NormParams& p, dynconv_dtype dt, bool vec, hipStream_t s) {
  const int rpb = kThreads / norm_plan(p.D, vec_elems(dt, vec)).lpr;
  return dispatch(p, dt, vec, false, (p.rows + rpb - 1) / rpb, s);
}

hipError_t norm_bwd(const NormParams& p, dynconv_dtype dt, bool vec, hipStream_t s) {
  return dispatch(p, dt, vec, true, norm_bwd_blocks(p.rows, p.D, dt, vec), s);
}

}  // namespace dynconv

// ---------------------------------------------------------------------------------
// C ABI
// ---------------------------------------------------------------------------------

using namespace dynconv;

namespace {

int elem_bytes(dynconv_dtype dt) { return dt == DYNCONV_F32 ? 4 : 2; }
bool aligned(const void* p, int64_t a) { return (reinterpret_cast<uintptr_t>(p) % uint64_t(a)) == 0; }

struct Shape {
  int64_t n[3], D;
};

dynconv_status check_shape(const Shape& z, dynconv_dtype dt, float eps) {
  if (dt != DYNCONV_F32 && dt != DYNCONV_BF16 && dt != DYNCONV_F16) return DYNCONV_ERR_INVALID_ARG;
  for (int64_t n : z.n)
    if (n < 0) return DYNCONV_ERR_INVALID_ARG;
  if (z.D < 0 || !(eps >= 0.f)) return DYNCONV_ERR_INVALID_ARG;
  for (int64_t n : z.n)
    if (n > INT32_MAX) return DYNCONV_ERR_UNSUPPORTED;
  if (z.D > (int64_t(1) << 24)) return DYNCONV_ERR_UNSUPPORTED;
  if (z.n[0] == 0 || z.n[1] == 0 || z.n[2] == 0) return DYNCONV_OK;
  if (z.n[0] > INT32_MAX / z.n[1] || z.n[0] * z.n[1] > INT32_MAX / z.n[2]) return DYNCONV_ERR_UNSUPPORTED;
  return DYNCONV_OK;
}

bool empty(const Shape& z) { return z.n[0] == 0 || z.n[1] == 0 || z.n[2] == 0 || z.D == 0; }

// Takes a tensor [n0,n1,n2,D] with strides s[0..3] into t; clears *vec when its rows do not
// allow 16-byte accesses.
dynconv_status take(NormTensor* t, const void* p, const int64_t* s, const Shape& z, int eb, bool required, bool output,
                    bool* vec) {
  if (p == nullptr) return required ? DYNCONV_ERR_INVALID_ARG : DYNCONV_OK;
  if (s == nullptr) return DYNCONV_ERR_INVALID_ARG;
  if (!aligned(p, eb) || (z.D > 1 && s[3] != 1)) return DYNCONV_ERR_UNSUPPORTED;
  if (!aligned(p, 16)) *vec = false;
  for (int i = 0; i < 3; ++i) {
    if (s[i] < 0) return DYNCONV_ERR_UNSUPPORTED;
    if (z.n[i] <= 1) continue;
    if (output && s[i] == 0) return DYNCONV_ERR_INVALID_ARG;
    if (s[i] * eb % 16 != 0) *vec = false;
  }
  t->p = p;
  t->s0 = s[0], t->s1 = s[1], t->s2 = s[2];
  return DYNCONV_OK;
}

dynconv_status take_weight(const void* w, int eb, bool* vec) {
  if (w == nullptr) return DYNCONV_OK;
  if (!aligned(w, eb)) return DYNCONV_ERR_UNSUPPORTED;
  if (!aligned(w, 16)) *vec = false;
  return DYNCONV_OK;
}

}  // namespace

extern "C" {

dynconv_status dynconv_norm_fwd(const void* x, const int64_t* xs, const void* weight, const void* gate,
                                const int64_t* gs, const void* residual, const int64_t* rs, int32_t residual_after,
                                float residual_scale, void* y, const int64_t* ys, void* h, const int64_t* hs, int64_t n0,
                                int64_t n1, int64_t n2, int64_t D, float eps, dynconv_dtype dtype, void* stream) {
  const Shape z{{n0, n1, n2}, D};
  dynconv_status st = check_shape(z, dtype, eps);
  if (st != DYNCONV_OK) return st;
  if (empty(z)) return DYNCONV_OK;
  const int eb = elem_bytes(dtype);
  NormParams p{};
  bool vec = D * eb % 16 == 0;
  p.before = residual != nullptr && !residual_after;
  p.after = residual != nullptr && residual_after;
  if ((st = take(&p.x, x, xs, z, eb, true, false, &vec)) != DYNCONV_OK) return st;
  if ((st = take(&p.gate, gate, gs, z, eb, false, false, &vec)) != DYNCONV_OK) return st;
  if ((st = take(&p.res, residual, rs, z, eb, false, false, &vec)) != DYNCONV_OK) return st;
  if ((st = take(&p.y, y, ys, z, eb, true, true, &vec)) != DYNCONV_OK) return st;
  if (p.before && (st = take(&p.h, h, hs, z, eb, true, true, &vec)) != DYNCONV_OK) return st;
  if ((st = take_weight(weight, eb, &vec)) != DYNCONV_OK) return st;
  for (const void* in : {x, weight, gate, residual})
    if (in != nullptr && (in == y || (p.before && in == h))) return DYNCONV_ERR_INVALID_ARG;
  if (p.before && y == h) return DYNCONV_ERR_INVALID_ARG;
  p.weight = weight;
  p.rows = n0 * n1 * n2;
  p.n1 = int32_t(n1), p.n2 = int32_t(n2), p.D = int32_t(D);
  p.alpha = residual_scale;
  p.eps = eps;
  const hipError_t e = norm_fwd(p, dtype, vec, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? DYNCONV_OK : record_hip_error(e);
}

size_t dynconv_norm_bwd_workspace_size(int64_t n0, int64_t n1, int64_t n2, int64_t D, dynconv_dtype dtype) {
  const Shape z{{n0, n1, n2}, D};
  if (check_shape(z, dtype, 0.f) != DYNCONV_OK || empty(z)) return 0;
  return size_t(norm_bwd_blocks_max(n0 * n1 * n2, D, dtype)) * size_t(D) * sizeof(float);
}

dynconv_status dynconv_norm_bwd(const void* x, const int64_t* xs, const void* weight, const void* gate,
                                const int64_t* gs, const void* dy, const int64_t* dys, const void* dh,
                                const int64_t* dhs, int32_t residual_at, float residual_scale, void* dx,
                                const int64_t* dxs, void* dresidual, const int64_t* drs, float* dweight, void* dgate,
                                const int64_t* dgs, int64_t n0, int64_t n1, int64_t n2, int64_t D, float eps,
                                dynconv_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const Shape z{{n0, n1, n2}, D};
  dynconv_status st = check_shape(z, dtype, eps);
  if (st != DYNCONV_OK) return st;
  if (residual_at < DYNCONV_NORM_NO_RESIDUAL || residual_at > DYNCONV_NORM_RESIDUAL_AFTER) return DYNCONV_ERR_INVALID_ARG;
  if (D == 0) return DYNCONV_OK;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (dweight != nullptr && !aligned(dweight, 4)) return DYNCONV_ERR_UNSUPPORTED;
  if (empty(z)) {
    const hipError_t e = dweight == nullptr ? hipSuccess : norm_dweight(nullptr, 0, int32_t(D), dweight, s);
    return e == hipSuccess ? DYNCONV_OK : record_hip_error(e);
  }
  const int eb = elem_bytes(dtype);
  NormParams p{};
  bool vec = D * eb % 16 == 0;
  p.before = residual_at == DYNCONV_NORM_RESIDUAL_BEFORE;
  p.after = residual_at == DYNCONV_NORM_RESIDUAL_AFTER;
  if (!p.before && (dh != nullptr || dresidual != nullptr)) return DYNCONV_ERR_INVALID_ARG;
  if ((st = take(&p.x, x, xs, z, eb, true, false, &vec)) != DYNCONV_OK) return st;
  if ((st = take(&p.gate, gate, gs, z, eb, false, false, &vec)) != DYNCONV_OK) return st;
  if ((st = take(&p.dy, dy, dys, z, eb, true, false, &vec)) != DYNCONV_OK) return st;
  if ((st = take(&p.dh, dh, dhs, z, eb, false, false, &vec)) != DYNCONV_OK) return st;
  if ((st = take(&p.dx, dx, dxs, z, eb, true, true, &vec)) != DYNCONV_OK) return st;
  if ((st = take(&p.dres, dresidual, drs, z, eb, false, true, &vec)) != DYNCONV_OK) return st;
  if ((st = take(&p.dgate, dgate, dgs, z, eb, gate != nullptr, true, &vec)) != DYNCONV_OK) return st;
  if (gate == nullptr && dgate != nullptr) return DYNCONV_ERR_INVALID_ARG;
  if ((st = take_weight(weight, eb, &vec)) != DYNCONV_OK) return st;
  const void* outs[4] = {dx, dresidual, dweight, dgate};
  for (int i = 0; i < 4; ++i) {
    if (outs[i] == nullptr) continue;
    for (const void* in : {x, weight, gate, dy, dh})
      if (in == outs[i]) return DYNCONV_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (outs[j] == outs[i]) return DYNCONV_ERR_INVALID_ARG;
  }
  p.weight = weight;
  p.rows = n0 * n1 * n2;
  p.n1 = int32_t(n1), p.n2 = int32_t(n2), p.D = int32_t(D);
  p.alpha = residual_scale;
  p.eps = eps;
  if (dweight != nullptr) {
    if (workspace == nullptr || workspace_bytes < dynconv_norm_bwd_workspace_size(n0, n1, n2, D, dtype))
      return DYNCONV_ERR_WORKSPACE;
    if (!aligned(workspace, 4)) return DYNCONV_ERR_UNSUPPORTED;
    p.dw_part = static_cast<float*>(workspace);
  }
  hipError_t e = norm_bwd(p, dtype, vec, s);
  if (e == hipSuccess && dweight != nullptr)
    e = norm_dweight(p.dw_part, norm_bwd_blocks(p.rows, D, dtype, vec), p.D, dweight, s);
  return e == hipSuccess ? DYNCONV_OK : record_hip_error(e);
}

}  // extern "C"
