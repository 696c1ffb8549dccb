// Gated delta rule: workspace layout and the decoding step (the chunked kernels are in
// dynconv_delta_kernels.hpp, compiled once per storage type).
#include "dynconv_common.hpp"
#include "dynconv_delta_internal.hpp"
#include "dynconv_internal.hpp"

namespace dynconv {

namespace {

constexpr size_t kPiece = 256;  // alignment of the workspace's pieces

struct DeltaSizes {
  size_t T, tok, S, U, dot, end, M;
};

DeltaSizes delta_sizes(int64_t B, int64_t T, int64_t Hv, int64_t dk, int64_t dv) {
  const size_t nC = size_t((T + kDeltaChunk - 1) / kDeltaChunk);
  const size_t n = size_t(B) * size_t(Hv) * nC;
  const size_t nCG = size_t((dv + kDeltaCols - 1) / kDeltaCols);
  DeltaSizes z;
  z.T = n * 3 * kTrapElems * sizeof(uint16_t);
  z.tok = n * kTokArrays * kDeltaChunk * sizeof(float);
  z.S = n * nCG * size_t(delta_dk_pad(int(dk))) * kDeltaCols * sizeof(float);
  z.U = n * nCG * kDeltaChunk * kDeltaCols * sizeof(float);
  z.dot = n * nCG * kDeltaChunk * sizeof(float);
  const size_t len = size_t(delta_segment_length(B * Hv, int64_t(nC), int64_t(nCG)));
  const size_t segs = size_t(B) * size_t(Hv) * ((nC + len - 1) / len);
  const size_t pad = size_t(delta_dk_pad(int(dk)));
  z.end = z.M = 0;
  if (nC > len) {
    z.end = segs * nCG * pad * kDeltaCols * sizeof(float);
    z.M = segs * pad * pad * sizeof(float);
  }
  return z;  // every size is a multiple of kPiece
}

}  // namespace

size_t delta_workspace(int64_t B, int64_t T, int64_t Hv, int64_t dk, int64_t dv, bool bwd) {
  const DeltaSizes z = delta_sizes(B, T, Hv, dk, dv);
  if (z.T == 0) return 0;
  return kPiece + z.T + z.tok + z.end + z.M + (bwd ? z.end + 2 * z.S + 2 * z.U + z.dot : 0);
}

void delta_carve(DeltaParams* p, void* ws, bool bwd) {
  const DeltaSizes z = delta_sizes(p->B, p->T, p->Hv, p->dkn, p->dvn);
  char* c = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(ws) + kPiece - 1) / kPiece * kPiece);
  auto take = [&](size_t n) {
    char* r = c;
    c += n;
    return r;
  };
  p->wT = reinterpret_cast<uint16_t*>(take(z.T));
  p->wTok = reinterpret_cast<float*>(take(z.tok));
  p->wEnd = reinterpret_cast<float*>(take(z.end));
  p->wM = reinterpret_cast<float*>(take(z.M));
  if (!bwd) return;
  p->wBegin = reinterpret_cast<float*>(take(z.end));
  p->wS = reinterpret_cast<float*>(take(z.S));
  p->wdS = reinterpret_cast<float*>(take(z.S));
  p->wU = reinterpret_cast<float*>(take(z.U));
  p->wR = reinterpret_cast<float*>(take(z.U));
  p->wDot = reinterpret_cast<float*>(take(z.dot));
}

namespace {

template <typename ET>
__device__ __forceinline__ float sldf(const void* p, int64_t i) {
  if constexpr (sizeof(ET) == 2) {
    return Cvt<ET>::of_bits(static_cast<const uint16_t*>(p)[i]);
  } else {
    return static_cast<const float*>(p)[i];
  }
}

constexpr int kStepCols = 32;                        // value columns of a workgroup
constexpr int kStepRowThreads = 256 * 4 / kStepCols;  // threads down the rows (4 columns each): 32
constexpr int kStepRows = kDeltaMaxDk / kStepRowThreads;

// One token: S' = a S + k u^T, u = beta (v - a S^T k), o = scale S'^T q, with
// S'^T q = a S^T q + (k.q) u, so one pass over S gives both sums and S is read once, kept in
// registers and written once. The state is the traffic (8 bytes per element against a few
// bytes of everything else), so a workgroup takes 32 columns (128-byte row pieces) and every
// thread issues its loads before anything else. Bound by HBM: 99 us for 128 sequences of 32 heads
// of 128 x 128, 5.4 TB/s; 5.6 us for one sequence of 16, of which nearly all is the launch.
template <typename ET, bool VEC>
__global__ __launch_bounds__(256) void k_delta_step(const DeltaStepParams p) {
  __shared__ float sq[kDeltaMaxDk], sk[kDeltaMaxDk], red[4][2][kStepCols], nrm[3];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int ncb = (p.dvn + kStepCols - 1) / kStepCols;
  const uint32_t bid = blockIdx.x;
  const int c0 = int(bid % ncb) * kStepCols;
  const int hv = int(bid / ncb % p.Hv), b = int(bid / ncb / p.Hv), hk = hv / p.group;
  const int col = c0 + (tid & 7) * 4, rg = tid >> 3;
  float* st = p.state + b * p.sts0 + hv * p.sts1;
  float S[kStepRows][4];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int row = rg + kStepRowThreads * i;
#pragma unroll
    for (int e = 0; e < 4; ++e) S[i][e] = 0.f;
    if (row < p.dkn) {
      if constexpr (VEC) {
        if (col < p.dvn) {
          const float4 x = *reinterpret_cast<const float4*>(st + row * p.sts2 + col);
          S[i][0] = x.x, S[i][1] = x.y, S[i][2] = x.z, S[i][3] = x.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < p.dvn) S[i][e] = st[row * p.sts2 + col + e];
      }
    }
  }
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = col + e < p.dvn ? sldf<ET>(p.v, b * p.vs0 + hv * p.vs1 + col + e) : 0.f;
  const float a = expf(p.g[b * p.gs0 + hv * p.gs1]), beta = sldf<ET>(p.beta, b * p.bs0 + hv * p.bs1);
  if (wave < 3) {  // wave 0: q and |q|^2, wave 1: k and |k|^2, wave 2: q.k
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int d = lane + 64 * i;
      const float x = d < p.dkn && wave != 1 ? sldf<ET>(p.q, b * p.qs0 + hk * p.qs1 + d) : 0.f;
      const float y = d < p.dkn && wave != 0 ? sldf<ET>(p.k, b * p.ks0 + hk * p.ks1 + d) : 0.f;
      if (wave == 0) sq[d] = x;
      if (wave == 1) sk[d] = y;
      s += wave == 0 ? x * x : wave == 1 ? y * y : x * y;
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m);
    if (lane == 0) nrm[wave] = s;
  }
  __syncthreads();
  const float rq = p.eps < 0.f ? 1.f : 1.f / sqrtf(nrm[0] + p.eps);
  const float rk = p.eps < 0.f ? 1.f : 1.f / sqrtf(nrm[1] + p.eps);
  float kS[4] = {0.f, 0.f, 0.f, 0.f}, qS[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const float kk = sk[rg + kStepRowThreads * i], qq = sq[rg + kStepRowThreads * i];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      kS[e] += kk * S[i][e];
      qS[e] += qq * S[i][e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll
    for (int m = 8; m < 64; m <<= 1) {
      kS[e] += __shfl_xor(kS[e], m);
      qS[e] += __shfl_xor(qS[e], m);
    }
    if (lane < 8) {
      red[wave][0][(tid & 7) * 4 + e] = kS[e];
      red[wave][1][(tid & 7) * 4 + e] = qS[e];
    }
  }
  __syncthreads();
  float u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int cc = (tid & 7) * 4 + e;
    const float ks = red[0][0][cc] + red[1][0][cc] + red[2][0][cc] + red[3][0][cc];
    const float qs = red[0][1][cc] + red[1][1][cc] + red[2][1][cc] + red[3][1][cc];
    u[e] = beta * (v[e] - a * rk * ks);
    const float o = p.scale * rq * (a * qs + nrm[2] * rk * u[e]);
    if (tid < 8 && col + e < p.dvn) {
      const int64_t at = b * p.os0 + hv * p.os1 + col + e;
      if constexpr (sizeof(ET) == 2) {
        static_cast<uint16_t*>(p.out)[at] = Cvt<ET>::bits(o);
      } else {
        static_cast<float*>(p.out)[at] = o;
      }
    }
    u[e] *= rk;
  }
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int row = rg + kStepRowThreads * i;
    if (row >= p.dkn) continue;
    const float kk = sk[row];
    if constexpr (VEC) {
      if (col < p.dvn)
        *reinterpret_cast<float4*>(st + row * p.sts2 + col) =
            make_float4(a * S[i][0] + kk * u[0], a * S[i][1] + kk * u[1], a * S[i][2] + kk * u[2], a * S[i][3] + kk * u[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < p.dvn) st[row * p.sts2 + col + e] = a * S[i][e] + kk * u[e];
    }
  }
}

template <typename ET>
void launch_step(const DeltaStepParams& p, hipStream_t s) {
  const int64_t blocks = int64_t(p.B) * p.Hv * ((p.dvn + kStepCols - 1) / kStepCols);
  if (p.vec) {
    hipLaunchKernelGGL((k_delta_step<ET, true>), dim3(unsigned(blocks)), dim3(256), 0, s, p);
  } else {
    hipLaunchKernelGGL((k_delta_step<ET, false>), dim3(unsigned(blocks)), dim3(256), 0, s, p);
  }
}

}  // namespace

hipError_t delta_step(const DeltaStepParams& p, dynconv_dtype dt, hipStream_t s) {
  if (dt == DYNCONV_BF16) {
    launch_step<bf16_t>(p, s);
  } else if (dt == DYNCONV_F16) {
    launch_step<f16_t>(p, s);
  } else {
    launch_step<float>(p, s);
  }
  return hipGetLastError();
}

}  // namespace dynconv
