// Gated linear scan, gfx950: kernels, compiled once per storage type.
//
//   s = sigmoid(decay),  a = exp(-rate s),  b = sqrt(1 - a^2),  u = b sigmoid(gate) x
//   h_t = a_t h_{t-1} + u_t                      (from zero at a document start)
// and backwards, with e_t = a_{t+1} dh_{t+1}:
//   dh_t = dy_t + e_t,  dx = dh b sigmoid(gate),  dgate = dx x (1 - sigmoid(gate)),
//   dg = a dh h_{t-1} - (a^2 / b) dh sigmoid(gate) x,  ddecay = -dg rate s (1 - s),  drate = -sum dg s
//
// A workgroup owns 64 channels of a sequence and walks along the tokens, a tile at a time. Within a
// tile each group of lanes takes a short run of tokens whose map h -> A h + H it forms from
// zero in registers; the 16 waves' maps meet in LDS, every wave folds those before its own (the same
// fixed order in each, so the carried state is the same bits in all), and the run is gone through
// again from its true start. Inputs are read once, outputs written once, one barrier per tile;
// the next tile's loads are under way meanwhile. The backward forms h and e that way side by side
// (both maps have the same A) from the kept states of every 128th token.
#pragma once

#include <type_traits>

#include "dynconv_common.hpp"
#include "dynconv_scan_internal.hpp"

namespace dynconv {

namespace scan {

constexpr int kThreads = kScanWaves * 64;
constexpr float kLog2e = 1.44269504088896340736f;

// Words that hold N bytes.
template <int N>
struct Word;
template <>
struct Word<1> {
  typedef uint8_t T;
};
template <>
struct Word<2> {
  typedef uint16_t T;
};
template <>
struct Word<4> {
  typedef uint32_t T;
};
template <>
struct Word<8> {
  typedef u32x2 T;
};

struct i8_t {
  int8_t bits;
};

template <typename ET, int V>
struct Elems {  // V adjacent elements of a storage type
  typedef typename Word<sizeof(ET) * V>::T W;
  static __device__ __forceinline__ void get(W w, float (&v)[V]) {
    if constexpr (sizeof(ET) == 4) {
      if constexpr (V == 1) {
        v[0] = __uint_as_float(w);
      } else {
        v[0] = __uint_as_float(w[0]), v[1] = __uint_as_float(w[1]);
      }
    } else if constexpr (sizeof(ET) == 2) {
      if constexpr (V == 1) {
        v[0] = Cvt<ET>::of_bits(w);
      } else {
        v[0] = Cvt<ET>::lo(w), v[1] = Cvt<ET>::hi(w);
      }
    } else {
      v[0] = float(int8_t(w & 0xff));
      if constexpr (V == 2) v[1] = float(int8_t(w >> 8));
    }
  }
  static __device__ __forceinline__ W put(const float (&v)[V]) {
    if constexpr (sizeof(ET) == 4) {
      if constexpr (V == 1) {
        return __float_as_uint(v[0]);
      } else {
        return W{__float_as_uint(v[0]), __float_as_uint(v[1])};
      }
    } else if constexpr (V == 1) {
      return Cvt<ET>::bits(v[0]);
    } else {
      return Cvt<ET>::pack2(v[0], v[1]);
    }
  }
};

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -kLog2e));
}

// (1 - e^-z) for z >= 0. Below a half the difference would cancel: a polynomial for (1 - e^-z) / z,
// interpolated at the six Chebyshev points of [0, 0.5] (5e-8 of the value in float32).
__device__ __forceinline__ float one_minus_exp(float z, float ez) {
  float p = -0x1.267e62p-10f;
  p = __builtin_fmaf(p, z, 0x1.0c5b76p-7f);
  p = __builtin_fmaf(p, z, -0x1.550898p-5f);
  p = __builtin_fmaf(p, z, 0x1.55531cp-3f);
  p = __builtin_fmaf(p, z, -0x1.fffff4p-2f);
  p = __builtin_fmaf(p, z, 1.f);
  return z < 0.5f ? p * z : 1.f - ez;
}

// One token's decay and input scale: a, 1/b (0 where b is 0) and b.
struct Decay {
  float a, rb, b;
};
__device__ __forceinline__ Decay decay_of(float s, float rate) {
  const float g = rate * s;  // -log a
  Decay d;
  d.a = __builtin_amdgcn_exp2f(g * -kLog2e);
  const float q = one_minus_exp(2.f * g, d.a * d.a);
  d.rb = q > 0.f ? __builtin_amdgcn_rsqf(q) : q;  // q of a NaN stays one
  d.b = q * d.rb;
  return d;
}

// Where a lane stands: its channels, its lane group's run of tokens.
template <int V>
struct Lane {
  static constexpr int kLanes = kScanCols / V;  // lanes side by side over the channels
  int wave, group, run, chl;                    // run: index of the lane group's run in the tile
  bool ok;                                      // the channels exist
  uint32_t ch;                                  // first channel within the block, one that exists
  __device__ __forceinline__ Lane(int D, int c0) {
    const int lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    group = lane / kLanes;
    run = wave * V + group;
    chl = (lane % kLanes) * V;
    ok = c0 + chl < D;
    ch = ok ? chl : D - V - c0;
  }
};

// A run's rows of one operand. Rows behind the last token repeat it.
template <typename ET, int V, int L>
struct Rows {
  typedef Elems<ET, V> E;
  typename E::W w[L];
  uint8_t sc[sizeof(ET) == 1 ? L : 1];

  // Tile rows start at token t0; `last` is the tile's last row that exists.
  __device__ __forceinline__ void load(const ScanTensor& t, int b, int t0, int c0, int run, uint32_t ch, int last) {
    const char* base = static_cast<const char*>(t.p) + (b * t.s0 + t0 * t.s1 + c0) * int64_t(sizeof(ET));
    const uint32_t pitch = uint32_t(t.s1) * uint32_t(sizeof(ET));
    const uint32_t end = uint32_t(last) * pitch + ch * uint32_t(sizeof(ET));
    uint32_t off = uint32_t(run * L) * pitch + ch * uint32_t(sizeof(ET));
#pragma unroll
    for (int j = 0; j < L; ++j) {
      w[j] = *reinterpret_cast<const typename E::W*>(base + (run * L + j < last ? off : end));
      off += pitch;
    }
    if constexpr (sizeof(ET) == 1) {
      const uint8_t* sb = t.sc + (b * t.c0 + t0 * t.c1 + c0 / kScanCols);
      const uint32_t sp = uint32_t(t.c1);
#pragma unroll
      for (int j = 0; j < L; ++j) sc[j] = sb[uint32_t(min(run * L + j, last)) * sp];
    }
  }
  __device__ __forceinline__ void get(int j, float (&v)[V]) const {
    E::get(w[j], v);
    if constexpr (sizeof(ET) == 1) {
      const float scale = __uint_as_float(uint32_t(sc[j]) << 23);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= scale;
    }
  }
};

template <typename ET, int V, int L>
__device__ __forceinline__ void store_row(const ScanTensor& t, int b, int t0, int c0, int run, int j, uint32_t ch,
                                          const float (&v)[V]) {
  char* base = static_cast<char*>(const_cast<void*>(t.p)) + (b * t.s0 + t0 * t.s1 + c0) * int64_t(sizeof(ET));
  const uint32_t off = uint32_t(run * L + j) * uint32_t(t.s1) * uint32_t(sizeof(ET)) + ch * uint32_t(sizeof(ET));
  *reinterpret_cast<typename Elems<ET, V>::W*>(base + off) = Elems<ET, V>::put(v);
}

// Document starts of a tile as a bit per token, one tile ahead of their use.
template <int TILE>
struct Starts {
  static constexpr int kWords = TILE / 64;
  static __device__ __forceinline__ void make(const ScanParams& p, int b, int t0, uint64_t* bits) {
    if (threadIdx.x < TILE) {
      const int t = t0 + int(threadIdx.x);
      bool first = false;
      if (t > 0 && t < p.T) {
        const int32_t* s = p.seg + b * p.ss0 + t * p.ss1;
        first = s[0] != s[-p.ss1];
      }
      const uint64_t m = __ballot(first);
      if ((threadIdx.x & 63) == 0) bits[threadIdx.x >> 6] = m;
    }
  }
  // The L bits of a run that lies in one word.
  static __device__ __forceinline__ uint32_t of_run(const uint64_t* bits, int run, int L) {
    return uint32_t(bits[run * L / 64] >> (run * L % 64)) & ((1u << L) - 1u);
  }
};

// h -> A h + H. A of zero (a document start, or a decay to nothing) forgets what came before, a
// NaN of another document too.
__device__ __forceinline__ float through(float A, float H, float h) { return A == 0.f ? H : __builtin_fmaf(A, h, H); }

// ---------------------------------------------------------------------------------
// Forward. MAPS: only the map of the segment, into p.maps; with segment 0 the initial state too.
// ---------------------------------------------------------------------------------
template <typename ET, int V, bool PACKED, bool MAPS>
__global__ __launch_bounds__(kThreads) void k_scan_fwd(const ScanParams p) {
  using IT = std::conditional_t<PACKED, i8_t, ET>;
  constexpr int L = 16 / V;
  __shared__ float maps[2][kScanWaves][kScanCols][2];
  __shared__ uint64_t starts[2][Starts<kScanTile>::kWords];
  const int nCols = (p.D + kScanCols - 1) / kScanCols;
  const int b = int(blockIdx.x) / nCols, c0 = (int(blockIdx.x) - b * nCols) * kScanCols, seg = blockIdx.y;
  const Lane<V> me(p.D, c0);
  const bool gated = p.gate.p != nullptr, docs = p.seg != nullptr;
  float rate[V], carry[V], total[V];
  const int cg = c0 + int(me.ch);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    rate[i] = p.rate[cg + i];
    carry[i] = 0.f;
    total[i] = 1.f;
  }
  if (p.nSeg > 1 && !MAPS) {
    const float2* m = p.maps + (int64_t(b) * p.nSeg) * p.D + cg;
#pragma unroll
    for (int i = 0; i < V; ++i) carry[i] = m[i].y;
    for (int q = 1; q <= seg; ++q) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 f = m[int64_t(q) * p.D + i];
        carry[i] = through(f.x, f.y, carry[i]);
      }
    }
  } else if (p.nSeg == 1 && p.state_in != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) carry[i] = p.state_in[b * p.sis + cg + i];
  }
  const int nTiles = (p.T + kScanTile - 1) / kScanTile;
  const int k0 = seg * p.segTiles, k1 = min(nTiles, k0 + p.segTiles);
  Rows<IT, V, L> rx, ra, rg;
  auto fetch = [&](int k) {
    const int t0 = k * kScanTile, last = min(p.T - t0, kScanTile) - 1;
    rx.load(p.x, b, t0, c0, me.run, me.ch, last);
    ra.load(p.decay, b, t0, c0, me.run, me.ch, last);
    if (gated) rg.load(p.gate, b, t0, c0, me.run, me.ch, last);
  };
  fetch(k0);
  if (docs) {
    Starts<kScanTile>::make(p, b, k0 * kScanTile, starts[k0 & 1]);
    __syncthreads();
  }
  for (int k = k0; k < k1; ++k) {
    const int t0 = k * kScanTile, last = min(p.T - t0, kScanTile) - 1;
    float a[L][V], u[L][V];
#pragma unroll
    for (int j = 0; j < L; ++j) {
      float x[V], r[V], g[V];
      rx.get(j, x);
      ra.get(j, r);
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] = 1.f;
      if (gated) {
        rg.get(j, g);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = sigmoid(g[i]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const Decay d = decay_of(sigmoid(r[i]), rate[i]);
        a[j][i] = d.a;
        u[j][i] = d.b * g[i] * x[i];
      }
    }
    if (last < kScanTile - 1) {  // tokens that do not exist leave the state as it is
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          a[j][i] = me.run * L + j > last ? 1.f : a[j][i];
          u[j][i] = me.run * L + j > last ? 0.f : u[j][i];
        }
    }
    if (docs) {
      const uint32_t m = Starts<kScanTile>::of_run(starts[k & 1], me.run, L);
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) a[j][i] = m >> j & 1 ? 0.f : a[j][i];
    }
    if (k + 1 < k1) fetch(k + 1);
    float A[V], H[V];
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = a[0][i], H[i] = u[0][i];
    if (docs) {
#pragma unroll
      for (int j = 1; j < L; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          H[i] = through(a[j][i], u[j][i], H[i]);
          A[i] = a[j][i] == 0.f ? 0.f : a[j][i] * A[i];
        }
    } else {
#pragma unroll
      for (int j = 1; j < L; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          H[i] = __builtin_fmaf(a[j][i], H[i], u[j][i]);
          A[i] *= a[j][i];
        }
    }
    // the wave's map: its lane groups' one behind the other
    float pA[V], pH[V];  // the map of the lane groups before this one
#pragma unroll
    for (int i = 0; i < V; ++i) pA[i] = 1.f, pH[i] = 0.f;
    if constexpr (V == 2) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float oA = __shfl_xor(A[i], 32), oH = __shfl_xor(H[i], 32);
        const float A0 = me.group ? oA : A[i], H0 = me.group ? oH : H[i];
        const float A1 = me.group ? A[i] : oA, H1 = me.group ? H[i] : oH;
        pA[i] = me.group ? A0 : 1.f;
        pH[i] = me.group ? H0 : 0.f;
        A[i] = A1 == 0.f ? 0.f : A1 * A0;
        H[i] = through(A1, H1, H0);
      }
    }
    if (me.group == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        maps[k & 1][me.wave][me.chl + i][0] = A[i];
        maps[k & 1][me.wave][me.chl + i][1] = H[i];
      }
    }
    if (docs && k + 1 < k1) Starts<kScanTile>::make(p, b, (k + 1) * kScanTile, starts[(k + 1) & 1]);
    __syncthreads();  // the other half's readers are past it: they read it before the barrier before
    float h[V];
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = 0.f;
#pragma unroll 4
    for (int w = 0; w < kScanWaves; ++w) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (w == me.wave) h[i] = carry[i];
        const float fA = maps[k & 1][w][me.chl + i][0], fH = maps[k & 1][w][me.chl + i][1];
        carry[i] = through(fA, fH, carry[i]);
        if constexpr (MAPS) total[i] = fA == 0.f ? 0.f : fA * total[i];
      }
    }
    if constexpr (!MAPS) {
      const int row = me.run * L;
      if (p.chunks != nullptr && me.group == 0 && row % kScanChunk == 0 && row <= last && me.ok) {
        const int nC = (p.T + kScanChunk - 1) / kScanChunk;
        float* out = p.chunks + (int64_t(b) * nC + (t0 + row) / kScanChunk) * p.D + cg;
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = h[i];
      }
      if (p.y.p != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = through(pA[i], pH[i], h[i]);
#pragma unroll
        for (int j = 0; j < L; ++j) {
#pragma unroll
          for (int i = 0; i < V; ++i)
            h[i] = docs ? through(a[j][i], u[j][i], h[i]) : __builtin_fmaf(a[j][i], h[i], u[j][i]);
          if (me.ok && row + j <= last) store_row<ET, V, L>(p.y, b, t0, c0, me.run, j, me.ch, h);
        }
      }
    }
  }
  if (!me.ok || threadIdx.x >= Lane<V>::kLanes) return;
  if constexpr (MAPS) {
    float2* m = p.maps + (int64_t(b) * p.nSeg) * p.D + cg;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (seg == 0) m[i] = float2{0.f, p.state_in != nullptr ? p.state_in[b * p.sis + cg + i] : 0.f};
      m[int64_t(seg + 1) * p.D + i] = float2{total[i], carry[i]};
    }
  } else if (p.state_out != nullptr && k1 == nTiles) {
#pragma unroll
    for (int i = 0; i < V; ++i) p.state_out[b * p.sos + cg + i] = carry[i];
  }
}

// ---------------------------------------------------------------------------------
// Backward, tiles from the last to the first. MAPS: only the segment's map of e.
// ---------------------------------------------------------------------------------
template <typename ET, int V, bool PACKED, bool MAPS>
__global__ __launch_bounds__(kThreads) void k_scan_bwd(const ScanParams p) {
  using IT = std::conditional_t<PACKED, i8_t, ET>;
  constexpr int L = 8 / V;
  __shared__ float maps[2][kScanWaves][kScanCols][MAPS ? 2 : 3];
  __shared__ uint64_t starts[2][Starts<kScanTileBwd>::kWords];
  const int nCols = (p.D + kScanCols - 1) / kScanCols;
  const int b = int(blockIdx.x) / nCols, c0 = (int(blockIdx.x) - b * nCols) * kScanCols;
  const int seg = int(blockIdx.y) + (MAPS ? 1 : 0);
  const Lane<V> me(p.D, c0);
  const bool gated = p.gate.p != nullptr, docs = p.seg != nullptr;
  const int cg = c0 + int(me.ch);
  float rate[V], carry[V], total[V];
  double drate[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    rate[i] = p.rate[cg + i];
    carry[i] = 0.f;
    total[i] = 1.f;
    drate[i] = 0.0;
  }
  if (p.nSeg > 1 && !MAPS) {
    const float2* m = p.maps + (int64_t(b) * p.nSeg) * p.D + cg;
#pragma unroll
    for (int i = 0; i < V; ++i) carry[i] = m[int64_t(p.nSeg - 1) * p.D + i].y;
    for (int q = p.nSeg - 2; q >= seg; --q) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 f = m[int64_t(q) * p.D + i];
        carry[i] = through(f.x, f.y, carry[i]);
      }
    }
  } else if (p.nSeg == 1 && p.dstate_out != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) carry[i] = p.dstate_out[b * p.dsos + cg + i];
  }
  const int nTiles = (p.T + kScanTileBwd - 1) / kScanTileBwd;
  const int k0 = seg * p.segTiles, k1 = min(nTiles, k0 + p.segTiles);
  Rows<IT, V, L> rx, ra, rg;
  Rows<ET, V, L> rd;
  float kept[V];
  auto fetch = [&](int k) {
    const int t0 = k * kScanTileBwd, last = min(p.T - t0, kScanTileBwd) - 1;
    ra.load(p.decay, b, t0, c0, me.run, me.ch, last);
    rd.load(p.dy, b, t0, c0, me.run, me.ch, last);
    if constexpr (!MAPS) {
      rx.load(p.x, b, t0, c0, me.run, me.ch, last);
      if (gated) rg.load(p.gate, b, t0, c0, me.run, me.ch, last);
      const float* c = p.chunks + (int64_t(b) * nTiles + k) * p.D + cg;
#pragma unroll
      for (int i = 0; i < V; ++i) kept[i] = c[i];
    }
  };
  fetch(k1 - 1);
  if (docs) {
    Starts<kScanTileBwd>::make(p, b, (k1 - 1) * kScanTileBwd, starts[(k1 - 1) & 1]);
    __syncthreads();
  }
  for (int k = k1 - 1; k >= k0; --k) {
    const int t0 = k * kScanTileBwd, last = min(p.T - t0, kScanTileBwd) - 1;
    const int row = me.run * L;
    float a[L][V], s[L][V], rb[L][V], b_[L][V], sg[L][V], x[L][V], hb[L][V], dy[L][V];
    float hk[V];
#pragma unroll
    for (int j = 0; j < L; ++j) {
      float r[V];
      ra.get(j, r);
      rd.get(j, dy[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) s[j][i] = sigmoid(r[i]);
      if constexpr (!MAPS) {
        rx.get(j, x[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) sg[j][i] = 1.f;
        if (gated) {
          rg.get(j, sg[j]);
#pragma unroll
          for (int i = 0; i < V; ++i) sg[j][i] = sigmoid(sg[j][i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const Decay d = decay_of(s[j][i], rate[i]);
          a[j][i] = d.a, rb[j][i] = d.rb, b_[j][i] = d.b;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) a[j][i] = __builtin_amdgcn_exp2f(rate[i] * s[j][i] * -kLog2e);
      }
    }
    if (last < kScanTileBwd - 1) {
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const bool gone = row + j > last;
          a[j][i] = gone ? 1.f : a[j][i];
          dy[j][i] = gone ? 0.f : dy[j][i];
          if constexpr (!MAPS) {
            s[j][i] = gone ? 0.f : s[j][i];
            x[j][i] = gone ? 0.f : x[j][i];
            b_[j][i] = gone ? 0.f : b_[j][i];
            rb[j][i] = gone ? 0.f : rb[j][i];
            sg[j][i] = gone ? 0.f : sg[j][i];
          }
        }
    }
    uint32_t first = 0;  // tokens that start a document: nothing passes through them, forwards or backwards
    if (docs) first = Starts<kScanTileBwd>::of_run(starts[k & 1], me.run, L);
#pragma unroll
    for (int i = 0; i < V; ++i) hk[i] = MAPS ? 0.f : kept[i];
    if (k > k0) fetch(k - 1);
    auto pass = [&](int j, int i) { return first >> j & 1 ? 0.f : a[j][i]; };
    float A[V], H[V], E[V];
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = 1.f, H[i] = 0.f, E[i] = 0.f;
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float f = pass(j, i);
        A[i] = f == 0.f ? 0.f : f * A[i];
        if constexpr (!MAPS) H[i] = through(f, b_[j][i] * sg[j][i] * x[j][i], H[i]);
      }
#pragma unroll
    for (int j = L - 1; j >= 0; --j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float f = pass(j, i);
        E[i] = f == 0.f ? 0.f : f * (dy[j][i] + E[i]);
      }
    float pA[V], pH[V], pE[V];  // A: the other lane group's; H before this one, E behind it
#pragma unroll
    for (int i = 0; i < V; ++i) pA[i] = 1.f, pH[i] = 0.f, pE[i] = 0.f;
    if constexpr (V == 2) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float oA = __shfl_xor(A[i], 32), oE = __shfl_xor(E[i], 32);
        const float A0 = me.group ? oA : A[i], A1 = me.group ? A[i] : oA;
        const float E0 = me.group ? oE : E[i], E1 = me.group ? E[i] : oE;
        pA[i] = oA;
        pE[i] = oE;
        A[i] = A0 == 0.f || A1 == 0.f ? 0.f : A1 * A0;
        E[i] = through(A0, E0, E1);
        if constexpr (!MAPS) {
          const float oH = __shfl_xor(H[i], 32);
          const float H0 = me.group ? oH : H[i], H1 = me.group ? H[i] : oH;
          pH[i] = oH;
          H[i] = through(A1, H1, H0);
        }
      }
    }
    if (me.group == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        maps[k & 1][me.wave][me.chl + i][0] = A[i];
        maps[k & 1][me.wave][me.chl + i][1] = E[i];
        if constexpr (!MAPS) maps[k & 1][me.wave][me.chl + i][2] = H[i];
      }
    }
    if (docs && k > k0) Starts<kScanTileBwd>::make(p, b, (k - 1) * kScanTileBwd, starts[(k - 1) & 1]);
    __syncthreads();
    float e[V], h[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = 0.f, h[i] = hk[i];
#pragma unroll 4
    for (int w = kScanWaves - 1; w >= 0; --w) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (w == me.wave) e[i] = carry[i];
        const float fA = maps[k & 1][w][me.chl + i][0], fE = maps[k & 1][w][me.chl + i][1];
        carry[i] = through(fA, fE, carry[i]);
        if constexpr (MAPS) total[i] = fA == 0.f ? 0.f : fA * total[i];
      }
    }
    if constexpr (!MAPS) {
#pragma unroll 1
      for (int w = 0; w < me.wave; ++w) {
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = through(maps[k & 1][w][me.chl + i][0], maps[k & 1][w][me.chl + i][2], h[i]);
      }
      if constexpr (V == 2) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (me.group) {
            h[i] = through(pA[i], pH[i], h[i]);
          } else {
            e[i] = through(pA[i], pE[i], e[i]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float f = pass(j, i);
          hb[j][i] = f == 0.f ? 0.f : h[i];
          h[i] = through(f, b_[j][i] * sg[j][i] * x[j][i], h[i]);
        }
      float sum[V];
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = 0.f;
#pragma unroll
      for (int j = L - 1; j >= 0; --j) {
        float dx[V], dr[V], dg[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float dh = dy[j][i] + e[i];
          const float dhs = dh * sg[j][i];
          dx[i] = dhs * b_[j][i];
          dg[i] = dx[i] * x[j][i] * (1.f - sg[j][i]);
          const float ad = a[j][i] * dh;
          const float dl = s[j][i] * __builtin_fmaf(ad, hb[j][i], -(a[j][i] * a[j][i]) * rb[j][i] * dhs * x[j][i]);
          sum[i] -= dl;
          dr[i] = -rate[i] * dl * (1.f - s[j][i]);
          e[i] = first >> j & 1 ? 0.f : ad;
        }
        if (me.ok && row + j <= last) {
          store_row<ET, V, L>(p.dx, b, t0, c0, me.run, j, me.ch, dx);
          store_row<ET, V, L>(p.ddecay, b, t0, c0, me.run, j, me.ch, dr);
          if (gated) store_row<ET, V, L>(p.dgate, b, t0, c0, me.run, j, me.ch, dg);
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) drate[i] += double(sum[i]);  // 64 bits: of any number of tiles
    }
  }
  if constexpr (MAPS) {
    if (!me.ok || threadIdx.x >= Lane<V>::kLanes) return;
    float2* m = p.maps + (int64_t(b) * p.nSeg) * p.D + cg;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (seg == p.nSeg - 1)
        m[int64_t(seg) * p.D + i] = float2{0.f, p.dstate_out != nullptr ? p.dstate_out[b * p.dsos + cg + i] : 0.f};
      m[int64_t(seg - 1) * p.D + i] = float2{total[i], carry[i]};
    }
  } else {
    // drate of the workgroup: the lane groups' sums in the order of their tokens
    __shared__ double sums[kScanWaves][kScanCols];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (V == 2) drate[i] += __shfl_xor(drate[i], 32);
      if (me.group == 0) sums[me.wave][me.chl + i] = drate[i];
    }
    __syncthreads();
    if (int(threadIdx.x) < kScanCols && c0 + int(threadIdx.x) < p.D) {
      double t = 0.0;
#pragma unroll
      for (int w = 0; w < kScanWaves; ++w) t += sums[w][threadIdx.x];
      p.drate_part[(int64_t(b) * p.nSeg + seg) * p.D + c0 + threadIdx.x] = float(t);
    }
    if (p.dstate != nullptr && k0 == 0 && me.ok && int(threadIdx.x) < Lane<V>::kLanes) {
#pragma unroll
      for (int i = 0; i < V; ++i) p.dstate[b * p.dsis + cg + i] = carry[i];
    }
  }
}

template <typename ET, int V, bool PACKED>
hipError_t launch_fwd(const ScanParams& p, hipStream_t s) {
  const unsigned blocks = unsigned((p.D + kScanCols - 1) / kScanCols) * unsigned(p.B);
  if (p.nSeg > 1) {
    hipLaunchKernelGGL((k_scan_fwd<ET, V, PACKED, true>), dim3(blocks, unsigned(p.nSeg - 1)), dim3(kThreads),
                       0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_scan_fwd<ET, V, PACKED, false>), dim3(blocks, unsigned(p.nSeg)), dim3(kThreads), 0, s,
                     p);
  return hipGetLastError();
}

template <typename ET, int V, bool PACKED>
hipError_t launch_bwd(const ScanParams& p, hipStream_t s) {
  const unsigned blocks = unsigned((p.D + kScanCols - 1) / kScanCols) * unsigned(p.B);
  if (p.nSeg > 1) {
    hipLaunchKernelGGL((k_scan_bwd<ET, V, PACKED, true>), dim3(blocks, unsigned(p.nSeg - 1)), dim3(kThreads),
                       0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_scan_bwd<ET, V, PACKED, false>), dim3(blocks, unsigned(p.nSeg)), dim3(kThreads), 0, s,
                     p);
  return hipGetLastError();
}

template <typename ET>
hipError_t fwd(const ScanParams& p, int vec, bool packed, hipStream_t s) {
  if (vec == 2) return packed ? launch_fwd<ET, 2, true>(p, s) : launch_fwd<ET, 2, false>(p, s);
  return packed ? launch_fwd<ET, 1, true>(p, s) : launch_fwd<ET, 1, false>(p, s);
}
template <typename ET>
hipError_t bwd(const ScanParams& p, int vec, bool packed, hipStream_t s) {
  if (vec == 2) return packed ? launch_bwd<ET, 2, true>(p, s) : launch_bwd<ET, 2, false>(p, s);
  return packed ? launch_bwd<ET, 1, true>(p, s) : launch_bwd<ET, 1, false>(p, s);
}

}  // namespace scan

}  // namespace dynconv
