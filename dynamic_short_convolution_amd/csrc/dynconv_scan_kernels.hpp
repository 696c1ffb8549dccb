// Gated linear scan, gfx950: kernels, compiled once per storage type.
//
//   s = sigmoid(decay),  a = exp(-rate s),  b = sqrt(1 - a^2),  u = b sigmoid(gate) x
//   h_t = a_t h_{t-1} + u_t                      (from zero at a document start)
// and backwards, with e_t = a_{t+1} dh_{t+1}:
//   dh_t = dy_t + e_t,  dx = dh b sigmoid(gate),  dgate = dx x (1 - sigmoid(gate)),
//   dg = a dh h_{t-1} - (a^2 / b) dh sigmoid(gate) x,  ddecay = -dg rate s (1 - s),  drate = -sum dg s
//
// A workgroup owns 64 channels of a sequence and walks along the tokens, a tile of 128 at a time. Within a
// tile each group of lanes takes a run of 8 or 16 tokens, whose map h -> A h + H it forms from zero in
// registers; the 8 waves' maps meet in LDS, every wave folds those before its own (the same fixed order in
// each, so the carried state is the same bits in all), and the run is gone through again from its true
// start. Inputs are read once, outputs written once, one barrier per tile. The backward forms h and e that
// way side by side (both maps have the same A) from the kept states of every 128th token.
//
// What bounds it is the time that its loads take to come: one workgroup per CU (its registers: 8 waves of up to
// 256) reads 128-byte pieces of rows that lie a row apart. The forward has two tiles' loads under way, the
// backward one. 8 sequences of 4096 tokens, 2048 channels, bf16 (537 MB forward, 940 MB backward): 128 to
// 134 us (4.0 to 4.2 TB/s; the same reads and writes with a sum in place of the scan take 118 to 122, however
// wide, deep or many the loads, and one after the other through memory 96), backward 206 to 226 us (4.2
// to 4.6 TB/s). Vector units are busy 48 % of the forward's time and 60 % of the backward's. Both directions
// when they took 342 us: with 32 channels per workgroup 438, with 16 waves of 8 elements per lane 394.
#pragma once

#include <type_traits>

#include "dynconv_common.hpp"
#include "dynconv_scan_internal.hpp"

namespace dynconv {

namespace scan {

constexpr int kThreads = kScanWaves * 64;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kAhead = 8;  // segments' maps whose loads are under way at a time

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
    } else {  // codes
      v[0] = float(int32_t(uint32_t(w) << 24) >> 24);
      if constexpr (V == 2) v[1] = float(int32_t(uint32_t(w) << 16) >> 24);
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

// 1 / (1 + 2^e): the sigmoid of -e log 2.
__device__ __forceinline__ float sigmoid_of(float e) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(e)); }
__device__ __forceinline__ float sigmoid(float z) { return sigmoid_of(z * -kLog2e); }
// 1 - s for s = 1 / (1 + p), without the difference, of which nothing is left for an open gate: p s, and 1 where p is
// infinite and s 0 (of infinity times 0, a NaN, the minimum is its other operand; where p is a NaN, s is one too).
__device__ __forceinline__ float rest_of(float p, float s) { return fminf(p * s, 1.f); }

// 1 - a^2 for a = 2^-v, v >= 0. At small v the difference would cancel: a polynomial for
// (1 - 2^-2v) / v, interpolated at the six Chebyshev points of [0, 0.36] (1.2e-7 of the value in float32);
// above, a^2 is at most 0.61.
__device__ __forceinline__ float one_minus_square(float v, float a) {
  float p = -0x1.0563dcp-7f;
  p = __builtin_fmaf(p, v, 0x1.57861ep-5f);
  p = __builtin_fmaf(p, v, -0x1.3ae43ap-3f);
  p = __builtin_fmaf(p, v, 0x1.c6ad9cp-2f);
  p = __builtin_fmaf(p, v, -0x1.ebfbd4p-1f);
  p = __builtin_fmaf(p, v, 0x1.62e430p+0f);
  float small = p * v, large = __builtin_fmaf(-a, a, 1.f);
  asm("" : "+v"(small), "+v"(large));  // both formed: without this the compiler makes a divergent branch of every element
  return v < 0.36f ? small : large;
}

// One token's decay and input scale: a, 1/b (0 where b is 0) and b. rate: in units of log 2. The instructions of
// roots and reciprocals take a denormal as zero, so b of a denormal 1 - a^2 is 0, as the forward's root has it, and
// 1/b must not become infinite.
struct Decay {
  float a, rb, b;
};
__device__ __forceinline__ Decay decay_of(float s, float rate) {
  const float v = rate * s;  // -log2 a
  Decay d;
  d.a = __builtin_amdgcn_exp2f(-v);
  const float q = one_minus_square(v, d.a);
  d.rb = __builtin_fabsf(q) < 0x1p-126f ? 0.f : __builtin_amdgcn_rsqf(q);
  d.b = q * d.rb;
  return d;
}

constexpr uint32_t kNowhere = 0x80000000u;  // an offset behind every buffer's range

// The (sequence, 64 channels) pair of a workgroup. Where the 64 channels of a row are not whole 128-byte lines,
// workgroups side by side share lines, so they go to one XCD and its L2 (64 sequences of 2000 tokens, 500 channels,
// bf16: forward 117 us, apart 147, backward 216 and 311; 8 of 4096 x 2048 from 8-bit inputs 551 and 558 in all).
// Else they go to the XCDs in turn (8 sequences of 1953 tokens, 4096 channels: forward 123 us, in one XCD 131,
// backward 214 and 229).
__device__ __forceinline__ int block_at(const ScanParams& p) {
  return int(p.shared ? xcd_logical_block(blockIdx.x, gridDim.x) : blockIdx.x);
}

// Where a lane stands: its channels, its lane group's run of tokens.
template <int V>
struct Lane {
  static constexpr int kLanes = kScanCols / V;  // lanes side by side over the channels
  static constexpr int kGroups = 64 / kLanes;
  int wave, group, run, chl;                    // run: index of the lane group's run in the tile
  bool ok;                                      // the channels exist
  int cg;                                       // the first of them, or the tensor's last
  __device__ __forceinline__ Lane(int D, int c0) {
    const int lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    group = lane / kLanes;
    run = wave * kGroups + group;
    chl = (lane % kLanes) * V;
    ok = c0 + chl < D;
    cg = ok ? c0 + chl : D - V;
  }
};

// A tile's rows of one tensor through buffer instructions: a uniform descriptor per tile whose range
// ends with the last row that exists, the lane's place in its first row as vector offset, the row as
// scalar offset (both count for the range), so rows and channels that do not exist read as zero and
// are not written, without a branch or an address per row.
template <typename ET, int V, int L>
struct Place {
  uint32_t off, pitch;
  __device__ __forceinline__ Place(const ScanTensor& t, const Lane<V>& me) {
    pitch = uint32_t(t.s1) * uint32_t(sizeof(ET));
    off = me.ok ? uint32_t(me.run * L) * pitch + uint32_t(me.chl) * uint32_t(sizeof(ET)) : kNowhere;
  }
  // Of tile k of k0 .. k1 - 1, or (another one, or no tensor) an empty range. Accesses without a branch
  // around them: where paths with and without loads meet, the compiler has to wait as if the later
  // ones had not been issued, which would undo the loads ahead.
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(const ScanTensor& t, int b, int k, int k0, int k1, int c0, int T, int D) const {
    const char* base = static_cast<const char*>(t.p) + (b * t.s0 + int64_t(k) * kScanTile * t.s1 + c0) * int64_t(sizeof(ET));
    const int last = min(T - k * kScanTile, kScanTile) - 1;
    uint32_t range = uint32_t(last) * pitch + uint32_t(min(D - c0, kScanCols)) * uint32_t(sizeof(ET));
    if (t.p == nullptr || k < k0 || k >= k1) range = 0;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, int(range), 0x00027000);
  }
};

// A run's rows of one operand.
template <typename ET, int V, int L>
struct Rows {
  typedef Elems<ET, V> E;
  typename E::W w[L];

  __device__ __forceinline__ void load(const Place<ET, V, L>& at, __amdgpu_buffer_rsrc_t r) {
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const int row = int(uint32_t(j) * at.pitch);
      if constexpr (sizeof(w[0]) == 1) {
        w[j] = __builtin_amdgcn_raw_buffer_load_b8(r, int(at.off), row, 0);
      } else if constexpr (sizeof(w[0]) == 2) {
        w[j] = __builtin_amdgcn_raw_buffer_load_b16(r, int(at.off), row, 0);
      } else if constexpr (sizeof(w[0]) == 4) {
        w[j] = __builtin_amdgcn_raw_buffer_load_b32(r, int(at.off), row, 0);
      } else {
        w[j] = __builtin_amdgcn_raw_buffer_load_b64(r, int(at.off), row, 0);
      }
    }
  }
  __device__ __forceinline__ void get(int j, float (&v)[V]) const { E::get(w[j], v); }
};

template <typename ET, int V, int L>
__device__ __forceinline__ void store_row(const Place<ET, V, L>& at, __amdgpu_buffer_rsrc_t r, int j, const float (&v)[V]) {
  const auto w = Elems<ET, V>::put(v);
  const int row = int(uint32_t(j) * at.pitch);
  if constexpr (sizeof(w) == 2) {
    __builtin_amdgcn_raw_buffer_store_b16(w, r, int(at.off), row, 0);
  } else if constexpr (sizeof(w) == 4) {
    __builtin_amdgcn_raw_buffer_store_b32(w, r, int(at.off), row, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b64(w, r, int(at.off), row, 0);
  }
}

// The steps of a tile's operands in 8 bits (those of decay and gate times -log2 e, as the exponential of
// their sigmoid takes them): a thread loads one of (operand, token), one tile before they are put into
// LDS, which is one tile before their use.
struct Steps {
  uint32_t held;
  __device__ __forceinline__ void load(const ScanParams& p, int b, int k, int c0) {
    const int which = threadIdx.x / kScanTile;
    const int64_t row = min(k * kScanTile + int(threadIdx.x % kScanTile), p.T - 1);
    const uint8_t* sc = p.x.sc + (b * p.x.c0 + row * p.x.c1);
    if (which == 1) sc = p.decay.sc + (b * p.decay.c0 + row * p.decay.c1);
    if (which == 2 && p.gate.sc != nullptr) sc = p.gate.sc + (b * p.gate.c0 + row * p.gate.c1);
    held = sc[c0 / kScanScaleCols];
  }
  __device__ __forceinline__ void put(float (&to)[3][kScanTile]) const {
    const int which = threadIdx.x / kScanTile;
    const float step = __uint_as_float(held << 23);
    if (which < 3) to[which][threadIdx.x % kScanTile] = which == 0 ? step : step * -kLog2e;
  }
};
// Document starts of a tile as a bit per token: a thread loads a token's id and the one before, one tile
// before the bits are put into LDS, which is one tile before their use.
struct Starts {
  static constexpr int kWords = kScanTile / 64;
  int32_t id, before;
  bool counts;
  __device__ __forceinline__ void load(const ScanParams& p, int b, int k) {
    const int t = k * kScanTile + int(threadIdx.x % kScanTile), at = min(t, p.T - 1);
    const int32_t* s = p.seg + b * p.ss0;
    id = s[at * p.ss1];
    before = s[max(at - 1, 0) * p.ss1];
    counts = t < p.T;  // token 0 differs from no id before it
  }
  __device__ __forceinline__ void put(uint64_t* bits) const {
    const uint64_t m = __ballot(counts && id != before);
    if (threadIdx.x < kScanTile && (threadIdx.x & 63) == 0) bits[threadIdx.x >> 6] = m;
  }
  // The L bits of a run that lies in one word.
  static __device__ __forceinline__ uint32_t of_run(const uint64_t* bits, int run, int L) {
    return uint32_t(bits[run * L / 64] >> (run * L % 64)) & ((1u << L) - 1u);
  }
};

// h -> A h + H. With documents a factor of -0 marks a map that holds a document's start: it forgets what came before,
// a NaN of another document too. Decays are positive, so a product of them that underflows is +0 and lets a NaN or
// infinity of its own document through.
__device__ __forceinline__ bool forgets(float A) { return __float_as_uint(A) == 0x80000000u; }
template <bool DOCS>
__device__ __forceinline__ float through(float A, float H, float h) {
  const float r = __builtin_fmaf(A, h, H);
  return DOCS && forgets(A) ? H : r;
}
// The product of two maps' factors: what either of them forgets is forgotten, whatever the other one is (the factors of
// a run serve both directions, in which a NaN is before or behind the document start).
template <bool DOCS>
__device__ __forceinline__ float chain(float A, float B) {
  return DOCS && (forgets(A) || forgets(B)) ? -0.f : A * B;
}

// Of the lane groups of a wave, one behind the other: the maps (A, H) become those of the group and all
// before it (or, REVERSE, behind it), and (pA, pH) those without its own.
template <int V, bool DOCS, bool REVERSE>
__device__ __forceinline__ void scan_groups(const Lane<V>& me, float (&A)[V], float (&H)[V], float (&pA)[V], float (&pH)[V]) {
  constexpr int kLanes = Lane<V>::kLanes, kGroups = Lane<V>::kGroups;
  auto from = [&](float v, int d) { return REVERSE ? __shfl_down(v, d * kLanes) : __shfl_up(v, d * kLanes); };
  const int rank = REVERSE ? kGroups - 1 - me.group : me.group;
#pragma unroll
  for (int d = 1; d < kGroups; d *= 2) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float oA = from(A[i], d), oH = from(H[i], d);
      const float h = through<DOCS>(A[i], H[i], oH), a = chain<DOCS>(A[i], oA);
      H[i] = rank >= d ? h : H[i];
      A[i] = rank >= d ? a : A[i];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    pA[i] = 1.f;
    pH[i] = 0.f;
    if constexpr (kGroups > 1) {
      const float oA = from(A[i], 1), oH = from(H[i], 1);
      pA[i] = rank > 0 ? oA : 1.f;
      pH[i] = rank > 0 ? oH : 0.f;
    }
  }
}

// The maps of the waves in LDS, read in pieces of a lane's channels.
template <int V>
__device__ __forceinline__ void read_map(const float (&m)[kScanCols], int chl, float (&v)[V]) {
  if constexpr (V == 2) {
    const float2 f = *reinterpret_cast<const float2*>(&m[chl]);
    v[0] = f.x, v[1] = f.y;
  } else {
    v[0] = m[chl];
  }
}
template <int V>
__device__ __forceinline__ void write_map(float (&m)[kScanCols], int chl, const float (&v)[V]) {
  if constexpr (V == 2) {
    *reinterpret_cast<float2*>(&m[chl]) = float2{v[0], v[1]};
  } else {
    m[chl] = v[0];
  }
}

// ---------------------------------------------------------------------------------
// Forward: the outputs (and the kept and last states), the kept states alone (for a backward that has to
// recompute them), or only the map of the segment, into p.maps; with segment 0 the initial state too. That pass
// goes from the last tile to the first, so that what it read last, which the memory-side cache still
// holds, is what the pass behind it reads first (32768 tokens of 2048 channels, 8 segments: 96 to 106 us and then
// 111 to 119; a call 209, the other way round 216 where it took 210). The states alone of 8 x 4096 x 2048: from 8-bit
// inputs 97 to 105 us, from bf16 113 to 119 (the outputs' variant, its stores switched off at run time, made a training
// step from 8-bit inputs 565 us that takes 554 with this one).
// ---------------------------------------------------------------------------------
enum Want { kOutputs, kStates, kMaps };
template <typename ET, int V, bool PACKED, bool DOCS, Want WANT>
__global__ __launch_bounds__(kThreads, 2) void k_scan_fwd(const ScanParams p) {
  constexpr bool MAPS = WANT == kMaps;
  using IT = std::conditional_t<PACKED, i8_t, ET>;
  constexpr int L = kScanElems / V;
  __shared__ float maps[2][2][kScanWaves][kScanCols];  // [tile & 1][A, H]
  __shared__ uint64_t starts[2][Starts::kWords];
  __shared__ __attribute__((aligned(16))) float steps[PACKED ? 2 : 1][3][PACKED ? kScanTile : 1];
  const int nCols = (p.D + kScanCols - 1) / kScanCols;
  const int at = block_at(p), b = at / nCols, c0 = (at - b * nCols) * kScanCols, seg = blockIdx.y;
  const Lane<V> me(p.D, c0);
  const bool gated = p.gate.p != nullptr;
  float rate[V], carry[V], total[V];
  const int cg = me.cg;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    rate[i] = p.rate[cg + i] * kLog2e;
    carry[i] = 0.f;
    total[i] = 1.f;
  }
  if (p.nSeg > 1 && !MAPS) {
    const float2* m = p.maps + (int64_t(b) * p.nSeg) * p.D + cg;
#pragma unroll
    for (int i = 0; i < V; ++i) carry[i] = m[i].y;
    for (int q0 = 1; q0 <= seg; q0 += kAhead) {
      float2 f[kAhead][V];
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) f[q][i] = m[int64_t(min(q0 + q, seg)) * p.D + i];
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) carry[i] = q0 + q <= seg ? through<DOCS>(f[q][i].x, f[q][i].y, carry[i]) : carry[i];
    }
  } else if (p.nSeg == 1 && p.state_in != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) carry[i] = p.state_in[b * p.sis + cg + i];
  }
  const int nTiles = (p.T + kScanTile - 1) / kScanTile;
  const int k0 = seg * p.segTiles, k1 = min(nTiles, k0 + p.segTiles);
  Rows<IT, V, L> rx[2], ra[2], rg[2];
  const Place<IT, V, L> px(p.x, me), pa(p.decay, me), pg(p.gate, me);
  const Place<ET, V, L> py(p.y, me);
  Steps sc;
  Starts first;
  const int n = k1 - k0;
  auto order = [&](int i) { return MAPS ? k1 - 1 - i : k0 + i; };  // the tile of turn i
  auto real = [&](int i) { return order(min(i, n - 1)); };
  auto fetch = [&](int i, Rows<IT, V, L>& x, Rows<IT, V, L>& a, Rows<IT, V, L>& g) {
    const int k = order(i);
    x.load(px, px.rows(p.x, b, k, k0, k1, c0, p.T, p.D));
    a.load(pa, pa.rows(p.decay, b, k, k0, k1, c0, p.T, p.D));
    g.load(pg, pg.rows(p.gate, b, k, k0, k1, c0, p.T, p.D));
  };
  if constexpr (PACKED) {
    sc.load(p, b, real(0), c0);
    sc.put(steps[0]);
    sc.load(p, b, real(1), c0);
  }
  if constexpr (DOCS) {
    first.load(p, b, real(0));
    first.put(starts[0]);
    first.load(p, b, real(1));
  }
  fetch(0, rx[0], ra[0], rg[0]);
  __builtin_amdgcn_sched_barrier(0);  // the loads return in order: those of the first tile first
  fetch(1, rx[1], ra[1], rg[1]);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (DOCS || PACKED) __syncthreads();

  auto tile = [&](int i, Rows<IT, V, L>& cx, Rows<IT, V, L>& ca, Rows<IT, V, L>& cgt) {
    const int k = order(i), t0 = k * kScanTile, last = min(p.T - t0, kScanTile) - 1, half = i & 1;
    float a[L][V], u[L][V];
    auto step = [&](int which, int j) { return PACKED ? steps[half][which][me.run * L + j] : 0.f; };
#pragma unroll
    for (int j = 0; j < L; ++j) {
      float x[V], r[V];
      cx.get(j, x);
      ca.get(j, r);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (PACKED) x[i] *= step(0, j), r[i] *= step(1, j);
        const float s = PACKED ? sigmoid_of(r[i]) : sigmoid(r[i]);
        const float v = rate[i] * s;
        a[j][i] = __builtin_amdgcn_exp2f(-v);
        u[j][i] = x[i] * __builtin_amdgcn_sqrtf(one_minus_square(v, a[j][i]));
      }
    }
    if (gated) {  // one branch: between branches the tokens' chains could not be interleaved
#pragma unroll
      for (int j = 0; j < L; ++j) {
        float g[V];
        cgt.get(j, g);
#pragma unroll
        for (int i = 0; i < V; ++i) u[j][i] *= PACKED ? sigmoid_of(g[i] * step(2, j)) : sigmoid(g[i]);
      }
    }
    fetch(i + 2, cx, ca, cgt);
    if (last < kScanTile - 1) {  // tokens that do not exist leave the state as it is
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          a[j][i] = me.run * L + j > last ? 1.f : a[j][i];
          u[j][i] = me.run * L + j > last ? 0.f : u[j][i];
        }
    }
    if constexpr (DOCS) {
      const uint32_t m = Starts::of_run(starts[half], me.run, L);
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) a[j][i] = m >> j & 1 ? -0.f : a[j][i];
    }
    float A[V], H[V];
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = a[0][i], H[i] = u[0][i];
#pragma unroll
    for (int j = 1; j < L; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        H[i] = through<DOCS>(a[j][i], u[j][i], H[i]);
        A[i] = chain<DOCS>(a[j][i], A[i]);
      }
    float pA[V], pH[V];  // the map of the lane groups before this one
    scan_groups<V, DOCS, false>(me, A, H, pA, pH);
    if (me.group == Lane<V>::kGroups - 1) {
      write_map<V>(maps[half][0][me.wave], me.chl, A);
      write_map<V>(maps[half][1][me.wave], me.chl, H);
    }
    if constexpr (DOCS) {
      first.put(starts[half ^ 1]);
      first.load(p, b, real(i + 2));
    }
    if constexpr (PACKED) {
      sc.put(steps[half ^ 1]);
      sc.load(p, b, real(i + 2), c0);
    }
    __syncthreads();  // what is overwritten next was read before the barrier before
    float h[V];
    if constexpr (MAPS) {
#pragma unroll
      for (int q = kScanWaves - 1; q >= 0; --q) {
        float fA[V], fH[V];
        read_map<V>(maps[half][0][q], me.chl, fA);
        read_map<V>(maps[half][1][q], me.chl, fH);
#pragma unroll
        for (int c = 0; c < V; ++c) {
          carry[c] = through<DOCS>(total[c], carry[c], fH[c]);
          total[c] = chain<DOCS>(total[c], fA[c]);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c) h[c] = carry[c];
#pragma unroll
      for (int q = 0; q < kScanWaves; ++q) {
        float fA[V], fH[V];
        read_map<V>(maps[half][0][q], me.chl, fA);
        read_map<V>(maps[half][1][q], me.chl, fH);
#pragma unroll
        for (int c = 0; c < V; ++c) {
          carry[c] = through<DOCS>(fA[c], fH[c], carry[c]);
          if (q < kScanWaves - 1) h[c] = q < me.wave ? carry[c] : h[c];
        }
      }
    }
    if constexpr (!MAPS) {
      if (p.chunks != nullptr && me.run == 0 && me.ok) {
        float* out = p.chunks + (int64_t(b) * nTiles + k) * p.D + cg;
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = h[i];
      }
    }
    if constexpr (WANT == kOutputs) {
      const __amdgpu_buffer_rsrc_t ry = py.rows(p.y, b, k, k0, k1, c0, p.T, p.D);
#pragma unroll
      for (int i = 0; i < V; ++i) h[i] = through<DOCS>(pA[i], pH[i], h[i]);
#pragma unroll
      for (int j = 0; j < L; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = through<DOCS>(a[j][i], u[j][i], h[i]);
        store_row(py, ry, j, h);
      }
    }
  };
  for (int i = 0;; i += 2) {
    tile(i, rx[0], ra[0], rg[0]);
    if (i + 1 >= n) break;
    tile(i + 1, rx[1], ra[1], rg[1]);
    if (i + 2 >= n) break;
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
// Backward, tiles from the last to the first. MAPS: only the segment's map of e, from the first to the last.
// From 8-bit inputs 202 to 215 us where 16-bit ones take 206 to 226 (8 x 4096 x 2048): the writes remain.
// ---------------------------------------------------------------------------------
template <typename ET, int V, bool PACKED, bool DOCS, bool MAPS>
__global__ __launch_bounds__(kThreads, 2) void k_scan_bwd(const ScanParams p) {
  using IT = std::conditional_t<PACKED, i8_t, ET>;
  constexpr int L = kScanElems / V;
  __shared__ float maps[2][MAPS ? 2 : 3][kScanWaves][kScanCols];  // [tile & 1][A, E, H]
  __shared__ uint64_t starts[2][Starts::kWords];
  __shared__ __attribute__((aligned(16))) float steps[PACKED ? 2 : 1][3][PACKED ? kScanTile : 1];
  const int nCols = (p.D + kScanCols - 1) / kScanCols;
  const int at = block_at(p), b = at / nCols, c0 = (at - b * nCols) * kScanCols;
  const int seg = int(blockIdx.y) + (MAPS ? 1 : 0);
  const Lane<V> me(p.D, c0);
  const bool gated = p.gate.p != nullptr;
  const int cg = me.cg, row = me.run * L;
  float rate[V], carry[V], total[V];
  double drate[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    rate[i] = p.rate[cg + i] * kLog2e;
    carry[i] = 0.f;
    total[i] = 1.f;
    drate[i] = 0.0;
  }
  if (p.nSeg > 1 && !MAPS) {
    const float2* m = p.maps + (int64_t(b) * p.nSeg) * p.D + cg;
#pragma unroll
    for (int i = 0; i < V; ++i) carry[i] = m[int64_t(p.nSeg - 1) * p.D + i].y;
    for (int q0 = p.nSeg - 2; q0 >= seg; q0 -= kAhead) {
      float2 f[kAhead][V];
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) f[q][i] = m[int64_t(max(q0 - q, seg)) * p.D + i];
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) carry[i] = q0 - q >= seg ? through<DOCS>(f[q][i].x, f[q][i].y, carry[i]) : carry[i];
    }
  } else if (p.nSeg == 1 && p.dstate_out != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) carry[i] = p.dstate_out[b * p.dsos + cg + i];
  }
  const int nTiles = (p.T + kScanTile - 1) / kScanTile;
  const int k0 = seg * p.segTiles, k1 = min(nTiles, k0 + p.segTiles), n = k1 - k0;
  auto order = [&](int i) { return MAPS ? k0 + i : k1 - 1 - i; };  // the tile of turn i
  auto real = [&](int i) { return order(min(i, n - 1)); };
  Rows<IT, V, L> rx, ra, rg;
  Rows<ET, V, L> rd;
  const Place<IT, V, L> px(p.x, me), pa(p.decay, me), pg(p.gate, me);
  const Place<ET, V, L> pd(p.dy, me), pdx(p.dx, me), pda(p.ddecay, me), pdg(p.dgate, me);
  Steps sc;
  Starts begin;
  float kept[V];
  auto fetch = [&](int i) {
    const int k = order(i);
    ra.load(pa, pa.rows(p.decay, b, k, k0, k1, c0, p.T, p.D));
    rd.load(pd, pd.rows(p.dy, b, k, k0, k1, c0, p.T, p.D));
    if constexpr (!MAPS) {
      rx.load(px, px.rows(p.x, b, k, k0, k1, c0, p.T, p.D));
      rg.load(pg, pg.rows(p.gate, b, k, k0, k1, c0, p.T, p.D));
      const float* c = p.chunks + (int64_t(b) * nTiles + real(i)) * p.D + cg;
#pragma unroll
      for (int v = 0; v < V; ++v) kept[v] = c[v];
    }
  };
  if constexpr (PACKED) {
    sc.load(p, b, real(0), c0);
    sc.put(steps[0]);
    sc.load(p, b, real(1), c0);
  }
  if constexpr (DOCS) {
    begin.load(p, b, real(0));
    begin.put(starts[0]);
    begin.load(p, b, real(1));
  }
  fetch(0);
  if constexpr (DOCS || PACKED) __syncthreads();
  for (int turn = 0; turn < n; ++turn) {
    const int k = order(turn), t0 = k * kScanTile, last = min(p.T - t0, kScanTile) - 1, half = turn & 1;
    // s = sigmoid(decay), sr = 1 - s; w = b sigmoid(gate); c = sigmoid(gate) x a^2 / b; xg = x (1 - sigmoid(gate)); hb: the
    // inputs b sigmoid(gate) x, then the states before the tokens
    float a[L][V], s[L][V], sr[L][V], w[L][V], c[L][V], xg[L][V], x[L][V], hb[L][V], dy[L][V], hk[V];
    auto step = [&](int which, int j) { return PACKED ? steps[half][which][me.run * L + j] : 0.f; };
#pragma unroll
    for (int j = 0; j < L; ++j) {
      float r[V];
      ra.get(j, r);
      rd.get(j, dy[j]);
      if constexpr (!MAPS) rx.get(j, x[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float pe = __builtin_amdgcn_exp2f(r[i] * (PACKED ? step(1, j) : -kLog2e));
        s[j][i] = __builtin_amdgcn_rcpf(1.f + pe);
        if constexpr (!MAPS) {
          if constexpr (PACKED) x[j][i] *= step(0, j);
          sr[j][i] = rest_of(pe, s[j][i]);
          const Decay d = decay_of(s[j][i], rate[i]);
          a[j][i] = d.a;
          w[j][i] = d.b;
          c[j][i] = d.a * d.a * d.rb;
          xg[j][i] = 0.f;
        } else {
          a[j][i] = __builtin_amdgcn_exp2f(-(rate[i] * s[j][i]));
        }
      }
    }
    if constexpr (!MAPS) {
      if (gated) {  // one branch: between branches the tokens' chains could not be interleaved
#pragma unroll
        for (int j = 0; j < L; ++j) {
          float g[V];
          rg.get(j, g);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float pg = __builtin_amdgcn_exp2f(g[i] * (PACKED ? step(2, j) : -kLog2e));
            const float sg = __builtin_amdgcn_rcpf(1.f + pg);
            w[j][i] *= sg;
            c[j][i] *= sg;
            xg[j][i] = rest_of(pg, sg);
          }
        }
      }
    }
    if (last < kScanTile - 1) {  // tokens that do not exist leave h and e as they are
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const bool gone = row + j > last;
          a[j][i] = gone ? 1.f : a[j][i];
          dy[j][i] = gone ? 0.f : dy[j][i];
          if constexpr (!MAPS) {
            x[j][i] = gone ? 0.f : x[j][i];
            w[j][i] = gone ? 0.f : w[j][i];
          }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) hk[i] = MAPS ? 0.f : kept[i];
    if constexpr (!MAPS) {
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {  // x itself is not kept
          hb[j][i] = w[j][i] * x[j][i];
          c[j][i] *= x[j][i];
          xg[j][i] *= x[j][i];
        }
    }
    fetch(turn + 1);
    uint32_t first = 0;  // tokens that start a document: nothing passes through them, forwards or backwards
    if constexpr (DOCS) first = Starts::of_run(starts[half], me.run, L);
    if constexpr (DOCS) {
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) a[j][i] = first >> j & 1 ? -0.f : a[j][i];
    }
    float A[V], H[V], E[V];
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = 1.f, H[i] = 0.f, E[i] = 0.f;
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float f = a[j][i];
        A[i] = chain<DOCS>(f, A[i]);
        if constexpr (!MAPS) {
          H[i] = through<DOCS>(f, hb[j][i], H[i]);
        }
      }
#pragma unroll
    for (int j = L - 1; j >= 0; --j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float f = a[j][i], dh = dy[j][i] + E[i];
        E[i] = DOCS && forgets(f) ? 0.f : f * dh;
      }
    float pA[V], pH[V], rA[V], rE[V], B[V];  // the maps of the lane groups before and behind this one
#pragma unroll
    for (int i = 0; i < V; ++i) B[i] = A[i];
    scan_groups<V, DOCS, true>(me, B, E, rA, rE);
    if (me.group == 0) {
      write_map<V>(maps[half][0][me.wave], me.chl, B);
      write_map<V>(maps[half][1][me.wave], me.chl, E);
    }
    if constexpr (!MAPS) {
      scan_groups<V, DOCS, false>(me, A, H, pA, pH);
      if (me.group == Lane<V>::kGroups - 1) write_map<V>(maps[half][2][me.wave], me.chl, H);
    }
    if constexpr (DOCS) {
      begin.put(starts[half ^ 1]);
      begin.load(p, b, real(turn + 2));
    }
    if constexpr (PACKED) {
      sc.put(steps[half ^ 1]);
      sc.load(p, b, real(turn + 2), c0);
    }
    __syncthreads();
    float e[V], h[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = carry[i], h[i] = hk[i];
    if constexpr (MAPS) {
#pragma unroll 2
      for (int q = 0; q < kScanWaves; ++q) {
        float fA[V], fE[V];
        read_map<V>(maps[half][0][q], me.chl, fA);
        read_map<V>(maps[half][1][q], me.chl, fE);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          carry[i] = through<DOCS>(total[i], carry[i], fE[i]);
          total[i] = chain<DOCS>(total[i], fA[i]);
        }
      }
    } else {
#pragma unroll 2
      for (int q = kScanWaves - 1; q >= 0; --q) {
        float fA[V], fE[V];
        read_map<V>(maps[half][0][q], me.chl, fA);
        read_map<V>(maps[half][1][q], me.chl, fE);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          carry[i] = through<DOCS>(fA[i], fE[i], carry[i]);
          e[i] = q > me.wave ? carry[i] : e[i];
        }
      }
    }
    if constexpr (!MAPS) {
#pragma unroll 2
      for (int q = 0; q < kScanWaves; ++q) {
        float fA[V], fH[V];
        read_map<V>(maps[half][0][q], me.chl, fA);
        read_map<V>(maps[half][2][q], me.chl, fH);
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = q < me.wave ? through<DOCS>(fA[i], fH[i], h[i]) : h[i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        h[i] = through<DOCS>(pA[i], pH[i], h[i]);
        e[i] = through<DOCS>(rA[i], rE[i], e[i]);
      }
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float f = a[j][i], before = DOCS && forgets(f) ? 0.f : h[i];
          h[i] = through<DOCS>(f, hb[j][i], h[i]);
          hb[j][i] = before;
        }
      const __amdgpu_buffer_rsrc_t rdx = pdx.rows(p.dx, b, k, k0, k1, c0, p.T, p.D);
      const __amdgpu_buffer_rsrc_t rda = pda.rows(p.ddecay, b, k, k0, k1, c0, p.T, p.D);
      const __amdgpu_buffer_rsrc_t rdg = pdg.rows(p.dgate, b, k, k0, k1, c0, p.T, p.D);
      float sum[V], back[V];
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = 0.f, back[i] = rate[i] * -0.693147180559945309417f;  // of log 2
#pragma unroll
      for (int j = L - 1; j >= 0; --j) {
        float dx[V], dr[V], dg[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float dh = dy[j][i] + e[i];
          dx[i] = dh * w[j][i];
          dg[i] = dx[i] * xg[j][i];
          const float ad = a[j][i] * dh;
          const float dl = s[j][i] * __builtin_fmaf(ad, hb[j][i], -c[j][i] * dh);
          sum[i] -= row + j > last ? 0.f : dl;  // of a token that does not exist it may be 0 times infinity
          dr[i] = back[i] * dl * sr[j][i];
          e[i] = DOCS && (first >> j & 1) ? 0.f : ad;
        }
        store_row(pdx, rdx, j, dx);
        store_row(pda, rda, j, dr);
        store_row(pdg, rdg, j, dg);
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
#pragma unroll
      for (int m = Lane<V>::kLanes; m < 64; m *= 2) drate[i] += __shfl_xor(drate[i], m);
      if (me.group == 0) sums[me.wave][me.chl + i] = drate[i];
    }
    __syncthreads();
    if (int(threadIdx.x) < kScanCols && c0 + int(threadIdx.x) < p.D) {
      double t = 0.0;
#pragma unroll
      for (int q = 0; q < kScanWaves; ++q) t += sums[q][threadIdx.x];
      p.drate_part[(int64_t(b) * p.nSeg + seg) * p.D + c0 + threadIdx.x] = float(t);
    }
    if (p.dstate != nullptr && k0 == 0 && me.ok && int(threadIdx.x) < Lane<V>::kLanes) {
#pragma unroll
      for (int i = 0; i < V; ++i) p.dstate[b * p.dsis + cg + i] = carry[i];
    }
  }
}

template <typename ET, int V, bool PACKED, bool DOCS>
hipError_t launch(const ScanParams& p, bool bwd, hipStream_t s) {
  const unsigned blocks = unsigned((p.D + kScanCols - 1) / kScanCols) * unsigned(p.B);
  const dim3 first(blocks, unsigned(p.nSeg - 1)), all(blocks, unsigned(p.nSeg));
  if (p.nSeg > 1) {
    if (bwd) {
      hipLaunchKernelGGL((k_scan_bwd<ET, V, PACKED, DOCS, true>), first, dim3(kThreads), 0, s, p);
    } else {
      hipLaunchKernelGGL((k_scan_fwd<ET, V, PACKED, DOCS, kMaps>), first, dim3(kThreads), 0, s, p);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (bwd) {
    hipLaunchKernelGGL((k_scan_bwd<ET, V, PACKED, DOCS, false>), all, dim3(kThreads), 0, s, p);
  } else if (p.y.p == nullptr) {
    hipLaunchKernelGGL((k_scan_fwd<ET, V, PACKED, DOCS, kStates>), all, dim3(kThreads), 0, s, p);
  } else if constexpr (!PACKED) {  // the forward of packed inputs only serves the backward
    hipLaunchKernelGGL((k_scan_fwd<ET, V, PACKED, DOCS, kOutputs>), all, dim3(kThreads), 0, s, p);
  }
  return hipGetLastError();
}

template <typename ET, int V, bool PACKED>
hipError_t launch_docs(const ScanParams& p, bool bwd, hipStream_t s) {
  return p.seg != nullptr ? launch<ET, V, PACKED, true>(p, bwd, s) : launch<ET, V, PACKED, false>(p, bwd, s);
}

// Two channels per lane where vec allows (calls of 8 sequences of 4096 tokens, 2048 channels, bf16, with documents:
// forward 137 us, with one 146, backward 237 and 245; from 8-bit inputs 351 and 373), but float32 inputs go one per
// lane: 64 lanes' 4 bytes are whole rows of a tile as well, and the backward with two would not fit its registers (8
// sequences of 2048 tokens: 200 us, with two 227, with documents 211 and 314; forward 116 and 113, 120 and 114). With
// float32 inputs in 8 bits two again (191 us, with one 198).
template <typename ET>
hipError_t run(const ScanParams& p, int vec, bool packed, bool bwd, hipStream_t s) {
  if (packed) return vec == 2 ? launch_docs<ET, 2, true>(p, bwd, s) : launch_docs<ET, 1, true>(p, bwd, s);
  if constexpr (sizeof(ET) == 2)
    if (vec == 2) return launch_docs<ET, 2, false>(p, bwd, s);
  return launch_docs<ET, 1, false>(p, bwd, s);
}

}  // namespace scan

}  // namespace dynconv
