// Group norm, channels last: plans, the sums that the storage types share, and the C ABI (argument checks
// before any HIP call; see include/dynconv.h for the contract).
#include <initializer_list>

#include "dynconv_groupnorm_internal.hpp"
#include "dynconv_internal.hpp"

namespace dynconv {

namespace {

constexpr int kThreads = 256;

// mean and 1 / sqrt(var + eps) of a (sequence, group) from its chunks' sums: a wave each, in a fixed order, eight
// loads of a lane under way at a time.
constexpr int kFinishAhead = 8;
struct Sums {
  double sum, sq;
};
__global__ __launch_bounds__(kThreads) void k_group_finish(const GroupParams p) {
  const int64_t i = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * (kThreads / 64) + threadIdx.x / 64;
  if (i >= int64_t(p.B) * p.G) return;
  const int lane = threadIdx.x & 63, b = int(i / p.G), g = int(i - int64_t(b) * p.G);
  double sum = 0.0, sq = 0.0;
  const Sums* part = reinterpret_cast<const Sums*>(p.part) + int64_t(b) * p.nChunk * p.G + g;
  for (int k = lane; k < p.nChunk; k += 64 * kFinishAhead) {
    Sums v[kFinishAhead];
#pragma unroll
    for (int u = 0; u < kFinishAhead; ++u) v[u] = part[int64_t(min(k + u * 64, p.nChunk - 1)) * p.G];
#pragma unroll
    for (int u = 0; u < kFinishAhead; ++u) {
      sum += k + u * 64 < p.nChunk ? v[u].sum : 0.0;
      sq += k + u * 64 < p.nChunk ? v[u].sq : 0.0;
    }
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    sum += __shfl_xor(sum, m);
    sq += __shfl_xor(sq, m);
  }
  int n = p.lengths != nullptr ? min(max(p.lengths[b], 0), p.T) : p.T;
  if (p.Cg == 0) n = 0;  // no channels
  if (lane != 0) return;
  const double count = double(n) * p.Cg;
  const double mean = n > 0 ? sum / count : 0.0, var = n > 0 ? sq / count - mean * mean : 0.0;
  p.stats[i * 2] = float(mean);
  // a NaN among the inputs stays one; without tokens there is nothing to scale
  p.stats[i * 2 + 1] = n > 0 ? float(1.0 / sqrt((var < 0.0 ? 0.0 : var) + double(p.eps))) : 0.f;
}

// Column sums over n partial rows of 2 C floats, in 64 bits and a fixed order, for each of gridDim.y
// batches of rows: the first C columns into out0, the others into out1 (either may be null). A workgroup
// takes 32 columns, its 32 thread groups every 32nd row, eight loads under way at a time.
constexpr int kSumCols = 32, kSumGroups = 32;
__global__ __launch_bounds__(kSumCols* kSumGroups) void k_group_sum(const float* __restrict__ part, int64_t n, int64_t C,
                                                                    float* out0, float* out1, int64_t outStride) {
  __shared__ double red[kSumGroups][kSumCols + 1];
  const int col = threadIdx.x % kSumCols, grp = threadIdx.x / kSumCols;
  const int64_t i = int64_t(blockIdx.x) * kSumCols + col, width = 2 * C;
  const float* rows = part + int64_t(blockIdx.y) * n * width;
  double s = 0.0;
  if (i < width) {
    for (int64_t c = grp; c < n; c += 8 * kSumGroups) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = rows[min(c + u * kSumGroups, n - 1) * width + i];
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
  if (col != 0 || o >= width) return;
  float* out = o < C ? out0 : out1;
  if (out != nullptr) out[int64_t(blockIdx.y) * outStride + (o < C ? o : o - C)] = float(s);
}

hipError_t group_sum(const float* part, int64_t n, int64_t C, int64_t batches, float* out0, float* out1, int64_t stride,
                     hipStream_t s) {
  // 2^15 batches at a time: the second dimension of a launch ends at 2^16
  constexpr int64_t most = int64_t(1) << 15;
  for (int64_t b = 0; b < batches; b += most) {
    const unsigned y = unsigned(batches - b < most ? batches - b : most);
    hipLaunchKernelGGL(k_group_sum, dim3(unsigned((2 * C + kSumCols - 1) / kSumCols), y), dim3(kSumCols * kSumGroups), 0, s,
                       part + b * n * 2 * C, n, C, out0 != nullptr ? out0 + b * stride : nullptr,
                       out1 != nullptr ? out1 + b * stride : nullptr, stride);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// The fewest lanes that hold a row in one piece each (groups of 16 bf16 channels on 4 lanes instead of 2: forward 91
// us, not 52): 2048 bf16 channels on 64 lanes of 4 pieces took the backward 190 us, on 256 lanes of one 107 (40
// million elements). Then more pieces per lane, which the backward pays for with its registers: two pieces on 256 lanes
// take 200 to 215 of them (4096 channels 120 us, the ragged 2050 244), four 370 to 398, one wave per SIMD (8192 channels
// 225, 4100 396); longer rows are read twice, with the column sums added to memory token by token (10001 channels 474,
// 20000 429). The forward of the same takes 48 to 108.
GroupPlan group_plan(int64_t Cg, int E) {
  const int64_t loads = (Cg + E - 1) / E;  // of the row
  for (int lpr : {1, 2, 4, 8, 16, 32, 64})
    if (loads <= lpr) return {lpr, 1};
  if (loads <= 128) return {64, 2};
  if (loads <= 256) return E == 8 ? GroupPlan{256, 1} : GroupPlan{64, 4};
  if (loads <= 512) return {256, 2};
  if (loads <= 1024) return {256, 4};
  return {256, 0};
}

int64_t group_token_blocks(int64_t tokens, int64_t G, int64_t Cg, int E, bool bwd, int32_t* gpw, int32_t* tpw) {
  const int64_t rpb = kThreads / group_plan(Cg, E).lpr;
  *gpw = int32_t(G < rpb ? G : rpb);
  *tpw = int32_t(rpb / *gpw);
  const int64_t need = (tokens + *tpw - 1) / *tpw, across = (G + *gpw - 1) / *gpw;
  // Workgroups per CU: eight in the forward; four in the backward, each of which leaves a row of
  // partial sums, and more where a lane would add over 512 rows to its float32 sums.
  const int64_t all = bwd ? 1024 : 2048;
  int64_t most = across < all ? all / across : 1;
  if (bwd && (need + 511) / 512 > most) most = (need + 511) / 512;
  return need < most ? need : most;
}

void group_sequence_plan(GroupParams* p, int E) {
  const int lanes = (p->Cg + E - 1) / E;
  p->lpg = lanes;
  p->gpb = lanes >= kThreads ? 1 : (p->G < kThreads / lanes ? p->G : kThreads / lanes);
  p->lpt = lanes >= kThreads ? kThreads : p->gpb * lanes;
  p->tps = kThreads / p->lpt;
  const int64_t across = int64_t(p->B) * ((p->G + p->gpb - 1) / p->gpb);
  // Workgroups per CU: eight (four are 5 % better where all have work, and 5 % worse where half of the tokens of a
  // batch do not exist: 8 sequences of 2048 bf16 channels, both directions 174 and 184 us), in the
  // gradient's two passes four, each of which leaves a row of column sums or begins with a sum over the
  // groups. Such a row is paid for by 16 of a lane's tokens (27 groups of 57 bf16 channels, 26000 tokens: 187 us,
  // with 32 212; 64 groups of 16 137 and 147), by 8 where there would be fewer than two workgroups per CU (8
  // sequences of 610 tokens, one group of 8192: 191, with 16 231, with 32 328). A lane adds up to `most` tokens to its sums:
  // any number in 64 bits, 512 to the gradient's float32 sums.
  auto cut = [&](int64_t all, int least, int64_t most, int32_t* chunk, int32_t* n) {
    const int64_t want = across < all ? all / across : 1;
    int64_t c = (int64_t(p->T) + want - 1) / want;
    if (c < least * p->tps) c = least * p->tps;
    if (c > most * p->tps) c = most * p->tps;
    *chunk = int32_t(c);
    *n = int32_t((p->T + c - 1) / c);
  };
  cut(2048, 8, INT32_MAX, &p->chunk, &p->nChunk);
  cut(1024, across * (p->T / (16 * p->tps)) >= 512 ? 16 : 8, 512, &p->gradChunk, &p->nGradChunk);
}

namespace {

constexpr int64_t kMaxC = int64_t(1) << 19;

struct Sizes {
  int64_t B, T, C, G;
  bool sequence;
};

int elem_bytes(dynconv_dtype dt) { return dt == DYNCONV_F32 ? 4 : 2; }
bool aligned(const void* p, int64_t a) { return (reinterpret_cast<uintptr_t>(p) % uint64_t(a)) == 0; }

dynconv_status check_sizes(const Sizes& z, dynconv_dtype dt, float eps) {
  if (dt != DYNCONV_F32 && dt != DYNCONV_BF16 && dt != DYNCONV_F16) return DYNCONV_ERR_INVALID_ARG;
  if (z.B < 0 || z.T < 0 || z.C < 0 || !(eps >= 0.f)) return DYNCONV_ERR_INVALID_ARG;
  if (z.G < 1 || z.C % z.G != 0) return DYNCONV_ERR_INVALID_ARG;
  if (z.C > kMaxC) return DYNCONV_ERR_UNSUPPORTED;
  if (z.B >= (int64_t(1) << 23) || z.T > INT32_MAX - 65536) return DYNCONV_ERR_UNSUPPORTED;
  if (z.B > 0 && z.T > INT32_MAX / z.B) return DYNCONV_ERR_UNSUPPORTED;
  return DYNCONV_OK;
}

bool empty(const Sizes& z) { return z.B == 0 || z.T == 0 || z.C == 0; }

dynconv_status take(GroupTensor* t, const void* p, const int64_t* s, const Sizes& z, int eb, int piece, bool output,
                    bool* whole) {
  if (p == nullptr || s == nullptr) return DYNCONV_ERR_INVALID_ARG;
  if (!aligned(p, eb) || (z.C > 1 && s[2] != 1) || s[0] < 0 || s[1] < 0) return DYNCONV_ERR_UNSUPPORTED;
  if (output && ((z.B > 1 && s[0] == 0) || (z.T > 1 && s[1] == 0))) return DYNCONV_ERR_INVALID_ARG;
  if (!aligned(p, piece) || (z.B > 1 && s[0] * eb % piece != 0) || (z.T > 1 && s[1] * eb % piece != 0)) *whole = false;
  t->p = p;
  t->s0 = s[0];
  t->s1 = s[1];
  return DYNCONV_OK;
}

dynconv_status take_vector(const void* w, int eb, bool* whole) {
  if (w == nullptr) return DYNCONV_OK;
  if (!aligned(w, eb)) return DYNCONV_ERR_UNSUPPORTED;
  if (!aligned(w, 16)) *whole = false;
  return DYNCONV_OK;
}

bool any_equal(const void* out, std::initializer_list<const void*> others) {
  if (out == nullptr) return false;
  for (const void* o : others)
    if (o == out) return true;
  return false;
}

size_t rounded(size_t n) { return (n + 255) / 256 * 256; }

GroupParams sized(const Sizes& z, int E) {
  GroupParams p{};
  p.B = int32_t(z.B), p.T = int32_t(z.T), p.C = int32_t(z.C), p.G = int32_t(z.G), p.Cg = int32_t(z.C / z.G);
  if (z.sequence) group_sequence_plan(&p, E);
  return p;
}

// Workspace: the statistics' partial sums and the statistics (unless given), the column sums.
struct Space {
  size_t part, stats, colpart, colsum;
  size_t total() const { return part + stats + colpart + colsum; }
};
Space space(const Sizes& z, int E, bool bwd, bool stats) {
  Space w{};
  const GroupParams p = sized(z, E);
  if (!z.sequence) {
    int32_t gpw, tpw;
    if (bwd) w.colpart = rounded(size_t(group_token_blocks(z.B * z.T, z.G, p.Cg, E, true, &gpw, &tpw)) * 2 * size_t(z.C) * sizeof(float));
    return w;
  }
  if (!(bwd && stats)) w.part = rounded(size_t(z.B) * size_t(p.nChunk) * size_t(z.G) * 2 * sizeof(double));
  if (!stats) w.stats = rounded(size_t(z.B) * size_t(z.G) * 2 * sizeof(float));
  if (bwd) {
    w.colpart = rounded(size_t(z.B) * size_t(p.nGradChunk) * 2 * size_t(z.C) * sizeof(float));
    w.colsum = rounded(size_t(z.B) * 2 * size_t(z.C) * sizeof(float));
  }
  return w;
}

hipError_t tokens(const GroupParams& p, dynconv_dtype dt, bool whole, bool packed, bool bwd, hipStream_t s) {
  return dt == DYNCONV_BF16  ? group_tokens_bf16(p, whole, packed, bwd, s)
         : dt == DYNCONV_F16 ? group_tokens_f16(p, whole, packed, bwd, s)
                             : group_tokens_f32(p, whole, packed, bwd, s);
}
hipError_t sequences(const GroupParams& p, dynconv_dtype dt, bool whole, bool packed, GroupStage stage, hipStream_t s) {
  return dt == DYNCONV_BF16  ? group_sequences_bf16(p, whole, packed, stage, s)
         : dt == DYNCONV_F16 ? group_sequences_f16(p, whole, packed, stage, s)
                             : group_sequences_f32(p, whole, packed, stage, s);
}

// Mean and scale of every (sequence, group) into p.stats, from the chunks' sums.
hipError_t finish(const GroupParams& p, hipStream_t s) {
  constexpr int64_t most = int64_t(1) << 23;  // a dimension of a launch has fewer than 2^32 threads
  const int64_t blocks = (int64_t(p.B) * p.G + kThreads / 64 - 1) / (kThreads / 64);
  const dim3 grid(unsigned(blocks < most ? blocks : most), unsigned((blocks + most - 1) / most));
  hipLaunchKernelGGL(k_group_finish, grid, dim3(kThreads), 0, s, p);
  return hipGetLastError();
}
hipError_t statistics(const GroupParams& p, dynconv_dtype dt, bool whole, bool packed, hipStream_t s) {
  const hipError_t e = sequences(p, dt, whole, packed, kGroupStats, s);
  return e == hipSuccess ? finish(p, s) : e;
}

dynconv_status done(hipError_t e) { return e == hipSuccess ? DYNCONV_OK : record_hip_error(e); }

}  // namespace

}  // namespace dynconv

using namespace dynconv;

extern "C" {

size_t dynconv_groupnorm_fwd_workspace_size(int64_t B, int64_t T, int64_t C, int64_t groups, int32_t over_sequence,
                                            int32_t with_stats, dynconv_dtype dtype) {
  const Sizes z{B, T, C, groups, over_sequence != 0};
  if (check_sizes(z, dtype, 0.f) != DYNCONV_OK || empty(z)) return 0;
  return space(z, 16 / elem_bytes(dtype), false, with_stats != 0).total();
}

dynconv_status dynconv_groupnorm_fwd(const void* x, const int64_t* xs, const void* weight, const void* bias,
                                     const void* gate, const int64_t* gs, const int32_t* lengths, void* y,
                                     const int64_t* ys, float* stats, int64_t B, int64_t T, int64_t C, int64_t groups,
                                     int32_t over_sequence, int32_t silu, float eps, dynconv_dtype dtype,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  const Sizes z{B, T, C, groups, over_sequence != 0};
  dynconv_status st = check_sizes(z, dtype, eps);
  if (st != DYNCONV_OK) return st;
  if (!z.sequence && (lengths != nullptr || stats != nullptr)) return DYNCONV_ERR_INVALID_ARG;
  const int eb = elem_bytes(dtype), E = 16 / eb;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (empty(z)) {  // the statistics of sequences without tokens
    if (stats == nullptr || B == 0) return DYNCONV_OK;
    if (!aligned(stats, 4) || groups > kMaxC) return DYNCONV_ERR_UNSUPPORTED;
    GroupParams p{};
    p.B = int32_t(B), p.G = int32_t(groups), p.Cg = int32_t(C / groups), p.stats = stats;
    return done(finish(p, s));
  }
  bool whole = C / groups % E == 0;
  GroupTensor tx{}, tg{}, ty{};
  if ((st = take(&tx, x, xs, z, eb, 16, false, &whole)) != DYNCONV_OK) return st;
  if (gate != nullptr && (st = take(&tg, gate, gs, z, eb, 16, false, &whole)) != DYNCONV_OK) return st;
  if ((st = take(&ty, y, ys, z, eb, 16, true, &whole)) != DYNCONV_OK) return st;
  if ((st = take_vector(weight, eb, &whole)) != DYNCONV_OK || (st = take_vector(bias, eb, &whole)) != DYNCONV_OK) return st;
  if (!aligned(lengths, 4) || !aligned(stats, 4)) return DYNCONV_ERR_UNSUPPORTED;
  if (any_equal(y, {x, weight, bias, gate, lengths, stats}) || any_equal(stats, {x, weight, bias, gate, lengths}))
    return DYNCONV_ERR_INVALID_ARG;
  GroupParams p = sized(z, E);
  p.x = tx, p.gate = tg, p.y = ty;
  p.weight = weight, p.bias = bias, p.lengths = lengths;
  p.silu = silu != 0;
  p.eps = eps;
  if (!z.sequence) return done(tokens(p, dtype, whole, false, false, s));
  const Space w = space(z, E, false, stats != nullptr);
  if (workspace == nullptr || workspace_bytes < w.total()) return DYNCONV_ERR_WORKSPACE;
  if (!aligned(workspace, 8)) return DYNCONV_ERR_UNSUPPORTED;
  p.part = static_cast<double*>(workspace);
  p.stats = stats != nullptr ? stats : reinterpret_cast<float*>(static_cast<char*>(workspace) + w.part);
  hipError_t e = statistics(p, dtype, whole, false, s);
  if (e == hipSuccess) e = sequences(p, dtype, whole, false, kGroupApply, s);
  return done(e);
}

size_t dynconv_groupnorm_bwd_workspace_size(int64_t B, int64_t T, int64_t C, int64_t groups, int32_t over_sequence,
                                            int32_t with_stats, dynconv_dtype dtype) {
  const Sizes z{B, T, C, groups, over_sequence != 0};
  if (check_sizes(z, dtype, 0.f) != DYNCONV_OK || empty(z)) return 0;
  return space(z, 16 / elem_bytes(dtype), true, with_stats != 0).total();
}

dynconv_status dynconv_groupnorm_bwd(const void* x, const int64_t* xs, const uint8_t* x_scales, const int64_t* xcs,
                                     const void* weight, const void* bias, const void* gate, const int64_t* gs,
                                     const int32_t* lengths, const float* stats, const void* dy, const int64_t* dys,
                                     void* dx, const int64_t* dxs, float* dweight, float* dbias, void* dgate,
                                     const int64_t* dgs, int64_t B, int64_t T, int64_t C, int64_t groups,
                                     int32_t over_sequence, int32_t silu, float eps, dynconv_dtype dtype,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  const Sizes z{B, T, C, groups, over_sequence != 0};
  dynconv_status st = check_sizes(z, dtype, eps);
  if (st != DYNCONV_OK) return st;
  if (!z.sequence && (lengths != nullptr || stats != nullptr)) return DYNCONV_ERR_INVALID_ARG;
  if (x_scales != nullptr && stats != nullptr) return DYNCONV_ERR_INVALID_ARG;  // the forward's are of another x
  if (C == 0) return DYNCONV_OK;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (!aligned(dweight, 4) || !aligned(dbias, 4)) return DYNCONV_ERR_UNSUPPORTED;
  const void* outs[4] = {dx, dweight, dbias, dgate};
  for (int i = 0; i < 4; ++i) {
    if (any_equal(outs[i], {x, x_scales, weight, bias, gate, lengths, stats, dy})) return DYNCONV_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (outs[i] != nullptr && outs[i] == outs[j]) return DYNCONV_ERR_INVALID_ARG;
  }
  if (empty(z)) {
    if (dweight == nullptr && dbias == nullptr) return DYNCONV_OK;
    return done(group_sum(nullptr, 0, C, 1, dweight, dbias, 0, s));
  }
  const int eb = elem_bytes(dtype), E = 16 / eb;
  bool whole = C / groups % E == 0;
  const bool packed = x_scales != nullptr;
  GroupTensor tx{}, tg{}, tdy{}, tdx{}, tdg{};
  if ((st = take(&tx, x, xs, z, packed ? 1 : eb, packed ? E : 16, false, &whole)) != DYNCONV_OK) return st;
  if (packed) {
    if (xcs == nullptr) return DYNCONV_ERR_INVALID_ARG;
    if (xcs[0] < 0 || xcs[1] < 0 || (C > 64 && xcs[2] != 1)) return DYNCONV_ERR_UNSUPPORTED;
    tx.sc = x_scales;
    tx.c0 = xcs[0];
    tx.c1 = xcs[1];
  }
  if (gate != nullptr && (st = take(&tg, gate, gs, z, eb, 16, false, &whole)) != DYNCONV_OK) return st;
  if ((st = take(&tdy, dy, dys, z, eb, 16, false, &whole)) != DYNCONV_OK) return st;
  if ((st = take(&tdx, dx, dxs, z, eb, 16, true, &whole)) != DYNCONV_OK) return st;
  if ((gate != nullptr) != (dgate != nullptr)) return DYNCONV_ERR_INVALID_ARG;
  if (gate != nullptr && (st = take(&tdg, dgate, dgs, z, eb, 16, true, &whole)) != DYNCONV_OK) return st;
  if ((st = take_vector(weight, eb, &whole)) != DYNCONV_OK || (st = take_vector(bias, eb, &whole)) != DYNCONV_OK) return st;
  if (!aligned(lengths, 4) || !aligned(stats, 4)) return DYNCONV_ERR_UNSUPPORTED;
  GroupParams p = sized(z, E);
  p.x = tx, p.gate = tg, p.dy = tdy, p.dx = tdx, p.dgate = tdg;
  p.weight = weight, p.bias = bias, p.lengths = lengths;
  p.silu = silu != 0;
  p.eps = eps;
  const bool params = dweight != nullptr || dbias != nullptr;
  const Space w = space(z, E, true, stats != nullptr);
  char* at = static_cast<char*>(workspace);
  if (z.sequence || params) {
    if (workspace == nullptr || workspace_bytes < w.total()) return DYNCONV_ERR_WORKSPACE;
    if (!aligned(workspace, 8)) return DYNCONV_ERR_UNSUPPORTED;
    p.part = reinterpret_cast<double*>(at);
    p.colpart = reinterpret_cast<float*>(at + w.part + w.stats);
    p.colsum = reinterpret_cast<float*>(at + w.part + w.stats + w.colpart);
  }
  hipError_t e;
  if (!z.sequence) {
    int32_t gpw, tpw;
    e = tokens(p, dtype, whole, packed, true, s);
    if (e == hipSuccess && params)
      e = group_sum(p.colpart, group_token_blocks(B * T, groups, p.Cg, E, true, &gpw, &tpw), C, 1, dweight, dbias, 0, s);
    return done(e);
  }
  if (stats != nullptr) {
    p.stats = const_cast<float*>(stats);
  } else {
    p.stats = reinterpret_cast<float*>(at + w.part);
    if ((e = statistics(p, dtype, whole, packed, s)) != hipSuccess) return done(e);
  }
  e = sequences(p, dtype, whole, packed, kGroupColumns, s);
  if (e == hipSuccess) e = group_sum(p.colpart, p.nGradChunk, C, B, p.colsum, p.colsum + C, 2 * C, s);
  if (e == hipSuccess && params) e = group_sum(p.colsum, B, C, 1, dweight, dbias, 0, s);
  if (e == hipSuccess) e = sequences(p, dtype, whole, packed, kGroupGradient, s);
  return done(e);
}

}  // extern "C"
