// C ABI of the gated linear scan: argument checks (before any HIP call) and dispatch. See
// include/dynconv.h for the contract of every entry point.
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "dynconv_internal.hpp"
#include "dynconv_norm_internal.hpp"
#include "dynconv_scan_internal.hpp"

using namespace dynconv;

namespace {

int elem_bytes(dynconv_dtype dt) { return dt == DYNCONV_F32 ? 4 : 2; }
bool aligned(const void* p, int64_t a) { return (reinterpret_cast<uintptr_t>(p) % uint64_t(a)) == 0; }

// The kernels address a tile's 128 rows with 32-bit byte offsets.
constexpr int64_t kScanMaxTokenStride = int64_t(1) << 22;

struct Sizes {
  int64_t B, T, D;
};

dynconv_status check_sizes(const Sizes& z, dynconv_dtype dt) {
  if (dt != DYNCONV_F32 && dt != DYNCONV_BF16 && dt != DYNCONV_F16) return DYNCONV_ERR_INVALID_ARG;
  if (z.B < 0 || z.T < 0 || z.D < 0) return DYNCONV_ERR_INVALID_ARG;
  if (z.B > INT32_MAX || z.T > INT32_MAX - 65536 || z.D > (int64_t(1) << 24)) return DYNCONV_ERR_UNSUPPORTED;
  // one workgroup of 512 threads per (sequence, 64 channels), a launch has fewer than 2^32 threads
  if (z.B * ((z.D + kScanCols - 1) / kScanCols) >= (int64_t(1) << 22)) return DYNCONV_ERR_UNSUPPORTED;
  return DYNCONV_OK;
}

// An activation [B,T,D] of eb-byte elements; clears *vec when two channels at a time are not aligned, sets
// *shared when 64 channels of a row are not whole 128-byte lines.
dynconv_status take(ScanTensor* t, const void* p, const int64_t* s, const Sizes& z, int eb, bool output, int* vec,
                    bool* shared) {
  if (p == nullptr || s == nullptr) return DYNCONV_ERR_INVALID_ARG;
  if (!aligned(p, eb) || (z.D > 1 && s[2] != 1) || s[0] < 0 || s[1] < 0) return DYNCONV_ERR_UNSUPPORTED;
  if (z.T > 1 && s[1] >= kScanMaxTokenStride) return DYNCONV_ERR_UNSUPPORTED;
  // an output's rows have places of their own (the kernels drop rows that do not exist by their offsets)
  if (output && ((z.B > 1 && s[0] == 0) || (z.T > 1 && s[1] < z.D))) return DYNCONV_ERR_INVALID_ARG;
  if (!aligned(p, 2 * eb) || (z.B > 1 && s[0] % 2 != 0) || (z.T > 1 && s[1] % 2 != 0)) *vec = 1;
  if (eb == 1 || !aligned(p, 128) || (z.B > 1 && s[0] * eb % 128 != 0) || (z.T > 1 && s[1] * eb % 128 != 0)) *shared = true;
  t->p = p;
  t->s0 = s[0];
  t->s1 = z.T > 1 ? s[1] : kScanCols;  // a single token's is not used: any that puts the next row out of the range
  return DYNCONV_OK;
}

dynconv_status take_scales(ScanTensor* t, const uint8_t* p, const int64_t* s, const Sizes& z) {
  if (p == nullptr || s == nullptr) return DYNCONV_ERR_INVALID_ARG;
  if (s[0] < 0 || s[1] < 0 || (z.D > kScanScaleCols && s[2] != 1)) return DYNCONV_ERR_UNSUPPORTED;
  if (z.T > 1 && s[1] >= kScanMaxTokenStride) return DYNCONV_ERR_UNSUPPORTED;
  t->sc = p;
  t->c0 = s[0];
  t->c1 = z.T > 1 ? s[1] : 0;
  return DYNCONV_OK;
}

dynconv_status take_state(const float* p, const int64_t* s, const Sizes& z, bool output) {
  if (p == nullptr) return DYNCONV_OK;
  if (s == nullptr) return DYNCONV_ERR_INVALID_ARG;
  if (!aligned(p, 4) || s[0] < 0 || (z.D > 1 && s[1] != 1)) return DYNCONV_ERR_UNSUPPORTED;
  if (output && z.B > 1 && s[0] == 0) return DYNCONV_ERR_INVALID_ARG;
  return DYNCONV_OK;
}

dynconv_status take_seg(ScanParams* p, const int32_t* seg, const int64_t* ss) {
  if (seg == nullptr) return DYNCONV_OK;
  if (ss == nullptr) return DYNCONV_ERR_INVALID_ARG;
  if (ss[0] < 0 || ss[1] < 0 || !aligned(seg, 4)) return DYNCONV_ERR_UNSUPPORTED;
  p->seg = seg;
  p->ss0 = ss[0];
  p->ss1 = ss[1];
  return DYNCONV_OK;
}

bool any_equal(const void* out, std::initializer_list<const void*> others) {
  if (out == nullptr) return false;
  for (const void* o : others)
    if (o == out) return true;
  return false;
}

size_t rounded(size_t n) { return (n + 255) / 256 * 256; }

int32_t segments(const Sizes& z, bool bwd) { return scan_segments(z.T, scan_segment_tiles(z.B, z.D, z.T, bwd)); }
void cut(ScanParams* p, const Sizes& z, bool bwd) {
  p->segTiles = scan_segment_tiles(z.B, z.D, z.T, bwd);
  p->nSeg = scan_segments(z.T, p->segTiles);
}

// The backward's hold the forward's too, which is cut into as many segments or none.
size_t maps_bytes(const Sizes& z, bool bwd) {
  const int32_t n = segments(z, bwd);
  return n > 1 ? rounded(size_t(z.B) * size_t(n) * size_t(z.D) * sizeof(float2)) : 0;
}

size_t chunks_bytes(const Sizes& z) {
  return rounded(size_t(z.B) * size_t((z.T + kScanChunk - 1) / kScanChunk) * size_t(z.D) * sizeof(float));
}

// Backward: partial sums of drate, the maps (the forward's and the backward's in turn), the states.
struct BwdSpace {
  size_t drate, maps, chunks;
  size_t total() const { return drate + maps + chunks; }
};
BwdSpace bwd_space(const Sizes& z, bool given) {
  BwdSpace w;
  w.drate = rounded(size_t(z.B) * size_t(segments(z, true)) * size_t(z.D) * sizeof(float));
  w.maps = maps_bytes(z, true);
  w.chunks = given ? 0 : chunks_bytes(z);
  return w;
}

hipError_t run_fwd(const ScanParams& p, dynconv_dtype dt, int vec, bool packed, hipStream_t s) {
  return dt == DYNCONV_BF16  ? scan_fwd_bf16(p, vec, packed, s)
         : dt == DYNCONV_F16 ? scan_fwd_f16(p, vec, packed, s)
                             : scan_fwd_f32(p, vec, packed, s);
}

dynconv_status done(hipError_t e) { return e == hipSuccess ? DYNCONV_OK : record_hip_error(e); }

}  // namespace

extern "C" {

size_t dynconv_scan_fwd_workspace_size(int64_t B, int64_t T, int64_t D, dynconv_dtype dtype) {
  const Sizes z{B, T, D};
  if (check_sizes(z, dtype) != DYNCONV_OK || B == 0 || T == 0 || D == 0) return 0;
  return maps_bytes(z, false);
}

dynconv_status dynconv_scan_fwd(const void* x, const int64_t* xs, const void* decay, const int64_t* as, const void* gate,
                                const int64_t* gs, const float* rate, const int32_t* seq_idx, const int64_t* ss,
                                const float* state_in, const int64_t* sis, void* y, const int64_t* ys, float* state_out,
                                const int64_t* sos, float* chunks, int64_t B, int64_t T, int64_t D, dynconv_dtype dtype,
                                void* workspace, size_t workspace_bytes, void* stream) {
  const Sizes z{B, T, D};
  dynconv_status st = check_sizes(z, dtype);
  if (st != DYNCONV_OK) return st;
  if (B == 0 || D == 0) return DYNCONV_OK;
  const int eb = elem_bytes(dtype);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  ScanParams p{};
  int vec = D % 2 == 0 ? 2 : 1;
  if ((st = take_state(state_in, sis, z, false)) != DYNCONV_OK) return st;
  if ((st = take_state(state_out, sos, z, true)) != DYNCONV_OK) return st;
  // the state may be carried in place when its rows have the same places
  if (state_out != nullptr && state_out == state_in && sis[0] != sos[0]) return DYNCONV_ERR_INVALID_ARG;
  if (T == 0) {
    if (state_out == nullptr || state_out == state_in) return DYNCONV_OK;
    return done(scan_copy_state(state_in, state_in != nullptr ? sis[0] : 0, state_out, sos[0], int32_t(B), int32_t(D), s));
  }
  if ((st = take(&p.x, x, xs, z, eb, false, &vec, &p.shared)) != DYNCONV_OK) return st;
  if ((st = take(&p.decay, decay, as, z, eb, false, &vec, &p.shared)) != DYNCONV_OK) return st;
  if (gate != nullptr && (st = take(&p.gate, gate, gs, z, eb, false, &vec, &p.shared)) != DYNCONV_OK) return st;
  if ((st = take(&p.y, y, ys, z, eb, true, &vec, &p.shared)) != DYNCONV_OK) return st;
  if ((st = take_seg(&p, seq_idx, ss)) != DYNCONV_OK) return st;
  if (rate == nullptr) return DYNCONV_ERR_INVALID_ARG;
  if (!aligned(rate, 4) || (chunks != nullptr && !aligned(chunks, 4))) return DYNCONV_ERR_UNSUPPORTED;
  if (any_equal(y, {x, decay, gate, rate, seq_idx, state_in, state_out, chunks}) ||
      any_equal(state_out, {x, decay, gate, rate, seq_idx, chunks}) ||
      any_equal(chunks, {x, decay, gate, rate, seq_idx, state_in}))
    return DYNCONV_ERR_INVALID_ARG;
  p.rate = rate;
  p.state_in = state_in, p.sis = state_in != nullptr ? sis[0] : 0;
  p.state_out = state_out, p.sos = state_out != nullptr ? sos[0] : 0;
  p.chunks = chunks;
  p.B = int32_t(B), p.T = int32_t(T), p.D = int32_t(D);
  cut(&p, z, false);
  const size_t need = maps_bytes(z, false);
  if (need != 0 && (workspace == nullptr || workspace_bytes < need)) return DYNCONV_ERR_WORKSPACE;
  if (need != 0 && !aligned(workspace, 8)) return DYNCONV_ERR_UNSUPPORTED;
  p.maps = static_cast<float2*>(workspace);
  return done(run_fwd(p, dtype, vec, false, s));
}

size_t dynconv_scan_bwd_workspace_size(int64_t B, int64_t T, int64_t D, int32_t with_chunks, dynconv_dtype dtype) {
  const Sizes z{B, T, D};
  if (check_sizes(z, dtype) != DYNCONV_OK || B == 0 || T == 0 || D == 0) return 0;
  return bwd_space(z, with_chunks != 0).total();
}

dynconv_status dynconv_scan_bwd(const void* x, const int64_t* xs, const void* decay, const int64_t* as, const void* gate,
                                const int64_t* gs, const uint8_t* x_scales, const int64_t* xcs,
                                const uint8_t* decay_scales, const int64_t* acs, const uint8_t* gate_scales,
                                const int64_t* gcs, const float* rate, const int32_t* seq_idx, const int64_t* ss,
                                const float* state_in, const int64_t* sis, const float* chunks, const void* dy,
                                const int64_t* dys, const float* dstate_out, const int64_t* dsos, void* dx,
                                const int64_t* dxs, void* ddecay, const int64_t* das, float* drate, void* dgate,
                                const int64_t* dgs, float* dstate_in, const int64_t* dsis, int64_t B, int64_t T,
                                int64_t D, dynconv_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const Sizes z{B, T, D};
  dynconv_status st = check_sizes(z, dtype);
  if (st != DYNCONV_OK) return st;
  if (D == 0) return DYNCONV_OK;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (drate == nullptr || rate == nullptr) return DYNCONV_ERR_INVALID_ARG;
  if (!aligned(drate, 4) || !aligned(rate, 4) || (chunks != nullptr && !aligned(chunks, 4))) return DYNCONV_ERR_UNSUPPORTED;
  if ((st = take_state(state_in, sis, z, false)) != DYNCONV_OK) return st;
  if ((st = take_state(dstate_out, dsos, z, false)) != DYNCONV_OK) return st;
  if ((st = take_state(dstate_in, dsis, z, true)) != DYNCONV_OK) return st;
  const void* outs[5] = {dx, ddecay, drate, dgate, dstate_in};
  for (int i = 0; i < 5; ++i) {
    if (any_equal(outs[i], {x, decay, gate, x_scales, decay_scales, gate_scales, rate, seq_idx, state_in, chunks, dy,
                            dstate_out}))
      return DYNCONV_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (outs[i] != nullptr && outs[i] == outs[j]) return DYNCONV_ERR_INVALID_ARG;
  }
  if (B == 0 || T == 0) {  // no token: drate is zero and the state's gradient passes through
    hipError_t e = norm_dweight(nullptr, 0, int32_t(D), drate, s);
    if (e == hipSuccess && dstate_in != nullptr && B > 0)
      e = scan_copy_state(dstate_out, dstate_out != nullptr ? dsos[0] : 0, dstate_in, dsis[0], int32_t(B), int32_t(D), s);
    return done(e);
  }
  const int eb = elem_bytes(dtype);
  const bool packed = x_scales != nullptr;
  ScanParams p{};
  int vec = D % 2 == 0 ? 2 : 1;
  // x, decay and gate are all of `dtype` or all in 8 bits
  if (packed != (decay_scales != nullptr) || (packed && gate != nullptr) != (gate_scales != nullptr))
    return DYNCONV_ERR_INVALID_ARG;
  if (packed && chunks != nullptr) return DYNCONV_ERR_INVALID_ARG;  // the forward's states are of other inputs
  const int ib = packed ? 1 : eb;
  if ((st = take(&p.x, x, xs, z, ib, false, &vec, &p.shared)) != DYNCONV_OK) return st;
  if ((st = take(&p.decay, decay, as, z, ib, false, &vec, &p.shared)) != DYNCONV_OK) return st;
  if (gate != nullptr && (st = take(&p.gate, gate, gs, z, ib, false, &vec, &p.shared)) != DYNCONV_OK) return st;
  if (packed) {
    if ((st = take_scales(&p.x, x_scales, xcs, z)) != DYNCONV_OK) return st;
    if ((st = take_scales(&p.decay, decay_scales, acs, z)) != DYNCONV_OK) return st;
    if (gate != nullptr && (st = take_scales(&p.gate, gate_scales, gcs, z)) != DYNCONV_OK) return st;
  }
  if ((st = take(&p.dy, dy, dys, z, eb, false, &vec, &p.shared)) != DYNCONV_OK) return st;
  if ((st = take(&p.dx, dx, dxs, z, eb, true, &vec, &p.shared)) != DYNCONV_OK) return st;
  if ((st = take(&p.ddecay, ddecay, das, z, eb, true, &vec, &p.shared)) != DYNCONV_OK) return st;
  if ((gate != nullptr) != (dgate != nullptr)) return DYNCONV_ERR_INVALID_ARG;
  if (gate != nullptr && (st = take(&p.dgate, dgate, dgs, z, eb, true, &vec, &p.shared)) != DYNCONV_OK) return st;
  if ((st = take_seg(&p, seq_idx, ss)) != DYNCONV_OK) return st;
  const BwdSpace w = bwd_space(z, chunks != nullptr);
  if (workspace == nullptr || workspace_bytes < w.total()) return DYNCONV_ERR_WORKSPACE;
  if (!aligned(workspace, 8)) return DYNCONV_ERR_UNSUPPORTED;
  char* at = static_cast<char*>(workspace);
  p.rate = rate;
  p.state_in = state_in, p.sis = state_in != nullptr ? sis[0] : 0;
  p.drate_part = reinterpret_cast<float*>(at);
  p.maps = reinterpret_cast<float2*>(at + w.drate);
  p.B = int32_t(B), p.T = int32_t(T), p.D = int32_t(D);
  cut(&p, z, false);
  hipError_t e;
  if (chunks != nullptr) {
    p.chunks = const_cast<float*>(chunks);
  } else {
    p.chunks = reinterpret_cast<float*>(at + w.drate + w.maps);
    if ((e = run_fwd(p, dtype, vec, packed, s)) != hipSuccess) return done(e);
  }
  cut(&p, z, true);
  p.dstate_out = dstate_out, p.dsos = dstate_out != nullptr ? dsos[0] : 0;
  p.dstate = dstate_in, p.dsis = dstate_in != nullptr ? dsis[0] : 0;
  const int64_t rows = int64_t(B) * p.nSeg;  // of drate's partial sums; a single one is the result
  if (rows == 1) p.drate_part = drate;
  e = dtype == DYNCONV_BF16  ? scan_bwd_bf16(p, vec, packed, s)
      : dtype == DYNCONV_F16 ? scan_bwd_f16(p, vec, packed, s)
                             : scan_bwd_f32(p, vec, packed, s);
  if (e == hipSuccess && rows > 1) e = norm_dweight(p.drate_part, rows, p.D, drate, s);
  return done(e);
}

dynconv_status dynconv_scan_step(const void* x, const int64_t* xs, const void* decay, const int64_t* as,
                                 const void* gate, const int64_t* gs, const float* rate, float* state,
                                 const int64_t* sts, void* y, const int64_t* ys, int64_t B, int64_t D,
                                 dynconv_dtype dtype, void* stream) {
  const Sizes z{B, 1, D};
  dynconv_status st = check_sizes(z, dtype);
  if (st != DYNCONV_OK) return st;
  if (B == 0 || D == 0) return DYNCONV_OK;
  const int eb = elem_bytes(dtype);
  int vec = D % 2 == 0 ? 2 : 1;
  ScanStepParams p{};
  auto row = [&](const void* t, const int64_t* s, bool output, int64_t* stride) {
    ScanTensor out;
    bool shared;
    if (t == nullptr || s == nullptr) return dynconv_status(DYNCONV_ERR_INVALID_ARG);
    const int64_t s3[3] = {s[0], 0, s[1]};
    const dynconv_status r = take(&out, t, s3, z, eb, output, &vec, &shared);
    *stride = s[0];
    return r;
  };
  if ((st = row(x, xs, false, &p.xs)) != DYNCONV_OK) return st;
  if ((st = row(decay, as, false, &p.as)) != DYNCONV_OK) return st;
  if (gate != nullptr && (st = row(gate, gs, false, &p.gs)) != DYNCONV_OK) return st;
  if ((st = row(y, ys, true, &p.ys)) != DYNCONV_OK) return st;
  if (rate == nullptr || state == nullptr) return DYNCONV_ERR_INVALID_ARG;
  if (!aligned(rate, 4)) return DYNCONV_ERR_UNSUPPORTED;
  if ((st = take_state(state, sts, z, true)) != DYNCONV_OK) return st;
  if (any_equal(y, {x, decay, gate, rate, state}) || any_equal(state, {x, decay, gate, rate})) return DYNCONV_ERR_INVALID_ARG;
  p.x = x, p.decay = decay, p.gate = gate, p.y = y, p.rate = rate, p.state = state, p.sts = sts[0];
  p.B = int32_t(B), p.D = int32_t(D);
  return done(scan_step(p, dtype, vec, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
