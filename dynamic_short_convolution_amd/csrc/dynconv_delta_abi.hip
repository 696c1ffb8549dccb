// C ABI of the gated delta rule: argument checks (before any HIP call) and dispatch. See
// include/dynconv.h for the contract of every entry point.
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "dynconv_delta_internal.hpp"
#include "dynconv_internal.hpp"

using namespace dynconv;

namespace {

int elem_bytes(dynconv_dtype dt) { return dt == DYNCONV_F32 ? 4 : 2; }
bool aligned(const void* p, int64_t a) { return (reinterpret_cast<uintptr_t>(p) % uint64_t(a)) == 0; }

// A tensor of n dimensions with extents e and strides s; `unit`: the last one has stride 1.
// Strides of inputs are at least 0; an output's elements have places of their own along
// every dimension of more than one.
dynconv_status check_tensor(const void* p, const int64_t* s, int n, const int64_t* e, int align, bool unit, bool output) {
  if (p == nullptr || s == nullptr) return DYNCONV_ERR_INVALID_ARG;
  if (!aligned(p, align)) return DYNCONV_ERR_UNSUPPORTED;
  if (unit && e[n - 1] > 1 && s[n - 1] != 1) return DYNCONV_ERR_UNSUPPORTED;
  for (int i = 0; i < n; ++i) {
    if (s[i] < 0) return DYNCONV_ERR_UNSUPPORTED;
    if (output && e[i] > 1 && s[i] == 0) return DYNCONV_ERR_INVALID_ARG;
  }
  return DYNCONV_OK;
}

// The kernels address a chunk's 64 rows with 32-bit byte offsets: token strides (s[1]) stay
// below this many elements.
constexpr int64_t kDeltaMaxTokenStride = int64_t(1) << 22;
bool far_tokens(const int64_t* s, int64_t T) { return T > 1 && s[1] >= kDeltaMaxTokenStride; }

// The token stride that the kernels get. With one token it has no meaning (0, 1 and far ones are
// common: an expanded row, channels first, a slice of one token), but the kernels tell the chunk's rows
// that do not exist by their offsets behind the first, which a shorter stride than a row would
// put into it.
int64_t token_stride(const int64_t* s, const int64_t* e) { return e[1] > 1 ? s[1] : e[3]; }

// Whether the rows of a chunk lie one behind the other (no token's row overlaps the next).
bool apart(const int64_t* s, const int64_t* e) { return e[1] <= 1 || s[1] >= e[3]; }

// Whether rows of the last dimension can be read in 16-byte pieces.
int wide(const void* p, const int64_t* s, int n, const int64_t* e, int eb) {
  if (!aligned(p, 16)) return 0;
  for (int i = 0; i + 1 < n; ++i)
    if (e[i] > 1 && s[i] * eb % 16 != 0) return 0;
  return 1;
}

dynconv_status check_sizes(int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, dynconv_dtype dt,
                           float eps = 0.f) {
  if (eps != eps) return DYNCONV_ERR_INVALID_ARG;  // neither with a norm nor without
  if (dt != DYNCONV_F32 && dt != DYNCONV_BF16 && dt != DYNCONV_F16) return DYNCONV_ERR_INVALID_ARG;
  if (B < 0 || T < 0 || Hk < 0 || Hv < 0 || dk < 0 || dv < 0) return DYNCONV_ERR_INVALID_ARG;
  if (B == 0 || Hv == 0 || dk == 0 || dv == 0) return DYNCONV_OK;
  if (Hk == 0 || Hv % Hk != 0) return DYNCONV_ERR_INVALID_ARG;
  if (dk > kDeltaMaxDk || dv > kDeltaMaxDv) return DYNCONV_ERR_UNSUPPORTED;
  if (B > INT32_MAX || T > INT32_MAX - 65536 || Hv > INT32_MAX) return DYNCONV_ERR_UNSUPPORTED;
  // Workgroups per launch: one per (sequence, head, 32 columns), of up to 512 threads (a launch
  // has fewer than 2^32), or per (sequence, head, chunk), where memory ends first: the forward's
  // 2^24 of 256 threads need 340 GB of workspace, the backward's 2^23 of 512 more.
  constexpr int64_t most = (int64_t(1) << 23) - 1;
  const int64_t bh = B * Hv;
  const int64_t per = (T + kDeltaChunk - 1) / kDeltaChunk;
  const int64_t cols = (dv + 31) / 32;
  if (bh > most || (per > 0 && bh > INT32_MAX / per) || bh > most / cols) return DYNCONV_ERR_UNSUPPORTED;
  return DYNCONV_OK;
}

bool empty(int64_t B, int64_t Hv, int64_t dk, int64_t dv) { return B == 0 || Hv == 0 || dk == 0 || dv == 0; }

// The inputs that both directions share, checked and set in p.
dynconv_status take_inputs(DeltaParams* p, const void* q, const int64_t* qs, const void* k, const int64_t* ks,
                           const void* v, const int64_t* vs, const float* g, const int64_t* gs, const void* beta,
                           const int64_t* bs, const int32_t* seg, const int64_t* ss, const float* state_in,
                           const int64_t* sis, int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv,
                           float scale, float eps, dynconv_dtype dt) {
  const int eb = elem_bytes(dt);
  const int64_t eq[4] = {B, T, Hk, dk}, ev[4] = {B, T, Hv, dv}, eg[3] = {B, T, Hv}, est[4] = {B, Hv, dk, dv};
  dynconv_status st;
  if (T > 0) {  // without tokens only the states are touched
    if ((st = check_tensor(q, qs, 4, eq, eb, true, false)) != DYNCONV_OK) return st;
    if ((st = check_tensor(k, ks, 4, eq, eb, true, false)) != DYNCONV_OK) return st;
    if ((st = check_tensor(v, vs, 4, ev, eb, true, false)) != DYNCONV_OK) return st;
    if ((st = check_tensor(g, gs, 3, eg, 4, false, false)) != DYNCONV_OK) return st;
    if ((st = check_tensor(beta, bs, 3, eg, eb, false, false)) != DYNCONV_OK) return st;
    if (far_tokens(qs, T) || far_tokens(ks, T) || far_tokens(vs, T)) return DYNCONV_ERR_UNSUPPORTED;
    if (seg != nullptr) {
      if (ss == nullptr) return DYNCONV_ERR_INVALID_ARG;
      if (ss[0] < 0 || ss[1] < 0 || !aligned(seg, 4)) return DYNCONV_ERR_UNSUPPORTED;
      p->seg = seg;
      p->ss0 = ss[0];
      p->ss1 = ss[1];
    }
    p->q = q, p->k = k, p->v = v, p->g = g, p->beta = beta;
    p->qs0 = qs[0], p->qs1 = token_stride(qs, eq), p->qs2 = qs[2];
    p->ks0 = ks[0], p->ks1 = token_stride(ks, eq), p->ks2 = ks[2];
    p->vs0 = vs[0], p->vs1 = token_stride(vs, ev), p->vs2 = vs[2];
    p->gs0 = gs[0], p->gs1 = gs[1], p->gs2 = gs[2];
    p->bs0 = bs[0], p->bs1 = bs[1], p->bs2 = bs[2];
    p->vec = dk % 8 == 0 && wide(q, qs, 4, eq, eb) && wide(k, ks, 4, eq, eb) && apart(qs, eq) && apart(ks, eq) &&
             apart(vs, ev);
  }
  if (state_in != nullptr) {
    if ((st = check_tensor(state_in, sis, 4, est, 4, true, false)) != DYNCONV_OK) return st;
    p->state_in = state_in;
    p->sis0 = sis[0], p->sis1 = sis[1], p->sis2 = sis[2];
  }
  p->B = int32_t(B), p->T = int32_t(T), p->Hk = int32_t(Hk), p->Hv = int32_t(Hv), p->group = int32_t(Hv / Hk);
  p->dkn = int32_t(dk), p->dvn = int32_t(dv);
  p->nC = int32_t((T + kDeltaChunk - 1) / kDeltaChunk);
  p->nCG = int32_t((dv + kDeltaCols - 1) / kDeltaCols);
  p->segLen = delta_segment_length(B * Hv, p->nC, p->nCG);
  p->nSeg = p->nC > 0 ? (p->nC + p->segLen - 1) / p->segLen : 1;
  p->scale = scale;
  p->eps = eps;
  return DYNCONV_OK;
}

bool any_equal(const void* out, std::initializer_list<const void*> others) {
  if (out == nullptr) return false;
  for (const void* o : others)
    if (o == out) return true;
  return false;
}

}  // namespace

extern "C" {

size_t dynconv_delta_fwd_workspace_size(int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv,
                                        dynconv_dtype dtype) {
  if (check_sizes(B, T, Hk, Hv, dk, dv, dtype) != DYNCONV_OK || empty(B, Hv, dk, dv) || T == 0) return 0;
  return delta_workspace(B, T, Hv, dk, dv, false);
}

dynconv_status dynconv_delta_fwd(const void* q, const int64_t* qs, const void* k, const int64_t* ks, const void* v,
                                 const int64_t* vs, const float* g, const int64_t* gs, const void* beta,
                                 const int64_t* bs, const int32_t* seq_idx, const int64_t* ss, const float* state_in,
                                 const int64_t* sis, void* o, const int64_t* os, float* state_out, const int64_t* sos,
                                 int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, float scale,
                                 float qk_norm_eps, dynconv_dtype dtype, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  dynconv_status st = check_sizes(B, T, Hk, Hv, dk, dv, dtype, qk_norm_eps);
  if (st != DYNCONV_OK) return st;
  if (empty(B, Hv, dk, dv)) return DYNCONV_OK;
  DeltaParams p{};
  st = take_inputs(&p, q, qs, k, ks, v, vs, g, gs, beta, bs, seq_idx, ss, state_in, sis, B, T, Hk, Hv, dk, dv, scale,
                   qk_norm_eps, dtype);
  if (st != DYNCONV_OK) return st;
  const int64_t ev[4] = {B, T, Hv, dv}, est[4] = {B, Hv, dk, dv};
  if (T > 0) {
    if ((st = check_tensor(o, os, 4, ev, elem_bytes(dtype), true, true)) != DYNCONV_OK) return st;
    if (far_tokens(os, T)) return DYNCONV_ERR_UNSUPPORTED;
    p.vec = p.vec && apart(os, ev);
    p.out = o;
    p.os0 = os[0], p.os1 = token_stride(os, ev), p.os2 = os[2];
  }
  if (state_out != nullptr) {
    if ((st = check_tensor(state_out, sos, 4, est, 4, true, true)) != DYNCONV_OK) return st;
    p.state_out = state_out;
    p.sos0 = sos[0], p.sos1 = sos[1], p.sos2 = sos[2];
  }
  if (any_equal(p.out, {q, k, v, g, beta, seq_idx, state_in, state_out}) ||
      any_equal(state_out, {q, k, v, g, beta, seq_idx}))
    return DYNCONV_ERR_INVALID_ARG;
  // the state may be carried in place when its rows have the same places
  if (state_out != nullptr && state_out == state_in && (sis[0] != sos[0] || sis[1] != sos[1] || sis[2] != sos[2]))
    return DYNCONV_ERR_INVALID_ARG;
  if (T == 0 && state_out == nullptr) return DYNCONV_OK;
  if (T > 0) {
    if (workspace == nullptr || workspace_bytes < delta_workspace(B, T, Hv, dk, dv, false)) return DYNCONV_ERR_WORKSPACE;
    delta_carve(&p, workspace, false);
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = dtype == DYNCONV_BF16  ? delta_fwd_bf16(p, s)
                       : dtype == DYNCONV_F16 ? delta_fwd_f16(p, s)
                                              : delta_fwd_f32(p, s);
  return e == hipSuccess ? DYNCONV_OK : record_hip_error(e);
}

size_t dynconv_delta_bwd_workspace_size(int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv,
                                        dynconv_dtype dtype) {
  if (check_sizes(B, T, Hk, Hv, dk, dv, dtype) != DYNCONV_OK || empty(B, Hv, dk, dv) || T == 0) return 0;
  return delta_workspace(B, T, Hv, dk, dv, true);
}

dynconv_status dynconv_delta_bwd(const void* q, const int64_t* qs, const void* k, const int64_t* ks, const void* v,
                                 const int64_t* vs, const float* g, const int64_t* gs, const void* beta,
                                 const int64_t* bs, const int32_t* seq_idx, const int64_t* ss, const float* state_in,
                                 const int64_t* sis, const void* dO, const int64_t* dos, const float* dstate_out,
                                 const int64_t* dsos, void* dq, const int64_t* dqs, void* dk_, const int64_t* dks,
                                 void* dv_, const int64_t* dvs, float* dg, const int64_t* dgs, void* dbeta,
                                 const int64_t* dbs, float* dstate_in, const int64_t* dsis, int64_t B, int64_t T,
                                 int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, float scale, float qk_norm_eps,
                                 dynconv_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  dynconv_status st = check_sizes(B, T, Hk, Hv, dk, dv, dtype, qk_norm_eps);
  if (st != DYNCONV_OK) return st;
  if (empty(B, Hv, dk, dv) || T == 0) return DYNCONV_OK;
  DeltaParams p{};
  st = take_inputs(&p, q, qs, k, ks, v, vs, g, gs, beta, bs, seq_idx, ss, state_in, sis, B, T, Hk, Hv, dk, dv, scale,
                   qk_norm_eps, dtype);
  if (st != DYNCONV_OK) return st;
  const int eb = elem_bytes(dtype);
  const int64_t eq[4] = {B, T, Hk, dk}, ev[4] = {B, T, Hv, dv}, eg[3] = {B, T, Hv}, est[4] = {B, Hv, dk, dv};
  if ((st = check_tensor(dO, dos, 4, ev, eb, true, false)) != DYNCONV_OK) return st;
  if ((st = check_tensor(dq, dqs, 4, eq, eb, true, true)) != DYNCONV_OK) return st;
  if ((st = check_tensor(dk_, dks, 4, eq, eb, true, true)) != DYNCONV_OK) return st;
  if ((st = check_tensor(dv_, dvs, 4, ev, eb, true, true)) != DYNCONV_OK) return st;
  if ((st = check_tensor(dg, dgs, 3, eg, 4, false, true)) != DYNCONV_OK) return st;
  if ((st = check_tensor(dbeta, dbs, 3, eg, eb, false, true)) != DYNCONV_OK) return st;
  if (far_tokens(dos, T) || far_tokens(dvs, T) || far_tokens(dqs, T) || far_tokens(dks, T)) return DYNCONV_ERR_UNSUPPORTED;
  p.dO = dO, p.dq = dq, p.dk = dk_, p.dv = dv_, p.dg = dg, p.dbeta = dbeta;
  p.dos0 = dos[0], p.dos1 = token_stride(dos, ev), p.dos2 = dos[2];
  p.dqs0 = dqs[0], p.dqs1 = token_stride(dqs, eq), p.dqs2 = dqs[2];
  p.dks0 = dks[0], p.dks1 = token_stride(dks, eq), p.dks2 = dks[2];
  p.dvs0 = dvs[0], p.dvs1 = token_stride(dvs, ev), p.dvs2 = dvs[2];
  p.dgs0 = dgs[0], p.dgs1 = dgs[1], p.dgs2 = dgs[2];
  p.dbs0 = dbs[0], p.dbs1 = dbs[1], p.dbs2 = dbs[2];
  p.vec = p.vec && dv % 8 == 0 && wide(dO, dos, 4, ev, eb) && apart(dos, ev) && apart(dvs, ev) &&
          apart(dqs, eq) && apart(dks, eq);
  if (dstate_out != nullptr) {
    if ((st = check_tensor(dstate_out, dsos, 4, est, 4, true, false)) != DYNCONV_OK) return st;
    p.dstate_out = dstate_out;
    p.dsos0 = dsos[0], p.dsos1 = dsos[1], p.dsos2 = dsos[2];
  }
  if (dstate_in != nullptr) {
    if ((st = check_tensor(dstate_in, dsis, 4, est, 4, true, true)) != DYNCONV_OK) return st;
    p.dstate = dstate_in;
    p.dsis0 = dsis[0], p.dsis1 = dsis[1], p.dsis2 = dsis[2];
  }
  const void* outs[6] = {dq, dk_, dv_, dg, dbeta, dstate_in};
  for (int i = 0; i < 6; ++i) {
    if (any_equal(outs[i], {q, k, v, g, beta, seq_idx, state_in, dO, dstate_out})) return DYNCONV_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (outs[i] != nullptr && outs[i] == outs[j]) return DYNCONV_ERR_INVALID_ARG;
  }
  if (workspace == nullptr || workspace_bytes < delta_workspace(B, T, Hv, dk, dv, true)) return DYNCONV_ERR_WORKSPACE;
  delta_carve(&p, workspace, true);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = dtype == DYNCONV_BF16  ? delta_bwd_bf16(p, s)
                       : dtype == DYNCONV_F16 ? delta_bwd_f16(p, s)
                                              : delta_bwd_f32(p, s);
  return e == hipSuccess ? DYNCONV_OK : record_hip_error(e);
}

dynconv_status dynconv_delta_step(const void* q, const int64_t* qs, const void* k, const int64_t* ks, const void* v,
                                  const int64_t* vs, const float* g, const int64_t* gs, const void* beta,
                                  const int64_t* bs, float* state, const int64_t* sts, void* o, const int64_t* os,
                                  int64_t B, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, float scale,
                                  float qk_norm_eps, dynconv_dtype dtype, void* stream) {
  dynconv_status st = check_sizes(B, 1, Hk, Hv, dk, dv, dtype, qk_norm_eps);
  if (st != DYNCONV_OK) return st;
  if (empty(B, Hv, dk, dv)) return DYNCONV_OK;
  const int eb = elem_bytes(dtype);
  const int64_t eq[3] = {B, Hk, dk}, ev[3] = {B, Hv, dv}, eg[2] = {B, Hv}, est[4] = {B, Hv, dk, dv};
  if ((st = check_tensor(q, qs, 3, eq, eb, true, false)) != DYNCONV_OK) return st;
  if ((st = check_tensor(k, ks, 3, eq, eb, true, false)) != DYNCONV_OK) return st;
  if ((st = check_tensor(v, vs, 3, ev, eb, true, false)) != DYNCONV_OK) return st;
  if ((st = check_tensor(g, gs, 2, eg, 4, false, false)) != DYNCONV_OK) return st;
  if ((st = check_tensor(beta, bs, 2, eg, eb, false, false)) != DYNCONV_OK) return st;
  if ((st = check_tensor(state, sts, 4, est, 4, true, true)) != DYNCONV_OK) return st;
  if ((st = check_tensor(o, os, 3, ev, eb, true, true)) != DYNCONV_OK) return st;
  if (any_equal(o, {q, k, v, g, beta, state}) || any_equal(state, {q, k, v, g, beta})) return DYNCONV_ERR_INVALID_ARG;
  DeltaStepParams p{};
  p.q = q, p.k = k, p.v = v, p.g = g, p.beta = beta, p.state = state, p.out = o;
  p.qs0 = qs[0], p.qs1 = qs[1], p.ks0 = ks[0], p.ks1 = ks[1], p.vs0 = vs[0], p.vs1 = vs[1];
  p.gs0 = gs[0], p.gs1 = gs[1], p.bs0 = bs[0], p.bs1 = bs[1], p.os0 = os[0], p.os1 = os[1];
  p.sts0 = sts[0], p.sts1 = sts[1], p.sts2 = sts[2];
  p.B = int32_t(B), p.Hk = int32_t(Hk), p.Hv = int32_t(Hv), p.group = int32_t(Hv / Hk);
  p.dkn = int32_t(dk), p.dvn = int32_t(dv);
  p.vec = dv % 4 == 0 && wide(state, sts, 4, est, 4);
  p.scale = scale;
  p.eps = qk_norm_eps;
  const hipError_t e = delta_step(p, dtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? DYNCONV_OK : record_hip_error(e);
}

}  // extern "C"
