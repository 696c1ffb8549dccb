// Internal interface of the gated delta rule: parameters, workspace layout, launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/dynconv.h"

namespace dynconv {

constexpr int kDeltaChunk = 64;     // tokens per chunk
constexpr int kDeltaMaxDk = 128;    // widest key head
constexpr int kDeltaMaxDv = 65536;  // widest value head
constexpr int kDeltaCols = 16;      // value columns of one wave

// Lower-triangular 64 x 64 matrices keep rows 0..31 in 32 columns and rows 32..63 in 64.
constexpr int kTrapElems = 32 * 32 + 32 * 64;
constexpr int kTokArrays = 8;  // per chunk and value head: float[64] each, in this order
enum { kTokGhi = 0, kTokGlo, kTokE, kTokD, kTokN, kTokRk, kTokRq, kTokBeta };

struct DeltaParams {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const void* beta;
  const int32_t* seg;
  const void* dO;
  void* out;  // o (forward)
  void* dq;
  void* dk;
  void* dv;
  float* dg;
  void* dbeta;
  const float* state_in;    // [B,Hv,dk,dv] or null
  float* state_out;         // or null
  const float* dstate_out;  // gradient of the final state, or null
  float* dstate;            // gradient of the initial state, or null
  int64_t qs0, qs1, qs2, ks0, ks1, ks2, vs0, vs1, vs2, gs0, gs1, gs2, bs0, bs1, bs2, ss0, ss1;
  int64_t dos0, dos1, dos2, os0, os1, os2, dqs0, dqs1, dqs2, dks0, dks1, dks2, dvs0, dvs1, dvs2;
  int64_t dgs0, dgs1, dgs2, dbs0, dbs1, dbs2;
  int64_t sis0, sis1, sis2, sos0, sos1, sos2, dsos0, dsos1, dsos2, dsis0, dsis1, dsis2;
  int32_t B, T, Hk, Hv, group, dkn, dvn;  // dkn, dvn: key and value head widths
  int32_t nC, nCG;                        // chunks per sequence, 16-column groups of a value head
  int32_t nSeg, segLen;                   // segments of a sequence's chunks, chunks of one (the last may be shorter)
  int32_t vec;                            // rows of q, k (and dO) allow 16-byte loads
  float scale, eps;                       // eps < 0: q and k as they are
  // workspace
  uint16_t* wT;   // [chunk][3][kTrapElems]: (I + A)^-1 in three 8-bit terms
  float* wTok;    // [chunk][kTokArrays][64]
  float* wS;      // [chunk][nCG][DK * 16]: state before the chunk, in fragment order
  float* wdS;     // the same, gradient of the state after the chunk
  float* wU;      // [chunk][nCG][1024]: u, in fragment order
  float* wR;      // the same, gradient of beta * (v - decayed prediction)
  float* wEnd;    // [sequence and head][nSeg][nCG][DK * 16]: state at a segment's end, in fragment order (last: initial)
  float* wBegin;  // the same, gradient at a segment's start
  float* wM;      // [sequence and head][nSeg][DK][DK]: a segment's transition
  float* wDot;    // [chunk][nCG][64]: sums of dR o V over the group's columns
};

constexpr int delta_dk_pad(int dk) { return dk <= 64 ? 64 : 128; }

// Segments that the scans cut a sequence's chunks into. They pay where one segment per sequence
// and head leaves most of the 256 CUs idle: with n segments of nC / n chunks the two passes take
// about 2 nC / n chunks' time, joining about a third of one per segment and the two more launches
// one, which is least for n = sqrt(6 nC); a segment has at least 2 chunks, and from 8 chunks and
// 3 segments on it is less than the nC of one pass (16 heads of 128 x 128, bf16, forward /
// backward in us, one segment and as many as here: T 400 45 / 95 and 51 / 98, T 512 47 / 104 and
// 47 / 91, T 1024 80 / 163 and 58 / 112, T 32768 forward 2500 and 681).
constexpr int delta_segment_length(int64_t bh, int64_t nC, int64_t nCG) {
  const int64_t blocks = bh * ((nCG + 3) / 4);
  int64_t n = blocks > 0 ? 256 / blocks : 1;
  if (n > nC / 2) n = nC / 2;
  while (n * n > 6 * nC) --n;
  if (n < 3 || nC < 8) return nC > 0 ? int(nC) : 1;
  return int((nC + n - 1) / n);
}

// Workspace bytes of the two directions (0 for sizes outside the limits).
size_t delta_workspace(int64_t B, int64_t T, int64_t Hv, int64_t dk, int64_t dv, bool bwd);
// Points p's workspace members into `ws` (256-byte aligned pieces).
void delta_carve(DeltaParams* p, void* ws, bool bwd);

hipError_t delta_fwd_f32(const DeltaParams& p, hipStream_t s);
hipError_t delta_fwd_bf16(const DeltaParams& p, hipStream_t s);
hipError_t delta_fwd_f16(const DeltaParams& p, hipStream_t s);
hipError_t delta_bwd_f32(const DeltaParams& p, hipStream_t s);
hipError_t delta_bwd_bf16(const DeltaParams& p, hipStream_t s);
hipError_t delta_bwd_f16(const DeltaParams& p, hipStream_t s);

struct DeltaStepParams {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const void* beta;
  float* state;
  void* out;
  int64_t qs0, qs1, ks0, ks1, vs0, vs1, gs0, gs1, bs0, bs1, sts0, sts1, sts2, os0, os1;
  int32_t B, Hk, Hv, group, dkn, dvn;
  int32_t vec;  // 16-byte state rows
  float scale, eps;
};
hipError_t delta_step(const DeltaStepParams& p, dynconv_dtype dt, hipStream_t s);

}  // namespace dynconv
