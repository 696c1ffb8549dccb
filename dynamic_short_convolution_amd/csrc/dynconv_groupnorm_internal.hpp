// Internal interface of the group norm: parameters, planning, launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/dynconv.h"

namespace dynconv {

// Activation [B,T,C] (channels adjacent); sc: the scales of an operand in 8 bits, [B,T,ceil(C/64)].
struct GroupTensor {
  const void* p;
  int64_t s0, s1;
  const uint8_t* sc;
  int64_t c0, c1;
};

struct GroupParams {
  GroupTensor x, gate;          // gate.p == null: none
  GroupTensor y;                // forward
  GroupTensor dy, dx, dgate;    // backward
  const void *weight, *bias;    // [C] or null
  const int32_t* lengths;       // [B] or null (sequences only)
  float* stats;                 // sequences: [B][G][2], mean and 1 / sqrt(var + eps)
  double* part;                 // sequences: [B][nChunk][G][2], sums of x and x^2
  float* colpart;               // backward: [rows][2][C] partial column sums (weight's and bias's gradient)
  float* colsum;                // backward over sequences: [B][2][C]
  int32_t B, T, C, G, Cg;
  int32_t silu;
  float eps;
  // Per token: groups and tokens that a workgroup works on at a time.
  int32_t gpw, tpw;
  // Sequences: groups of a workgroup, lanes of a group and of a token, tokens at a time, tokens of a workgroup
  // (and how many such chunks) in the forward's passes and in the gradient's.
  int32_t gpb, lpg, lpt, tps, chunk, nChunk, gradChunk, nGradChunk;
};

// Lanes per row and vectors per lane (nv 0: the looping form) of a group of Cg channels.
struct GroupPlan {
  int lpr, nv;
};
GroupPlan group_plan(int64_t Cg, int E);
// Workgroups along the tokens, each with one row of partial sums in the backward.
int64_t group_token_blocks(int64_t tokens, int64_t G, int64_t Cg, int E, bool bwd, int32_t* gpw, int32_t* tpw);
// Sets gpb to nGradChunk.
void group_sequence_plan(GroupParams* p, int E);

hipError_t group_tokens_f32(const GroupParams&, bool whole, bool packed, bool bwd, hipStream_t);
hipError_t group_tokens_bf16(const GroupParams&, bool whole, bool packed, bool bwd, hipStream_t);
hipError_t group_tokens_f16(const GroupParams&, bool whole, bool packed, bool bwd, hipStream_t);
enum GroupStage { kGroupStats, kGroupApply, kGroupColumns, kGroupGradient };
hipError_t group_sequences_f32(const GroupParams&, bool whole, bool packed, GroupStage, hipStream_t);
hipError_t group_sequences_bf16(const GroupParams&, bool whole, bool packed, GroupStage, hipStream_t);
hipError_t group_sequences_f16(const GroupParams&, bool whole, bool packed, GroupStage, hipStream_t);
}  // namespace dynconv
