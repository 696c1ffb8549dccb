// Internal interface of the gated linear scan: parameters, the segment rule, launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/dynconv.h"

namespace dynconv {

constexpr int kScanCols = 64;    // channels of a workgroup
constexpr int kScanScaleCols = 64;  // channels that share a scale of an operand in 8 bits
constexpr int kScanWaves = 8;    // waves of a workgroup, one after the other along the tokens
constexpr int kScanElems = 16;   // elements of a tile per lane: 16 tokens of one channel or 8 of two
constexpr int kScanTile = kScanWaves * kScanElems * 64 / kScanCols;  // tokens of a workgroup's tile
constexpr int kScanChunk = 128;  // tokens between two kept states
static_assert(kScanTile == kScanChunk, "kept states start tiles");

// Activation [B,T,D] (channels adjacent); sc: the scales of an operand in 8 bits, [B,T,ceil(D/64)].
struct ScanTensor {
  const void* p;
  int64_t s0, s1;
  const uint8_t* sc;
  int64_t c0, c1;
};

struct ScanParams {
  ScanTensor x, decay, gate, dy;   // gate.p == null: none
  ScanTensor y, dx, ddecay, dgate; // forward output (p == null: none); backward outputs
  const float* rate;               // [D]
  const int32_t* seg;              // document ids or null
  int64_t ss0, ss1;
  const float* state_in;           // [B,D] or null
  int64_t sis;
  float* state_out;                // forward
  int64_t sos;
  float* chunks;                   // [B, ceil(T/128), D]: written by the forward, read by the backward; or null
  const float* dstate_out;         // backward: [B,D] or null
  int64_t dsos;
  float* dstate;
  int64_t dsis;
  float* drate_part;               // [B * nSeg][D]
  // Segments of a sequence that run at the same time (nSeg > 1): [B][nSeg][D] pairs. Forward: place 0
  // holds the initial state, place s the product of decays and the state from zero of segment
  // s - 1. Backward: place nSeg - 1 the gradient from behind the last token, place s those of
  // segment s + 1, in reverse.
  float2* maps;
  int32_t B, T, D, nSeg, segTiles;  // segTiles: tiles per segment
  bool shared;                      // workgroups side by side share 128-byte lines of a tensor
};

// Tiles per segment. A workgroup walks its tiles one behind the other; with few (sequence, 64
// channels) pairs the CUs would idle, so the sequence is cut, at the price of a first pass that
// reads the inputs of the maps once more: all three of the forward, two of the backward's four, which therefore
// is cut into two already (bf16, whole / cut, us: 128 pairs of 7812 tokens 176 / 180 forward and 326 / 242
// backward, of 2048 tokens 47 / 50 and 83 / 67; 85 pairs of 11764 tokens into three 245 / 170 and 456 / 227;
// 32 of 31250 into eight 658 / 183 and 1215 / 255, into four 328 / 423, into sixteen 201 / 267).
inline int32_t scan_segment_tiles(int64_t B, int64_t D, int64_t T, bool bwd) {
  const int64_t blocks = B * ((D + kScanCols - 1) / kScanCols), tiles = (T + kScanTile - 1) / kScanTile;
  int64_t want = blocks > 0 ? 256 / blocks : 1;  // one workgroup per CU
  if (want < (bwd ? 2 : 3) || tiles < 4) return int32_t(tiles > 0 ? tiles : 1);
  if (want > tiles) want = tiles;
  if (want > 64) want = 64;
  return int32_t((tiles + want - 1) / want);
}
inline int32_t scan_segments(int64_t T, int32_t segTiles) {
  const int64_t tiles = (T + kScanTile - 1) / kScanTile;
  return int32_t(tiles > 0 ? (tiles + segTiles - 1) / segTiles : 1);
}

// vec: channels per lane (1, or 2 where alignment and D allow); packed: x, decay and gate in 8 bits.
hipError_t scan_fwd_f32(const ScanParams&, int vec, bool packed, hipStream_t);
hipError_t scan_fwd_bf16(const ScanParams&, int vec, bool packed, hipStream_t);
hipError_t scan_fwd_f16(const ScanParams&, int vec, bool packed, hipStream_t);
hipError_t scan_bwd_f32(const ScanParams&, int vec, bool packed, hipStream_t);
hipError_t scan_bwd_bf16(const ScanParams&, int vec, bool packed, hipStream_t);
hipError_t scan_bwd_f16(const ScanParams&, int vec, bool packed, hipStream_t);

// dst [B,D] (row stride ds) = src (row stride ss), or zeros without src.
hipError_t scan_copy_state(const float* src, int64_t ss, float* dst, int64_t ds, int32_t B, int32_t D, hipStream_t s);

struct ScanStepParams {
  const void *x, *decay, *gate;
  void* y;
  int64_t xs, as, gs, ys, sts;
  const float* rate;
  float* state;
  int32_t B, D;
};
hipError_t scan_step(const ScanStepParams&, dynconv_dtype dt, int vec, hipStream_t);

}  // namespace dynconv
