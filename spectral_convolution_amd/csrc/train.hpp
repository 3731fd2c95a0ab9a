// train.hpp - arguments and launchers of the training operators around a block
// (checkpoint.hip, norm.hip, mix_train.hip). Apart from common.hpp: the counter
// summaries of the layer's kernels name the sources those are built from.
#pragma once

#include "common.hpp"

namespace fno {

// 8-bit checkpoint of rows x n values (checkpoint.hpp): pack reads x, unpack
// writes y.
struct CkArgs {
  const void *x;
  void *y;
  uint8_t *codes;  // [rows][32 nb]
  int8_t *exps;    // [rows][nb]
  long rows, n, nb;
};

// Norms around a block (norm.hip). Parameters may be NULL (weights, gate and
// scale then 1, biases 0).
struct NormArgs {
  const void *w_post, *b_post, *gate, *scale, *w_pre, *b_pre;
  int kind;  // 0: root mean square, 1: layer norm
  float eps;
  int B, C;
  long P;
  const void *x, *v;         // fields; NULL in a backward from checkpoints
  void *y, *u;               // forward outputs (u may be NULL)
  uint8_t *xq, *vq;          // codes of x and v: written by a forward, read by a backward; NULL: none
  int8_t *xe, *ve;           // their exponents
  const void *gy, *gu;       // gu may be NULL (no gradient through u)
  void *gx, *gv;             // NULL: not wanted
  void *g_w_post, *g_b_post, *g_gate, *g_scale, *g_w_pre, *g_b_pre;  // NULL: not wanted
  float *part;               // runs' sums; NULL when no parameter gradient is wanted
  int per;                   // fields: tiles of a run (set by the launcher)
};

// Channel mix of a training step (mix_train.hip): [B][I][P] -> [B][O][P].
struct MixTrainArgs {
  const void *x, *add;  // forward (add may be NULL)
  const void *A, *bias; // bias may be NULL
  void *y;
  uint8_t *xq, *aq;     // codes of x and add: written by the forward, read by the backward; aq NULL: add not kept
  int8_t *xe, *ae;      // their exponents
  const void *gy;
  void *gx, *gadd, *gA, *gbias;  // NULL: not wanted
  float *part;                   // workgroups' sums; NULL when neither gA nor gbias is wanted
  int B, I, O;
  long P;
  int act;
  int tpb, tiles, per;  // tiles of a sample, in all, of a workgroup (set by the launcher)
};

hipError_t launch_checkpoint(const CkArgs &a, bool pack, int dtype, hipStream_t s);
constexpr int kNormMaxField = 512;   // norms: channels of a field (P > 1)
constexpr long kNormMaxPixels = 1L << 27;  // lane offsets of 7 rows fit 32 bits
constexpr int kNormMaxToken = 8192;  // channels of a token (P = 1)
size_t norm_workspace_bytes(int B, int C, long P, int dtype);
hipError_t launch_norm_fwd(const NormArgs &a, int dtype, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs &a, int dtype, hipStream_t s);
constexpr int kMixTrainMax = 128;    // training channel mix: channels on either side
constexpr long kMixTrainPixels = 1L << 26, kMixTrainTiles = 1L << 30;  // lane offsets and tile numbers in 32 bits
size_t mix_train_workspace_bytes(int B, int I, int O, long P, int dtype);
hipError_t launch_mix_save(const MixTrainArgs &a, int dtype, hipStream_t s);
hipError_t launch_mix_bwd(const MixTrainArgs &a, int dtype, hipStream_t s);

}  // namespace fno
