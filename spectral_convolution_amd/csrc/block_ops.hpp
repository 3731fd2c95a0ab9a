// block_ops.hpp - arguments and launchers of the operators of a regularised block and
// of its 4-bit serving form (gnorm.hip, drop.hip, mx4.hip, mx4_mix.hip).
#pragma once

#include "common.hpp"

namespace fno {

// dropout of a call (drop.hpp); thr 0: none
enum : int { kDropElement = 0, kDropChannel = 1, kDropSample = 2 };
struct Drop {
  uint32_t thr;  // of 65536
  float scale;
  int unit;
  uint64_t seed, offset;
  const uint64_t *step;  // device memory, added to the offset; may be NULL
};

// y = x + D(v), x may be NULL. The field is rows of n contiguous values: [B C][P], or
// channels last [B P][C].
struct DropArgs {
  const void *x, *v;
  void *y;
  long rows, n;      // element and sample units: one row of everything
  int B, C;
  long P;
  int last;
  Drop drop;
};

hipError_t launch_drop(const DropArgs &a, int dtype, hipStream_t s);

// group norm with an activation and dropout (gnorm.hip)
struct GnArgs {
  const void *x, *gy;    // gy: backward
  void *y, *gx;          // forward, backward (gx may be NULL)
  const void *w, *b;     // may be NULL
  void *gw, *gb;         // NULL: not wanted
  float2 *stats;         // [B][G] (mean, 1 / sqrt(variance + eps))
  float2 *part;          // sums of rows or runs
  float2 *gpart;         // channels last: [B][S][G] sums of the groups in the pieces
  float2 *gsum;          // [B][G] backward: means of w gz and of w gz x^
  int B, C, G, Cg;
  long P;
  int act, last;
  float eps;
  Drop drop;
  int S;                 // pieces of a row (channels first) or of a sample (channels last), or runs
  long per;              // 16-byte chunks of such a piece (channels first), rows of it (channels last)
  long sb, sc, ss;       // strides of part: sample, channel, piece
  int whole;             // channels last: the first pass leaves gpart (a workgroup has all channels)
  int main;              // channels first: workgroups of the rows, in front of those of the parameters' sums
};

constexpr int kGnMaxChannels = 8192;
constexpr long kGnMaxPixels = 1L << 27;
size_t gnorm_workspace_bytes(const GnArgs &a, int dtype);  // of the shape: B, C, G, Cg, P, last
hipError_t launch_gnorm(const GnArgs &a, bool fwd, void *workspace, int dtype, hipStream_t s);

constexpr int kMx4MaxChannels = 65536;
constexpr long kMx4MaxRows = 1L << 31;
// microscaled 4-bit floats (mx4.hpp): rows (b, p) of C values along the channels
struct Mx4Args {
  const void *x;   // pack reads [B][C][P]
  void *y;         // unpack writes it
  uint8_t *codes;  // [B P][16 nb]
  uint8_t *exps;   // [B P][nb], 2^(exp - 127)
  int B, C;
  long P, nb;
  int step;        // fields: blocks that a workgroup packs at a time (set by the launcher)
};
hipError_t launch_mx4(const Mx4Args &a, bool pack, int dtype, hipStream_t s);

// y[b][o][p] = act(sum_i A[o][i] x[b][p][i] + bias[o] + add[b][o][p])
struct Mx4MixArgs {
  const uint8_t *xq, *xe;  // [B P][16 nb], [B P][nb]
  const uint8_t *aq, *ae;  // [O][16 nb], [O][nb]
  const void *bias, *add;  // may be NULL
  void *y;
  int B, I, O;
  long P, nb;
  int act;
};
hipError_t launch_mx4_mix(const Mx4MixArgs &a, int dtype, hipStream_t s);

}  // namespace fno
