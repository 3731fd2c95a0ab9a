// gnorm.hip - group norm with an activation and dropout behind it, forward and backward, on
// fields with the channels first ([B][C][P]) or last ([B][P][C]).
//
// Over a group g of C / G channels and all pixels of a sample, n values:
//   m = mean(x),  r = 1 / sqrt(mean((x - m)^2) + eps),  x^ = (x - m) r
//   y = D(act(w[c] x^ + b[c]))            D: dropout (drop.hpp); act: none, GELU or SiLU
// Backward at gy = dL/dy, z = w x^ + b, gz = D(gy) act'(z), with the sums over a channel's pixels
//   s1[b][c] = sum gz,  s2[b][c] = sum gz x^:
//   gb = sum_b s1,  gw = sum_b s2,
//   gx = r (w gz - M1 - x^ M2),  M1 = sum_c w s1 / n,  M2 = sum_c w s2 / n.
// The mask of D is computed again. Statistics and sums are fp32. A group that is read once has its mean corrected by its values'
// deviations from it, so the mean is off by half a step; pieces of a larger one have their squares summed about a value from among
// those summed, which an outlier or a large mean does not cost digits, and are joined by Chan's formula, where each join
// moves the mean by up to half a step. No atomics: results repeat bit for bit.
//
// A group that fits a workgroup's registers is read once (fno_gnorm_small). Of larger ones a first
// kernel leaves the moments (forward) or s1, s2 (backward) of every channel's pieces, a small one joins
// them, a third reads the field again. A backward of small groups still needs s1, s2 for the
// parameters, summed over runs of whole rows. Bound by memory and by the vector units alike: a step of 20 x 64 x 256^2 fp16 with
// GELU takes 254 us, its kernels at their fastest 33 (the moments, 5.1 TB/s), 66 (values, 5.1), 73 (sums, 4.6) and 90 (gx, 5.6), vector
// issue 94 and 97 % in the middle two; of 4 x 64^3 x 32 fp32, channels last, dropout, 215 us: 28, 54, 56 and 70 (5.8 TB/s).

#include <algorithm>

#include "gnorm.hpp"

namespace fno {

namespace {
// Workgroups that fill the chip, each with as much to read as pays for its start (channels first, 20 x 64 x 256^2
// fp16, a step: 1024 / 2048 / 3000 of them 294 / 280 / 300 us; last, 4 x 64^3 x 32 fp32: 211 / 215 / 237)
constexpr long kUnits = 2048, kLastUnits = 1024;
constexpr long kParts = 1L << 22;     // sums that pieces beyond one a sample may take
}  // namespace

GnPlan gn_plan(const GnArgs &a, int dtype) {
  GnPlan p{};
  const long V = gn_vec(dtype);
  p.last = a.last || a.P == 1;
  const long len = p.last ? a.Cg : a.P, rows = p.last ? a.P : a.Cg, chunks = up(len, V) * rows;
  p.team = chunks <= 16 ? 8 : chunks <= 64 ? 16 : chunks <= 256 ? 64 : chunks <= 1024 ? 256 : chunks <= 4096 ? 1024 : chunks <= 8192 ? 2048 : 0;
  // one compute unit a group: few large ones would leave the others idle
  if (p.team >= 1024 && (long)a.B * a.G < 96) p.team = 0;
  p.bteam = chunks <= 4096 ? p.team : 0;  // the backward holds two fields
  const long bc = (long)a.B * a.C;
  if (!p.last) {
    const long cpr = up(a.P, V);
    p.T = cpr <= 16 ? 8 : cpr <= 256 ? 64 : 256;
    p.S = 1, p.per = cpr;
    if (p.T == 256) {  // at least two chunks a lane, at most 64
      const long want = std::max(std::min(up(kUnits, bc), up(cpr, 512)), up(cpr, 64 * 256));
      p.per = up(up(cpr, want), 256) * 256;
      p.S = (int)up(cpr, p.per);
    }
    p.parts = (size_t)bc * p.S;
    return p;
  }
  const long cpr = up(a.C, V), lanes = std::max(1L, (long)kThreads / std::min(cpr, (long)kThreads));
  const long blocks = up(cpr, kThreads), most = std::max(1L, kParts / bc);
  // long samples in more pieces, of 256 rows a lane (3 x 64 x 22 M fp16, forward: 4.8 ms, 6.5 by 1024 workgroups)
  const long S = std::min({std::max(up(kLastUnits, a.B * blocks), up(a.P, 256 * lanes)), up(a.P, 4 * lanes), most});
  p.per = up(a.P, S);
  p.S = (int)up(a.P, p.per);
  const long all = a.B * a.P;
  // half as many runs: twice the sums cost more than the second half of the workgroups gains (8192 x 1024 bf16 in 8
  // groups, a step: 50 us with all, 45 with half)
  const long R = std::min({up(kLastUnits / 2, blocks), up(all, 4 * lanes), std::max(1L, kParts / a.C)});
  p.per_run = up(all, R);
  p.runs = (int)up(all, p.per_run);
  p.parts = std::max(p.bteam ? 0 : (size_t)bc * p.S, (size_t)a.C * p.runs);
  p.gparts = !p.bteam && blocks == 1 ? (size_t)a.B * p.S * a.G : 0;
  return p;
}

size_t gnorm_workspace_bytes(const GnArgs &a, int dtype) {
  const GnPlan p = gn_plan(a, dtype);
  return (p.parts + p.gparts + (p.bteam ? 0 : (size_t)a.B * a.G)) * sizeof(float2);
}

hipError_t gnorm_f32(const GnArgs &a, bool fwd, void *workspace, hipStream_t s);
hipError_t gnorm_f16(const GnArgs &a, bool fwd, void *workspace, hipStream_t s);
hipError_t gnorm_bf16(const GnArgs &a, bool fwd, void *workspace, hipStream_t s);

hipError_t launch_gnorm(const GnArgs &a, bool fwd, void *workspace, int dtype, hipStream_t s) {
  if (dtype == DT_F32) return gnorm_f32(a, fwd, workspace, s);
  return dtype == DT_F16 ? gnorm_f16(a, fwd, workspace, s) : gnorm_bf16(a, fwd, workspace, s);
}

}  // namespace fno
