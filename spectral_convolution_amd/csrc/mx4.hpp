// mx4.hpp - microscaled 4-bit floats: the format, and its instructions.
//
// A packed operand is rows of C values cut into blocks of 32 (the last may be short). A block has one
// power of two, 2^(s - 127), s its byte: with M the block's largest magnitude s - 127 =
// max(floor(log2 M) - 2, -127), -127 where M = 0. A value x is kept as the nearest of 0, 1/2, 1, 3/2, 2, 3,
// 4, 6 to |x| 2^(127 - s), ties to the even code, 6 past it, with x's sign in bit 3 of its code: off by at most
// 2^(s - 127) up to the cut at 6, by less than twice that past it. A block with an infinity
// or a NaN has s = 255 and codes 0, and reads back as NaN throughout; so does every product that it enters.
// These are the element and scale formats E2M1 and E8M0 of the OCP Microscaling Formats specification (MX, 1.0).
// Layout: codes [rows][16 nb], nb = ceil(C / 32), value 2 i of a block in the low half of its byte i, zero
// past C; then, from the next multiple of 256 bytes, s [rows][nb]; the whole rounded up to 256 bytes.
#pragma once

#include "block_ops.hpp"
#include "checkpoint.hpp"

namespace fno {

constexpr int kMx4Block = 32;
constexpr uint32_t kMx4Bad = 255;  // scale byte of a block with a non-finite value

struct Mx4Layout {
  long nb;       // blocks of a row
  size_t exps;   // where the scale bytes begin
  size_t bytes;
};
inline __host__ __device__ Mx4Layout mx4_layout(long rows, long C) {
  Mx4Layout l;
  l.nb = (C + kMx4Block - 1) / kMx4Block;
  const size_t codes = (size_t)rows * l.nb * 16, exps = (size_t)rows * l.nb;
  l.exps = (codes + 255) / 256 * 256;
  l.bytes = l.exps + (exps + 255) / 256 * 256;
  return l;
}

// a block's scale byte from the fp32 bits of its largest magnitude (NaN bits are past infinity's)
__device__ __forceinline__ uint32_t mx4_scale(uint32_t bits) {
  const int E = (int)(bits >> 23);  // M = f 2^(E - 127), 1 <= f < 2; 0 below the normal numbers
  return E == 255 ? kMx4Bad : (uint32_t)max(E - 2, 0);
}
// the operand by which the conversions divide and multiply: its exponent field is the scale byte
__device__ __forceinline__ float mx4_factor(uint32_t s) { return __uint_as_float(s << 23); }

}  // namespace fno
