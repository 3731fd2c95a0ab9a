// checkpoint.hip - packing a field into the 8-bit checkpoint format and
// unpacking it (the format: checkpoint.hpp).
//
// Both are streams: a lane owns 8 consecutive values of a row (one or two
// 16-byte accesses on the field's side, 8 bytes of codes), 4 lanes a block;
// the block's largest magnitude goes round the 4 lanes with two DPP moves.
// Bound by memory: the field plus 1 1/32 bytes a value, each moved once (84 M bf16
// values: pack 50 us, unpack 38 us, 5.1 and 6.7 TB/s).

#include <algorithm>

#include "checkpoint.hpp"

namespace fno {

namespace {
constexpr int kCkThreads = 256;
constexpr int kCkRuns = 4;  // runs of 256 units a workgroup handles
constexpr long kCkRow = 1L << 22;  // workgroups in the grid's first dimension, which takes fewer than 2^32 threads
}  // namespace

// (row, unit in row) of unit base + local, base's row and remainder known
__device__ __forceinline__ void ck_place(long row0, uint32_t rem0, uint32_t upr, uint32_t local, long &row,
                                         uint32_t &u) {
  const uint32_t v = rem0 + local;  // < upr + kCkThreads * kCkRuns
  const uint32_t d = upr > kCkThreads * kCkRuns ? (v >= upr ? 1u : 0u) : v / upr;
  row = row0 + d;
  u = v - d * upr;
}

template <int DT, bool PACK>
__global__ __launch_bounds__(kCkThreads) void fno_checkpoint(CkArgs a) {
  const uint32_t upr = (uint32_t)(4 * a.nb);  // units per row
  const long base = ((long)blockIdx.y * kCkRow + blockIdx.x) * (kCkThreads * kCkRuns), total = a.rows * (long)upr;
  const long row0 = base / upr;
  const uint32_t rem0 = (uint32_t)(base - row0 * upr);
#pragma unroll
  for (int k = 0; k < kCkRuns; ++k) {
    const uint32_t local = k * kCkThreads + threadIdx.x;
    if (base + local >= total) return;  // rows are whole groups of 4 lanes: a block's lanes stay together
    long row;
    uint32_t u;
    ck_place(row0, rem0, upr, local, row, u);
    const long p = 8L * u, n = a.n - p;  // n <= 0: past the row's end (block padding)
    const size_t at = (size_t)row * a.n + p;
    uint2 *cd = reinterpret_cast<uint2 *>(a.codes + (size_t)row * a.nb * kCkBlock + p);
    int8_t *ex = a.exps + (size_t)row * a.nb + (u >> 2);
    if constexpr (PACK) {
      const ck_u32x4 r0 = ck_load<DT>(a.x, at, n);
      uint32_t key = ck_maxkey<DT>(r0);
      uint2 q;
      if constexpr (DT == DT_F32) {
        const ck_u32x4 r1 = ck_load<DT>(a.x, at + 4, n - 4);
        key = ck_groupmax<4>(max(key, ck_maxkey<DT>(r1)));
        const int e = ck_exponent<DT>(key);
        q.x = ck_codes<DT>(r0, e).x;
        q.y = ck_codes<DT>(r1, e).x;
        if ((u & 3) == 0) *ex = (int8_t)e;
      } else {
        key = ck_groupmax<4>(key);
        const int e = ck_exponent<DT>(key);
        q = ck_codes<DT>(r0, e);
        if ((u & 3) == 0) *ex = (int8_t)e;
      }
      *cd = q;
    } else {
      const uint2 q = *cd;
      const int e = *ex;
      if constexpr (DT == DT_F32) {
        ck_store<DT>(a.y, at, n, ck_decode<DT>(make_uint2(q.x, 0), e));
        ck_store<DT>(a.y, at + 4, n - 4, ck_decode<DT>(make_uint2(q.y, 0), e));
      } else {
        ck_store<DT>(a.y, at, n, ck_decode<DT>(q, e));
      }
    }
  }
}

hipError_t launch_checkpoint(const CkArgs &a, bool pack, int dtype, hipStream_t s) {
  FNO_BOUNDS(check_checkpoint(a, pack, dtype);)
  const long total = a.rows * 4 * a.nb, per = kCkThreads * kCkRuns;
  const long groups = (total + per - 1) / per;
  const dim3 grid((unsigned)std::min(groups, kCkRow), (unsigned)((groups + kCkRow - 1) / kCkRow));
  CkArgs arg = a;
  void *args[] = {(void *)&arg};
  const void *k;
  if (pack)
    k = dtype == DT_F32 ? (const void *)fno_checkpoint<DT_F32, true>
        : dtype == DT_F16 ? (const void *)fno_checkpoint<DT_F16, true>
                          : (const void *)fno_checkpoint<DT_BF16, true>;
  else
    k = dtype == DT_F32 ? (const void *)fno_checkpoint<DT_F32, false>
        : dtype == DT_F16 ? (const void *)fno_checkpoint<DT_F16, false>
                          : (const void *)fno_checkpoint<DT_BF16, false>;
  return hipLaunchKernel(k, grid, dim3(kCkThreads), args, 0, s);
}

}  // namespace fno
