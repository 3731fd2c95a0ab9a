// drop.hip - dropout, alone or into a residual stream: y = x + D(v) (drop.hpp has D).
//
// A stream: a lane has 16 bytes of v (and of x) in hand, four such chunks in flight while it
// computes their random bits. 16-bit chunks of eight values are one block of the generator; two
// lanes with four fp32 values each compute the same block, which costs no time, since
// their values are twice the bytes. Dropped channels and samples are not read. Bound by memory: 32 x 64 x 256^2 fp16 into a
// residual in 123 us, 805 MB at 6.5 TB/s (two streams read, one written; a copy reaches 5.1).
// The backward is the same call: dL/dv = D(dL/dy), dL/dx = dL/dy.

#include <algorithm>

#include "checkpoint.hpp"
#include "drop.hpp"

namespace fno {

namespace {
constexpr int kDropThreads = 256;
constexpr int kDropRuns = 4;  // chunks a lane has at a time
constexpr int kDropSpan = kDropThreads * kDropRuns;
constexpr long kDropRow = 1L << 22;  // workgroups in the grid's first dimension, which takes fewer than 2^32 threads
enum : int { kFlat = 0, kRows = 1, kColumns = 2 };
}  // namespace

template <int DT>
__device__ __forceinline__ ck_u32x4 drop_apply(const ck_u32x4 &x, const ck_u32x4 &v, uint32_t keep, float scale) {
  constexpr int V = ck_vec<DT>();
  float o[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {  // a dropped value is 0 whatever it was: not multiplied
    const float f = ck_get<DT>(v, e) * scale;
    o[e] = ck_get<DT>(x, e) + (keep >> e & 1 ? f : 0.f);
  }
  return ck_raw<DT>(o);
}

// MODE kFlat: the field is one row and a value is a unit. kRows: a row is a unit (a channel
// of a field, a sample). kColumns: channels last, a row's values belong to units of their own, shared
// by the rows of a sample.
template <int DT, int MODE>
__global__ __launch_bounds__(kDropThreads) void fno_drop(DropArgs a) {
  constexpr int V = ck_vec<DT>();
  const long cpr = (a.n + V - 1) / V;  // chunks of a row
  const long base = ((long)blockIdx.y * kDropRow + blockIdx.x) * kDropSpan, total = a.rows * cpr;
  const long row0 = MODE == kFlat ? 0 : base / cpr, rem0 = base - row0 * cpr;
  const long b0 = MODE == kColumns ? row0 / a.P : 0;
  const uint32_t prem = (uint32_t)(row0 - b0 * a.P);
  const DropKey key = drop_key(a.drop);
  const uint32_t thr = a.drop.thr;
  const float scale = a.drop.scale;

  long row[kDropRuns], k[kDropRuns];
#pragma unroll
  for (int i = 0; i < kDropRuns; ++i) {
    const long v = rem0 + i * kDropThreads + threadIdx.x;
    long d = 0;
    if constexpr (MODE != kFlat) d = cpr > kDropSpan ? (v >= cpr ? 1 : 0) : (uint32_t)v / (uint32_t)cpr;
    row[i] = row0 + d;
    k[i] = v - d * cpr;
  }
  auto kept = [&](int i) -> uint32_t {
    if constexpr (MODE == kFlat) {
      const uint64_t u = (uint64_t)k[i] * V;
      return drop_block(key, thr, u >> 3) >> (u & 7);
    } else if constexpr (MODE == kRows) {
      return drop_one(key, thr, (uint64_t)row[i]);
    } else {
      const long b = b0 + (prem + (uint32_t)(row[i] - row0)) / (uint32_t)a.P;
      return drop_units(key, thr, (uint64_t)b * a.C + k[i] * V, V);
    }
  };
  const ck_u32x4 none{0u, 0u, 0u, 0u};
  const ck_u32x4 *xs = reinterpret_cast<const ck_u32x4 *>(a.x), *vs = reinterpret_cast<const ck_u32x4 *>(a.v);
  ck_u32x4 *ys = reinterpret_cast<ck_u32x4 *>(a.y);
  // whole chunks only: their places are those of a flat field
  const bool whole = (MODE == kFlat ? (base + kDropSpan) * V <= a.n : base + kDropSpan <= total && a.n % V == 0);
  if (whole) {
    const long at = base + threadIdx.x;
    ck_u32x4 x[kDropRuns], v[kDropRuns];
    uint32_t m[kDropRuns];
    if constexpr (MODE == kRows)
#pragma unroll
      for (int i = 0; i < kDropRuns; ++i) m[i] = kept(i);
#pragma unroll
    for (int i = 0; i < kDropRuns; ++i) {
      v[i] = none;
      if (MODE != kRows || m[i]) v[i] = __builtin_nontemporal_load(vs + at + i * kDropThreads);
    }
    if (a.x) {
#pragma unroll
      for (int i = 0; i < kDropRuns; ++i) x[i] = __builtin_nontemporal_load(xs + at + i * kDropThreads);
    } else {
#pragma unroll
      for (int i = 0; i < kDropRuns; ++i) x[i] = none;
    }
#pragma unroll
    for (int i = 0; i < kDropRuns; ++i) {
      if constexpr (MODE != kRows) m[i] = kept(i);
      __builtin_nontemporal_store(drop_apply<DT>(x[i], v[i], m[i], scale), ys + at + i * kDropThreads);
    }
    return;
  }
  // Rows that end inside a chunk: 16 bytes all the same, which end inside the field except in the last workgroups.
  const long tail = rem0 + kDropSpan - 1, down = tail / cpr;  // the workgroup's last chunk
  if (base + kDropSpan <= total && (row0 + down) * a.n + (tail - down * cpr + 1) * V <= a.rows * a.n) {
    ck_u32x4 x[kDropRuns], v[kDropRuns];
    size_t at[kDropRuns];
#pragma unroll
    for (int i = 0; i < kDropRuns; ++i) {
      at[i] = (size_t)row[i] * a.n + k[i] * V;
      v[i] = ck_load<DT>(a.v, at[i], V);
    }
#pragma unroll
    for (int i = 0; i < kDropRuns; ++i) x[i] = a.x ? ck_load<DT>(a.x, at[i], V) : none;
#pragma unroll
    for (int i = 0; i < kDropRuns; ++i)
      ck_store_row<DT>(a.y, at[i], a.n - k[i] * V, drop_apply<DT>(x[i], v[i], kept(i), scale));
    return;
  }
#pragma unroll 1
  for (int i = 0; i < kDropRuns; ++i) {
    if (base + i * kDropThreads + threadIdx.x >= total) return;
    const long n = a.n - k[i] * V;
    const size_t at = (size_t)row[i] * a.n + k[i] * V;
    const uint32_t m = kept(i);
    const ck_u32x4 v = m ? ck_load<DT>(a.v, at, n) : none;
    const ck_u32x4 x = a.x ? ck_load<DT>(a.x, at, n) : none;
    ck_store<DT>(a.y, at, n, drop_apply<DT>(x, v, m, scale));
  }
}

hipError_t launch_drop(const DropArgs &a, int dtype, hipStream_t s) {
  DropArgs arg = a;
  int mode = kFlat;
  // one pixel: a channel of a sample is a value
  if (a.drop.unit == kDropElement || (a.drop.unit == kDropChannel && a.P == 1)) {
    arg.rows = 1, arg.n = (long)a.B * a.C * a.P;
  } else if (a.drop.unit == kDropSample) {
    arg.rows = a.B, arg.n = a.C * a.P;
    mode = kRows;
  } else if (a.last) {
    arg.rows = a.B * a.P, arg.n = a.C;
    mode = kColumns;
  } else {
    arg.rows = (long)a.B * a.C, arg.n = a.P;
    mode = kRows;
  }
  const int V = dtype == DT_F32 ? 4 : 8;
  FNO_BOUNDS(check_drop(arg, mode, dtype);)
  const long total = arg.rows * ((arg.n + V - 1) / V), groups = (total + kDropSpan - 1) / kDropSpan;
  const dim3 grid((unsigned)std::min(groups, kDropRow), (unsigned)((groups + kDropRow - 1) / kDropRow));
#define FNO_PICK(DT) \
  (mode == kFlat ? (const void *)fno_drop<DT, kFlat> \
                 : mode == kRows ? (const void *)fno_drop<DT, kRows> : (const void *)fno_drop<DT, kColumns>)
  const void *k = dtype == DT_F32 ? FNO_PICK(DT_F32) : dtype == DT_F16 ? FNO_PICK(DT_F16) : FNO_PICK(DT_BF16);
#undef FNO_PICK
  void *args[] = {(void *)&arg};
  return hipLaunchKernel(k, grid, dim3(kDropThreads), args, 0, s);
}

}  // namespace fno
