// checkpoint.hpp - the 8-bit checkpoint format of a field, and the device
// helpers that quantise into it and read it back.
//
// A field is seen as rows of n contiguous values, each row as blocks of 32
// (the last one may be short). With M the largest magnitude of a block, its
// exponent is e = max(floor(log2 M) - 6, low) (low for M = 0) and a value is
// kept as q = rint(x 2^-e), clamped to [-127, 127]: M 2^-e < 128 (and 64 or more but where e is
// low), so a value is off by at most half of 2^e, and by 2^e where the clamp acts. low
// is -24 for fp16 (every value is a multiple of 2^-24, so tiny blocks are
// kept exactly) and -126 for fp32 / bf16 (2^e and 2^-e stay normal numbers).
// A block that holds an infinity or a NaN has e = 127, which reads back as
// NaN throughout: a poisoned block cannot pass for a finite one.
// q 2^e has at most 7 significant bits and e >= low, so what is read back is
// exact in all three storage types.
//
// Codes are int8 [rows][32 nb], nb = ceil(n / 32), zeros past n; exponents
// int8 [rows][nb]; each part starts on a multiple of 256 bytes.
#pragma once

#include "train.hpp"

namespace fno {

constexpr int kCkBlock = 32;
constexpr int kCkBad = 127;  // exponent of a block with a non-finite value

typedef unsigned ck_u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at any element's address: rows of odd length start off the 16-byte
// grid, and gfx950's global accesses need no alignment beyond the dword's
// halves (measured: the kernels below reach the same rate on odd rows)
typedef unsigned ck_u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned short ck_u16x2 __attribute__((ext_vector_type(2)));

template <int DT>
constexpr int ck_low() { return DT == DT_F16 ? -24 : -126; }

// storage elements in 16 bytes
template <int DT>
constexpr int ck_vec() { return DT == DT_F32 ? 4 : 8; }

// element e of 16 raw bytes as fp32
template <int DT>
__device__ __forceinline__ float ck_get(const ck_u32x4 &r, int e) {
  if constexpr (DT == DT_F32) return __uint_as_float(r[e]);
  const uint32_t h = (e & 1) ? r[e >> 1] >> 16 : r[e >> 1] & 0xffffu;
  if constexpr (DT == DT_F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
  return (e & 1) ? __uint_as_float(r[e >> 1] & 0xffff0000u) : __uint_as_float(r[e >> 1] << 16);
}

// two fp32 into the halves of a dword (fp16 / bf16, round to nearest even)
template <int DT>
__device__ __forceinline__ uint32_t ck_pair(float lo, float hi) {
  if constexpr (DT == DT_F16) {
    half2_t h;
    h.x = (_Float16)lo;
    h.y = (_Float16)hi;
    return __builtin_bit_cast(uint32_t, h);
  } else {
    return f32x2_to_bf16x2(lo, hi);
  }
}

// fp32 values -> 16 raw storage bytes
template <int DT>
__device__ __forceinline__ ck_u32x4 ck_raw(const float *v) {
  ck_u32x4 r;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == DT_F32) r[k] = __float_as_uint(v[k]);
    else r[k] = ck_pair<DT>(v[2 * k], v[2 * k + 1]);
  }
  return r;
}

// n of the 16 bytes' elements at p[i] (n <= 0: none), zeros for the others
template <int DT>
__device__ __forceinline__ ck_u32x4 ck_load(const void *p, size_t i, long n) {
  if constexpr (DT == DT_F32) {
    const float *s = reinterpret_cast<const float *>(p) + i;
    if (n >= 4) return *reinterpret_cast<const ck_u32x4_any *>(s);
    ck_u32x4 r{0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) r[e] = __float_as_uint(s[e]);
    return r;
  } else {
    const uint16_t *s = reinterpret_cast<const uint16_t *>(p) + i;
    if (n >= 8) return *reinterpret_cast<const ck_u32x4_any *>(s);
    // a row's tail: one element at a time through a 128-bit shift, small code
    // where every access of a kernel has such a path
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int e = (int)n - 1; e >= 0; --e) {
      hi = hi << 16 | lo >> 48;
      lo = lo << 16 | s[e];
    }
    return ck_u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  }
}

template <int DT>
__device__ __forceinline__ void ck_store(void *p, size_t i, long n, const ck_u32x4 &r) {
  if constexpr (DT == DT_F32) {
    float *d = reinterpret_cast<float *>(p) + i;
    if (n >= 4) {
      *reinterpret_cast<ck_u32x4_any *>(d) = r;
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) d[e] = __uint_as_float(r[e]);
    }
  } else {
    uint16_t *d = reinterpret_cast<uint16_t *>(p) + i;
    if (n >= 8) {
      *reinterpret_cast<ck_u32x4_any *>(d) = r;
    } else {
      uint64_t lo = (uint64_t)r[1] << 32 | r[0], hi = (uint64_t)r[3] << 32 | r[2];
#pragma unroll 1
      for (int e = 0; e < (int)n; ++e) {
        d[e] = (uint16_t)lo;
        lo = lo >> 16 | hi << 48;
        hi >>= 16;
      }
    }
  }
}

// 128 bits moved down by whole bytes, zeros from above (16 or more: all)
__device__ __forceinline__ ck_u32x4 ck_shift(const ck_u32x4 &r, int bytes) {
  uint64_t lo = (uint64_t)r[1] << 32 | r[0], hi = (uint64_t)r[3] << 32 | r[2];
  const bool far = bytes >= 8;
  const int s = 8 * (bytes & 7);
  lo = far ? hi : lo;
  hi = far ? 0 : hi;
  lo = lo >> s | (s ? hi << (64 - s) : 0);
  hi >>= s;
  if (bytes >= 16) lo = hi = 0;
  return ck_u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// the first n of the elements to p[i] .. (n <= 0: none)
template <int DT>
__device__ __forceinline__ void ck_store_row(void *p, size_t i, long n, const ck_u32x4 &r) {
  typedef unsigned u32_any __attribute__((aligned(2)));
  typedef unsigned u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
  constexpr int V = ck_vec<DT>(), ES = DT == DT_F32 ? 4 : 2;
  char *d = static_cast<char *>(p) + i * ES;
  if (n >= V) {
    *reinterpret_cast<ck_u32x4_any *>(d) = r;
  } else if (n > 0) {
    const int bytes = (int)n * ES;
    uint32_t a = r[0], b = r[1];
    if (bytes & 8) {
      *reinterpret_cast<u32x2_any *>(d) = u32x2_any{a, b};
      d += 8;
      a = r[2];
      b = r[3];
    }
    if (bytes & 4) {
      *reinterpret_cast<u32_any *>(d) = a;
      d += 4;
      a = b;
    }
    if (ES == 2 && (bytes & 2)) *reinterpret_cast<uint16_t *>(d) = (uint16_t)a;
  }
}

// ---- quantising

// The largest magnitude of 16 raw bytes' elements as a key that orders like
// the magnitudes (NaN above infinity above all finite): the storage bits
// without the sign. Fields of 16 bits are compared two at a time.
template <int DT>
__device__ __forceinline__ uint32_t ck_maxkey(const ck_u32x4 &r) {
  if constexpr (DT == DT_F32) {
    return max(max(r[0] & 0x7fffffffu, r[1] & 0x7fffffffu), max(r[2] & 0x7fffffffu, r[3] & 0x7fffffffu));
  } else {
    ck_u16x2 m = __builtin_bit_cast(ck_u16x2, r[0] & 0x7fff7fffu);
#pragma unroll
    for (int k = 1; k < 4; ++k)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(ck_u16x2, r[k] & 0x7fff7fffu));
    return max((uint32_t)m.x, (uint32_t)m.y);
  }
}

template <int CTRL>
__device__ __forceinline__ uint32_t ck_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
constexpr int kDppXor1 = 0xb1, kDppXor2 = 0x4e, kDppHalfMirror = 0x141, kDppRor8 = 0x128;

// max over aligned groups of 4 (N = 4) or 8 lanes
template <int N>
__device__ __forceinline__ uint32_t ck_groupmax(uint32_t m) {
  m = max(m, ck_dpp<kDppXor1>(m));
  m = max(m, ck_dpp<kDppXor2>(m));
  if constexpr (N == 8) m = max(m, ck_dpp<kDppHalfMirror>(m));
  return m;
}

// a block's exponent from its key
template <int DT>
__device__ __forceinline__ int ck_exponent(uint32_t key) {
  uint32_t b;
  if constexpr (DT == DT_F32) b = key;
  else if constexpr (DT == DT_F16) b = __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)key));
  else b = key << 16;
  // M = f 2^(E - 127), 1 <= f < 2: e = E - 133
  const int E = (int)(b >> 23);
  return E == 255 ? kCkBad : max(E - 133, ck_low<DT>());
}

// four values -> four codes, first value in the low byte. inv = 2^-e; the
// addition of 1.5 2^23 rounds to nearest even and leaves the integer in the
// low bits.
__device__ __forceinline__ uint32_t ck_codes4(float a, float b, float c, float d, float inv) {
  const float g = 12582912.f;
  const uint32_t ua = __float_as_uint(__builtin_amdgcn_fmed3f(a * inv, -127.f, 127.f) + g);
  const uint32_t ub = __float_as_uint(__builtin_amdgcn_fmed3f(b * inv, -127.f, 127.f) + g);
  const uint32_t uc = __float_as_uint(__builtin_amdgcn_fmed3f(c * inv, -127.f, 127.f) + g);
  const uint32_t ud = __float_as_uint(__builtin_amdgcn_fmed3f(d * inv, -127.f, 127.f) + g);
  const uint32_t lo = __builtin_amdgcn_perm(ub, ua, 0x0c0c0400u), hi = __builtin_amdgcn_perm(ud, uc, 0x04000c0cu);
  return lo | hi;
}

__device__ __forceinline__ float ck_inv(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

// codes of the elements of 16 raw bytes: 4 (fp32) or 8 bytes
template <int DT>
__device__ __forceinline__ uint2 ck_codes(const ck_u32x4 &r, int e) {
  const float inv = ck_inv(e);
  const uint32_t keep = e == kCkBad ? 0u : ~0u;
  uint2 q;
  q.x = keep & ck_codes4(ck_get<DT>(r, 0), ck_get<DT>(r, 1), ck_get<DT>(r, 2), ck_get<DT>(r, 3), inv);
  q.y = 0;
  if constexpr (DT != DT_F32)
    q.y = keep & ck_codes4(ck_get<DT>(r, 4), ck_get<DT>(r, 5), ck_get<DT>(r, 6), ck_get<DT>(r, 7), inv);
  return q;
}

// ---- reading back

// 2^e, NaN for the exponent of a poisoned block
__device__ __forceinline__ float ck_step(int e) {
  return e == kCkBad ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 + e) << 23);
}

__device__ __forceinline__ float ck_value(uint32_t q4, int k, float step) {
  return (float)(int8_t)(q4 >> (8 * k)) * step;
}

// 4 (fp32) or 8 codes -> 16 raw storage bytes (exact)
template <int DT>
__device__ __forceinline__ ck_u32x4 ck_decode(uint2 q, int e) {
  const float s = ck_step(e);
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = ck_value(q.x, k, s);
    v[4 + k] = DT == DT_F32 ? 0.f : ck_value(q.y, k, s);
  }
  return ck_raw<DT>(v);
}

// where the parts of a checkpoint of rows x n lie
struct CkLayout {
  long nb;         // blocks per row
  size_t exps;     // byte offset of the exponents
  size_t bytes;    // whole checkpoint
};
inline __host__ __device__ CkLayout ck_layout(long rows, long n) {
  CkLayout l;
  l.nb = (n + kCkBlock - 1) / kCkBlock;
  l.exps = ((size_t)rows * l.nb * kCkBlock + 255) / 256 * 256;
  l.bytes = l.exps + ((size_t)rows * l.nb + 255) / 256 * 256;
  return l;
}

}  // namespace fno
