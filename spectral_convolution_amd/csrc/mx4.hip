// mx4.hip - packing fields and tokens into 4-bit floats, and unpacking them (the format: mx4.hpp).
//
// Blocks run along the channels, the axis that a channel mix sums over. Tokens have it contiguous: a lane
// has 8 values, 4 lanes a block, as in checkpoint.hip. A field [B][C][P] is transposed on the
// way, to rows of one pixel: a lane takes 8 bytes of pixels (4 in 16 bits, 2 in fp32) of a block's 32
// channels into registers, so a block's maximum and its codes need no other lane, and loads cover 512
// bytes of a channel. The hardware conversions round to the nearest even code (checked over all
// scales, v_cvt_scalef32_pk_fp4_{f32,f16,bf16}). Bound by memory: 20 x 64 x 256^2 fp16 to 4 bits in 41 us and back in
// 37, 212 MB each.

#include <algorithm>

#include "mx4.hpp"

namespace fno {

namespace {
constexpr int kMx4Threads = 256;
constexpr int kMx4Runs = 4;         // token units a lane handles
constexpr long kMx4Row = 1L << 22;  // workgroups in the grid's first dimension, which takes fewer than 2^32 threads
typedef unsigned u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
}  // namespace

// the codes of two storage values into byte SEL of `old`; pair: both in a dword (16 bits), or fp32 a, b
template <int DT, int SEL>
__device__ __forceinline__ uint32_t mx4_pair(uint32_t old, uint32_t pair, float f) {
  if constexpr (DT == DT_F16) return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(half2_t, pair), f, SEL);
  else return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2_t, pair), f, SEL);
}
template <int SEL>
__device__ __forceinline__ uint32_t mx4_pair(uint32_t old, float a, float b, float f) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, f, SEL);
}

// ------------------------------------------------------------------- tokens

template <int DT, bool PACK>
__global__ __launch_bounds__(kMx4Threads) void fno_mx4_tokens(Mx4Args a) {
  constexpr int V = ck_vec<DT>();
  const long upr = 4 * a.nb, rows = (long)a.B * a.P, total = rows * upr;  // units of 8 values
  const long base = ((long)blockIdx.y * kMx4Row + blockIdx.x) * (kMx4Threads * kMx4Runs);
  const long row0 = base / upr, rem0 = base - row0 * upr;
#pragma unroll
  for (int k = 0; k < kMx4Runs; ++k) {
    const long local = k * kMx4Threads + threadIdx.x;
    if (base + local >= total) return;  // rows are whole groups of 4 lanes: a block's lanes stay together
    const uint32_t v = (uint32_t)(rem0 + local);
    const uint32_t d = v / (uint32_t)upr, u = v - d * (uint32_t)upr;
    const long row = row0 + d, n = (long)a.C - 8L * u;
    const size_t at = (size_t)row * a.C + 8L * u, block = (size_t)row * a.nb + (u >> 2);
    uint32_t *code = reinterpret_cast<uint32_t *>(a.codes + block * 16) + (u & 3);
    if constexpr (PACK) {
      const ck_u32x4 r0 = ck_load<DT>(a.x, at, n);
      ck_u32x4 r1{0u, 0u, 0u, 0u};
      uint32_t key = ck_maxkey<DT>(r0), q = 0;
      if constexpr (DT == DT_F32) {
        r1 = ck_load<DT>(a.x, at + V, n - V);
        key = max(key, ck_maxkey<DT>(r1));
      }
      key = ck_groupmax<4>(key);
      uint32_t bits = key;
      if constexpr (DT == DT_F16) bits = __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)key));
      if constexpr (DT == DT_BF16) bits = key << 16;
      const uint32_t s = mx4_scale(bits);
      const float f = mx4_factor(s);
      if constexpr (DT == DT_F32) {
        q = mx4_pair<0>(q, ck_get<DT>(r0, 0), ck_get<DT>(r0, 1), f);
        q = mx4_pair<1>(q, ck_get<DT>(r0, 2), ck_get<DT>(r0, 3), f);
        q = mx4_pair<2>(q, ck_get<DT>(r1, 0), ck_get<DT>(r1, 1), f);
        q = mx4_pair<3>(q, ck_get<DT>(r1, 2), ck_get<DT>(r1, 3), f);
      } else {
        q = mx4_pair<DT, 0>(q, r0[0], f);
        q = mx4_pair<DT, 1>(q, r0[1], f);
        q = mx4_pair<DT, 2>(q, r0[2], f);
        q = mx4_pair<DT, 3>(q, r0[3], f);
      }
      *code = s == kMx4Bad ? 0u : q;
      if ((u & 3) == 0) a.exps[block] = (uint8_t)s;
    } else {
      const uint32_t q = *code, s = a.exps[block];
      const float f = mx4_factor(s), bad = __uint_as_float(0x7fc00000u);
      float o[8];
      const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, f, 1),
                  p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, f, 3);
      o[0] = p0.x, o[1] = p0.y, o[2] = p1.x, o[3] = p1.y, o[4] = p2.x, o[5] = p2.y, o[6] = p3.x, o[7] = p3.y;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = s == kMx4Bad ? bad : o[e];
      ck_store<DT>(a.y, at, n, ck_raw<DT>(o));
      if constexpr (DT == DT_F32) ck_store<DT>(a.y, at + V, n - V, ck_raw<DT>(o + V));
    }
  }
}

// ------------------------------------------------------------------- fields

// A lane has NP pixels of a sample: chunk q of them is chunk q % ppr of sample q / ppr. Packing, two blocks of a
// workgroup's pixels at a time go through LDS, so that neighbouring lanes store neighbouring 16 bytes: each
// storing its own pixels' took twice as long (20 x 64 x 256^2 fp16 79 us, so 41). Pixels of odd rows
// strung together over the samples, so that they go through LDS too, were no faster (16 x 64 x 61^2 bf16 14 us, so 13).
template <int DT, bool PACK>
__global__ __launch_bounds__(kMx4Threads) void fno_mx4_field(Mx4Args a) {
  constexpr int NP = DT == DT_F32 ? 2 : 4, PIX = NP * kMx4Threads, KB = 2;
  __shared__ ck_u32x4 stage[PACK ? PIX * KB : 1];
  __shared__ uint8_t scales[PACK ? PIX * KB : 1];
  const long ppr = (a.P + NP - 1) / NP, total = a.B * ppr;
  const long q0 = (long)blockIdx.x * kMx4Threads, q = q0 + threadIdx.x, qc = min(q, total - 1);
  if (!PACK && q >= total) return;
  const long b = qc / ppr, p = (qc - b * ppr) * NP;
  const int n = q < total ? (int)min((long)NP, a.P - p) : 0;
  using E = typename std::conditional<DT == DT_F32, uint32_t, uint16_t>::type;
  // unit u of the stage, so placed that lanes 8 units apart meet other banks
  auto at = [](int u) { return u ^ (u >> 3 & 7); };
  // Where all lanes have whole chunks of pixels the workgroup's rows follow each other, over samples' ends too.
  const bool whole = a.P % NP == 0 && q0 + kMx4Threads <= total;
  const int step = PACK ? a.step : 1;  // blocks at a time
  for (long kb0 = (long)blockIdx.y * step; kb0 < a.nb; kb0 += (long)gridDim.y * step) {
    if constexpr (PACK) {
      const int kn = (int)min((long)step, a.nb - kb0);
      for (int kk = 0; kk < kn; ++kk) {
        const long kb = kb0 + kk;
        const int c0 = (int)kb * kMx4Block, nc = min(kMx4Block, a.C - c0);
        const E *src = reinterpret_cast<const E *>(a.x) + ((size_t)b * a.C + c0) * a.P + p;
        u32x2 r[kMx4Block];
        if (n == NP) {
#pragma unroll
          for (int i = 0; i < kMx4Block; ++i)
            r[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x2_any *>(src + (size_t)min(i, nc - 1) * a.P));
        } else {
#pragma unroll
          for (int i = 0; i < kMx4Block; ++i) {
            const E *s = src + (size_t)min(i, nc - 1) * a.P;
            r[i] = u32x2{0u, 0u};
            if (n > 0) r[i][0] = s[0];
            if constexpr (DT != DT_F32) {
              if (n > 1) r[i][0] |= (uint32_t)s[1] << 16;
              if (n > 2) r[i][1] = s[2];
            }
          }
        }
        if (nc < kMx4Block)
#pragma unroll
          for (int i = 0; i < kMx4Block; ++i)
            if (i >= nc) r[i] = u32x2{0u, 0u};
        uint32_t key[NP];
        if constexpr (DT == DT_F32) {
          key[0] = key[1] = 0;
#pragma unroll
          for (int i = 0; i < kMx4Block; ++i)
#pragma unroll
            for (int j = 0; j < NP; ++j) key[j] = max(key[j], r[i][j] & 0x7fffffffu);
        } else {  // two pixels a word
          u16x2 m[2] = {u16x2{0, 0}, u16x2{0, 0}};
#pragma unroll
          for (int i = 0; i < kMx4Block; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              m[j] = __builtin_elementwise_max(m[j], __builtin_bit_cast(u16x2, r[i][j] & 0x7fff7fffu));
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            key[j] = m[j / 2][j & 1];
            if constexpr (DT == DT_F16) key[j] = __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)key[j]));
            else key[j] <<= 16;
          }
        }
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          ck_u32x4 code;
          const uint32_t s = mx4_scale(key[j]);
          const float f = mx4_factor(s);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t v = 0;
            if constexpr (DT == DT_F32) {
              auto val = [&](int i) { return __uint_as_float(r[8 * w + i][j]); };
              v = mx4_pair<0>(v, val(0), val(1), f);
              v = mx4_pair<1>(v, val(2), val(3), f);
              v = mx4_pair<2>(v, val(4), val(5), f);
              v = mx4_pair<3>(v, val(6), val(7), f);
            } else {  // the halves of two channels' dwords side by side
              auto val = [&](int i) {
                return __builtin_amdgcn_perm(r[8 * w + i + 1][j / 2], r[8 * w + i][j / 2], j & 1 ? 0x07060302u : 0x05040100u);
              };
              v = mx4_pair<DT, 0>(v, val(0), f);
              v = mx4_pair<DT, 1>(v, val(2), f);
              v = mx4_pair<DT, 2>(v, val(4), f);
              v = mx4_pair<DT, 3>(v, val(6), f);
            }
            code[w] = s == kMx4Bad ? 0u : v;
          }
          if (whole) {
            const int u = (threadIdx.x * NP + j) * kn + kk;
            stage[at(u)] = code;
            scales[u] = (uint8_t)s;
          } else if (j < n) {
            const size_t block = ((size_t)b * a.P + p + j) * a.nb + kb;
            *reinterpret_cast<ck_u32x4 *>(a.codes + block * 16) = code;
            a.exps[block] = (uint8_t)s;
          }
        }
      }
      if (whole) {
        __syncthreads();
        const size_t first = (size_t)q0 * NP;
        for (int u = threadIdx.x; u < PIX * kn; u += kMx4Threads) {
          const int px = kn == KB ? u / KB : u, kk = u - px * kn;
          *reinterpret_cast<ck_u32x4 *>(a.codes + ((first + px) * a.nb + kb0 + kk) * 16) = stage[at(u)];
          a.exps[(first + px) * a.nb + kb0 + kk] = scales[u];
        }
        __syncthreads();
      }
    } else {
      const long kb = kb0;
      const int c0 = (int)kb * kMx4Block, nc = min(kMx4Block, a.C - c0);
      const size_t row = (size_t)b * a.P + p;
      ck_u32x4 code[NP];
      uint32_t s[NP];
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const size_t block = (row + min(j, n - 1)) * a.nb + kb;
        code[j] = *reinterpret_cast<const ck_u32x4 *>(a.codes + block * 16);
        s[j] = a.exps[block];
      }
      E *dst = reinterpret_cast<E *>(a.y) + ((size_t)b * a.C + c0) * a.P + p;
      // two channels of all pixels at a time
      auto pair = [&](auto sel, int w) {
        constexpr int SEL = decltype(sel)::value;
        float o0[NP], o1[NP];
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[j][w], mx4_factor(s[j]), SEL);
          const bool bad = s[j] == kMx4Bad;
          o0[j] = bad ? __uint_as_float(0x7fc00000u) : v.x;
          o1[j] = bad ? __uint_as_float(0x7fc00000u) : v.y;
        }
        const int i = 8 * w + 2 * SEL;
        auto put = [&](int c, const float *o) {
          if (c >= nc) return;
          u32x2 t;
          if constexpr (DT == DT_F32) t = u32x2{__float_as_uint(o[0]), __float_as_uint(o[1])};
          else t = u32x2{ck_pair<DT>(o[0], o[1]), ck_pair<DT>(o[2], o[3])};
          E *d = dst + (size_t)c * a.P;
          if (n == NP) {
            __builtin_nontemporal_store((u32x2_any)t, reinterpret_cast<u32x2_any *>(d));
          } else {
            d[0] = (E)t[0];
            if constexpr (DT != DT_F32) {
              if (n > 1) d[1] = (E)(t[0] >> 16);
              if (n > 2) d[2] = (E)t[1];
            }
          }
        };
        put(i, o0);
        put(i + 1, o1);
      };
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        pair(std::integral_constant<int, 0>{}, w);
        pair(std::integral_constant<int, 1>{}, w);
        pair(std::integral_constant<int, 2>{}, w);
        pair(std::integral_constant<int, 3>{}, w);
      }
    }
  }
}

hipError_t launch_mx4(const Mx4Args &a, bool pack, int dtype, hipStream_t s) {
  Mx4Args arg = a;
  void *args[] = {(void *)&arg};
  FNO_BOUNDS(check_mx4(a, pack, dtype);)
  const void *k;
  dim3 grid;
#define FNO_PICK(DT, K) (pack ? (const void *)K<DT, true> : (const void *)K<DT, false>)
  if (a.P == 1) {
    const long groups = (4 * a.nb * a.B + kMx4Threads * kMx4Runs - 1) / (kMx4Threads * kMx4Runs);
    grid = dim3((unsigned)std::min(groups, kMx4Row), (unsigned)((groups + kMx4Row - 1) / kMx4Row));
    k = dtype == DT_F32 ? FNO_PICK(DT_F32, fno_mx4_tokens)
        : dtype == DT_F16 ? FNO_PICK(DT_F16, fno_mx4_tokens) : FNO_PICK(DT_BF16, fno_mx4_tokens);
  } else {
    const long np = dtype == DT_F32 ? 2 : 4, groups = (a.B * ((a.P + np - 1) / np) + kMx4Threads - 1) / kMx4Threads;
    // a workgroup has all of its pixels' blocks, so that rows are written whole, unless the chip would stay empty;
    // two at a time where they go through LDS and there are enough (5 x 200 x 1001 fp32, which has neither: 4.5 us, not 8.6)
    arg.step = pack && a.P % np == 0 && groups * ((a.nb + 1) / 2) >= 512 ? 2 : 1;
    grid = dim3((unsigned)groups, (unsigned)std::min((a.nb + arg.step - 1) / arg.step, std::max(1L, 1024 / groups)));
    k = dtype == DT_F32 ? FNO_PICK(DT_F32, fno_mx4_field)
        : dtype == DT_F16 ? FNO_PICK(DT_F16, fno_mx4_field) : FNO_PICK(DT_BF16, fno_mx4_field);
  }
#undef FNO_PICK
  return hipLaunchKernel(k, grid, dim3(kMx4Threads), args, 0, s);
}

}  // namespace fno
