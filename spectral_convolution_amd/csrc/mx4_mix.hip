// mx4_mix.hip - the channel mix of two operands in 4-bit floats (mx4.hpp),
//   y[b][o][p] = act(sum_i A[o][i] x[b][i][p] + bias[o] + add[b][o][p]),
// on the scaled matrix instructions v_mfma_scale_f32_16x16x128_f8f6f4, which take the blocks' powers of two with
// the codes: lane l has row l % 16 and block l / 16 of four, 16 bytes of codes and one scale byte of either operand.
// Products of codes are exact, sums are fp32 (a product of 128 off by up to 4e-8 of its terms' sizes, measured).
// 8192 x 4096 x 4096 bf16 with GELU: 96 us, 2.9 PFLOP/s; the instruction alone runs at 6.6 on random codes, at 8 to 9 on
// constant ones. On zeros it takes 71 to 79 us, again less than half of the instruction's rate, so power is not what bounds it: a step of
// 64 of a 256^2 tile's sum reads 48 KB of LDS and fills 16, 512 clocks at 128 bytes, as long as its matrix instructions
// take, and the tile's GELU runs behind the last of them. One token, 8192 x 8192: 10 us
// for 36 MB. 32 x 64 x 64 x 256^2 fp16, GELU and addition: 203 us, 3 TB/s, bound by GELU behind one step of products.
//
// The rows that are neighbours in y are the instruction's first operand (pixels of a field, output
// channels of tokens): a lane then has four neighbouring results.

#include <algorithm>

#include "gelu.hpp"
#include "mx4.hpp"
#include "norm_common.hpp"

namespace fno {

namespace {

constexpr int kThreads = 256;
constexpr long kMaxGrid = 1L << 22;

typedef int v8i __attribute__((ext_vector_type(8)));

// first operand f, second operand s: y[b][s][f] with strides ybatch, ys, 1
struct Gemm {
  const uint8_t *fq, *fe, *sq, *se;
  const void *bias, *add;
  void *y;
  long nf, ns, nb, batches;
  long ybatch, ys;
  int act;
  int bias_f;  // bias belongs to f (tokens), else to s
};

__device__ __forceinline__ v4f mx4_product(const ck_u32x4 &a, uint32_t sa, const ck_u32x4 &b, uint32_t sb, const v4f &c) {
  const v8i x{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0}, y{(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

template <int DT>
__device__ __forceinline__ float value_at(const void *p, size_t i) {
  if constexpr (DT == DT_F32) return reinterpret_cast<const float *>(p)[i];
  else if constexpr (DT == DT_F16) return (float)reinterpret_cast<const _Float16 *>(p)[i];
  else return bf16_to_f32(reinterpret_cast<const uint16_t *>(p)[i]);
}

template <int DT>
__device__ __forceinline__ float bias_at(const Gemm &g, long i, long n) {
  return g.bias ? value_at<DT>(g.bias, (size_t)min(i, n - 1)) : 0.f;
}

// neighbouring sums o of row s at y[at] .., n of them there: bias (bf: of their f), addition, activation
template <int DT, int N>
__device__ __forceinline__ void mx4_finish(const Gemm &g, float (&o)[N], const float *bf, long s, size_t at, int n) {
  static_assert(N == ck_vec<DT>(), "16 bytes");
  const float bs = g.bias_f ? 0.f : bias_at<DT>(g, s, g.ns);
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] += bf[e] + bs;
  if (g.add) {
    const ck_u32x4 d = ck_load<DT>(g.add, at, n);
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] += ck_get<DT>(d, e);
  }
  if (g.act)
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = gelu_train(o[e]);
  ck_store_row<DT>(g.y, at, n, ck_raw<DT>(o));
}

}  // namespace

// Short sums: a wave has 16 F f x 16 S s, four waves side by side along f; operands straight from memory to
// registers, the next step's loaded before this one's products.
template <int DT, int F, int S>
__global__ __launch_bounds__(kThreads, 3) void fno_mx4_mix(Gemm g) {
  __shared__ __attribute__((aligned(16))) float stage[4][16 * (16 * F + 4)];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, quad = lane >> 4;
  const long ft = (g.nf + 64 * F - 1) / (64 * F), st = (g.ns + 16 * S - 1) / (16 * S), tiles = ft * st * g.batches, steps = (g.nb + 3) / 4;
  for (long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const long si = t % st, fb = t / st, b = fb / ft, f0 = (fb - b * ft) * (64 * F) + wave * (16 * F), s0 = si * (16 * S);
    if (f0 >= g.nf) continue;
    size_t fr[F], sr[S];
#pragma unroll
    for (int i = 0; i < F; ++i) fr[i] = (size_t)(b * g.nf + min(f0 + 16 * i + l16, g.nf - 1)) * g.nb;
#pragma unroll
    for (int j = 0; j < S; ++j) sr[j] = (size_t)min(s0 + 16 * j + l16, g.ns - 1) * g.nb;
    v4f acc[F][S];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < S; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    ck_u32x4 fc[F], sc[S];
    uint32_t fx[F], sx[S];
    auto load = [&](long k) {
      const long kb = 4 * k + quad, kc = min(kb, g.nb - 1);
#pragma unroll
      for (int i = 0; i < F; ++i) {
        fc[i] = *reinterpret_cast<const ck_u32x4 *>(g.fq + (fr[i] + kc) * 16);
        fx[i] = g.fe[fr[i] + kc];
      }
#pragma unroll
      for (int j = 0; j < S; ++j) {
        sc[j] = *reinterpret_cast<const ck_u32x4 *>(g.sq + (sr[j] + kc) * 16);
        sx[j] = g.se[sr[j] + kc];
      }
      if (kb >= g.nb) {  // no such block: codes of 0, a scale that makes 0 of them
#pragma unroll
        for (int i = 0; i < F; ++i) fc[i] = ck_u32x4{0u, 0u, 0u, 0u}, fx[i] = 127;
#pragma unroll
        for (int j = 0; j < S; ++j) sc[j] = ck_u32x4{0u, 0u, 0u, 0u}, sx[j] = 127;
      }
    };
    load(0);
    for (long k = 0; k < steps; ++k) {
      ck_u32x4 fn[F], sn[S];
      uint32_t fxn[F], sxn[S];
#pragma unroll
      for (int i = 0; i < F; ++i) fn[i] = fc[i], fxn[i] = fx[i];
#pragma unroll
      for (int j = 0; j < S; ++j) sn[j] = sc[j], sxn[j] = sx[j];
      if (k + 1 < steps) load(k + 1);
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < S; ++j) acc[i][j] = mx4_product(fn[i], fxn[i], sn[j], sxn[j], acc[i][j]);
    }
    // 16 columns at a time through LDS, so that lanes finish and store whole 16 bytes of neighbours
    constexpr int N = ck_vec<DT>(), FW = 16 * F, PITCH = FW + 4, LANES = FW / N;
    const long fl = f0 + lane % LANES * N;
    const int there = (int)max(0L, min((long)N, g.nf - fl));
    float bf[N];
#pragma unroll
    for (int e = 0; e < N; ++e) bf[e] = g.bias_f && there > 0 ? bias_at<DT>(g, fl + e, g.nf) : 0.f;
    float *part = stage[wave];
#pragma unroll
    for (int j = 0; j < S; ++j) {
#pragma unroll
      for (int i = 0; i < F; ++i) *reinterpret_cast<v4f *>(part + l16 * PITCH + 16 * i + 4 * quad) = acc[i][j];
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int c = lane / LANES; c < 16; c += 64 / LANES) {
        const long s = s0 + 16 * j + c;
        if (s >= g.ns || there == 0) continue;
        float o[N];
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          const v4f v = *reinterpret_cast<const v4f *>(part + c * PITCH + lane % LANES * N + e);
#pragma unroll
          for (int r = 0; r < 4; ++r) o[e + r] = v[r];
        }
        mx4_finish<DT>(g, o, bf, s, (size_t)(b * g.ybatch + s * g.ys + fl), there);
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// Few second rows (one token, a handful): a workgroup has 16 f and all 16 NS s, its eight waves an
// eighth of the steps each, joined through LDS. Every load of a wave's next four steps is in flight at a time: bound by
// the first operand's bytes (28672 x 8192: 125 MB). WHOLE: rows of whole steps (nb % 4 == 0), whose
// scales of four steps are one load; a load of four bytes for each took a third more time.
template <int DT, int NS, bool WHOLE>
__global__ __launch_bounds__(512) void fno_mx4_mix_few(Gemm g) {
  constexpr int W = 8, U = 4;
  __shared__ v4f red[W][NS][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, quad = lane >> 4;
  const long ft = (g.nf + 15) / 16, tiles = ft * g.batches, steps = (g.nb + 3) / 4, per = (steps + W - 1) / W;
  const long k0 = wave * per, k1 = min(steps, k0 + per);
  size_t sr[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) sr[j] = (size_t)min(16L * j + l16, g.ns - 1) * g.nb;
  // the scales of steps k .. k + 3 of the row at block `row`, a lane's own in the low byte of each later
  auto scales = [&](const uint8_t *e, size_t row, long k, uint32_t *x) __attribute__((always_inline)) {
    if (WHOLE && k + U <= steps) {
      typedef unsigned u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));
      const u32x4_4 v = *reinterpret_cast<const u32x4_4 *>(e + row + 4 * k);
#pragma unroll
      for (int u = 0; u < U; ++u) x[u] = v[u];
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long step = min(k + u, k1 - 1);
        x[u] = WHOLE ? *reinterpret_cast<const uint32_t *>(e + row + 4 * step) : e[row + min(4 * step + quad, g.nb - 1)];
      }
    }
  };
  for (long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const long b = t / ft, f0 = (t - b * ft) * 16;
    const size_t fr = (size_t)(b * g.nf + min(f0 + l16, g.nf - 1)) * g.nb;
    v4f acc[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (long k = k0; k < k1; k += U) {
      ck_u32x4 fc[U], sc[NS][U];
      uint32_t fx[U], sx[NS][U];
      scales(g.fe, fr, k, fx);
#pragma unroll
      for (int j = 0; j < NS; ++j) scales(g.se, sr[j], k, sx[j]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long kb = 4 * min(k + u, k1 - 1) + quad, kc = WHOLE ? kb : min(kb, g.nb - 1);
        fc[u] = *reinterpret_cast<const ck_u32x4 *>(g.fq + (fr + kc) * 16);
#pragma unroll
        for (int j = 0; j < NS; ++j) sc[j][u] = *reinterpret_cast<const ck_u32x4 *>(g.sq + (sr[j] + kc) * 16);
      }
      __builtin_amdgcn_sched_barrier(0);  // all loads first
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // no such step or block: codes of 0 on one side, scales that make 0 of them on both
        const bool none = k + u >= k1 || (!WHOLE && 4 * (k + u) + quad >= g.nb);
        fc[u] = none ? ck_u32x4{0u, 0u, 0u, 0u} : fc[u];
        fx[u] = none ? 127u : WHOLE ? fx[u] >> 8 * quad : fx[u];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          sx[j][u] = none ? 127u : WHOLE ? sx[j][u] >> 8 * quad : sx[j][u];
          acc[j] = mx4_product(fc[u], fx[u], sc[j][u], sx[j][u], acc[j]);
        }
      }
    }
    __syncthreads();  // the last tile's sums have been read
#pragma unroll
    for (int j = 0; j < NS; ++j) red[wave][j][lane] = acc[j];
    __syncthreads();
    if (wave < NS) {
      v4f v = red[0][wave][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) v += red[w][wave][lane];
      const long s = 16 * wave + l16, f = f0 + 4 * quad;
      if (s < g.ns) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (f + r < g.nf) {
            const size_t at = (size_t)(b * g.ybatch + s * g.ys + f + r);
            float o = v[r] + (g.bias_f ? bias_at<DT>(g, f + r, g.nf) : bias_at<DT>(g, s, g.ns));
            if (g.add) o += value_at<DT>(g.add, at);
            put<DT>(g.y, at, g.act ? gelu_train(o) : o);
          }
      }
    }
  }
}

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

// SIZE bytes a lane from p to LDS at `to` + SIZE lane
template <int SIZE>
__device__ __forceinline__ void mx4_to_lds(const uint8_t *p, uint8_t *to) {
  const auto from = (const __attribute__((address_space(1))) void *)p;
  const auto at = (__attribute__((address_space(3))) void *)to;
  static_assert(SIZE == 16 || SIZE == 4, "the builtin takes a literal");
  if constexpr (SIZE == 16) __builtin_amdgcn_global_load_lds(from, at, 16, 0, 0);
  else __builtin_amdgcn_global_load_lds(from, at, 4, 0, 0);
}

// the unit of row r that lies at place l % 8 of its 128 bytes, and the other way round
__device__ __forceinline__ int mx4_unit(int r, int l) { return (l & 7) ^ ((r >> 1 & 3) | (r >> 4 & 1) << 2); }

// A barrier that also waits for the wave's loads to LDS, whose end only the count of loads tells
__device__ __forceinline__ void mx4_barrier() {
  __builtin_amdgcn_s_waitcnt(0);
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

// The scheduler's order for a step: M products with R reads of LDS (MASK 0x100) or loads from memory (0x10) between them
template <int MASK, int R, int M>
__device__ __forceinline__ void mx4_interleave() {
#pragma unroll
  for (int m = 0; m < M; ++m) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(MASK, (R + M - 1) / M, 0);
  }
}

// Workgroups go round the eight XCDs, each with an L2 of its own: an XCD gets neighbouring tiles, eight rows of them
// at a time, so that its 32 workgroups share operands' rows on both sides.
struct Mx4Tile {
  int b, f, s;
};
__device__ __forceinline__ Mx4Tile mx4_tile(uint32_t group, uint32_t ft, uint32_t st, uint32_t tiles) {
  const uint32_t xcd = group % 8, t = xcd * (tiles / 8) + min(xcd, tiles % 8) + group / 8, per = ft * st, b = t / per, r = t - b * per;
  const uint32_t band = r / (8 * st), high = min(8u, ft - 8 * band), in = r - band * 8 * st, s = in / high;
  return Mx4Tile{(int)b, (int)(8 * band + in - s * high), (int)s};
}

}  // namespace

// Large products: a workgroup has a tile of 64 WF x 64 WF, its waves 32 WF x 32 WS each on
// v_mfma_scale_f32_32x32x64_f8f6f4 (lane l: row l % 32, block l / 32 of two). Codes of 256 of the sum's values go from
// memory straight to LDS, the next ones while these are multiplied: rows of 128 bytes, whose 16-byte units are
// swapped by row so that a fragment's reads meet no bank twice (a pass serves rows r .. r + 7 and r + 16 .. r + 23).
// Fragments are read a step of 64 values ahead; the barrier between two buffers stands before the last step's
// products, which cover the first reads from the new one. Rows of whole 128 values (nb % 4 == 0).
template <int DT, int WF, int WS>
__global__ __launch_bounds__(256 * WF / WS) __attribute__((amdgpu_waves_per_eu(2, 2)))
void fno_mx4_mix_tiles(Gemm g) {
  constexpr int T = 64 * WF, ROWS = 2 * T, NW = 4 * WF / WS;   // waves: two along f, the others along s
  constexpr int NL = ROWS / 8 / NW, NX = ROWS / 16 / NW;       // loads of a wave: codes of a stage, scales of two
  __shared__ __attribute__((aligned(128))) uint8_t buf0[ROWS * 128], buf1[ROWS * 128], sx0[ROWS * 16], sx1[ROWS * 16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l32 = lane & 31, half = lane >> 5;
  const int wf = wave & 1, ws = wave >> 1;
  const uint32_t ft = (uint32_t)((g.nf + T - 1) / T), st = (uint32_t)((g.ns + T - 1) / T), tiles = ft * st * (uint32_t)g.batches;
  const int stages = (int)((g.nb + 7) / 8), pairs = (stages + 1) / 2;
  const Mx4Tile tile = mx4_tile(blockIdx.x, ft, st, tiles);
  const long b = tile.b, f0 = (long)tile.f * T, s0 = (long)tile.s * T;
  // the first half of the waves fetches the first operand's rows, the others the second's
  const bool first = wave < NW / 2;
  const long row0 = first ? b * g.nf + f0 : s0;
  const int rows = (int)min((long)T, (first ? g.nf - f0 : g.ns - s0)), mine = wave % (NW / 2) * (2 * T / NW);
  const uint8_t *codes = (first ? g.fq : g.sq) + (size_t)row0 * g.nb * 16, *scales = (first ? g.fe : g.se) + (size_t)row0 * g.nb;
  uint32_t off[NL], xoff[NX];
#pragma unroll
  for (int n = 0; n < NL; ++n) {
    const int r = mine + 8 * n + (lane >> 3), unit = mx4_unit(r, lane);
    off[n] = (uint32_t)(min(r, rows - 1) * (int)g.nb + unit) * 16;
  }
#pragma unroll
  for (int n = 0; n < NX; ++n) xoff[n] = (uint32_t)(min(mine + 16 * n + (lane >> 2), rows - 1) * (int)g.nb);
  const int at = (first ? 0 : T) + mine;  // the wave's first row in LDS

  // A row that ends in half a stage is fetched 64 bytes past its end, at the last row into the scales behind the
  // codes: nobody multiplies them. Past the last stage it is fetched again, so that a stage has no branch.
  auto fetch = [&](uint8_t *to, int stage) __attribute__((always_inline)) {
    const uint8_t *p = codes + (size_t)min(stage, stages - 1) * 128;
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      uint32_t o = off[n];
      asm volatile("" : "+v"(o));  // one base in scalar registers and 32 bits a lane, not an address for each load
      mx4_to_lds<16>(p + o, to + (at + 8 * n) * 128);
    }
  };
  auto fetch_scales = [&](uint8_t *to, int pair) __attribute__((always_inline)) {
    const uint32_t x = (uint32_t)min(16 * min(pair, pairs - 1) + 4 * (lane & 3), (int)g.nb - 4);
#pragma unroll
    for (int n = 0; n < NX; ++n) mx4_to_lds<4>(scales + (xoff[n] + x), to + (at + 16 * n) * 16);
  };

  v16f acc[WF][WS];
#pragma unroll
  for (int i = 0; i < WF; ++i)
#pragma unroll
    for (int j = 0; j < WS; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  // a lane's row within 32, and its unit's place: rows of a fragment differ by multiples of 32, which the swap ignores
  const int swap = mx4_unit(l32, 0);
  const int frow = wf * (32 * WF) + l32, srow = T + ws * (32 * WS) + l32;
  ck_u32x4 fc[2][WF], sc[2][WS];
  uint2 fx[2][WF], sx[2][WS];  // scales of this stage and the next, the lane's own at bytes 0, 2 of either word
  auto read = [&](const uint8_t *from, int step, int slot) __attribute__((always_inline)) {
    const int u = ((2 * step + half) ^ swap) * 16;
#pragma unroll
    for (int i = 0; i < WF; ++i) fc[slot][i] = *reinterpret_cast<const ck_u32x4 *>(from + (frow + 32 * i) * 128 + u);
#pragma unroll
    for (int j = 0; j < WS; ++j) sc[slot][j] = *reinterpret_cast<const ck_u32x4 *>(from + (srow + 32 * j) * 128 + u);
  };
  auto read_scales = [&](const uint8_t *from, int odd, int slot) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < WF; ++i) fx[slot][i] = *reinterpret_cast<const uint2 *>(from + (frow + 32 * i) * 16 + 8 * odd);
#pragma unroll
    for (int j = 0; j < WS; ++j) sx[slot][j] = *reinterpret_cast<const uint2 *>(from + (srow + 32 * j) * 16 + 8 * odd);
  };
  auto own_scales = [&](int slot) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < WF; ++i) fx[slot][i] = make_uint2(fx[slot][i].x >> 8 * half, fx[slot][i].y >> 8 * half);
#pragma unroll
    for (int j = 0; j < WS; ++j) sx[slot][j] = make_uint2(sx[slot][j].x >> 8 * half, sx[slot][j].y >> 8 * half);
  };
  auto multiply = [&](auto step, int slot, int xslot) __attribute__((always_inline)) {
    constexpr int STEP = decltype(step)::value, SEL = STEP & 1 ? 2 : 0;
#pragma unroll
    for (int i = 0; i < WF; ++i)
#pragma unroll
      for (int j = 0; j < WS; ++j) {
        const v8i x{(int)fc[slot][i][0], (int)fc[slot][i][1], (int)fc[slot][i][2], (int)fc[slot][i][3], 0, 0, 0, 0};
        const v8i y{(int)sc[slot][j][0], (int)sc[slot][j][1], (int)sc[slot][j][2], (int)sc[slot][j][3], 0, 0, 0, 0};
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc[i][j], 4, 4, SEL, (int)(STEP & 2 ? fx[xslot][i].y : fx[xslot][i].x),
                                                                    SEL, (int)(STEP & 2 ? sx[xslot][j].y : sx[xslot][j].x));
      }
  };
  // A stage that another follows: every step's products go on while the next step's fragments are read. X: the
  // scales' registers of this stage.
  auto stage = [&](auto xslot, const uint8_t *now, const uint8_t *next, uint8_t *freed, const uint8_t *xnext, int odd_next,
                   int s) __attribute__((always_inline)) {
    constexpr int X = decltype(xslot)::value;
    read(now, 1, 1);
    multiply(std::integral_constant<int, 0>{}, 0, X);
    mx4_interleave<0x100, WF + WS, WF * WS>();
    __builtin_amdgcn_sched_barrier(0);
    read(now, 2, 0);
    multiply(std::integral_constant<int, 1>{}, 1, X);
    mx4_interleave<0x100, WF + WS, WF * WS>();
    __builtin_amdgcn_sched_barrier(0);
    read(now, 3, 1);
    multiply(std::integral_constant<int, 2>{}, 0, X);
    mx4_interleave<0x100, WF + WS, WF * WS>();
    __builtin_amdgcn_sched_barrier(0);
    mx4_barrier();  // what is fetched has landed, and this stage's fragments have been read
    read(next, 0, 0);
    read_scales(xnext, odd_next, 1 - X);
    fetch(freed, s + 2);
    multiply(std::integral_constant<int, 3>{}, 1, X);
    mx4_interleave<0x100, 2 * (WF + WS), (WF * WS + 1) / 2>();  // reads of LDS stay in front of loads to it
    mx4_interleave<0x010, NL, (WF * WS + 1) / 2>();
    __builtin_amdgcn_sched_barrier(0);
    own_scales(1 - X);
  };
  constexpr std::integral_constant<int, 0> X0{};
  constexpr std::integral_constant<int, 1> X1{};

  fetch_scales(sx0, 0);
  fetch(buf0, 0);
  mx4_barrier();
  fetch(buf1, 1);
  fetch_scales(sx1, 1);
  read(buf0, 0, 0);
  read_scales(sx0, 0, 0);
  own_scales(0);
  const int whole = (int)(g.nb / 8);
  // The pair's scales and the next one's change places; reads of them stand right behind a barrier, where no fetch is
  // under way that the compiler would wait for, not knowing which of the two they come from.
  uint8_t *xnow = sx0, *xnext = sx1;
  int s = 0;
  for (; s + 2 <= whole; s += 2) {
    stage(X0, buf0, buf1, buf0, xnow, 1, s);
    stage(X1, buf1, buf0, buf1, xnext, 0, s + 1);
    fetch_scales(xnow, s / 2 + 2);
    uint8_t *const x = xnow;
    xnow = xnext, xnext = x;
  }
#pragma unroll 1
  for (long k = 8 * s + half; k < g.nb; k += 2) {  // up to 12 blocks more: straight from memory, two at a time
#pragma unroll
    for (int i = 0; i < WF; ++i) {
      const size_t at = (size_t)(b * g.nf + min(f0 + frow + 32 * i, g.nf - 1)) * g.nb + k;
      fc[0][i] = *reinterpret_cast<const ck_u32x4 *>(g.fq + at * 16);
      fx[0][i].x = g.fe[at];
    }
#pragma unroll
    for (int j = 0; j < WS; ++j) {
      const size_t at = (size_t)min(s0 + srow - T + 32 * j, g.ns - 1) * g.nb + k;
      sc[0][j] = *reinterpret_cast<const ck_u32x4 *>(g.sq + at * 16);
      sx[0][j].x = g.se[at];
    }
    multiply(std::integral_constant<int, 0>{}, 0, 0);
  }
  // A lane has rows f = 8 q + 4 half .. + 3 of a fragment (q = 0 .. 3) in column s. Up to 64 rows of 32 columns at a time
  // go through LDS, so that lanes finish and store whole 16 bytes of neighbours, 128 bytes a column (16 bits).
  mx4_barrier();
  constexpr int PI = WF >= 2 ? 2 : 1, N = ck_vec<DT>(), PITCH = 32 * PI + 4, LANES = 32 * PI / N;  // lanes of a column
  float *part = reinterpret_cast<float *>(first ? buf0 : buf1) + wave % (NW / 2) * 32 * PITCH;
  static_assert(NW / 2 * 32 * PITCH * 4 <= (int)sizeof(buf0), "half of the waves' parts fit a buffer");
#pragma unroll 1
  for (int h = 0; h < WF / PI; ++h) {
    const long fl = f0 + wf * (32 * WF) + 32 * PI * h + lane % LANES * N;
    const int there = (int)max(0L, min((long)N, g.nf - fl));
    float bf[N];
#pragma unroll
    for (int e = 0; e < N; ++e) bf[e] = g.bias_f && there > 0 ? bias_at<DT>(g, fl + e, g.nf) : 0.f;
#pragma unroll 1
    for (int j = 0; j < WS; ++j) {  // one copy of what follows: straight-line code of all parts costs more than it does
#pragma unroll
      for (int k = 0; k < WF / PI * WS; ++k)
        if (k == h * WS + j)
#pragma unroll
          for (int i = 0; i < PI; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const v16f &c = acc[PI * (k / WS) + i][k % WS];
              *reinterpret_cast<v4f *>(part + l32 * PITCH + 32 * i + 8 * q + 4 * half) =
                  v4f{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
            }
      __builtin_amdgcn_wave_barrier();
#pragma unroll 2
      for (int c = lane / LANES; c < 32; c += 64 / LANES) {
        const long s = s0 + ws * (32 * WS) + 32 * j + c;
        if (s >= g.ns || there == 0) continue;
        float o[N];
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          const v4f v = *reinterpret_cast<const v4f *>(part + c * PITCH + lane % LANES * N + e);
#pragma unroll
          for (int r = 0; r < 4; ++r) o[e + r] = v[r];
        }
        mx4_finish<DT>(g, o, bf, s, (size_t)(b * g.ybatch + s * g.ys + fl), there);
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

namespace {

template <int DT>
const void *few_kernel(const Gemm &g) {
  const bool whole = g.nb % 4 == 0;
  if (g.ns <= 16) return whole ? (const void *)fno_mx4_mix_few<DT, 1, true> : (const void *)fno_mx4_mix_few<DT, 1, false>;
  if (g.ns > 32) return (const void *)fno_mx4_mix_few<DT, 4, false>;
  return whole ? (const void *)fno_mx4_mix_few<DT, 2, true> : (const void *)fno_mx4_mix_few<DT, 2, false>;
}

template <int DT>
const void *tiles_kernel(int w) {
  return w == 4 ? (const void *)fno_mx4_mix_tiles<DT, 4, 2>
         : w == 2 ? (const void *)fno_mx4_mix_tiles<DT, 2, 2> : (const void *)fno_mx4_mix_tiles<DT, 1, 1>;
}

}  // namespace

hipError_t launch_mx4_mix(const Mx4MixArgs &a, int dtype, hipStream_t s) {
  Gemm g{};
  g.bias = a.bias, g.add = a.add, g.y = a.y, g.nb = a.nb, g.act = a.act;
  if (a.P == 1) {
    g.fq = a.aq, g.fe = a.ae, g.sq = a.xq, g.se = a.xe;
    g.nf = a.O, g.ns = a.B, g.batches = 1, g.ybatch = 0, g.ys = a.O, g.bias_f = 1;
  } else {
    g.fq = a.xq, g.fe = a.xe, g.sq = a.aq, g.se = a.ae;
    g.nf = a.P, g.ns = a.O, g.batches = a.B, g.ybatch = a.O * a.P, g.ys = a.P, g.bias_f = 0;
  }
  FNO_BOUNDS(check_mx4_mix(a, dtype);)
  void *args[] = {(void *)&g};
  // few rows: 1 x 8192 x 8192 97 us as below, 11 so; from 33 on tiles are as fast where rows are whole steps
  // (64 x 8192 x 8192: 42 us so, 27 in tiles)
  if (g.nb >= 32 && g.ns <= (g.nb % 4 == 0 ? 32 : 64)) {
    const void *k = dtype == DT_F32 ? few_kernel<DT_F32>(g) : dtype == DT_F16 ? few_kernel<DT_F16>(g) : few_kernel<DT_BF16>(g);
    return hipLaunchKernel(k, dim3((unsigned)std::min((g.nf + 15) / 16 * g.batches, kMaxGrid)), dim3(512), args, 0, s);
  }
  auto tiles = [&](long T) { return (g.nf + T - 1) / T * ((g.ns + T - 1) / T) * g.batches; };
  if (g.nb % 4 == 0 && g.nb >= 16 && g.ns > 32 && tiles(64) <= kMaxGrid) {
    // The largest tiles that still give three quarters of the 256 compute units one (bf16, random codes; tiles of
    // 256 / 128 / 64): 4096^3 59 / 68 / 106 us, 2048 x 4096 x 4096 44 / 34 / 56, 512 x 4096 x 4096 39 / 19 / 14.
    const int w = tiles(256) >= 192 ? 4 : tiles(128) >= 192 ? 2 : 1;
    const void *k = dtype == DT_F32 ? tiles_kernel<DT_F32>(w) : dtype == DT_F16 ? tiles_kernel<DT_F16>(w) : tiles_kernel<DT_BF16>(w);
    return hipLaunchKernel(k, dim3((unsigned)tiles(64 * w)), dim3(w == 4 ? 512 : 256), args, 0, s);
  }
  // tiles of 128 x 64 (of 256 x 64, whose registers leave a compute unit half the waves, 32 x 64 x 64 x 65536 fp16 takes
  // 245 us, so 203), or of 64 x 32 where those would leave compute units idle (5 x 200 x 72 x 1001 fp32: 17 us, 8)
  auto count = [&](long f, long r) { return (g.nf + f - 1) / f * ((g.ns + r - 1) / r) * g.batches; };
  const bool wide = count(128, 64) >= 256;
#define FNO_PICK(DT) (wide ? (const void *)fno_mx4_mix<DT, 2, 4> : (const void *)fno_mx4_mix<DT, 1, 2>)
  const void *k = dtype == DT_F32 ? FNO_PICK(DT_F32) : dtype == DT_F16 ? FNO_PICK(DT_F16) : FNO_PICK(DT_BF16);
#undef FNO_PICK
  return hipLaunchKernel(k, dim3((unsigned)std::min(wide ? count(128, 64) : count(64, 32), kMaxGrid)), dim3(kThreads), args, 0, s);
}

}  // namespace fno
