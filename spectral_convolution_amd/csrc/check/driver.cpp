// driver.cpp - the bounds-check build's driver: every public entry point on a
// spread of shapes (matrix-core and VALU planes, 2D and 3D, the three dtypes,
// ragged modes and channels, both launch shapes, the half exchange, the
// backward pass (from x and from saved spectra), weight repacking, the
// allocation-free entry, the FNO block, the full FNO2d network and the
// training operators around a block). Each launch is checked by its launcher's
// bounds hook against the recording runtime's allocations; the program exits
// non-zero if any span or assumption was broken. With the argument `kernels` it
// prints the kernels of the library, with `trace` the launches (kernel | grid x, y, workgroup) of the training
// operators' calls that standard input lists, a line each:
//   norm DTYPE KIND BATCH CHANNELS PIXELS  |  mix DTYPE BATCH C_IN C_OUT PIXELS ACT ADD  |  checkpoint DTYPE ROWS N
// Host code only.

#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>
#include <string>
#include <vector>

#include "../../../include/fno.h"
#include "../block_ops.hpp"
#include "../train.hpp"

long check_launches();
long check_reports();
void *check_reserve(size_t n);
void check_trace(bool on);
void check_list_kernels();

namespace {

int n_fail = 0;

void expect(bool ok, const char *what, int line) {
  if (!ok) {
    std::fprintf(stderr, "driver: line %d: %s\n", line, what);
    ++n_fail;
  }
}
#define EXPECT(c) expect((c), #c, __LINE__)

size_t es_of(fno_dtype_t d) { return d == FNO_F32 ? 4 : 2; }

struct Buf {
  void *p = nullptr;
  explicit Buf(size_t n);
  ~Buf();
};

}  // namespace

Buf::Buf(size_t n) {
  if (hipMalloc(&p, n) != hipSuccess) p = nullptr;
}
Buf::~Buf() { (void)hipFree(p); }

namespace {

void run_layer(int ndim, int B, int Ci, int Co, std::vector<int> grid, std::vector<int> modes, fno_dtype_t dt) {
  fno_plan_t p = nullptr;
  const fno_status_t st = fno_plan_create(&p, ndim, B, Ci, Co, grid.data(), modes.data(), dt, 0);
  if (st == FNO_ERR_UNSUPPORTED) return;
  EXPECT(st == FNO_OK);
  if (st != FNO_OK) return;
  size_t px = 1, K = ndim == 2 ? 2 : 4;
  for (int d = 0; d < ndim; ++d) {
    px *= (size_t)grid[d];
    K *= (size_t)modes[d];
  }
  const size_t es = es_of(dt);
  Buf x((size_t)B * Ci * px * es), y((size_t)B * Co * px * es), w(K * Ci * Co * 2 * es);
  Buf gy((size_t)B * Co * px * es), gx((size_t)B * Ci * px * es), gw(K * Ci * Co * 2 * es);
  auto conv = ndim == 2 ? fno_spectral_conv2d : fno_spectral_conv3d;
  EXPECT(conv(p, x.p, w.p, y.p, nullptr) == FNO_OK);
  auto bwd = ndim == 2 ? fno_spectral_conv2d_backward : fno_spectral_conv3d_backward;
  EXPECT(bwd(p, x.p, w.p, gy.p, gx.p, gw.p, nullptr) == FNO_OK);
  EXPECT(bwd(p, x.p, w.p, gy.p, gx.p, nullptr, nullptr) == FNO_OK);
  EXPECT(bwd(p, x.p, w.p, gy.p, nullptr, gw.p, nullptr) == FNO_OK);
  // the saved-spectra pair, where the plan has a saved format
  size_t sb = 0;
  const fno_status_t ss = fno_plan_saved_bytes(p, &sb);
  EXPECT(ss == FNO_OK || ss == FNO_ERR_UNSUPPORTED);
  if (ss == FNO_OK) {
    Buf sv(sb);
    EXPECT(fno_spectral_conv_forward_save(p, x.p, w.p, y.p, sv.p, nullptr) == FNO_OK);
    EXPECT(fno_spectral_conv_backward_saved(p, sv.p, w.p, gy.p, gx.p, gw.p, nullptr) == FNO_OK);
    EXPECT(fno_spectral_conv_backward_saved(p, sv.p, nullptr, gy.p, nullptr, gw.p, nullptr) == FNO_OK);
  }
  const fno_status_t na = fno_spectral_conv_noalloc(p, x.p, w.p, y.p, nullptr);
  EXPECT(na == FNO_OK || na == FNO_ERR_UNSUPPORTED);
  int nl = 0;
  EXPECT(fno_plan_num_launches(p, &nl) == FNO_OK);
  for (int i = 0; i < nl; ++i) EXPECT(fno_plan_run_launch(p, i, x.p, w.p, y.p, nullptr) == FNO_OK);
  if (fno_plan_set_launch_shape(p, FNO_LAUNCH_FUSED) == FNO_OK) {
    EXPECT(conv(p, x.p, w.p, y.p, nullptr) == FNO_OK);
    if (fno_plan_set_launch_shape(p, FNO_LAUNCH_FUSED_STALL_TEST) == FNO_OK) (void)conv(p, x.p, w.p, y.p, nullptr);
    EXPECT(fno_plan_set_launch_shape(p, FNO_LAUNCH_SEPARATE) == FNO_OK);
  }
  const size_t n = K * Ci * Co;
  Buf re(n * es), im(n * es), corners(2 * n * es);
  EXPECT(fno_weights_pack(p, FNO_WEIGHTS_SPLIT, re.p, im.p, w.p, nullptr) == FNO_OK);
  EXPECT(fno_weights_unpack(p, FNO_WEIGHTS_SPLIT, w.p, re.p, im.p, nullptr) == FNO_OK);
  EXPECT(fno_weights_pack(p, FNO_WEIGHTS_CORNERS, corners.p, nullptr, w.p, nullptr) == FNO_OK);
  EXPECT(fno_weights_unpack(p, FNO_WEIGHTS_CORNERS, w.p, corners.p, nullptr, nullptr) == FNO_OK);
  if (ndim == 2) {
    Buf A((size_t)Co * Ci * es), bias((size_t)Co * es);
    const fno_status_t b0 = fno_block2d(p, x.p, w.p, A.p, bias.p, 1, y.p, nullptr);
    EXPECT(b0 == FNO_OK || b0 == FNO_ERR_UNSUPPORTED);
    if (b0 == FNO_OK) EXPECT(fno_block2d(p, x.p, w.p, A.p, nullptr, 0, y.p, nullptr) == FNO_OK);
  }
  EXPECT(fno_plan_destroy(p) == FNO_OK);
}

void run_model(int B, int H, int W, int in, int ch, int layers, int m1, int m2, int proj, int out, fno_dtype_t dt) {
  fno_model2d_t m = nullptr;
  const fno_status_t st = fno_model2d_create(&m, B, H, W, in, ch, layers, m1, m2, proj, out, dt, 0);
  EXPECT(st == FNO_OK);
  if (st != FNO_OK) return;
  const size_t es = es_of(dt), px = (size_t)H * W, K = (size_t)2 * m1 * m2;
  std::vector<Buf *> bufs;
  auto mk = [&](size_t n) {
    bufs.push_back(new Buf(n * es));
    return bufs.back()->p;
  };
  std::vector<const void *> params;
  params.push_back(mk((size_t)ch * in));
  params.push_back(mk(ch));
  for (int l = 0; l < layers; ++l) {
    params.push_back(mk(K * ch * ch * 2));
    params.push_back(mk((size_t)ch * ch));
    params.push_back(mk(ch));
  }
  params.push_back(mk((size_t)proj * ch));
  params.push_back(mk(proj));
  params.push_back(mk((size_t)out * proj));
  params.push_back(mk(out));
  void *f = mk((size_t)B * in * px), *o = mk((size_t)B * out * px);
  EXPECT(fno_model2d_forward(m, f, params.data(), o, nullptr) == FNO_OK);
  EXPECT(fno_model2d_set_graph(m, 1) == FNO_OK);
  EXPECT(fno_model2d_forward(m, f, params.data(), o, nullptr) == FNO_OK);
  EXPECT(fno_model2d_destroy(m) == FNO_OK);
  for (Buf *b : bufs) delete b;
}

void run_checkpoint(long rows, long n, fno_dtype_t dt) {
  size_t bytes = 0;
  EXPECT(fno_checkpoint_bytes(rows, n, &bytes) == FNO_OK);
  Buf x((size_t)rows * n * es_of(dt)), s(bytes);
  EXPECT(fno_checkpoint_pack(x.p, s.p, rows, n, dt, nullptr) == FNO_OK);
  EXPECT(fno_checkpoint_unpack(s.p, x.p, rows, n, dt, nullptr) == FNO_OK);
}

// more values than the host could hold: nothing behind the buffers
void run_checkpoint_far(long rows, long n, fno_dtype_t dt) {
  size_t bytes = 0;
  EXPECT(fno_checkpoint_bytes(rows, n, &bytes) == FNO_OK);
  void *x = check_reserve((size_t)rows * n * es_of(dt)), *s = check_reserve(bytes);
  EXPECT(fno_checkpoint_pack(x, s, rows, n, dt, nullptr) == FNO_OK);
  EXPECT(fno_checkpoint_unpack(s, x, rows, n, dt, nullptr) == FNO_OK);
}

void run_norm(int B, int C, long P, int kind, bool params, fno_dtype_t dt) {
  const size_t es = es_of(dt), n = (size_t)B * C * P * es, nc = C * es;
  size_t sb = 0, wb = 0;
  EXPECT(fno_norm_residual_saved_bytes(B, C, P, &sb) == FNO_OK);
  EXPECT(fno_norm_residual_workspace_bytes(B, C, P, dt, &wb) == FNO_OK);
  Buf x(n), v(n), y(n), u(n), gy(n), gu(n), gx(n), gv(n), saved(sb), ws(wb);
  Buf p0(nc), p1(nc), p2(nc), p3(nc), p4(nc), pg(B * nc), g0(nc), g1(nc), g2(nc), g3(nc), g4(nc), gg(B * nc);
  fno_norm_params_t p{kind, 1e-5f, p0.p, p1.p, pg.p, p2.p, p3.p, p4.p};
  fno_norm_grads_t g{g0.p, g1.p, gg.p, g2.p, g3.p, g4.p};
  if (!params) {
    p = fno_norm_params_t{kind, 1e-5f, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
    g = fno_norm_grads_t{};
  }
  EXPECT(fno_norm_residual(&p, x.p, v.p, y.p, u.p, B, C, P, dt, nullptr) == FNO_OK);
  EXPECT(fno_norm_residual(&p, x.p, v.p, y.p, nullptr, B, C, P, dt, nullptr) == FNO_OK);
  EXPECT(fno_norm_residual_save(&p, x.p, v.p, y.p, u.p, saved.p, B, C, P, dt, nullptr) == FNO_OK);
  EXPECT(fno_norm_residual_backward(&p, x.p, v.p, gy.p, gu.p, gx.p, gv.p, &g, ws.p, B, C, P, dt, nullptr) == FNO_OK);
  EXPECT(fno_norm_residual_backward_saved(&p, saved.p, gy.p, gu.p, gx.p, nullptr, params ? &g : nullptr, ws.p, B, C, P,
                                          dt, nullptr) == FNO_OK);
}

void run_mix(int B, int I, int O, long P, int act, bool add, fno_dtype_t dt) {
  const size_t es = es_of(dt), nx = (size_t)B * I * P * es, ny = (size_t)B * O * P * es;
  size_t sb = 0, wb = 0;
  EXPECT(fno_channel_mix_saved_bytes(B, I, O, P, act, add, &sb) == FNO_OK);
  EXPECT(fno_channel_mix_workspace_bytes(B, I, O, P, dt, &wb) == FNO_OK);
  Buf x(nx), A((size_t)O * I * es), bias(O * es), ad(ny), y(ny), saved(sb), gy(ny), gx(nx), gA((size_t)O * I * es),
      gb(O * es), gadd(ny), ws(wb);
  EXPECT(fno_channel_mix_save(x.p, A.p, bias.p, add ? ad.p : nullptr, y.p, saved.p, B, I, O, P, act, dt, nullptr) ==
         FNO_OK);
  EXPECT(fno_channel_mix_backward_saved(saved.p, A.p, bias.p, gy.p, gx.p, gA.p, gb.p, add ? gadd.p : nullptr, ws.p, B, I,
                                        O, P, act, add, dt, nullptr) == FNO_OK);
  EXPECT(fno_channel_mix_backward_saved(saved.p, A.p, nullptr, gy.p, gx.p, nullptr, nullptr, nullptr, nullptr, B, I, O,
                                        P, act, add, dt, nullptr) == FNO_OK);
}

// dropout alone and into a residual, in every unit; nothing behind the buffers
void run_drop(int B, int C, long P, fno_dtype_t dt) {
  const size_t n = (size_t)B * C * P * es_of(dt);
  void *x = check_reserve(n), *v = check_reserve(n), *y = check_reserve(n), *step = check_reserve(8);
  for (int unit = 0; unit < 3; ++unit)
    for (int last = 0; last < 2; ++last) {
      const fno_dropout_t d{0.25f, unit, 1, 2, last ? static_cast<uint64_t *>(step) : nullptr};
      EXPECT(fno_dropout_residual(&d, last ? x : nullptr, v, y, B, C, P, last, dt, nullptr) == FNO_OK);
    }
}

// group norm, forward and backward, with every gradient and with one; nothing behind the buffers
void run_gnorm(int B, int C, long P, int G, int last, fno_dtype_t dt) {
  const size_t es = es_of(dt), n = (size_t)B * C * P * es, nc = C * es;
  size_t wb = 0;
  EXPECT(fno_group_norm_workspace_bytes(B, C, P, G, last, dt, &wb) == FNO_OK);
  auto far = [](size_t k) { return check_reserve(k); };
  void *x = far(n), *y = far(n), *ws = far(wb), *gy = far(n), *gx = far(n);
  float *stats = static_cast<float *>(far((size_t)B * G * 8));
  const fno_dropout_t d{0.25f, FNO_DROP_ELEMENT, 1, 2, nullptr};
  const fno_group_norm_params_t p{G, 1, last, 1e-5f, far(nc), far(nc)}, q{G, 2, last, 1e-5f, nullptr, nullptr};
  EXPECT(fno_group_norm(&p, &d, x, y, stats, ws, B, C, P, dt, nullptr) == FNO_OK);
  EXPECT(fno_group_norm(&q, nullptr, x, y, nullptr, ws, B, C, P, dt, nullptr) == FNO_OK);
  EXPECT(fno_group_norm_backward(&p, &d, x, stats, gy, gx, far(nc), far(nc), ws, B, C, P, dt, nullptr) == FNO_OK);
  EXPECT(fno_group_norm_backward(&p, &d, x, stats, gy, nullptr, far(nc), nullptr, ws, B, C, P, dt, nullptr) == FNO_OK);
  EXPECT(fno_group_norm_backward(&q, nullptr, x, stats, gy, gx, nullptr, nullptr, ws, B, C, P, dt, nullptr) == FNO_OK);
}

// a field to 4-bit floats and back, and a channel mix of it; nothing behind the buffers
void run_mx4(int B, int I, int O, long P, fno_dtype_t dt) {
  size_t xb = 0, ab = 0;
  EXPECT(fno_mx4_bytes(B, I, P, &xb) == FNO_OK);
  EXPECT(fno_mx4_bytes(O, I, 1, &ab) == FNO_OK);
  const size_t es = es_of(dt), nx = (size_t)B * I * P * es, ny = (size_t)B * O * P * es;
  void *x = check_reserve(nx), *xq = check_reserve(xb), *aq = check_reserve(ab), *y = check_reserve(ny), *add = check_reserve(ny),
       *bias = check_reserve(O * es);
  EXPECT(fno_mx4_pack(x, xq, B, I, P, dt, nullptr) == FNO_OK);
  EXPECT(fno_mx4_unpack(xq, x, B, I, P, dt, nullptr) == FNO_OK);
  EXPECT(fno_channel_mix_mx4(xq, aq, bias, add, y, B, I, O, P, 1, dt, nullptr) == FNO_OK);
  EXPECT(fno_channel_mix_mx4(xq, aq, nullptr, nullptr, y, B, I, O, P, 0, dt, nullptr) == FNO_OK);
}

// one call of a training operator, forward and backward, with nothing behind its buffers
void trace_call(const std::string &op, int dt, const std::vector<long> &v) {
  const auto d = (fno_dtype_t)dt;
  const size_t es = es_of(d);
  size_t sb = 0, wb = 0;
  auto far = [](size_t n) { return check_reserve(n); };
  if (op == "norm") {
    const int kind = (int)v[0], B = (int)v[1], C = (int)v[2];
    const long P = v[3];
    EXPECT(fno_norm_residual_saved_bytes(B, C, P, &sb) == FNO_OK);
    EXPECT(fno_norm_residual_workspace_bytes(B, C, P, d, &wb) == FNO_OK);
    const size_t n = (size_t)B * C * P * es, nc = C * es, ng = (size_t)B * nc;
    const fno_norm_params_t p{kind, 1e-5f, far(nc), far(nc), far(ng), far(nc), far(nc), far(nc)};
    const fno_norm_grads_t g{far(nc), far(nc), far(ng), far(nc), far(nc), far(nc)};
    void *saved = far(sb);
    EXPECT(fno_norm_residual_save(&p, far(n), far(n), far(n), far(n), saved, B, C, P, d, nullptr) == FNO_OK);
    EXPECT(fno_norm_residual_backward_saved(&p, saved, far(n), far(n), far(n), far(n), &g, far(wb), B, C, P, d, nullptr) == FNO_OK);
  } else if (op == "mix") {
    const int B = (int)v[0], I = (int)v[1], O = (int)v[2], act = (int)v[4], add = (int)v[5];
    const long P = v[3];
    EXPECT(fno_channel_mix_saved_bytes(B, I, O, P, act, add, &sb) == FNO_OK);
    EXPECT(fno_channel_mix_workspace_bytes(B, I, O, P, d, &wb) == FNO_OK);
    const size_t nx = (size_t)B * I * P * es, ny = (size_t)B * O * P * es, na = (size_t)O * I * es;
    void *saved = far(sb), *A = far(na), *bias = far(O * es);
    EXPECT(fno_channel_mix_save(far(nx), A, bias, add ? far(ny) : nullptr, far(ny), saved, B, I, O, P, act, d, nullptr) == FNO_OK);
    EXPECT(fno_channel_mix_backward_saved(saved, A, bias, far(ny), far(nx), far(na), far(O * es), add ? far(ny) : nullptr,
                                          far(wb), B, I, O, P, act, add, d, nullptr) == FNO_OK);
  } else if (op == "gnorm") {
    run_gnorm((int)v[0], (int)v[1], v[2], (int)v[3], (int)v[4], d);
  } else if (op == "drop") {
    run_drop((int)v[0], (int)v[1], v[2], d);
  } else if (op == "mx4") {
    run_mx4((int)v[0], (int)v[1], (int)v[2], v[3], d);
  } else {
    run_checkpoint_far(v[0], v[1], d);
  }
}

void trace_calls() {
  check_trace(true);
  char op[16];
  int dt;
  while (std::scanf("%15s %d", op, &dt) == 2) {
    const std::string name = op;
    std::vector<long> v(name == "norm" || name == "mx4" ? 4 : name == "mix" ? 6 : name == "gnorm" ? 5 : name == "drop" ? 3 : 2);
    for (long &x : v) EXPECT(std::scanf("%ld", &x) == 1);
    trace_call(name, dt, v);
  }
}

}  // namespace

int main(int argc, char **argv) {
  if (argc > 1 && !std::strcmp(argv[1], "kernels")) {
    check_list_kernels();
    return 0;
  }
  if (argc > 1 && !std::strcmp(argv[1], "trace")) {
    trace_calls();
    return check_reports() == 0 && n_fail == 0 ? 0 : 1;
  }
  const fno_dtype_t dts[3] = {FNO_F32, FNO_F16, FNO_BF16};
  // 2D: matrix-core planes (64 .. 256) and the VALU planes (small and
  // non-power-of-two grids), ragged and maximal modes, small and large batches
  struct L2 { int B, Ci, Co, H, W, m1, m2; };
  const L2 l2[] = {
      {2, 4, 4, 16, 16, 4, 4},      {16, 32, 32, 128, 128, 16, 16}, {32, 64, 64, 256, 256, 32, 32},
      {3, 5, 7, 64, 64, 5, 7},      {1, 3, 64, 128, 128, 16, 16},   {20, 64, 64, 256, 256, 24, 24},
      {17, 33, 20, 64, 128, 20, 24}, {2, 8, 12, 32, 48, 6, 9},      {16, 64, 68, 256, 128, 32, 17},
      {1, 1, 1, 64, 64, 1, 1},      {4, 16, 16, 256, 64, 32, 32},   {2, 64, 65, 128, 256, 9, 3},
  };
  for (const L2 &c : l2)
    for (fno_dtype_t dt : dts) run_layer(2, c.B, c.Ci, c.Co, {c.H, c.W}, {c.m1, c.m2}, dt);
  struct L3 { int B, Ci, Co, X, Y, Z, m1, m2, m3; };
  const L3 l3[] = {
      {4, 32, 32, 64, 64, 64, 16, 16, 16}, {2, 3, 5, 16, 16, 16, 4, 4, 4}, {1, 8, 8, 32, 64, 64, 6, 10, 17},
  };
  for (const L3 &c : l3)
    for (fno_dtype_t dt : dts) run_layer(3, c.B, c.Ci, c.Co, {c.X, c.Y, c.Z}, {c.m1, c.m2, c.m3}, dt);
  run_model(2, 64, 64, 3, 32, 2, 8, 8, 16, 1, FNO_F16);
  run_model(20, 256, 256, 3, 64, 4, 24, 24, 128, 1, FNO_F16);
  run_model(1, 64, 64, 3, 64, 4, 12, 12, 128, 1, FNO_BF16);
  run_model(2, 32, 32, 3, 16, 1, 4, 4, 8, 2, FNO_F32);
  run_model(2, 64, 64, 3, 16, 0, 4, 4, 8, 1, FNO_F16);
  const long ck[][2] = {{1, 1}, {7, 31}, {96, 3721}, {5, 32}, {1280, 1000}, {3, 40000}};
  for (const auto &c : ck)
    for (fno_dtype_t dt : dts) run_checkpoint(c[0], c[1], dt);
  const long far[][2] = {{1L << 33, 1}, {(1L << 32) + 7, 31}, {512, 1L << 31}, {1L << 40, 1}, {1L << 35, 32}};
  for (const auto &c : far)
    for (fno_dtype_t dt : dts) run_checkpoint_far(c[0], c[1], dt);
  struct N { int B, C; long P; };
  const N nn[] = {{2, 4, 256}, {1, 1, 2}, {3, 7, 33}, {1, 16, 1000}, {20, 64, 4096}, {3, 48, 3721}, {2, 65, 100},
                  {2, 130, 64}, {1, 256, 777}, {1, 512, 65}, {300, 8, 5}, {1, 1, 1}, {5, 64, 1}, {9, 257, 1},
                  {700, 512, 1}, {3, 1025, 1}, {2, 3001, 1}, {2, 8192, 1}, {8192, 40, 1}};
  for (const N &c : nn)
    for (fno_dtype_t dt : dts)
      for (int kind = 0; kind < 2; ++kind) run_norm(c.B, c.C, c.P, kind, kind == 0 || c.C != 64, dt);
  // the largest rows and batches the header allows: nothing behind the buffers
  const N nf[] = {{1, 512, fno::kNormMaxPixels}, {65535, 100, 70}, {65535, 512, 31}, {4, 64, fno::kNormMaxPixels - 5}, {3, 9, (1L << 27) - 31},
                  {2000000000, 64, 1}, {134217728, 8192, 1}, {65535, 256, 65536}};
  for (const N &c : nf)
    for (int dt = 0; dt < 3; ++dt)
      for (int kind = 0; kind < 2; ++kind) trace_call("norm", dt, {kind, c.B, c.C, c.P});
  struct M { int B, I, O; long P; };
  const M mm[] = {{2, 4, 4, 256}, {1, 1, 1, 1}, {3, 5, 70, 33}, {2, 40, 72, 1001}, {1, 64, 64, 4096}, {1, 128, 128, 300},
                  {2, 128, 3, 100}, {1, 17, 33, 7}, {4, 32, 32, 1024}, {70, 8, 16, 500}};
  for (const M &c : mm)
    for (fno_dtype_t dt : dts)
      for (int k = 0; k < 4; ++k) run_mix(c.B, c.I, c.O, c.P, k & 1, (k & 2) != 0, dt);
  const M mf[] = {{1, 128, 128, fno::kMixTrainPixels}, {1024, 128, 128, fno::kMixTrainPixels}, {1 << 30, 3, 5, 64}, {1 << 29, 128, 128, 65},
                  {7, 33, 20, fno::kMixTrainPixels - 3}};
  for (const M &c : mf)
    for (int dt = 0; dt < 3; ++dt)
      for (int k = 0; k < 4; ++k) trace_call("mix", dt, {c.B, c.I, c.O, c.P, k & 1, k >> 1});
  struct D { int B, C; long P; };
  const D dd[] = {{1, 1, 1}, {2, 4, 256}, {3, 7, 33}, {5, 1001, 1}, {32, 64, 65536}, {4, 3, 3721}, {7, 130, 9}, {1, 1, 1L << 31},
                  {1 << 30, 1, 1024}, {15, 189, 2622}, {2000, 3, 3}, {1, 37, 5000}, {2, 8192, 1L << 26}, {65536, 4096, 4096}, {2000000000, 3, 5}};
  for (const D &c : dd)
    for (fno_dtype_t dt : dts) run_drop(c.B, c.C, c.P, dt);
  struct G { int B, C; long P; int G; };
  const G gg[] = {{2, 4, 256, 2}, {1, 1, 1, 1}, {1, 1, 2, 1}, {5, 64, 1, 8}, {3, 6, 2, 3}, {2, 48, 33, 3}, {1, 61, 97, 1}, {32, 64, 9, 16},
                  {3, 33, 1, 3}, {9, 257, 1, 1}, {1, 96, 1000, 3}, {2, 48, 3721, 3}, {1, 3, 70000, 1}, {2, 512, 300, 1}, {1, 4096, 20, 2}, {300, 40, 1, 5},
                  {1, 8192, 1, 1}, {2, 8192, 9, 4}, {20, 64, 65536, 8}, {16, 128, 16384, 32}, {8192, 1024, 1, 16},
                  {1, 8192, fno::kGnMaxPixels, 1}, {3, 5, fno::kGnMaxPixels - 3, 5}, {1 << 30, 4, 3, 1}, {1 << 28, 8, 511, 4}, {1 << 22, 1, 8200, 1}, {1 << 22, 16, 1500, 1},
                  {2, 8191, 65537, 1}, {1000000, 100, 70, 100}, {5, 61, 20000, 1}, {5, 4, 56935, 2}, {1, 3, 90001, 1}, {1, 2057, 9001, 1}, {134217728, 8192, 1, 8}};
  for (const G &c : gg)
    for (fno_dtype_t dt : dts)
      for (int last = 0; last < 2; ++last) run_gnorm(c.B, c.C, c.P, c.G, last, dt);
  struct X { int B, I, O; long P; };
  const X xx[] = {{1, 1, 1, 1}, {2, 4, 4, 256}, {3, 33, 70, 7}, {5, 200, 72, 1001}, {8192, 4096, 4096, 1}, {1, 8192, 8192, 1},
                  {32, 64, 64, 65536}, {16, 65536, 3, 1}, {2, 31, 129, 2}, {700, 96, 40, 1}, {1, 64, 512, 1L << 31},
                  {2147483647, 32, 64, 1}, {1 << 20, 17, 5, 2047},
                  {3, 1100, 70, 1}, {1, 4001, 300, 1}, {20, 1024, 31, 1}, {2, 1056, 16, 33}};
  for (const X &c : xx)
    for (fno_dtype_t dt : dts) run_mx4(c.B, c.I, c.O, c.P, dt);
  const long reports = check_reports();
  // the checker itself: spans past the end of a buffer must be reported
  {
    Buf x(64 * 2), A(4 * 2), y(64 * 2);
    std::fprintf(stderr, "self-test: three planted out-of-range spans follow\n");
    const long before = check_reports();
    fno::check_channel_mix(x.p, A.p, nullptr, nullptr, y.p, 1, 1, 4, 16, fno::DT_F16);  // in range
    EXPECT(check_reports() == before);
    fno::check_channel_mix(x.p, A.p, nullptr, nullptr, y.p, 1, 1, 4, 17, fno::DT_F16);  // y 4 elements short
    EXPECT(check_reports() == before + 1);
    fno::check_channel_mix(x.p, A.p, nullptr, nullptr, y.p, 1, 1, 5, 16, fno::DT_F16);  // A and y a row short
    EXPECT(check_reports() == before + 3);
  }
  {
    std::fprintf(stderr, "self-test: a norm's planted mistakes follow\n");
    const size_t n = (size_t)2 * 20 * 100 * 4;
    fno::NormArgs a{};
    a.eps = 1e-5f, a.B = 2, a.C = 20, a.P = 100, a.per = 4;
    a.x = check_reserve(n), a.v = check_reserve(n), a.y = check_reserve(n);
    long before = check_reports();
    auto more = [&](long k) {
      const bool hit = check_reports() - before >= (k ? 1 : 0) && (k || check_reports() == before);
      before = check_reports();
      return hit;
    };
    fno::check_norm(a, true, 1, fno::DT_F32, 256, 4, 0, 1, 3);  // as launched
    EXPECT(more(0));
    fno::check_norm(a, true, 1, fno::DT_F32, 256, 4, 0, 1, 2);  // a group of channels short
    EXPECT(more(1));
    fno::check_norm(a, true, 1, fno::DT_F32, 256, 4, 0, 1, 4);  // a group that has no channel
    EXPECT(more(1));
    fno::check_norm(a, true, 1, fno::DT_F16, 256, 4, 0, 2, 2);  // waves that are not there
    EXPECT(more(1));
    a.per = 2;
    fno::check_norm(a, true, 1, fno::DT_F32, 256, 4, 0, 1, 3);  // tiles left out
    EXPECT(more(1));
  }
  std::printf("launches checked: %ld, bounds reports: %ld, driver failures: %d\n", check_launches(), reports,
              n_fail);
  return (reports == 0 && n_fail == 0 && check_launches() > 0) ? 0 : 1;
}
