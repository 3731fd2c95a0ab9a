// block_checks.cpp - the bounds-check build's model of the block operators' launches
// (gnorm_kernels.hpp, drop.hip, mx4.hip, mx4_mix.hip), as launch_checks.cpp has those of the others. Host code only.

#include <algorithm>

#include "../gnorm.hpp"
#include "../mx4.hpp"

namespace fno {

namespace {

size_t es_of(int dtype) { return dtype == DT_F32 ? 4 : 2; }

struct Ctx {
  const char *name;
  void span(const char *what, const void *p, size_t n) const {
    if (n && (!p || !bounds::inside(p, n))) bounds::report(name, what);
  }
  void opt(const char *what, const void *p, size_t n) const {
    if (p) span(what, p, n);
  }
  void need(const char *what, bool ok) const {
    if (!ok) bounds::report(name, what);
  }
};

size_t values(const GnArgs &a) { return (size_t)a.B * a.C * a.P; }

void gn_spans(const Ctx &c, const GnArgs &a, bool bwd, bool out, int dtype) {
  const size_t es = es_of(dtype), n = values(a) * es, groups = (size_t)a.B * a.G;
  c.span("x", a.x, n);
  if (bwd) c.span("gy", a.gy, n);
  if (out && !(bwd && !a.gx)) c.span(bwd ? "gx" : "y", bwd ? a.gx : a.y, n);
  c.opt("weight", a.w, a.C * es);
  c.opt("bias", a.b, a.C * es);
  c.opt("step", a.drop.step, 8);
  if (bwd || out) c.opt("stats", a.stats, groups * 8);
  c.need("groups of whole channels", a.G >= 1 && a.Cg * a.G == a.C);
  c.need("threshold", a.drop.thr <= 65536);
}

}  // namespace

void check_drop(const DropArgs &a, int mode, int dtype) {
  const Ctx c{"fno_drop"};
  const size_t es = es_of(dtype), n = (size_t)a.B * a.C * a.P * es;
  const long V = dtype == DT_F32 ? 4 : 8, span = 1024, cpr = (a.n + V - 1) / V, total = a.rows * cpr;
  c.opt("x", a.x, n);
  c.span("v", a.v, n);
  c.span("y", a.y, n);
  c.opt("step", a.drop.step, 8);
  c.need("rows are the field", a.rows >= 1 && a.n >= 1 && a.rows * a.n == (long)a.B * a.C * a.P);
  // the chunks of the first and last workgroups, placed as the kernel does
  const long groups = (total + span - 1) / span;
  for (long g : {0L, 1L, groups / 2, groups - 2, groups - 1}) {
    if (g < 0 || g >= groups) continue;
    const long base = g * span, row0 = mode == 0 ? 0 : base / cpr, rem0 = base - row0 * cpr;
    const bool whole = mode == 0 ? (base + span) * V <= a.n : base + span <= total && a.n % V == 0;
    if (whole) {
      c.need("whole chunks inside the field", (base + span) * V <= a.rows * a.n);
      if (mode != 0) c.need("whole chunks where a flat field has them", base * V == row0 * a.n + rem0 * V);
    }
    const long tail = rem0 + span - 1, down = tail / cpr, end = a.rows * a.n;
    // rows that end inside a chunk: 16 bytes all the same where the workgroup's last chunk has them
    const bool wide = !whole && base + span <= total && (row0 + down) * a.n + (tail - down * cpr + 1) * V <= end;
    bool loads = true;
    for (long local = 0; local < span && base + local < total; ++local) {
      const long v = rem0 + local, d = mode == 0 ? 0 : cpr > span ? (v >= cpr ? 1 : 0) : (uint32_t)v / (uint32_t)cpr;
      const long k = v - d * cpr, at = whole ? (base + local) * V : (row0 + d) * a.n + k * V;
      loads = loads && at >= 0 && at + (whole || wide ? V : std::min(a.n - k * V, V)) <= end;
      loads = loads && k >= 0 && (whole || a.n - k * V > 0);  // a store of a row's own values
    }
    c.need("loads inside the field", loads);
    for (long local : {0L, 1L, 255L, 256L, 1022L, 1023L}) {
      if (base + local >= total) continue;
      const long v = rem0 + local, d = mode == 0 ? 0 : cpr > span ? (v >= cpr ? 1 : 0) : (uint32_t)v / (uint32_t)cpr;
      const long row = row0 + d, k = v - d * cpr;
      c.need("chunk in its row", row < a.rows && k >= 0 && k < cpr && row * cpr + k == base + local);
      if (mode == 2) {
        const long b0 = row0 / a.P, prem = row0 - b0 * a.P;
        c.need("sample of a row", prem + d < 1L << 32 && b0 + (prem + d) / a.P == row / a.P);
      }
    }
  }
}

void check_gnorm_small(const GnArgs &a, bool last, bool bwd, int T, int NC, int dtype) {
  const Ctx c{bwd ? "fno_gnorm_small backward" : "fno_gnorm_small"};
  gn_spans(c, a, bwd, true, dtype);
  const long V = dtype == DT_F32 ? 4 : 8, len = last ? a.Cg : a.P, rows = last ? a.P : a.Cg;
  const long cpr = (len + V - 1) / V, chunks = rows * cpr, groups = (long)a.B * a.G, n = (long)values(a);
  c.need("a team holds a group", chunks <= (long)T * NC && T <= 1024);
  c.need("groups in 31 bits", groups < 1L << 31);
  c.need("one pixel: channels last", last || a.P > 1);
  bool in = true, loads = true, params = true;
  for (long id : {0L, groups / 2, groups - 1}) {
    const long b = id / a.G, c0 = (id - b * a.G) * a.Cg, pitch = last ? a.C : a.P;
    const long first = last ? b * a.P * a.C + c0 : (b * a.C + c0) * a.P;
    for (long q = 0; q < (long)T * NC; ++q) {  // a lane's slots, those behind the group's last chunk too: they load it again
      const long qc = std::min(q, chunks - 1), row = (long)((uint64_t)(2 * qc) * ((0x80000000u + cpr - 1) / cpr) >> 32), k = (qc - row * cpr) * V;
      in = in && row == qc / cpr;
      const long nv = q < chunks ? std::min(len - k, V) : 0, at = first + row * pitch + k;
      in = in && at >= 0 && at + nv <= n;
      // the values that its load takes, by the kernel's three branches
      const long back = len % V != 0 && len >= V ? V - std::min(len - k, V) : 0, from = at - back;
      const long wide = len >= V || at + V <= n ? V : nv;
      loads = loads && from >= 0 && from + wide <= n;
      params = params && (last ? c0 + k + std::min(len - k, V) <= a.C : c0 + row < a.C);
    }
  }
  c.need("loads inside the field", loads);
  c.need("chunks inside the field", in);
  c.need("parameters of existing channels", params);
}

void check_gnorm_rows(const GnArgs &a, bool bwd, bool out, bool fold, bool params, int T, int dtype) {
  const Ctx c{bwd ? "fno_gnorm_rows backward" : "fno_gnorm_rows"};
  gn_spans(c, a, bwd, out, dtype);
  const long V = dtype == DT_F32 ? 4 : 8, cpr = (a.P + V - 1) / V, rows = (long)a.B * a.C;
  c.need("pieces cover the row", a.S >= 1 && a.per >= 1 && a.S * a.per >= cpr && (a.S - 1) * a.per < cpr);
  c.need("a row of lanes or a workgroup", T == 8 || T == 64 || T == 256);
  c.need("offsets of a row in 32 bits", cpr * V + 4L * T * V < 1L << 32);
  c.need("whole chunks inside the row", a.P / V * V <= a.P && a.P - (cpr - 1) * V >= 1);
  if (!out || fold) c.span("sums", a.part, (size_t)rows * a.S * 8);
  if (bwd && out && !fold) c.span("group sums", a.gsum, (size_t)a.B * a.G * 8);
  c.need("strides of the sums", a.sb == (long)a.C * a.S && a.sc == a.S && a.ss == 1);
  c.need("workgroups", a.main + (params ? 1 : 0) >= 1 && (long)a.main + (a.C + 7) / 8 < 1L << 24);
  if (fold) {
    c.need("no empty piece, a second pass", out && (a.S - 1) * a.per * V < a.P);
    c.need("a group's sums in 31 bits", (long)a.Cg * a.S + 256 < 1L << 31);
  }
  if (params) {
    c.need("behind a folded backward", fold && bwd);
    c.opt("gw", a.gw, a.C * es_of(dtype));
    c.opt("gb", a.gb, a.C * es_of(dtype));
    c.need("a channel's sums in 32 bits", (long)a.B * a.S + 256 < 1L << 32);
  }
}

void check_gnorm_cols(const GnArgs &a, bool bwd, bool out, bool runs, int dtype) {
  const Ctx c{bwd ? "fno_gnorm_cols backward" : "fno_gnorm_cols"};
  gn_spans(c, a, bwd, out, dtype);
  const long V = dtype == DT_F32 ? 4 : 8, cpr = (a.C + V - 1) / V, rows = runs ? a.B * a.P : a.P;
  c.need("pieces cover the rows", a.S >= 1 && a.per >= 1 && a.S * a.per >= rows && (a.S - 1) * a.per < rows);
  for (long kb = 0; kb < cpr; kb += 256) {
    const long kn = std::min(256L, cpr - kb), PL = 256 / kn;
    c.need("lanes of a row", PL >= 1 && ((PL - 1) * V + V - 1) * kn + kn - 1 < 256 * V && (kb + kn - 1) * V < a.C);
    // the loads of a lane: 16 bytes of its channels in the rows below `safe`, its own values in the others
    bool loads = true;
    const long all = (long)a.B * a.P, units = runs ? a.S : (long)a.B * a.S;
    for (long u : {0L, units / 2, units - 1}) {
      const long b = runs ? 0 : u / a.S, p0 = runs ? u * a.per : (u - b * a.S) * a.per;
      const long r0 = runs ? p0 : b * a.P + p0, r1 = runs ? std::min(all, p0 + a.per) : b * a.P + std::min(a.P, p0 + a.per);
      loads = loads && r0 >= 0 && r0 < r1 && r1 <= all;
      for (long kl = 0; kl < kn; ++kl) {
        const long c0 = (kb + kl) * V, nv = std::min(V, a.C - c0);
        const long safe = nv == V ? r1 : all * a.C < V + c0 ? 0 : std::min(r1, (all * a.C - V - c0) / a.C + 1);
        loads = loads && nv >= 1 && safe <= r1 && (safe <= r0 || (safe - 1) * a.C + c0 + V <= all * a.C);
      }
    }
    c.need("loads inside the field", loads);
  }
  if (!out) c.span("sums", a.part, (size_t)(runs ? 1 : a.B) * a.S * a.C * 8);
  if (!out && a.whole) {
    c.need("a workgroup has all channels", cpr <= 256 && !runs);
    c.span("groups' sums", a.gpart, (size_t)a.B * a.S * a.G * 8);
  }
  if (bwd && out) c.span("group sums", a.gsum, (size_t)a.B * a.G * 8);
  c.need("strides of the sums", a.sb == (runs ? 0 : (long)a.C * a.S) && a.sc == 1 && a.ss == a.C);
}

void check_gnorm_join(const GnArgs &a, bool bwd, bool group, int samples, int dtype) {
  const Ctx c{bwd ? "fno_gnorm_join backward" : "fno_gnorm_join"};
  const size_t groups = (size_t)a.B * a.G, es = es_of(dtype);
  c.need("something to join", group || samples);
  if (group) {
    c.span("sums", a.part, (size_t)a.B * a.C * a.S * 8);
    if (a.whole) c.span("groups' sums", a.gpart, (size_t)a.B * a.S * a.G * 8);
    c.span(bwd ? "group sums" : "stats", bwd ? a.gsum : a.stats, groups * 8);
    c.need("last sum of a sample", (a.C - 1) * a.sc + (a.S - 1) * a.ss < a.sb && a.sb == (long)a.C * a.S);
    const long piece = a.last ? a.per : a.per * (dtype == DT_F32 ? 4 : 8);
    c.need("no empty piece", (a.S - 1) * piece < a.P);
    c.need("a group's sums in 32 bits", (long)a.Cg * a.S + 4096 < 1L << 32);
  }
  if (samples) {
    c.opt("gw", a.gw, a.C * es);
    c.opt("gb", a.gb, a.C * es);
    c.span("sums", a.part, (size_t)samples * a.S * a.C * 8);
    c.need("last sum", (samples - 1) * a.sb + (a.C - 1) * a.sc + (a.S - 1) * a.ss < (long)samples * a.S * a.C);
    c.need("a channel's sums in 32 bits", (long)samples * a.S + 512 < 1L << 32);
  }
}

void check_mx4(const Mx4Args &a, bool pack, int dtype) {
  const Ctx c{pack ? "fno_mx4_pack" : "fno_mx4_unpack"};
  const long rows = a.B * a.P;
  c.span("field", pack ? a.x : a.y, (size_t)a.B * a.C * a.P * es_of(dtype));
  c.span("codes", a.codes, (size_t)rows * a.nb * 16);
  c.span("scales", a.exps, (size_t)rows * a.nb);
  c.need("blocks cover the row", a.nb == (a.C + 31) / 32);
  c.need("codes 16-byte aligned", ((uintptr_t)a.codes & 15) == 0);
  c.need("units of a row in 32 bits, rows in 31", 4 * a.nb + 1024 < 1L << 31 && rows <= 1L << 31);
  if (a.P > 1) {  // the lanes of the first and last workgroups, placed as the kernel does
    const long np = dtype == DT_F32 ? 2 : 4, ppr = (a.P + np - 1) / np, total = a.B * ppr;
    for (long q : {0L, ppr - 1, total - 1}) {
      const long b = q / ppr, p = (q - b * ppr) * np, n = std::min(np, a.P - p);
      c.need("pixels of a lane", b < a.B && p >= 0 && n >= 1 && p + n <= a.P);
    }
    c.need("lanes for the grid", total + 256 < 1L << 32);
  }
}

void check_mx4_mix(const Mx4MixArgs &a, int dtype) {
  const Ctx c{"fno_mx4_mix"};
  const size_t es = es_of(dtype), n = (size_t)a.B * a.O * a.P * es, rows = (size_t)a.B * a.P;
  c.span("codes of x", a.xq, rows * a.nb * 16);
  c.span("scales of x", a.xe, rows * a.nb);
  c.span("codes of A", a.aq, (size_t)a.O * a.nb * 16);
  c.span("scales of A", a.ae, (size_t)a.O * a.nb);
  c.opt("bias", a.bias, a.O * es);
  c.opt("add", a.add, n);
  c.span("y", a.y, n);
  c.need("blocks cover the row", a.nb == (a.I + 31) / 32);
  c.need("codes 16-byte aligned", (((uintptr_t)a.xq | (uintptr_t)a.aq) & 15) == 0);
  if (a.nb >= 32) {  // what a lane of fno_mx4_mix_few reads of its two rows: whole and clamped steps of four blocks
    const bool steps4 = a.nb % 4 == 0;
    const long steps = (a.nb + 3) / 4, per = (steps + 7) / 8;
    bool codes = true, scales = true;
    for (long wave = 0; wave < 8; ++wave) {
      const long k0 = wave * per, k1 = std::min(steps, k0 + per);
      for (long k = k0; k < k1; k += 4)
        for (long u = 0; u < 4; ++u)
          for (long quad = 0; quad < 4; ++quad) {
            const long step = std::min(k + u, k1 - 1), kb = 4 * step + quad, kc = steps4 ? kb : std::min(kb, a.nb - 1);
            codes = codes && step >= k0 && kc < a.nb;
            scales = scales && (steps4 ? (k + 4 <= steps ? 4 * k + 16 : 4 * step + 4) <= a.nb : kc < a.nb);
          }
    }
    c.need("few rows: codes inside the row", codes);
    c.need("few rows: scales inside the row", scales);
  }
  if (a.nb % 4 == 0 && a.nb >= 16) {  // what fno_mx4_mix_tiles fetches of a row, in bytes, and its LDS reads
    const long stages = (a.nb + 7) / 8, pairs = (stages + 1) / 2;
    const size_t past = 8 * stages > a.nb ? 64 : 0;  // half a stage's units behind the last row
    c.span("codes of x as fetched", a.xq, rows * a.nb * 16 + past);
    c.span("codes of A as fetched", a.aq, (size_t)a.O * a.nb * 16 + past);
    for (long pair : {0L, pairs - 1})
      for (long d = 0; d < 4; ++d) c.need("scales inside the row", std::min(16 * pair + 4 * d, a.nb - 4) + 4 <= a.nb);
    c.need("offsets of a tile in 32 bits", 256L * a.nb * 16 + 128 < 1L << 31);
  }
}

}  // namespace fno
