// Host side of the C ABI, continued: the operators around the step that work on a model's gradients and
// activations. Arguments are validated completely before the first HIP call, as in qgalore.hip.
#include <algorithm>
#include <memory>
#include <new>

#include "qg_host.hpp"

using namespace qg_host;

// ================================================ gradient norm and clipping ===

namespace {

int64_t dtype_bytes(int32_t dtype) { return dtype == QG_DTYPE_BF16 ? 2 : 4; }

constexpr int64_t kClipMaxN = int64_t(1) << 40;

qg_status check_clip(const qg_clip_desc* d, const qg_grad* grads, int32_t count, bool clip) {
  if (!d || !grads) return QG_ERR_NULL;
  if (count < 1 || count > 65536) return QG_ERR_ARG;
  if ((d->kind != QG_GRAD_L2 && d->kind != QG_GRAD_MAX) ||
      (d->zero_nonfinite != 0 && d->zero_nonfinite != 1))
    return QG_ERR_ARG;
  if (clip && (!finite(d->max_norm) || d->max_norm < 0.f || !finite(d->eps) || d->eps < 0.f))
    return QG_ERR_ARG;
  for (int32_t k = 0; k < count; ++k) {
    const qg_grad& g = grads[k];
    if (g.dtype != QG_DTYPE_BF16 && g.dtype != QG_DTYPE_FP32) return QG_ERR_ARG;
    if (g.n < 0 || g.n > kClipMaxN) return QG_ERR_SHAPE;
    if (g.n == 0) continue;
    if (!g.g || (clip && !g.out)) return QG_ERR_NULL;
    if (!aligned(g.g, dtype_bytes(g.dtype)) || (clip && !aligned(g.out, dtype_bytes(g.dtype))))
      return QG_ERR_ALIGN;
  }
  return QG_OK;
}

// Whether a result lies over anything but the gradient that it is made from: the spans by their start,
// each against the furthest end of those before it.
struct ClipSpan {
  uintptr_t from, to;
  bool written;
};
qg_status clip_clash(const qg_grad* grads, int32_t count, std::initializer_list<ClipSpan> more) {
  const std::unique_ptr<ClipSpan[]> v(new (std::nothrow) ClipSpan[2 * (size_t)count + more.size()]);
  if (!v) {
    g_last_error = "no host memory for the list of gradients";
    return QG_ERR_HIP;
  }
  ClipSpan* last = std::copy(more.begin(), more.end(), v.get());
  for (int32_t k = 0; k < count; ++k) {
    const qg_grad& g = grads[k];
    if (g.n == 0) continue;
    const uintptr_t bytes = (uintptr_t)(g.n * dtype_bytes(g.dtype));
    const uintptr_t in = reinterpret_cast<uintptr_t>(g.g), out = reinterpret_cast<uintptr_t>(g.out);
    *last++ = {out, out + bytes, true};
    if (in != out) *last++ = {in, in + bytes, false};
  }
  std::sort(v.get(), last, [](const ClipSpan& a, const ClipSpan& b) { return a.from < b.from; });
  uintptr_t end = 0, written = 0;
  for (const ClipSpan* s = v.get(); s != last; ++s) {
    if (s->from < (s->written ? end : written)) return QG_ERR_ARG;
    end = std::max(end, s->to);
    if (s->written) written = std::max(written, s->to);
  }
  return QG_OK;
}
ClipSpan clip_span(const void* p, int64_t bytes, bool written) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, p ? a + (uintptr_t)bytes : a, written};
}

// f(args) for each launch: up to kClipTensors tensors and a number of chunks that fits 31 bits.
template <class F>
hipError_t clip_launches(qg::ClipArgs& a, const qg_grad* grads, int32_t count, F&& f) {
  int32_t k = 0;
  do {
    a.count = 0;
    a.first[0] = 0;
    a.in_place = 1;
    std::memset(a.bf16, 0, sizeof(a.bf16));
    for (; k < count && a.count < qg::kClipTensors; ++k) {
      const qg_grad& g = grads[k];
      if (g.n == 0) continue;
      const int64_t chunks = a.first[a.count] + cdiv(g.n, qg::kClipChunk);
      if (chunks > kMaxDim) break;
      a.t[a.count] = {g.g, g.out, g.n};
      a.in_place &= g.g == g.out;
      if (g.dtype == QG_DTYPE_BF16) a.bf16[a.count >> 5] |= 1u << (a.count & 31);
      a.first[++a.count] = (uint32_t)chunks;
    }
    const hipError_t e = f();
    if (e != hipSuccess) return e;
  } while (k < count);
  return hipSuccess;
}

qg::ClipArgs clip_args(const qg_clip_desc* d) {
  qg::ClipArgs a;
  std::memset(&a, 0, sizeof(a));
  a.part = static_cast<double*>(d->workspace);
  a.kind = d->kind;
  a.zero = d->zero_nonfinite;
  a.max_norm = d->max_norm;
  a.eps = d->eps;
  return a;
}

// The first pass: every launch's partial results.
hipError_t clip_partials(qg::ClipArgs& a, const qg_grad* grads, int32_t count, hipStream_t s) {
  return clip_launches(a, grads, count, [&] {
    const hipError_t e = qg::launch_grad_norm(a, s);
    a.filled = std::max(a.filled, (int32_t)qg::clip_grid(a.first[a.count]));
    a.slots = a.filled;
    return e;
  });
}

constexpr int64_t kClipBytes = qg::kClipSlots * (int64_t)sizeof(double);

}  // namespace

extern "C" size_t qgalore_grad_workspace_bytes(void) { return (size_t)kClipBytes; }

extern "C" qg_status qgalore_grad_norm(const qg_clip_desc* d, const qg_grad* grads, int32_t count,
                                       float* norm_out, double* total_out) {
  qg_status st = check_clip(d, grads, count, false);
  if (st != QG_OK) return st;
  if (!norm_out && !total_out) return QG_ERR_NULL;
  if (!aligned(norm_out, 4) || !aligned(total_out, 8)) return QG_ERR_ALIGN;
  if ((st = check_scratch(d->workspace, d->workspace_bytes, kClipBytes)) != QG_OK) return st;
  if (clash({norm_out, 4}, {{total_out, 8}, {d->workspace, kClipBytes}}) ||
      clash({total_out, 8}, {{d->workspace, kClipBytes}}))
    return QG_ERR_ARG;
  for (int32_t k = 0; k < count; ++k) {   // the results are written while no gradient is read
    const Span g{grads[k].n ? grads[k].g : nullptr, grads[k].n * dtype_bytes(grads[k].dtype)};
    if (clash({d->workspace, kClipBytes}, {g}) || clash({norm_out, 4}, {g}) ||
        clash({total_out, 8}, {g}))
      return QG_ERR_ARG;
  }
  if ((st = device_present()) != QG_OK) return st;
  qg::ClipArgs a = clip_args(d);
  const hipStream_t s = static_cast<hipStream_t>(d->stream);
  hipError_t e = clip_partials(a, grads, count, s);
  if (e == hipSuccess) {
    a.norm_out = norm_out;
    a.total_out = total_out;
    e = qg::launch_grad_total(a, s);
  }
  return e == hipSuccess ? QG_OK : hip_fail(e, "gradient norm kernels");
}

extern "C" qg_status qgalore_grad_clip(const qg_clip_desc* d, const qg_grad* grads, int32_t count,
                                       const double* total, float* norm_out) {
  qg_status st = check_clip(d, grads, count, true);
  if (st != QG_OK) return st;
  if (!aligned(norm_out, 4) || !aligned(total, 8)) return QG_ERR_ALIGN;
  if (!total && (st = check_scratch(d->workspace, d->workspace_bytes, kClipBytes)) != QG_OK)
    return st;
  const ClipSpan scratch = clip_span(total ? nullptr : d->workspace, kClipBytes, true);
  if ((st = clip_clash(grads, count, {scratch, clip_span(total, 8, false),
                                      clip_span(norm_out, 4, true)})) != QG_OK)
    return st;
  if ((st = device_present()) != QG_OK) return st;
  qg::ClipArgs a = clip_args(d);
  a.total = total;
  const hipStream_t s = static_cast<hipStream_t>(d->stream);
  hipError_t e = total ? hipSuccess : clip_partials(a, grads, count, s);
  if (e == hipSuccess) {
    a.norm_out = norm_out;
    e = clip_launches(a, grads, count, [&] {
      const hipError_t r = qg::launch_grad_scale(a, s);
      a.norm_out = nullptr;
      return r;
    });
  }
  return e == hipSuccess ? QG_OK : hip_fail(e, "gradient clipping kernels");
}

// ============================================== norms around a block, gate and scales ===

namespace {

qg_status check_resnorm(const qg_resnorm_desc* d, bool gate) {
  if (d->T < 1 || d->n < 1 || d->n > qg::kNormMaxN || d->T > kMaxDim / d->n) return QG_ERR_SHAPE;
  if (gate && d->per < 1) return QG_ERR_SHAPE;
  if (!finite(d->eps) || d->eps < 0.f || !finite(d->alpha) || (d->center != 0 && d->center != 1) ||
      (d->dtype != QG_DTYPE_BF16 && d->dtype != QG_DTYPE_FP32) ||
      d->gate_act < QG_GATE_IDENTITY || d->gate_act > QG_GATE_TANH)
    return QG_ERR_ARG;
  return QG_OK;
}

// Tokens for each row of the gate; one without a gate, and no more than there are.
int64_t res_per(const qg_resnorm_desc* d, bool gate) {
  return gate ? std::min(d->per, d->T) : 1;
}

// The workspace: two means of each long row, a row of each parameter's sums for every workgroup, and the
// gate's parts.
int64_t res_mean_bytes(const qg_resnorm_desc* d) {
  return d->n > qg::kResLong ? round_up(d->T * (int64_t)sizeof(float2), 256) : 0;
}
int64_t res_sum_bytes(const qg_resnorm_desc* d, const qg::ResSplit& s) {
  return s.slabs > 1 ? round_up((int64_t)s.slabs * d->n * 4, 256) : 0;
}
int64_t res_bytes(const qg_resnorm_desc* d, bool gate) {
  const qg::ResSplit s = qg::res_split(d->T, d->n, res_per(d, gate));
  return res_mean_bytes(d) + qg::kResSums * res_sum_bytes(d, s) +
         (s.parts > 1 ? round_up((int64_t)s.strands * d->n * 4, 256) : 0);
}

qg::ResArgs res_args(const qg_resnorm_desc* d, const qg_resnorm_params* p) {
  qg::ResArgs a;
  std::memset(&a, 0, sizeof(a));
  a.g1 = p->gamma1;
  a.b1 = p->gamma1 ? p->beta1 : nullptr;
  a.g2 = p->gamma2;
  a.b2 = p->gamma2 ? p->beta2 : nullptr;
  a.rho = p->rho;
  a.z = p->z;
  a.T = d->T;
  a.n = d->n;
  a.per = res_per(d, p->z != nullptr);
  a.alpha = d->alpha;
  a.eps = d->eps;
  a.bf16 = d->dtype == QG_DTYPE_BF16;
  a.center = d->center;
  a.act = d->gate_act;
  return a;
}

bool all_aligned(std::initializer_list<const void*> ps, size_t a) {
  for (const void* p : ps)
    if (!aligned(p, a)) return false;
  return true;
}

}  // namespace

extern "C" size_t qgalore_resnorm_bwd_workspace_bytes(const qg_resnorm_desc* d) {
  if (!d || check_resnorm(d, false) != QG_OK) return 0;
  return (size_t)std::max(res_bytes(d, false), d->per < 1 ? 0 : res_bytes(d, true));
}

extern "C" qg_status qgalore_resnorm_fwd(const qg_resnorm_desc* d, const qg_resnorm_params* p,
                                         const void* u, const void* x, void* h, void* y,
                                         float* stats) {
  if (!d || !p || !u || !x || !h || !stats || (p->gamma2 != nullptr) != (y != nullptr))
    return QG_ERR_NULL;
  qg_status st = check_resnorm(d, p->z != nullptr);
  if (st != QG_OK) return st;
  qg::ResArgs a = res_args(d, p);
  if (!all_aligned({u, x, h, y, a.z, a.g1, a.b1, a.g2, a.b2, a.rho}, 16) || !aligned(stats, 4))
    return QG_ERR_ALIGN;
  const int64_t bytes = d->T * d->n * dtype_bytes(d->dtype), vec = d->n * 4;
  const Span su{u, bytes}, sx{x, bytes}, sh{h, bytes}, sy{y, bytes}, ss{stats, d->T * 16},
      sz{a.z, cdiv(d->T, a.per) * d->n * dtype_bytes(d->dtype)}, g1{a.g1, vec}, b1{a.b1, vec},
      g2{a.g2, vec}, b2{a.b2, vec}, rho{a.rho, vec};
  // a row is in registers before it is written, so h and y may lie over u and x
  for (const Span& out : {sh, sy})
    if ((out.p != u && clash(out, {su})) || (out.p != x && clash(out, {sx})) ||
        clash(out, {sz, g1, b1, g2, b2, rho, ss}))
      return QG_ERR_ARG;
  if (clash(sh, {sy}) || clash(ss, {su, sx, sz, g1, b1, g2, b2, rho})) return QG_ERR_ARG;
  if ((st = device_present()) != QG_OK) return st;
  a.u = a.safe = u;
  a.x = x;
  a.h = h;
  a.y = y;
  a.stats_out = stats;
  const hipError_t e = qg::launch_resnorm_fwd(a, static_cast<hipStream_t>(d->stream));
  return e == hipSuccess ? QG_OK : hip_fail(e, "residual norm forward kernel");
}

extern "C" qg_status qgalore_resnorm_bwd(const qg_resnorm_desc* d, const qg_resnorm_params* p,
                                         const void* dh, const void* dy, const void* u,
                                         const void* h, const float* stats,
                                         const qg_resnorm_grads* g) {
  if (!d || !p || !g || !stats || !g->du || !g->dx) return QG_ERR_NULL;
  const bool norm1 = p->gamma1 != nullptr, norm2 = p->gamma2 != nullptr;
  if (!norm1 && !p->z && !p->rho)
    u = nullptr;   // no gradient depends on it
  else if (!u)
    return QG_ERR_NULL;
  if ((norm2 && (!h || !dy)) || (p->z != nullptr) != (g->dz != nullptr) ||
      (p->rho != nullptr) != (g->drho != nullptr) || norm1 != (g->dgamma1 != nullptr) ||
      norm2 != (g->dgamma2 != nullptr))
    return QG_ERR_NULL;
  qg_status st = check_resnorm(d, p->z != nullptr);
  if (st != QG_OK) return st;
  // a beta's gradient without its norm is refused as one that is not wanted
  if ((!norm1 && g->dbeta1) || (!norm2 && g->dbeta2)) return QG_ERR_ARG;
  qg::ResArgs a = res_args(d, p);
  if (!norm2) dy = h = nullptr;
  if (!all_aligned({dh, dy, u, h, a.z, a.g1, a.b1, a.g2, a.rho, g->du, g->dx, g->dz, g->drho,
                    g->dgamma1, g->dbeta1, g->dgamma2, g->dbeta2}, 16) ||
      !aligned(stats, 4))
    return QG_ERR_ALIGN;
  const int64_t need = res_bytes(d, p->z != nullptr);
  if ((st = check_scratch(d->workspace, d->workspace_bytes, need)) != QG_OK) return st;
  const int64_t bytes = d->T * d->n * dtype_bytes(d->dtype), vec = d->n * 4;
  const int64_t zb = cdiv(d->T, a.per) * d->n * dtype_bytes(d->dtype);
  const Span in[] = {{dh, bytes}, {dy, bytes}, {u, bytes}, {h, bytes}, {a.z, zb}, {a.g1, vec},
                     {a.b1, vec}, {a.g2, vec}, {a.rho, vec}, {stats, d->T * 16}};
  const Span out[] = {{g->du, bytes}, {g->dx, bytes}, {g->dz, zb}, {g->drho, vec},
                      {g->dgamma1, vec}, {g->dbeta1, vec}, {g->dgamma2, vec}, {g->dbeta2, vec},
                      {need ? d->workspace : nullptr, need}};
  for (const Span& o : out) {
    for (const Span& i : in) {
      const bool may = o.p == i.p && ((o.p == g->dx && i.p == dh) ||
                                      (o.p == g->du && (i.p == dy || i.p == u)));
      if (!may && clash(o, {i})) return QG_ERR_ARG;
    }
    for (const Span& q : out)
      if (&q != &o && clash(o, {q})) return QG_ERR_ARG;
  }
  if ((st = device_present()) != QG_OK) return st;
  a.dh = dh;
  a.dy = dy;
  a.u = u;
  a.safe = u ? u : g->dx;   // what is read there is not used
  a.h_in = h;
  a.stats = stats;
  a.du = g->du;
  a.dx = g->dx;
  a.dz = g->dz;
  a.split = qg::res_split(d->T, d->n, a.per);
  float* const sums[] = {g->drho, g->dgamma1, g->dbeta1, g->dgamma2, g->dbeta2};
  char* ws = static_cast<char*>(d->workspace);
  a.row_means = reinterpret_cast<float2*>(ws);
  ws += res_mean_bytes(d);
  for (int k = 0; k < qg::kResSums; ++k) {
    a.sum[k] = sums[k];
    if (!sums[k]) continue;
    a.part[k] = a.split.slabs > 1 ? reinterpret_cast<float*>(ws) : sums[k];
    ws += res_sum_bytes(d, a.split);
  }
  if (a.z && a.split.parts > 1) a.part_z = reinterpret_cast<float*>(ws);
  const hipError_t e = qg::launch_resnorm_bwd(a, static_cast<hipStream_t>(d->stream));
  return e == hipSuccess ? QG_OK : hip_fail(e, "residual norm backward kernels");
}

// ================================================ FP8 with a scale for 128 values ===

namespace {

constexpr int64_t kF8MaxK = int64_t(1) << 20;

// Bytes of a matrix's codes and scales.
int64_t f8_codes(int64_t rows, int64_t cols) { return rows * qg::f8_pitch(cols); }
int64_t f8_scales(int64_t rows, int64_t cols, bool block) {
  return qg::f8_blocks(cols) * (block ? qg::f8_blocks(rows) : rows) * 4;
}
bool f8_size(int64_t rows, int64_t cols) {
  return rows >= 1 && cols >= 1 && rows <= kMaxDim && cols <= kMaxDim && rows * cols <= kMaxDim &&
         f8_codes(rows, cols) <= kMaxDim && f8_codes(cols, rows) <= kMaxDim;
}
// Bytes of a matrix of values within the limit.
bool f8_value_bytes(int64_t rows, int64_t cols, int64_t each) {
  return rows * cols <= kMaxDim / each;
}
bool f8_format(int32_t f) { return f == QG_FP8_E4M3 || f == QG_FP8_E5M2; }

qg_status check_f8_mm(int64_t M, int64_t N, int64_t K, int64_t each) {
  return f8_size(M, K) && f8_size(N, K) && M <= kMaxDim / N && f8_value_bytes(M, N, each) &&
                 K <= kF8MaxK
             ? QG_OK
             : QG_ERR_SHAPE;
}

qg::F8Quant f8_quant(const void* src, int64_t rows, int64_t cols, int32_t source, int32_t format) {
  qg::F8Quant a;
  std::memset(&a, 0, sizeof(a));
  a.src = src;
  a.rows = rows;
  a.cols = cols;
  a.source = source;
  a.format = format;
  return a;
}

// What a linear layer keeps in its workspace: the quantized tokens along their rows, and behind them along
// their columns.
// Behind those lie the parts of its products, which run one after another.
struct F8Scratch {
  int64_t off_s, off_qt, off_st, rows, both;   // bytes of the first alone, and of both
};
F8Scratch f8_scratch(int64_t T, int64_t c) {
  F8Scratch z;
  z.off_s = round_up(f8_codes(T, c), 256);
  z.rows = z.off_qt = z.off_s + round_up(f8_scales(T, c, false), 256);
  z.off_st = z.off_qt + round_up(f8_codes(c, T), 256);
  z.both = z.off_st + round_up(f8_scales(c, T, false), 256);
  return z;
}
int64_t f8_fwd_bytes(int64_t T, int64_t m, int64_t n) {
  return qg::f8_few_fits(T, n) ? 0 : f8_scratch(T, n).rows + qg::f8_part_bytes(T, m, n);
}
int64_t f8_bwd_bytes(int64_t T, int64_t m, int64_t n) {
  return f8_scratch(T, m).both + std::max(qg::f8_part_bytes(T, n, m), qg::f8_part_bytes(m, n, T));
}
qg_status check_f8_linear(int64_t T, int64_t m, int64_t n, bool backward) {
  qg_status st = check_f8_mm(T, m, n, 2);
  if (st == QG_OK && !f8_value_bytes(T, n, 2)) st = QG_ERR_SHAPE;
  if (st != QG_OK || !backward) return st;
  if ((st = check_f8_mm(T, n, m, 2)) != QG_OK) return st;
  return check_f8_mm(m, n, T, 2);
}

}  // namespace

extern "C" qg_status qgalore_fp8_quantize(const qg_fp8_desc* d, const void* src,
                                          const float* src_scale, uint8_t* Q, float* S,
                                          uint8_t* Qt, float* St) {
  if (!d || !src || (!Q && !Qt) || !Q != !S || !Qt != !St) return QG_ERR_NULL;
  if (!f8_format(d->format) || d->source < QG_FP8_FROM_BF16 || d->source > QG_FP8_FROM_INT8 ||
      (d->block != 0 && d->block != 1))
    return QG_ERR_ARG;
  const bool int8 = d->source == QG_FP8_FROM_INT8;
  if (int8 != (src_scale != nullptr)) return QG_ERR_NULL;
  const int64_t each = int8 ? 1 : d->source == QG_FP8_FROM_BF16 ? 2 : 4;
  if (!f8_size(d->rows, d->cols) || !f8_value_bytes(d->rows, d->cols, each)) return QG_ERR_SHAPE;
  if (!all_aligned({src, Q, Qt}, 16) || !all_aligned({src_scale, S, St}, 4)) return QG_ERR_ALIGN;
  const int64_t numel = d->rows * d->cols;
  const Span in{src, numel * each}, is{src_scale, cdiv(numel, qg::kGroup) * 4},
      q{Q, f8_codes(d->rows, d->cols)}, s{S, f8_scales(d->rows, d->cols, d->block)},
      qt{Qt, f8_codes(d->cols, d->rows)}, st{St, f8_scales(d->cols, d->rows, d->block)};
  if (clash(q, {in, is, s, qt, st}) || clash(s, {in, is, qt, st}) || clash(qt, {in, is, st}) ||
      clash(st, {in, is}))
    return QG_ERR_ARG;
  qg_status r;
  if ((r = device_present()) != QG_OK) return r;
  qg::F8Quant a = f8_quant(src, d->rows, d->cols, d->source, d->format);
  a.src_scale = src_scale;
  a.q = Q;
  a.s = S;
  a.qt = Qt;
  a.st = St;
  a.block = d->block;
  const hipError_t e = qg::launch_f8_quantize(a, static_cast<hipStream_t>(d->stream));
  return e == hipSuccess ? QG_OK : hip_fail(e, "FP8 quantization kernel");
}

extern "C" qg_status qgalore_fp8_dequantize(const qg_fp8_desc* d, const uint8_t* Q, const float* S,
                                            void* out) {
  if (!d || !Q || !S || !out) return QG_ERR_NULL;
  if (!f8_format(d->format) || (d->source != QG_FP8_FROM_BF16 && d->source != QG_FP8_FROM_FP32) ||
      (d->block != 0 && d->block != 1))
    return QG_ERR_ARG;
  const int64_t each = d->source == QG_FP8_FROM_BF16 ? 2 : 4;
  if (!f8_size(d->rows, d->cols) || !f8_value_bytes(d->rows, d->cols, each)) return QG_ERR_SHAPE;
  if (!all_aligned({Q, out}, 16) || !aligned(S, 4)) return QG_ERR_ALIGN;
  if (clash({out, d->rows * d->cols * each},
            {{Q, f8_codes(d->rows, d->cols)}, {S, f8_scales(d->rows, d->cols, d->block)}}))
    return QG_ERR_ARG;
  qg_status r;
  if ((r = device_present()) != QG_OK) return r;
  const qg::F8Values a{Q, S, out, d->rows, d->cols, d->format, d->block,
                       d->source == QG_FP8_FROM_BF16};
  const hipError_t e = qg::launch_f8_dequantize(a, static_cast<hipStream_t>(d->stream));
  return e == hipSuccess ? QG_OK : hip_fail(e, "FP8 dequantization kernel");
}

extern "C" size_t qgalore_fp8_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return check_f8_mm(M, N, K, 2) == QG_OK ? (size_t)qg::f8_part_bytes(M, N, K) : 0;
}

extern "C" qg_status qgalore_fp8_matmul(const qg_fp8_mm_desc* d, const uint8_t* A, const float* SA,
                                        const uint8_t* B, const float* SB, void* out) {
  if (!d || !A || !SA || !B || !SB || !out) return QG_ERR_NULL;
  if (!f8_format(d->a_format) || (d->b_block != 0 && d->b_block != 1) ||
      (d->out_dtype != QG_DTYPE_BF16 && d->out_dtype != QG_DTYPE_FP32))
    return QG_ERR_ARG;
  const int64_t each = dtype_bytes(d->out_dtype);
  qg_status st = check_f8_mm(d->M, d->N, d->K, each);
  if (st != QG_OK) return st;
  if (!all_aligned({A, B, out}, 16) || !all_aligned({SA, SB}, 4)) return QG_ERR_ALIGN;
  const int64_t need = d->workspace ? qg::f8_part_bytes(d->M, d->N, d->K) : 0;
  if ((st = check_scratch(d->workspace, d->workspace_bytes, need)) != QG_OK) return st;
  const Span ws{need ? d->workspace : nullptr, need}, in[] = {
      {A, f8_codes(d->M, d->K)}, {SA, f8_scales(d->M, d->K, false)},
      {B, f8_codes(d->N, d->K)}, {SB, f8_scales(d->N, d->K, d->b_block)}};
  if (clash({out, d->M * d->N * each}, {ws, in[0], in[1], in[2], in[3]}) ||
      clash(ws, {in[0], in[1], in[2], in[3]}))
    return QG_ERR_ARG;
  if ((st = device_present()) != QG_OK) return st;
  const qg::F8Mm a{A, SA, B, SB, out, nullptr, d->M, d->N, d->K, d->a_format, d->b_block,
                   d->out_dtype == QG_DTYPE_BF16, need ? static_cast<float*>(d->workspace) : nullptr};
  const hipError_t e = qg::launch_f8_mm(a, static_cast<hipStream_t>(d->stream));
  return e == hipSuccess ? QG_OK : hip_fail(e, "FP8 product kernel");
}

extern "C" size_t qgalore_fp8_linear_fwd_workspace_bytes(int64_t T, int64_t m, int64_t n) {
  return check_f8_linear(T, m, n, false) == QG_OK ? (size_t)f8_fwd_bytes(T, m, n) : 0;
}
extern "C" size_t qgalore_fp8_linear_bwd_workspace_bytes(int64_t T, int64_t m, int64_t n) {
  return check_f8_linear(T, m, n, true) == QG_OK ? (size_t)f8_bwd_bytes(T, m, n) : 0;
}

extern "C" qg_status qgalore_fp8_linear_fwd(const qg_fp8_linear_desc* d, const uint16_t* X,
                                            const uint8_t* W, const float* S, uint16_t* Y) {
  if (!d || !X || !W || !S || !Y) return QG_ERR_NULL;
  qg_status st = check_f8_linear(d->T, d->m, d->n, false);
  if (st != QG_OK) return st;
  if (!all_aligned({X, W, Y}, 16) || !aligned(S, 4)) return QG_ERR_ALIGN;
  const bool few = qg::f8_few_fits(d->T, d->n);
  const F8Scratch z = f8_scratch(d->T, d->n);
  const int64_t need = f8_fwd_bytes(d->T, d->m, d->n);
  if ((st = check_scratch(d->workspace, d->workspace_bytes, need)) != QG_OK) return st;
  const Span ws{need ? d->workspace : nullptr, need}, y{Y, d->T * d->m * 2}, x{X, d->T * d->n * 2},
      w{W, f8_codes(d->m, d->n)}, s{S, f8_scales(d->m, d->n, true)};
  if (clash(y, {ws, x, w, s}) || clash(ws, {x, w, s})) return QG_ERR_ARG;
  if ((st = device_present()) != QG_OK) return st;
  const hipStream_t stream = static_cast<hipStream_t>(d->stream);
  qg::F8Mm a{nullptr, nullptr, W, S, Y, X, d->T, d->m, d->n, qg::kF8E4M3, 1, 1, nullptr};
  hipError_t e = hipSuccess;
  if (!few) {
    qg::F8Quant q = f8_quant(X, d->T, d->n, qg::kF8FromBf16, qg::kF8E4M3);
    q.q = static_cast<uint8_t*>(d->workspace);
    q.s = reinterpret_cast<float*>(q.q + z.off_s);
    e = qg::launch_f8_quantize(q, stream);
    a.A = q.q;
    a.sa = q.s;
    a.X = nullptr;
    if (need > z.rows) a.part = reinterpret_cast<float*>(q.q + z.rows);
  }
  if (e == hipSuccess) e = qg::launch_f8_mm(a, stream);
  return e == hipSuccess ? QG_OK : hip_fail(e, "FP8 linear forward kernels");
}

extern "C" qg_status qgalore_fp8_linear_bwd(const qg_fp8_linear_desc* d, const uint16_t* dY,
                                            const uint8_t* Wt, const float* St, const uint8_t* Xt,
                                            const float* Sx, uint16_t* dX, uint16_t* G) {
  if (!d || !dY || (!dX && !G) || (dX && (!Wt || !St)) || (G && (!Xt || !Sx))) return QG_ERR_NULL;
  if (!f8_format(d->format)) return QG_ERR_ARG;
  qg_status st = check_f8_linear(d->T, d->m, d->n, true);
  if (st != QG_OK) return st;
  if (!dX) Wt = nullptr, St = nullptr;
  if (!G) Xt = nullptr, Sx = nullptr;
  if (!all_aligned({dY, Wt, Xt, dX, G}, 16) || !all_aligned({St, Sx}, 4)) return QG_ERR_ALIGN;
  const F8Scratch z = f8_scratch(d->T, d->m);
  const int64_t need = f8_bwd_bytes(d->T, d->m, d->n);
  if ((st = check_scratch(d->workspace, d->workspace_bytes, need)) != QG_OK) return st;
  const Span ws{d->workspace, need}, dx{dX, d->T * d->n * 2}, g{G, d->m * d->n * 2},
      dy{dY, d->T * d->m * 2}, wt{Wt, f8_codes(d->n, d->m)}, s{St, f8_scales(d->n, d->m, true)},
      xt{Xt, f8_codes(d->n, d->T)}, sx{Sx, f8_scales(d->n, d->T, false)};
  if (clash(dx, {ws, g, dy, wt, s, xt, sx}) || clash(g, {ws, dy, wt, s, xt, sx}) ||
      clash(ws, {dy, wt, s, xt, sx}))
    return QG_ERR_ARG;
  if ((st = device_present()) != QG_OK) return st;
  const hipStream_t stream = static_cast<hipStream_t>(d->stream);
  uint8_t* base = static_cast<uint8_t*>(d->workspace);
  qg::F8Quant q = f8_quant(dY, d->T, d->m, qg::kF8FromBf16, d->format);
  if (dX) {
    q.q = base;
    q.s = reinterpret_cast<float*>(base + z.off_s);
  }
  if (G) {
    q.qt = base + z.off_qt;
    q.st = reinterpret_cast<float*>(base + z.off_st);
  }
  hipError_t e = qg::launch_f8_quantize(q, stream);
  float* part = need > z.both ? reinterpret_cast<float*>(base + z.both) : nullptr;
  const qg::F8Mm x{q.q, q.s, Wt, St, dX, nullptr, d->T, d->n, d->m, d->format, 1, 1, part};
  const qg::F8Mm w{q.qt, q.st, Xt, Sx, G, nullptr, d->m, d->n, d->T, d->format, 0, 1, part};
  if (e == hipSuccess)
    e = dX && G ? qg::launch_f8_mm_pair(x, w, stream) : qg::launch_f8_mm(dX ? x : w, stream);
  return e == hipSuccess ? QG_OK : hip_fail(e, "FP8 linear backward kernels");
}
