// C ABI of the token-level operators: rotary positions and decay attention
// (validation and dispatch; the contract is in include/vdn.h).
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "common.cuh"
#include "decay.h"
#include "internal.h"

using namespace vdn;

namespace {

vdn_status fail(vdn_status st, const char *fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  set_last_error(msg);
  return st;
}

#define VDN_TRY(x)                 \
  do {                             \
    vdn_status st_ = (x);          \
    if (st_ != VDN_OK) return st_; \
  } while (0)

#define VDN_CUDA(x, where)                                                                            \
  do {                                                                                                \
    cudaError_t e_ = (x);                                                                             \
    if (e_ != cudaSuccess) return fail(VDN_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e_)); \
  } while (0)

bool misaligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

vdn_status need(const void *p, const char *name, bool required) {
  if (!required) return VDN_OK;
  if (!p) return fail(VDN_ERR_INVALID, "%s is NULL", name);
  if (misaligned(p, 16)) return fail(VDN_ERR_INVALID, "%s is not 16-byte aligned", name);
  return VDN_OK;
}
vdn_status maybe(const void *p, const char *name, size_t a = 16) {
  if (p && misaligned(p, a)) return fail(VDN_ERR_INVALID, "%s is not %zu-byte aligned", name, a);
  return VDN_OK;
}

// The token sequence of a (batch, head) pair: its T * U tokens in order.
vdn_status token_count(const vdn_shape *s, long long *n) {
  set_last_error("");
  VDN_TRY(validate_shape(s));
  *n = (long long)s->T * s->U;
  if (*n > 0x7fffffffLL - kDecayC) return fail(VDN_ERR_UNSUPPORTED, "T*U = %lld tokens exceed 2^31-1-%d", *n, kDecayC);
  return VDN_OK;
}

// Blocks of a launch (the grid's x extent).
vdn_status check_grid(long long blocks) {
  return blocks > 0x7fffffffLL ? fail(VDN_ERR_UNSUPPORTED, "too many (batch, head) pairs") : VDN_OK;
}

DecaySplit split_of(const vdn_shape *s, long long n, int nops, int nsums, bool ragged) {
  const long long BH = (long long)s->B * s->H;
  return decay_split(nops * BH, nsums * BH, n, decay_slots(s->in_dtype, s->out_dtype, s->dk),
                     decay_tc_supported(s->in_dtype, s->out_dtype), ragged);
}

void fill_args(const vdn_shape *s, long long n, int nops, int nsums, const DecaySplit &split, DecayArgs *a) {
  a->BH = (long long)s->B * s->H;
  a->H = s->H;
  a->N = (int)n;
  a->d = s->dk;
  a->nops = nops;
  a->nsums = nsums;
  a->nseg = split.nseg;
  a->seglen = split.seglen;
  a->nsub = split.nsub;
}

// The states in front of the segments. A query knows no lengths: the larger of
// the two splits.
size_t state_bytes(const vdn_shape *s, int nsums, const DecaySplit &split) {
  if (split.nseg <= 1) return 0;
  const size_t n = (size_t)nsums * s->B * s->H * split.nseg * split.nsub * s->dk * s->dk * sizeof(float);
  return (n + 255) & ~size_t(255);
}
size_t query_bytes(const vdn_shape *s, long long n, int nops, int nsums) {
  if ((long long)s->B * s->H == 0) return 0;
  const size_t a = state_bytes(s, nsums, split_of(s, n, nops, nsums, false));
  const size_t b = state_bytes(s, nsums, split_of(s, n, nops, nsums, true));
  return a > b ? a : b;
}

vdn_status check_workspace(const void *ws, size_t have, size_t want) {
  if (want == 0) return VDN_OK;
  if (!ws) return fail(VDN_ERR_INVALID, "workspace is NULL");
  if (misaligned(ws, 256)) return fail(VDN_ERR_INVALID, "workspace is not 256-byte aligned");
  if (have < want) return fail(VDN_ERR_INVALID, "workspace of %zu bytes < %zu required", have, want);
  return VDN_OK;
}

// No tokens: the state passes through.
vdn_status copy_state(const vdn_shape *s, const float *from, float *to, cudaStream_t st) {
  const size_t bytes = (size_t)s->B * s->H * s->dk * s->dk * sizeof(float);
  if (!to || to == from) return VDN_OK;
  if (from)
    VDN_CUDA(cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, st), "copy of the state");
  else
    VDN_CUDA(cudaMemsetAsync(to, 0, bytes, st), "clearing of the state");
  return VDN_OK;
}

vdn_status run_decay(const vdn_shape *s, DecayArgs &a, cudaStream_t st) {
  const bool tc = decay_tc_supported(s->in_dtype, s->out_dtype);
  auto walk = [&](bool sums) {
    return tc ? launch_decay_tc(a, sums, st) : launch_decay_simt(a, s->in_dtype, s->out_dtype, sums, st);
  };
  if (a.nseg > 1) {
    VDN_CUDA(walk(true), "decay segment sums");
    VDN_CUDA(launch_decay_prefix(a, st), "decay segment states");
  }
  VDN_CUDA(walk(false), "decay attention");
  return VDN_OK;
}

// A number of about 106 bits as a sum of two doubles (Dekker, "A floating-point
// technique for extending the available precision", 1971), for the rotary
// frequencies: a position of 2^52 turns them into angles with float32's accuracy.
struct Twofold {
  double hi, lo;
};
Twofold operator*(const Twofold &a, const Twofold &b) {
  const double p = a.hi * b.hi, e = fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi), s = p + e;
  return {s, e - (s - p)};
}
constexpr Twofold kInv2Pi = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / (2 pi)
// theta^(-1/n): the double next to it, and a Newton step on y^n theta = 1.
Twofold inverse_root(double theta, int n) {
  if (n <= 1) return {n ? 1.0 / theta : 1.0, 0.0};  // not used by an axis of one pair
  const double y = pow(theta, -1.0 / n);
  Twofold power = {1.0, 0.0}, square = {y, 0.0};
  for (int e = n; e; e >>= 1) {
    if (e & 1) power = power * square;
    square = square * square;
  }
  const Twofold r = power * Twofold{theta, 0.0};
  const double step = -y * ((r.hi - 1.0) + r.lo) / n;
  return isfinite(step) ? Twofold{y, step} : Twofold{y, 0.0};
}

// y's rows may not overlap: walking its axes from the smallest stride up, each
// stride passes the extent of those below.
bool disjoint_rows(const long long *stride, const long long *count, int d) {
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (stride[order[j]] < stride[order[i]]) {
        const int t = order[i];
        order[i] = order[j];
        order[j] = t;
      }
  long long extent = d;
  for (int i = 0; i < 3; ++i) {
    const int k = order[i];
    if (count[k] <= 1) continue;
    if (stride[k] < extent) return false;
    extent += (count[k] - 1) * stride[k];
  }
  return true;
}

}  // namespace

extern "C" {

vdn_status vdn_rotary(const vdn_shape *s, const vdn_rotary_args *r, const vdn_rotary_io *io, int32_t n_io,
                      vdn_stream_t stream) {
  long long n;
  VDN_TRY(token_count(s, &n));
  if (!r) return fail(VDN_ERR_INVALID, "rotary arguments are NULL");
  if (n_io < 1 || n_io > kRotaryIo) return fail(VDN_ERR_INVALID, "n_io = %d not in [1, %d]", n_io, kRotaryIo);
  if (!io) return fail(VDN_ERR_INVALID, "io is NULL");
  const int dims[3] = {r->dim_t, r->dim_h, r->dim_w};
  const double scales[3] = {r->scale_t, r->scale_h, r->scale_w};
  RotaryArgs a{};
  int at = 0;
  long long sum = 0;
  double most = 0.0;  // turns per position
  for (int x = 0; x < 3; ++x) {
    if (dims[x] < 0 || dims[x] % 2) return fail(VDN_ERR_INVALID, "axis of %d channels: even and >= 0 is needed", dims[x]);
    sum += dims[x];
  }
  if (sum > s->dk) return fail(VDN_ERR_INVALID, "the axes' %lld channels exceed d = %d", sum, s->dk);
  if (!(r->theta > 0.0) || !isfinite(r->theta)) return fail(VDN_ERR_INVALID, "theta must be positive and finite");
  if ((r->interleaved != 0 && r->interleaved != 1) || (r->inverse != 0 && r->inverse != 1))
    return fail(VDN_ERR_INVALID, "interleaved and inverse must be 0 or 1");
  for (int x = 0; x < 3; ++x) {
    if (!isfinite(scales[x])) return fail(VDN_ERR_INVALID, "scale must be finite");
    a.npairs[x] = dims[x] / 2;
    // theta^(-2 i / n) as powers of theta^(-2 / n)
    const Twofold step = inverse_root(r->theta, a.npairs[x]);
    Twofold f = {1.0, 0.0};
    for (int i = 0; i < a.npairs[x]; ++i, f = f * step) {
      const Twofold turn = f * Twofold{scales[x], 0.0} * kInv2Pi;
      if (!isfinite(turn.hi) || fabs(turn.hi) > 1e6)
        return fail(VDN_ERR_INVALID, "theta and scale turn a pair by more than 1e6 turns");
      a.turn[at] = turn.hi;
      most = fmax(most, fabs(turn.hi));
      a.turn_lo[at++] = isfinite(turn.lo) ? turn.lo : 0.0;
    }
  }
  const bool any = (long long)s->B * s->H * n > 0;
  if (!r->pos) {
    if (any && (r->grid_h < 1 || r->grid_w < 1 || (long long)r->grid_h * r->grid_w != s->U))
      return fail(VDN_ERR_INVALID, "grid %d x %d does not hold U = %d tokens", r->grid_h, r->grid_w, s->U);
    if (r->frame0 > (1LL << 52) || r->frame0 < -(1LL << 52)) return fail(VDN_ERR_INVALID, "frame0 beyond 2^52");
  }
  VDN_TRY(maybe(r->pos, "pos", 4));
  const long long step = s->in_dtype == VDN_BF16 ? 8 : 4;
  const long long count[3] = {s->B, s->H, n};
  for (int k = 0; k < n_io; ++k) {
    RotaryIo &o = a.io[k];
    VDN_TRY(need(io[k].x, "io.x", any));
    VDN_TRY(need(io[k].y, "io.y", any));
    if (io[k].rotate != 0 && io[k].rotate != 1) return fail(VDN_ERR_INVALID, "io[%d].rotate must be 0 or 1", k);
    o.x = io[k].x;
    o.y = io[k].y;
    o.rotate = io[k].rotate;
    for (int x = 0; x < 3; ++x) {
      o.xs[x] = io[k].x_stride[x];
      o.ys[x] = io[k].y_stride[x];
      if (count[x] > 1 && (o.xs[x] < 0 || o.xs[x] % step || o.ys[x] % step))
        return fail(VDN_ERR_INVALID, "io[%d]: strides must be multiples of 16 bytes, not negative", k);
      if (count[x] > 1 && (o.xs[x] > (1LL << 60) / count[x] || o.ys[x] > (1LL << 60) / count[x]))
        return fail(VDN_ERR_INVALID, "io[%d]: stride too large", k);
    }
    if (any && !disjoint_rows(o.ys, count, s->dk)) return fail(VDN_ERR_INVALID, "io[%d]: rows of y overlap", k);
    if (any && o.x == o.y)
      for (int x = 0; x < 3; ++x)
        if (count[x] > 1 && o.xs[x] != o.ys[x])
          return fail(VDN_ERR_INVALID, "io[%d]: in place needs equal strides", k);
    for (int m = 0; m < n_io; ++m)
      if (any && m != k && (io[m].y == io[k].y || io[m].x == io[k].y))
        return fail(VDN_ERR_INVALID, "io[%d].y is another tensor of the call", k);
  }
  if (!any) return VDN_OK;
  if (s->B > 65535) return fail(VDN_ERR_UNSUPPORTED, "B = %d > 65535", s->B);
  if ((long long)n_io * s->H > 65535) return fail(VDN_ERR_UNSUPPORTED, "H = %d too large", s->H);
  a.nio = n_io;
  a.B = s->B;
  a.H = s->H;
  a.d = s->dk;
  a.U = s->U;
  a.gw = r->pos ? 1 : r->grid_w;
  a.interleaved = r->interleaved;
  a.inverse = r->inverse;
  a.N = n;
  a.frame0 = r->frame0;
  a.pos = r->pos;
  const double first = fabs((double)r->frame0), last = fabs((double)r->frame0 + s->T), side = fmax(a.gw, s->U);
  a.far = most * (r->pos ? 0x1p31 : fmax(side, fmax(first, last))) >= 0x1p20;
  VDN_CUDA(launch_rotary(a, s->in_dtype, (cudaStream_t)stream), "rotary");
  return VDN_OK;
}

size_t vdn_decay_attn_workspace_bytes(const vdn_shape *s) {
  long long n;
  if (token_count(s, &n) != VDN_OK) return 0;
  return query_bytes(s, n, 1, 1);
}

vdn_status vdn_decay_attn(const vdn_shape *s, const void *Q, const void *K, const void *V, const float *log_decay,
                          const int32_t *lens, const float *S_in, void *O, float *S_out, void *workspace,
                          size_t workspace_bytes, int32_t *info, vdn_stream_t stream) {
  long long n;
  VDN_TRY(token_count(s, &n));
  const long long BH = (long long)s->B * s->H;
  const bool any = BH * n > 0;
  VDN_TRY(need(Q, "Q", any));
  VDN_TRY(need(K, "K", any));
  VDN_TRY(need(V, "V", any));
  VDN_TRY(need(O, "O", any));
  VDN_TRY(need(log_decay, "log_decay", BH > 0));
  VDN_TRY(maybe(lens, "lens", 4));
  VDN_TRY(maybe(S_in, "S_in"));
  VDN_TRY(maybe(S_out, "S_out"));
  VDN_TRY(maybe(info, "info", 4));
  if (any && (O == Q || O == K || O == V)) return fail(VDN_ERR_INVALID, "O is an input");
  if (BH == 0) return VDN_OK;
  if (n == 0) return copy_state(s, S_in, S_out, (cudaStream_t)stream);
  const DecaySplit split = split_of(s, n, 1, 1, lens != nullptr);
  VDN_TRY(check_workspace(workspace, workspace_bytes, query_bytes(s, n, 1, 1)));
  VDN_TRY(check_grid(BH * split.nseg * split.nsub));
  DecayArgs a{};
  fill_args(s, n, 1, 1, split, &a);
  a.t[0] = const_cast<void *>(Q);
  a.t[1] = const_cast<void *>(K);
  a.t[2] = const_cast<void *>(V);
  a.t[4] = O;
  a.op[0] = DecayOp{0, 1, 2, 4, 0, 0, 0, 0, S_in, S_out};
  a.g = log_decay;
  a.lens = lens;
  a.info = info;
  a.ws = (float *)workspace;
  return run_decay(s, a, (cudaStream_t)stream);
}

size_t vdn_decay_attn_backward_workspace_bytes(const vdn_shape *s) {
  long long n;
  if (token_count(s, &n) != VDN_OK) return 0;
  return query_bytes(s, n, 3, 2);
}

vdn_status vdn_decay_attn_backward(const vdn_shape *s, const void *Q, const void *K, const void *V,
                                   const float *log_decay, const int32_t *lens, const float *S_in, const void *dO,
                                   const float *dS_out, void *dQ, void *dK, void *dV, float *dS_in, void *workspace,
                                   size_t workspace_bytes, int32_t *info, vdn_stream_t stream) {
  long long n;
  VDN_TRY(token_count(s, &n));
  if (s->in_dtype != s->out_dtype) return fail(VDN_ERR_UNSUPPORTED, "the backward pass needs in_dtype == out_dtype");
  const long long BH = (long long)s->B * s->H;
  const bool any = BH * n > 0;
  const void *in[4] = {Q, K, V, dO};
  void *out[3] = {dQ, dK, dV};
  const char *names[7] = {"Q", "K", "V", "dO", "dQ", "dK", "dV"};
  for (int i = 0; i < 4; ++i) VDN_TRY(need(in[i], names[i], any));
  for (int i = 0; i < 3; ++i) VDN_TRY(need(out[i], names[4 + i], any));
  VDN_TRY(need(log_decay, "log_decay", BH > 0));
  VDN_TRY(maybe(lens, "lens", 4));
  VDN_TRY(maybe(S_in, "S_in"));
  VDN_TRY(maybe(dS_out, "dS_out"));
  VDN_TRY(maybe(dS_in, "dS_in"));
  VDN_TRY(maybe(info, "info", 4));
  for (int o = 0; any && o < 3; ++o) {
    for (int i = 0; i < 4; ++i)
      if (out[o] == in[i]) return fail(VDN_ERR_INVALID, "%s is an input", names[4 + o]);
    for (int i = 0; i < o; ++i)
      if (out[o] == out[i]) return fail(VDN_ERR_INVALID, "%s and %s are the same", names[4 + i], names[4 + o]);
  }
  if (dS_in && (dS_in == S_in || dS_in == dS_out)) return fail(VDN_ERR_INVALID, "dS_in is an input");
  if (BH == 0) return VDN_OK;
  if (n == 0) return copy_state(s, dS_out, dS_in, (cudaStream_t)stream);
  const DecaySplit split = split_of(s, n, 3, 2, lens != nullptr);
  VDN_TRY(check_workspace(workspace, workspace_bytes, query_bytes(s, n, 3, 2)));
  VDN_TRY(check_grid(3 * BH * split.nseg * split.nsub));
  DecayArgs a{};
  fill_args(s, n, 3, 2, split, &a);
  for (int i = 0; i < 4; ++i) a.t[i] = const_cast<void *>(in[i]);
  for (int i = 0; i < 3; ++i) a.t[4 + i] = out[i];
  a.op[0] = DecayOp{3, 2, 1, 4, 0, 1, 0, 0, S_in, nullptr};    // dQ
  a.op[1] = DecayOp{1, 0, 3, 6, 1, 0, 1, 0, dS_out, dS_in};    // dV
  a.op[2] = DecayOp{2, 3, 0, 5, 1, 1, 1, 1, dS_out, nullptr};  // dK: the transposed states of dV's walk
  a.g = log_decay;
  a.lens = lens;
  a.info = info;
  a.ws = (float *)workspace;
  return run_decay(s, a, (cudaStream_t)stream);
}

vdn_status vdn_decay_step(const vdn_shape *s, const void *Q, const void *K, const void *V, const float *log_decay,
                          const int32_t *active, const float *S_in, void *O, float *S_out, vdn_stream_t stream) {
  long long n;
  VDN_TRY(token_count(s, &n));
  const long long BH = (long long)s->B * s->H;
  if (n != 1) return fail(VDN_ERR_INVALID, "vdn_decay_step takes one token per (batch, head): T = U = 1");
  VDN_TRY(need(Q, "Q", BH > 0));
  VDN_TRY(need(K, "K", BH > 0));
  VDN_TRY(need(V, "V", BH > 0));
  VDN_TRY(need(log_decay, "log_decay", BH > 0));
  VDN_TRY(maybe(active, "active", 4));
  VDN_TRY(need(S_in, "S_in", BH > 0));
  VDN_TRY(need(O, "O", BH > 0));
  VDN_TRY(need(S_out, "S_out", BH > 0));
  if (BH > 0 && (O == Q || O == K || O == V)) return fail(VDN_ERR_INVALID, "O is an input");
  if (BH == 0) return VDN_OK;
  VDN_TRY(check_grid(BH * 8));
  VDN_CUDA(launch_decay_step(Q, K, V, log_decay, active, S_in, O, S_out, BH, s->H, s->dk, s->in_dtype, s->out_dtype,
                             (cudaStream_t)stream),
           "decay step");
  return VDN_OK;
}

}  // extern "C"
