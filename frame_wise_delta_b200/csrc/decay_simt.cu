// Decay attention on the CUDA cores: the chunked form for the types that the
// tensor-core kernel does not take, the join of the segments' states, and the
// form for single tokens.
//
// Chunked form, per chunk of 64 tokens with local indexes i, j, n valid rows
// and the state X in front of it (forward walk):
//   o_i  = sum_{j <= i} l^{i-j} (q_i . k_j) v_j + l^{i+1} X q_i
//   X'   = l^n X + sum_j l^{n-1-j} v_j k_j^T
// and on the walk back
//   o_i  = sum_{j >= i} l^{j-i} (q_i . k_j) v_j + l^{n-1-i} Z q_i
//   Z'   = l^n Z + sum_j l^{j+1} v_j k_j^T.
// Powers with whole exponents >= 0 only, each at most 1, so nothing overflows.
// All sums are in float32; everything outside j <= i or behind the last token
// is selected away, not multiplied by 0.
//
// Per chunk four products of 64 x 64 x d or 64 x d x d, 4 x 4 values a thread,
// from shared memory. What bounds it is that memory, its rate (half of it is
// used) and its latency under 8 to 16 warps per SM: about 2 of 4 instructions
// per cycle are issued and 30 to 44 % of the FMA pipe is used. 16 warps with
// half the values each, packed pairs of FMAs over transposed tiles (half the
// instructions), more CTAs per SM at d <= 32 and fetching ahead in the walk at
// d = 128 were all no faster. Measured, float32: 4
// heads of 5120 tokens, d = 64, 45 us; 2 x 8 heads of 2000 tokens, d = 128,
// 144 us.
#include <cuda_bf16.h>

#include "common.cuh"
#include "decay.h"
#include "internal.h"

namespace vdn {
namespace {

constexpr int kC = kDecayC;

constexpr int kThreads = 256;
// CTAs per SM. At d >= 64 one, with 255 registers a thread to read ahead into
// (4 heads of 5120 tokens, d = 64: 45 us, 56 us with two of 128 registers); at
// d <= 32 two (3 x 4 ragged heads, d = 32, gradients: 23 us, 26 us with one).
constexpr int simt_ctas(int d) { return d >= 64 ? 1 : 2; }

template <int D>
struct SimtSmem {
  float q[kC][D + 4], k[kC][D + 4], v[kC][D + 4];
  float wk[kC][D + 4];  // the keys times their weights in the chunk's sum
  float st[D][D + 4];   // the state, st[key][value]
  float p[kC][kC + 4];
  float pw[kC + 1];     // l^n
  float carry[2][2];    // l^n of a whole chunk and of the segment's last one, as two floats each
};

template <int W>
__device__ __forceinline__ void lds(const float *p, float (&r)[W]) {
  if constexpr (W == 4) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    r[0] = x.x, r[1] = x.y, r[2] = x.z, r[3] = x.w;
  } else if constexpr (W == 2) {
    const float2 x = *reinterpret_cast<const float2 *>(p);
    r[0] = x.x, r[1] = x.y;
  } else {
    r[0] = p[0];
  }
}

template <int W>
__device__ __forceinline__ void sts(float *p, const float *r) {
  if constexpr (W == 4)
    *reinterpret_cast<float4 *>(p) = make_float4(r[0], r[1], r[2], r[3]);
  else if constexpr (W == 2)
    *reinterpret_cast<float2 *>(p) = make_float2(r[0], r[1]);
  else
    p[0] = r[0];
}

// A chunk's rows on their way to shared memory: all of a thread's loads are in
// flight before the first is used.
template <typename T, int D>
struct Rows {
  static constexpr int V = 16 / sizeof(T), kPer = D / V, N = (kC * kPer + kThreads - 1) / kThreads;
  uint4 x[N];
  __device__ __forceinline__ void fetch(const T *src, int rows) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = threadIdx.x + i * kThreads, r = e / kPer, c = (e % kPer) * V;
      x[i] = make_uint4(0, 0, 0, 0);
      if (r < rows) x[i] = *reinterpret_cast<const uint4 *>(src + (long long)r * D + c);
    }
  }
  // dst = the rows times weight(row)
  template <typename W>
  __device__ __forceinline__ void stash(float (*dst)[D + 4], W weight) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = threadIdx.x + i * kThreads, r = e / kPer, c = (e % kPer) * V;
      const T *y = reinterpret_cast<const T *>(&x[i]);
      if (r < kC) {
        const float f = weight(r);
#pragma unroll
        for (int q = 0; q < V; q += 4)
          *reinterpret_cast<float4 *>(&dst[r][c + q]) =
              make_float4(f * to_f32(y[q]), f * to_f32(y[q + 1]), f * to_f32(y[q + 2]), f * to_f32(y[q + 3]));
      }
    }
  }
  __device__ __forceinline__ void stash(float (*dst)[D + 4]) const {
    stash(dst, [](int) { return 1.f; });
  }
};

// SUMS: only the state that a segment adds (from zero), into the workspace.
// A warp is a grid of 4 x 8 threads over rows x columns of each product: its
// 16-byte reads of either operand then touch 64 and 128 bytes of different
// banks, one pass of the shared memory each.
template <typename TI, typename TO, int D, bool SUMS>
__global__ void __launch_bounds__(kThreads, simt_ctas(D)) decay_simt_kernel(const DecayArgs p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem<D> &s = *reinterpret_cast<SimtSmem<D> *>(smem_raw);
  constexpr int TY = kThreads / 16;            // threads over rows; 16 over columns
  constexpr int R = kC / TY;                   // rows per thread of the scores and outputs
  constexpr int VW = D / 16 < 4 ? D / 16 : 4;  // value channels per vector
  constexpr int NV = D / (16 * VW);            // vectors per thread
  constexpr int NK = D / TY;                   // key channels per thread of the state
  constexpr int KW = NK < 4 ? NK : 4, NKV = NK / KW;  // in vectors
  const DecayWork w = decay_work(p, blockIdx.x, SUMS);
  const DecayOp &op = p.op[w.op];
  const int back = op.back;
  launch_dependents();
  if (SUMS && !decay_before_final(w, back)) return;
  const bool fin = w.seg == decay_final_seg(w, back);
  if (!SUMS && w.nch == 0 && !fin) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tx = (warp & 1) * 8 + (lane & 7), ty = (warp >> 1) * 4 + (lane >> 3);
  constexpr long long DD = (long long)D * D;

  const long long base = w.bh * (long long)p.N;
  // the next chunk is fetched under this one's arithmetic where registers hold it
  constexpr bool kEarly = D <= 64 || SUMS;
  Rows<TI, D> q, k, v;
  auto fetch = [&](int it) {
    const int t0 = w.begin + (back ? w.nch - 1 - it : it) * kC, n = min(kC, w.end - t0);
    const long long row = (base + t0) * D;
    if (!SUMS) q.fetch((const TI *)p.t[op.q] + row, n);
    k.fetch((const TI *)p.t[op.k] + row, n);
    v.fetch((const TI *)p.t[op.v] + row, n);
  };
  if (kEarly && w.nch > 0) fetch(0);

  const float g = p.g[w.h];
  if (threadIdx.x <= kC) {
    s.pw[threadIdx.x] = (float)decay_pow(g, threadIdx.x);
  } else if (threadIdx.x >= 96 && threadIdx.x < 98) {
    const int set = threadIdx.x - 96;
    const double l = decay_pow(g, set ? w.end - w.begin - (w.nch - 1) * kC : kC);
    s.carry[set][0] = (float)l;
    s.carry[set][1] = (float)(l - (double)(float)l);
  }

  // the state: this thread's key channels KW (TY a + ty) + e, value channels VW (16 c + tx) + x
  float X[NK][NV * VW];
  const float *src = nullptr;
  bool tr = false;
  if (!SUMS) {
    src = decay_start(p, op, w, tr);
    wait_for_launches();
  }
  // by way of shared memory, so that memory is read along its rows
  if (src) {
    constexpr int kAhead = D * D / kThreads < 16 ? D * D / kThreads : 16;  // loads in flight
    for (int e0 = threadIdx.x; e0 < D * D; e0 += kAhead * kThreads) {
      float y[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) y[x] = src[e0 + x * kThreads];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int e = e0 + x * kThreads, r = e / D, c = e % D;
        s.st[tr ? r : c][tr ? c : r] = y[x];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int a = 0; a < NK; ++a)
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int e = 0; e < VW; ++e)
        X[a][c * VW + e] = src ? s.st[KW * (TY * (a / KW) + ty) + a % KW][VW * (16 * c + tx) + e] : 0.f;
  auto put_state = [&]() {
#pragma unroll
    for (int a = 0; a < NK; ++a)
#pragma unroll
      for (int c = 0; c < NV; ++c) sts<VW>(&s.st[KW * (TY * (a / KW) + ty) + a % KW][VW * (16 * c + tx)], &X[a][c * VW]);
  };

  for (int it = 0; it < w.nch; ++it) {
    const int c0 = back ? w.nch - 1 - it : it;
    const int t0 = w.begin + c0 * kC, n = min(kC, w.end - t0);
    const long long row = (base + t0) * D;
    if (!kEarly) fetch(it);
    if (!SUMS) {
      q.stash(s.q);
      k.stash(s.k);
      put_state();
    }
    k.stash(s.wk, [&](int j) { return j < n ? s.pw[back ? j + 1 : n - 1 - j] : 0.f; });
    v.stash(s.v);
    if (kEarly && it + 1 < w.nch) fetch(it + 1);
    __syncthreads();
    if (!SUMS) {
      // the scores: rows ty + TY r, columns tx + 16 c
      float sc[R][4] = {};
#pragma unroll 4
      for (int x = 0; x < D; x += 4) {
        float a[R][4], b[4][4];
#pragma unroll
        for (int r = 0; r < R; ++r) lds<4>(&s.q[ty + TY * r][x], a[r]);
#pragma unroll
        for (int c = 0; c < 4; ++c) lds<4>(&s.k[tx + 16 * c][x], b[c]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[r][c] = fmaf(a[r][e], b[c][e], sc[r][c]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int i = ty + TY * r, j = tx + 16 * c, gap = back ? j - i : i - j;
          s.p[i][j] = gap >= 0 && j < n ? sc[r][c] * s.pw[gap] : 0.f;
        }
      __syncthreads();
      // the outputs: rows as the scores', value channels as the state's
      float o[R][NV * VW] = {};
      auto product = [&](const float *a0, int lda, const float (*b0)[D + 4], int len) {
#pragma unroll 4
        for (int x = 0; x < len; x += 4) {
          float a[R][4];
#pragma unroll
          for (int r = 0; r < R; ++r) lds<4>(a0 + (ty + TY * r) * lda + x, a[r]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < NV; ++c) {
              float b[VW];
              lds<VW>(&b0[x + e][VW * (16 * c + tx)], b);
#pragma unroll
              for (int r = 0; r < R; ++r)
#pragma unroll
                for (int y = 0; y < VW; ++y) o[r][c * VW + y] = fmaf(a[r][e], b[y], o[r][c * VW + y]);
            }
        }
      };
      product(&s.q[0][0], D + 4, s.st, D);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int i = ty + TY * r;
        const float f = i < n ? s.pw[back ? n - 1 - i : i + 1] : 0.f;
#pragma unroll
        for (int x = 0; x < NV * VW; ++x) o[r][x] *= f;
      }
      product(&s.p[0][0], kC + 4, s.v, kC);
      TO *out = (TO *)p.t[op.o] + row;
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (ty + TY * r < n) {
#pragma unroll
          for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int x = 0; x < VW; ++x)
              store_val(out + (long long)(ty + TY * r) * D + VW * (16 * c + tx) + x, o[r][c * VW + x]);
        }
    }
    // the state behind the chunk
    float u[NK][NV * VW] = {};
#pragma unroll(D >= 64 ? 8 : 4)
    for (int j = 0; j < kC; ++j) {
      float a[NK], b[NV * VW];
#pragma unroll
      for (int c = 0; c < NKV; ++c) lds<KW>(&s.wk[j][KW * (TY * c + ty)], *reinterpret_cast<float(*)[KW]>(&a[c * KW]));
#pragma unroll
      for (int c = 0; c < NV; ++c) lds<VW>(&s.v[j][VW * (16 * c + tx)], *reinterpret_cast<float(*)[VW]>(&b[c * VW]));
#pragma unroll
      for (int y = 0; y < NK; ++y)
#pragma unroll
        for (int x = 0; x < NV * VW; ++x) u[y][x] = fmaf(a[y], b[x], u[y][x]);
    }
    const float l0 = s.carry[c0 == w.nch - 1][0], l1 = s.carry[c0 == w.nch - 1][1];
#pragma unroll
    for (int a = 0; a < NK; ++a)
#pragma unroll
      for (int x = 0; x < NV * VW; ++x) X[a][x] = fmaf(X[a][x], l0, fmaf(X[a][x], l1, u[a][x]));
    __syncthreads();
  }

  float *dst = SUMS ? p.ws + blockIdx.x * DD : (fin && op.s_out ? op.s_out + w.bh * DD : nullptr);
  if (dst) {
    put_state();
    __syncthreads();
    for (int e = threadIdx.x; e < D * D; e += kThreads) dst[e] = s.st[e % D][e / D];
  }
}

// ws[part] becomes the state in front of that part on the walk: it held what
// the part itself adds. A thread takes V neighbouring values of a pair's state
// through the parts in 64 bits: a chain of dependent loads and FMAs, so kAhead
// of the loads are in flight at once, behind a start of several us (lengths,
// decay, powers: worked out by two threads for the block). So one value a
// thread and the shortest chain where all blocks run at a time, four where they
// would come in waves. Alone, one against four: 10 and 17 us for 40 parts of 4 x
// 64 x 64 values, 34 and 13 us for 4 parts of 48 x 128 x 128.
template <int V>
__global__ void __launch_bounds__(256) decay_prefix_kernel(const DecayArgs p, int dd) {
  __shared__ struct {
    const float *src;
    float *ws;
    double full, tail;
    int count, last, back, tr;
  } b;
  const int per = (dd + 256 * V - 1) / (256 * V), pair = blockIdx.x / per, e = (blockIdx.x % per * 256 + threadIdx.x) * V;
  launch_dependents();
  if (threadIdx.x % 32 == 0 && threadIdx.x < 64) {
    const DecayWork w = decay_work(p, (long long)pair * p.nseg, false);
    const DecayOp &op = p.op[w.op];
    const int plen = p.seglen / p.nsub, last = decay_last_part(p, w.len);
    const float g = p.g[w.h];
    if (threadIdx.x == 0) {
      b.src = op.s_in ? op.s_in + w.bh * dd : nullptr;
      b.ws = p.ws + ((long long)pair * (p.nseg * p.nsub) + (op.back ? last : 0)) * dd;
      b.full = decay_pow(g, plen);
      // parts to pass up to the final segment's first
      b.count = op.back ? last - min(p.nsub - 1, last) : w.last_seg * p.nsub;
      b.last = last;
      b.back = op.back;
      b.tr = op.s_in_t;
    } else {
      b.tail = decay_pow(g, w.len - (long long)last * plen);
    }
  }
  __syncthreads();
  const int count = b.count, last = b.back ? 0 : b.last;  // the step that passes the sequence's last part
  const double full = b.full, tail = b.tail;
  if (e >= dd) return;
  double s[V];
#pragma unroll
  for (int y = 0; y < V; ++y) {
    const int r = (e + y) / p.d, c = (e + y) % p.d;
    s[y] = b.src ? b.src[b.tr ? c * p.d + r : e + y] : 0.f;
  }
  const long long step = b.back ? -dd : dd;
  float *ws = b.ws + e;
  wait_for_launches();
  constexpr int kAhead = V == 1 ? 16 : 8;  // parts in flight
  for (int n0 = 0; n0 <= count; n0 += kAhead) {
    float u[kAhead][V];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      if (n0 + x < count)
        lds<V>(ws + (n0 + x) * step, u[x]);
      else
        for (int y = 0; y < V; ++y) u[x][y] = 0.f;
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int n = n0 + x;
      if (n > count) break;
      float o[V];
#pragma unroll
      for (int y = 0; y < V; ++y) {
        o[y] = (float)s[y];
        s[y] = fma(s[y], n == last ? tail : full, (double)u[x][y]);
      }
      sts<V>(ws + n * step, o);
    }
  }
}

template <typename TI, typename TO, int D, bool SUMS>
cudaError_t launch_simt_t(const DecayArgs &a, cudaStream_t st) {
  constexpr size_t smem = sizeof(SimtSmem<D>);
  auto *kern = decay_simt_kernel<TI, TO, D, SUMS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long grid = SUMS ? a.nsums * a.BH * a.nseg * a.nsub : a.nops * a.BH * a.nseg;
  return launch_after(kern, grid, kThreads, smem, st, !SUMS && a.nseg > 1, a);
}

template <typename TI, typename TO, bool SUMS>
cudaError_t launch_simt_d(const DecayArgs &a, cudaStream_t st) {
  switch (a.d) {
    case 16: return launch_simt_t<TI, TO, 16, SUMS>(a, st);
    case 32: return launch_simt_t<TI, TO, 32, SUMS>(a, st);
    case 64: return launch_simt_t<TI, TO, 64, SUMS>(a, st);
    case 128: return launch_simt_t<TI, TO, 128, SUMS>(a, st);
  }
  return cudaErrorInvalidValue;
}

// ------------------------------------------------------------ single tokens
// S' = l S + v k^T, o = S' q: bound by reading and writing the state once
// (8 d^2 bytes per pair against 5 d^2 operations). A warp takes whole rows of
// S, kLanes lanes to a row and 16 bytes per lane and load, so each load of a
// warp covers full 128-byte lines; the row's product with q is summed over its
// lanes by shuffles.
// Measured: 72 of 96 sequences x 24 states of 128 x 128 in 55 us (49 us of it
// the kernel), 85 % of a plain copy's rate; the 24 states of one sequence take
// 5 us, a launch and two reads behind one another.
constexpr int kStepThreads = 128;
template <typename TI, typename TO, int D>
__global__ void __launch_bounds__(kStepThreads)
    decay_step_kernel(const TI *Q, const TI *K, const TI *V, const float *g, const int32_t *active, const float *s_in,
                      TO *O, float *s_out, long long rows, int H) {
  constexpr int kLanes = D / 4 < 8 ? D / 4 : 8;  // lanes per row
  constexpr int NV = D / (4 * kLanes);           // 16-byte vectors per lane
  constexpr int RW = 32 / kLanes;                // rows per warp
  const int lane = threadIdx.x & 31, sub = lane % kLanes;
  const long long row = ((long long)blockIdx.x * (kStepThreads / 32) + (threadIdx.x >> 5)) * RW + lane / kLanes;
  const bool there = row < rows;
  float4 s[NV];
#pragma unroll
  for (int c = 0; c < NV; ++c)
    if (there) s[c] = *reinterpret_cast<const float4 *>(s_in + row * D + 4 * (sub + kLanes * c));
  const long long bh = (there ? row : 0) / D;
  const bool on = there && (!active || active[bh / H] != 0);
  float acc = 0.f;
  if (on) {
    const double l = exp((double)g[bh % H]);
    const float l0 = (float)l, l1 = (float)(l - (double)l0);
    const float v = to_f32(V[row]);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const long long at = bh * D + 4 * (sub + kLanes * c);
      float *x = reinterpret_cast<float *>(&s[c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = fmaf(x[e], l0, fmaf(x[e], l1, v * to_f32(K[at + e])));
        acc = fmaf(x[e], to_f32(Q[at + e]), acc);
      }
    }
  }
#pragma unroll
  for (int m = kLanes / 2; m > 0; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
  if (there && (on || s_out != s_in)) {
#pragma unroll
    for (int c = 0; c < NV; ++c) *reinterpret_cast<float4 *>(s_out + row * D + 4 * (sub + kLanes * c)) = s[c];
  }
  if (on && sub == 0) store_val(O + row, acc);
}

template <typename TI, typename TO, int D>
cudaError_t launch_step_t(const void *Q, const void *K, const void *V, const float *g, const int32_t *active,
                          const float *s_in, void *O, float *s_out, long long BH, int H, cudaStream_t st) {
  constexpr int kLanes = D / 4 < 8 ? D / 4 : 8;
  constexpr int kRows = (32 / kLanes) * (kStepThreads / 32);  // rows per CTA
  const long long rows = BH * D, grid = (rows + kRows - 1) / kRows;
  decay_step_kernel<TI, TO, D><<<(unsigned)grid, kStepThreads, 0, st>>>(
      (const TI *)Q, (const TI *)K, (const TI *)V, g, active, s_in, (TO *)O, s_out, rows, H);
  return cudaGetLastError();
}

template <typename TI, typename TO>
cudaError_t launch_step_d(const void *Q, const void *K, const void *V, const float *g, const int32_t *active,
                          const float *s_in, void *O, float *s_out, long long BH, int H, int d, cudaStream_t st) {
  switch (d) {
    case 16: return launch_step_t<TI, TO, 16>(Q, K, V, g, active, s_in, O, s_out, BH, H, st);
    case 32: return launch_step_t<TI, TO, 32>(Q, K, V, g, active, s_in, O, s_out, BH, H, st);
    case 64: return launch_step_t<TI, TO, 64>(Q, K, V, g, active, s_in, O, s_out, BH, H, st);
    case 128: return launch_step_t<TI, TO, 128>(Q, K, V, g, active, s_in, O, s_out, BH, H, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

DecaySplit decay_split(long long pairs, long long sums, long long n, int slots, bool tc, bool ragged) {
  // Times in halves of a chunk's: a wave of CTAs walks `len` chunks of its
  // segment after a start of kStart chunks' time; more than one segment adds
  // a pass for the states in front of the segments (half the traffic, no
  // outputs; each segment cut into parts until the card is full) and their
  // join. Ragged sequences are half full on average, and the CTAs of short
  // ones leave their place at once: then the longest walk or half of the whole
  // work counts, whichever is more.
  // A launch and a start cost the tensor-core kernel (1.4 to 2 us a chunk) several
  // chunks' time, the CUDA-core one (10 us) less than one.
  // Measured: 24 heads of 102 816 tokens, d = 128: 6 segments 0.82 to 0.95 ms (a single
  // one would be 1607 chunks of 1.9 us in a row, 3 ms); 8 x 16 ragged heads of
  // up to 4099 tokens, d = 64: a single segment 92 us, two about 12 % more.
  const long long chunks = n > 0 ? (n + kDecayC - 1) / kDecayC : 1;
  DecaySplit best{1, (int)(chunks * kDecayC), 1};
  if (pairs > 8LL * slots) return best;  // several waves of whole walks
  const int kStart = tc ? 6 : 1, kJoin = tc ? 20 : 1, ch = (int)chunks, np = (int)pairs, ns = (int)sums;
  // four waves of CTAs at most
  const int most = ch < 4 * slots / np + 1 ? ch : 4 * slots / np + 1;
  long long cost = -1;
  for (int want = 1; want <= most; ++want) {
    int len = (ch + want - 1) / want, nsub = 1;
    if (want > 1) {
      nsub = slots / (ns * (want - 1));
      nsub = nsub < 1 ? 1 : nsub > len ? len : nsub;
      len = (len + nsub - 1) / nsub * nsub;
    }
    const int nseg = (ch + len - 1) / len;
    auto pass = [&](int ctas, int walk) {
      if (!ragged) return (long long)((ctas + slots - 1) / slots) * walk;
      const long long all = ((long long)ctas * walk / 2 + slots - 1) / slots;
      return all > walk ? all : (long long)walk;
    };
    long long c = 2 * pass(np * nseg, len + kStart);
    if (nseg > 1) c += pass(ns * (nseg - 1) * nsub, len / nsub + 2 * kStart) + 2 * kJoin;
    if (cost < 0 || c < cost) {
      cost = c;
      best = DecaySplit{nseg, len * kDecayC, nsub};
    }
  }
  return best;
}

int decay_slots(int in_dtype, int out_dtype, int d) {
  return 148 * (decay_tc_supported(in_dtype, out_dtype) ? 1 : simt_ctas(d));
}

cudaError_t launch_decay_simt(const DecayArgs &a, int in_dtype, int out_dtype, bool sums, cudaStream_t st) {
  if (in_dtype == VDN_F32) {
    if (sums) return launch_simt_d<float, float, true>(a, st);
    return out_dtype == VDN_F32 ? launch_simt_d<float, float, false>(a, st)
                                : launch_simt_d<float, __nv_bfloat16, false>(a, st);
  }
  if (sums) return launch_simt_d<__nv_bfloat16, float, true>(a, st);
  return out_dtype == VDN_F32 ? launch_simt_d<__nv_bfloat16, float, false>(a, st) : cudaErrorInvalidValue;
}

cudaError_t launch_decay_prefix(const DecayArgs &a, cudaStream_t st) {
  const int dd = a.d * a.d;
  const long long pairs = a.nsums * a.BH, blocks = pairs * (dd / 256);
  if (blocks <= 8 * 148) return launch_after(decay_prefix_kernel<1>, blocks, 256, 0, st, true, a, dd);
  return launch_after(decay_prefix_kernel<4>, pairs * ((dd + 1023) / 1024), 256, 0, st, true, a, dd);
}

cudaError_t launch_decay_step(const void *Q, const void *K, const void *V, const float *g, const int32_t *active,
                              const float *s_in, void *O, float *s_out, long long BH, int H, int d, int in_dtype,
                              int out_dtype, cudaStream_t st) {
  if (in_dtype == VDN_F32)
    return out_dtype == VDN_F32
               ? launch_step_d<float, float>(Q, K, V, g, active, s_in, O, s_out, BH, H, d, st)
               : launch_step_d<float, __nv_bfloat16>(Q, K, V, g, active, s_in, O, s_out, BH, H, d, st);
  return out_dtype == VDN_F32
             ? launch_step_d<__nv_bfloat16, float>(Q, K, V, g, active, s_in, O, s_out, BH, H, d, st)
             : launch_step_d<__nv_bfloat16, __nv_bfloat16>(Q, K, V, g, active, s_in, O, s_out, BH, H, d, st);
}

}  // namespace vdn
