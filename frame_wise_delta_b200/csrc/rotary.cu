// Rotary positions over several axes (time, height, width).
//
// The head's channels are cut into one section per axis (dim_t, dim_h, dim_w;
// what is left over passes through). Pair i of an axis with n channels turns
// by the angle pos * scale * theta^(-2 i / n):
//   y_a = x_a cos - x_b sin,   y_b = x_a sin + x_b cos
// with (a, b) = (2 i, 2 i + 1) of the section (interleaved) or (i, i + n / 2).
//
// Angles: turns per position come as a sum of two doubles; pos * turns is formed
// as a product, beyond 2^20 turns with its exact remainder (fma) and the second
// double's share, and reduced to the nearest whole turn. So every position a call
// takes keeps float32's accuracy: the product alone is 2^-32 turns off at 2^20
// turns, but 2^-12 at 2^40, and arbitrary at 2^52. Calls whose positions stay
// below 2^20 turns have a kernel without the rest: it costs 0.9 us of 13 in the
// small float32 case, a choice for each block or angle 0.7 us. The sine and
// cosine of what is left are taken in float32 (sincospif). A block forms them
// once for its tokens, in shared memory, and applies them to every head of
// every tensor.
//
// Bound by memory: each value is read and written once (2 d * size bytes per
// row against 3 d operations), so a thread moves 16 bytes per access: whole
// pairs when they are interleaved, the same stretch of both halves otherwise.
// Sections that do not start on such a stretch take the widest one that divides
// every section's half.
//
// Measured: Q and K of 102 816 tokens x 24 heads x 128 channels in bf16, 2.5 GB
// moved, 0.40 ms (6.3 TB/s, 97 % of a plain copy's rate); Q, K and V of 5040
// tokens, token-major, in stretches of 8 bytes, 40.5 us (186 MB, 4.6 TB/s): there
// the angles cost about as much as turning five heads. Sixteen tokens in
// float32 and the like are one launch, 5 us behind 12 us of the caller's.
#include <cuda_bf16.h>

#include "common.cuh"
#include "decay.h"
#include "internal.h"

namespace vdn {
namespace {

constexpr int kThreads = 256;

template <int BYTES> struct VecOf;
template <> struct VecOf<2> { using T = uint16_t; };
template <> struct VecOf<4> { using T = uint32_t; };
template <> struct VecOf<8> { using T = uint2; };
template <> struct VecOf<16> { using T = uint4; };

template <typename T, int W>
struct alignas(sizeof(T) * W) Pack {
  T v[W];
};

template <typename T, int W>
__device__ __forceinline__ Pack<T, W> load(const T *p) {
  using V = typename VecOf<sizeof(T) * W>::T;
  const V x = *reinterpret_cast<const V *>(p);
  return *reinterpret_cast<const Pack<T, W> *>(&x);
}
template <typename T, int W>
__device__ __forceinline__ void store(T *p, const Pack<T, W> &x) {
  using V = typename VecOf<sizeof(T) * W>::T;
  *reinterpret_cast<V *>(p) = *reinterpret_cast<const V *>(&x);
}

// One unit: PW pairs, either 2 PW neighbouring channels or PW channels of each
// half. P: pairs per head (d / 2), the last `rest` of them pass through.
template <typename T, int PW, bool INTER, bool FAR>
__global__ void __launch_bounds__(kThreads, PW == 1 || INTER ? 4 : 3)
    rotary_kernel(const __grid_constant__ RotaryArgs p, int tokens, int slices) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const int P = p.d >> 1;
  float2 *cs = reinterpret_cast<float2 *>(smem_raw);                     // [tokens][P]
  double *turn = reinterpret_cast<double *>(cs + (size_t)tokens * P);    // [P]
  double *where = turn + P;                                              // [tokens][3]
  const int b = blockIdx.z;
  const long long n0 = (long long)blockIdx.x * tokens;
  const int nt = (int)min((long long)tokens, p.N - n0);
  const int rot = p.npairs[0] + p.npairs[1] + p.npairs[2];

  for (int i = threadIdx.x; i < rot; i += kThreads) turn[i] = p.turn[i];
  if ((int)threadIdx.x < nt) {
    const long long n = n0 + threadIdx.x;
    double *at = where + 3 * threadIdx.x;
    if (p.pos) {
      const int32_t *q = p.pos + ((long long)b * p.N + n) * 3;
      at[0] = q[0], at[1] = q[1], at[2] = q[2];
    } else {
      const uint32_t f = (uint32_t)n / (uint32_t)p.U, u = (uint32_t)n - f * (uint32_t)p.U, row = u / (uint32_t)p.gw;
      at[0] = (double)(p.frame0 + f), at[1] = row, at[2] = u - row * (uint32_t)p.gw;
    }
  }
  __syncthreads();
  // thread: pairs i, i + step, ..; tokens t, t + kThreads / step, ..
  const int step = P < kThreads ? P : kThreads;  // P is a power of two
  for (int i = threadIdx.x & (step - 1); i < rot; i += step) {
    const int axis = i < p.npairs[0] ? 0 : i < p.npairs[0] + p.npairs[1] ? 1 : 2;
    const double per = turn[i];
    for (int t = threadIdx.x / step; t < nt; t += kThreads / step) {
      const double x = where[3 * t + axis];
      double a = __dmul_rn(x, per);  // not taken into an fma with what follows
      const double left = FAR ? fma(x, p.turn_lo[i], fma(x, per, -a)) : 0.0;
      a -= rint(a);
      if (FAR) a += left, a -= rint(a);
      float s, c;
      sincospif(2.f * (float)a, &s, &c);
      cs[t * P + i] = make_float2(c, p.inverse ? -s : s);
    }
  }
  __syncthreads();

  // units of a row, then rows (tokens), then slices (tensor, head)
  constexpr int kAhead = sizeof(T) * PW >= 16 ? 2 : 4;
  const int UR = P / PW;
  const int per = nt * UR;
  const int s0 = blockIdx.y * slices, s1 = min(s0 + slices, p.nio * p.H);
  const int first1 = p.npairs[0], first2 = first1 + p.npairs[1];
  for (int e = threadIdx.x; e < per; e += kThreads) {
    const int t = e / UR, i = (e - t * UR) * PW;  // token, first pair
    int lo, hi;                                   // channels of the first pair
    if (INTER) {
      lo = 2 * i;
      hi = lo + PW;  // the second vector
    } else {
      const int f = i < first1 ? 0 : i < first2 ? first1 : i < rot ? first2 : rot;
      const int n = i < first1 ? first1 : i < first2 ? p.npairs[1] : i < rot ? p.npairs[2] : P - rot;
      lo = f + i;  // 2 f + (i - f)
      hi = lo + n;
    }
    float2 w[PW];
#pragma unroll
    for (int x = 0; x < PW; ++x) w[x] = i + x < rot ? cs[t * P + i + x] : make_float2(1.f, 0.f);
    // the slices of one tensor at a time: head by head along its stride
    for (int sl = s0; sl < s1;) {
      const int k = sl / p.H, h0 = sl - k * p.H, h1 = min(p.H, h0 + s1 - sl);
      const RotaryIo &io = p.io[k];
      const long long xh = io.xs[1], yh = io.ys[1];
      const T *x = (const T *)io.x + b * io.xs[0] + h0 * xh + (n0 + t) * io.xs[2];
      T *y = (T *)io.y + b * io.ys[0] + h0 * yh + (n0 + t) * io.ys[2];
      const bool rotate = io.rotate != 0;
      sl += h1 - h0;
      // kAhead heads' loads are in flight before the first store (rows do not
      // overlap, which the compiler cannot know)
      for (int h = h0; h < h1; h += kAhead, x += kAhead * xh, y += kAhead * yh) {
        Pack<T, PW> A[kAhead], B[kAhead];
#pragma unroll
        for (int g = 0; g < kAhead; ++g)
          if (h + g < h1) {
            A[g] = load<T, PW>(x + g * xh + lo);
            B[g] = load<T, PW>(x + g * xh + hi);
          }
#pragma unroll
        for (int g = 0; g < kAhead; ++g) {
          if (h + g >= h1) break;
          if (rotate) {
#pragma unroll
            for (int q = 0; q < PW; ++q) {
              // pairs that pass through are copied, not turned by 0: 0 * inf is no number
              if (i + q < rot) {
                T &ra = INTER ? (2 * q < PW ? A[g].v[(2 * q) % PW] : B[g].v[(2 * q) % PW]) : A[g].v[q];
                T &rb = INTER ? (2 * q + 1 < PW ? A[g].v[(2 * q + 1) % PW] : B[g].v[(2 * q + 1) % PW]) : B[g].v[q];
                const float fa = to_f32(ra), fb = to_f32(rb);
                store_val(&ra, fa * w[q].x - fb * w[q].y);
                store_val(&rb, fa * w[q].y + fb * w[q].x);
              }
            }
          }
          store<T, PW>(y + g * yh + lo, A[g]);
          store<T, PW>(y + g * yh + hi, B[g]);
        }
      }
    }
  }
}

template <typename T, int PW, bool INTER>
cudaError_t launch_t(const RotaryArgs &a, cudaStream_t st) {
  // tokens per block: enough for one unit per thread, 8 at least (the angles
  // of a block are shared by all heads, so few tokens per block recompute
  // nothing); the (tensor, head) slices are spread over blocks until each SM
  // gets eight of them, as long as eight slices share a block's angles, and
  // then until every SM has four. (Three tensors of 5040 tokens x 24 heads:
  // 42 us with eight blocks per SM, 43 us with twelve, 49 us with sixteen.)
  const int P = a.d / 2, UR = P / PW;
  int tokens = (kThreads + UR - 1) / UR;
  if (tokens < 8) tokens = 8;
  if ((long long)tokens > a.N) tokens = (int)a.N;
  const long long tiles = (a.N + tokens - 1) / tokens;
  const int all = a.nio * a.H;
  int parts = 1;
  while (parts * 8 < all && tiles * a.B * parts < 8 * 148) ++parts;
  while (parts < all && tiles * a.B * parts < 4 * 148) ++parts;
  const int slices = (all + parts - 1) / parts;
  const dim3 grid((unsigned)tiles, (unsigned)((all + slices - 1) / slices), (unsigned)a.B);
  const size_t smem = (size_t)tokens * P * sizeof(float2) + (size_t)(P + 3 * tokens) * sizeof(double);
  auto *kern = a.far ? rotary_kernel<T, PW, INTER, true> : rotary_kernel<T, PW, INTER, false>;
  kern<<<grid, kThreads, smem, st>>>(a, tokens, slices);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_d(const RotaryArgs &a, cudaStream_t st) {
  constexpr int W = 16 / sizeof(T);
  if (a.interleaved) return launch_t<T, W, true>(a, st);
  // the widest stretch that divides every section's start and half
  int m = W;
  const int rest = a.d / 2 - a.npairs[0] - a.npairs[1] - a.npairs[2];
  for (const int n : {a.npairs[0], a.npairs[1], a.npairs[2], rest})
    while (n % m) m /= 2;
  if (m == 8) return launch_t<T, W, false>(a, st);
  if (m == 4) return launch_t<T, 4, false>(a, st);
  if (m == 2) return launch_t<T, 2, false>(a, st);
  return launch_t<T, 1, false>(a, st);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a, int dtype, cudaStream_t st) {
  return dtype == VDN_BF16 ? launch_d<__nv_bfloat16>(a, st) : launch_d<float>(a, st);
}

}  // namespace vdn
