// Decay attention (token-level linear attention with one decay per head):
// what its kernels and their dispatch share.
//
// Every direction is one operator over the tokens of a (batch, head) pair.
// Walking forward from a state X (value channels x key channels),
//   X_i = l X_{i-1} + v_i k_i^T,   o_i = X_i q_i,                l = exp(g_h),
// and walking back from a state Z that has not decayed yet,
//   Z_i = l Z_{i+1} + v_i k_i^T (Z_last = Z + v k^T),  o_i = Z_i q_i,
// with l Z_first left behind. The forward pass is the first with (Q, K, V); the backward pass is
//   dQ: forward with (dO, V, K) from S_in^T,
//   dK: back with (V, dO, Q) from dS_out^T,    dV: back with (K, Q, dO) from dS_out, leaving dS_in.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "vdn.h"

namespace vdn {

constexpr int kDecayC = 64;      // tokens per chunk of both chunked kernels
constexpr int kDecayOps = 3;     // operators per launch, at most
constexpr int kDecayTensors = 7; // Q, K, V, dO and three outputs

// One operator: indexes into DecayArgs.t.
struct DecayOp {
  int q, k, v, o;
  int back;           // walk from the last token to the first
  int s_in_t;         // s_in is read transposed
  int ws, ws_t;       // whose segment states it starts from, read transposed or not
  const float *s_in;  // [BH, d, d] or null (zero)
  float *s_out;       // [BH, d, d] or null
};

struct DecayArgs {
  DecayOp op[kDecayOps];
  void *t[kDecayTensors];  // [BH, N, d] each
  const float *g;          // [H]
  const int32_t *lens;     // [B] or null
  int32_t *info;           // or null
  float *ws;               // [nsums * BH, nseg * nsub, d, d] with nseg > 1
  long long BH;
  int H, N, d, nops;
  int nsums;               // the first operators: those whose segments are summed
  int nseg, seglen;        // segments of a sequence; seglen is a multiple of nsub * kDecayC
  int nsub;                // parts of a segment that are summed on their own
};

// The split of the sequences over CTAs.
struct DecaySplit {
  int nseg, seglen, nsub;
};
// pairs, sums: (operator, batch, head) pairs of the walk and of the pass for the
// states in front of the segments; slots: CTAs that run at a time; ragged: the sequences end anywhere within n.
DecaySplit decay_split(long long pairs, long long sums, long long n, int slots, bool tc, bool ragged);
int decay_slots(int in_dtype, int out_dtype, int d);

// What a CTA works on: block -> (operator, b*h, segment); `sums`: a segment's part.
struct DecayWork {
  int op, seg, h, len, begin, end, nch, last_seg;
  long long bh;
};
__device__ __forceinline__ DecayWork decay_work(const DecayArgs &p, long long block, bool sums) {
  DecayWork w;
  const int parts = sums ? p.nseg * p.nsub : p.nseg, plen = sums ? p.seglen / p.nsub : p.seglen;
  const int part = (int)(block % parts);
  w.seg = sums ? part / p.nsub : part;
  const long long r = block / parts;
  w.bh = r % p.BH;
  w.op = (int)(r / p.BH);
  w.h = (int)(w.bh % p.H);
  w.len = p.N;
  if (p.lens) w.len = min(max(p.lens[w.bh / p.H], 0), p.N);
  w.begin = min((long long)part * plen, (long long)w.len);
  w.end = min(((long long)part + 1) * plen, (long long)w.len);
  w.nch = (w.end - w.begin + kDecayC - 1) / kDecayC;
  w.last_seg = w.len > 0 ? (w.len - 1) / p.seglen : 0;
  return w;
}
// The segment a walk ends in, and whether a segment lies before it on the way.
__device__ __forceinline__ int decay_final_seg(const DecayWork &w, int back) { return back ? 0 : w.last_seg; }
__device__ __forceinline__ bool decay_before_final(const DecayWork &w, int back) {
  return back ? (w.seg > 0 && w.seg <= w.last_seg) : w.seg < w.last_seg;
}

// exp(g n) for a whole n >= 0 (g = -inf included), in 64 bits: l^n multiplies
// a state once per chunk for thousands of chunks, so a power rounded to 32
// bits would drift by its own error each time.
__device__ __forceinline__ double decay_pow(float g, long long n) {
  return n == 0 ? 1.0 : exp((double)g * (double)n);
}

__device__ __forceinline__ int decay_last_part(const DecayArgs &p, int len) {
  return len > 0 ? (len - 1) / (p.seglen / p.nsub) : 0;
}
// Where a walk's segment finds the state in front of it.
__device__ __forceinline__ const float *decay_start(const DecayArgs &p, const DecayOp &op, const DecayWork &w, bool &tr) {
  const long long dd = (long long)p.d * p.d;
  if (p.nseg > 1) {
    tr = op.ws_t;
    // the segment's first part on the way
    const int part = op.back ? min(w.seg * p.nsub + p.nsub - 1, decay_last_part(p, w.len)) : w.seg * p.nsub;
    return p.ws + ((op.ws * p.BH + w.bh) * (p.nseg * p.nsub) + part) * dd;
  }
  tr = op.s_in_t;
  return op.s_in ? op.s_in + w.bh * dd : nullptr;
}

// The passes of one call overlap at their ends: a launch with `early` starts
// while the kernel before it still runs (once every block of that one has
// called launch_dependents or left), and waits for its results where it first
// reads them. Before that it only reads what was there before the call.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_launches() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), long long grid, int threads, size_t smem, cudaStream_t st, bool early,
                         const A &...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_decay_simt(const DecayArgs &a, int in_dtype, int out_dtype, bool sums, cudaStream_t st);
// bf16 in and out: the tensor cores.
bool decay_tc_supported(int in_dtype, int out_dtype);
cudaError_t launch_decay_tc(const DecayArgs &a, bool sums, cudaStream_t st);
cudaError_t launch_decay_prefix(const DecayArgs &a, cudaStream_t st);
cudaError_t launch_decay_step(const void *Q, const void *K, const void *V, const float *g, const int32_t *active,
                              const float *s_in, void *O, float *s_out, long long BH, int H, int d, int in_dtype,
                              int out_dtype, cudaStream_t st);

// One tensor of a rotary call; strides in elements (batch, head, token).
struct RotaryIo {
  const void *x;
  void *y;
  long long xs[3], ys[3];
  int rotate;
};
constexpr int kRotaryIo = 3;
constexpr int kRotaryPairs = 64;  // d / 2, at most
struct RotaryArgs {
  RotaryIo io[kRotaryIo];
  int nio, B, H, d, U, gw, interleaved, inverse;
  long long N, frame0;
  int npairs[3];              // rotated pairs of each axis
  const int32_t *pos;         // [B, N, 3] or null
  // turns per position of each pair, as a sum of two doubles
  double turn[kRotaryPairs], turn_lo[kRotaryPairs];
  int far;                    // positions may take 2^20 turns or more (rotary.cu)
};
cudaError_t launch_rotary(const RotaryArgs &a, int dtype, cudaStream_t st);

}  // namespace vdn
