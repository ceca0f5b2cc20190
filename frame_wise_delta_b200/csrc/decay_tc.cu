// Decay attention in chunks on the 5th-generation tensor cores (tcgen05 + TMEM
// + TMA), bf16 in and out, d in {16, 32, 64, 128}; sums and state in float32.
//
// Per chunk of 64 tokens (local indexes i, j; n valid rows; X the state in
// front of it, rows = value channels):
//   o_i = f_i (X q_i + sum_j c_ij s_ij v_j),   s_ij = q_i . k_j,   c_ij = l^{|i-j|} / f_i
//   X'  = l^n X + sum_j (w_j v_j) k_j^T
// forward: j <= i, f_i = l^{i+1}, w_j = l^{n-1-j}; back: j >= i, f_i = l^{n-1-i}, w_j = l^{j+1}. With
// f_i taken out, c_ij = c_j depends on the column alone (l^{-(j+1)}, or l^{-(n-1-j)} back), and both
// products share one accumulator. A head that decays by more than 2^-60 over a chunk would overflow
// there: it takes f_i >= 2^-60 and c_ij entry by entry (the state then enters its late rows with
// 2^-60 in place of something smaller, far below a rounding of o_i).
//
// Four products per chunk, all with 128 TMEM lanes:
//   SC[i][j]  = Q K^T              A = Q, B = K (K-major tiles as TMA brings them; rows 64.. unused)
//   U[v][k]   = (w v)^T K          A = the weighted values in TMEM, B = K (MN-major)
//   O[v][i]   = X Q^T + V^T P^T    A = X in TMEM as bf16 hi and lo parts, B = Q; A = V (MN-major),
//                                  B = P = c SC as bf16, in shared memory
// The state stays in registers in float32 and is written to TMEM once per chunk, so it never passes
// through shared memory; the outputs come transposed (lane = channel) and leave through a swizzled
// staging tile by TMA. The weighted values enter U as three bf16 parts (2^-24 together): two would
// leave 3e-6 in the float32 state. P is rounded to bf16 (an error of the size of the output's own).
//
// One CTA of 16 warps walks one segment of one (operator, batch, head):
//   warps 0, 1  : scores SC -> P (TMEM lanes 0..63)
//   warp 2      : TMA producer
//   warp 3      : TMEM allocation, one lane issues the MMAs
//   warps 4..11 : the state: lane = value channel (warp % 4), column half (warp - 4) / 4
//   warps 12..15: the weighted values of the next chunk, then the outputs of this one
// SUMS: only what a segment adds to the state (from zero), for the walk's later segments.
// Every wait is bounded.
#include <cudaTypedefs.h>

#include "common.cuh"
#include "decay.h"
#include "internal.h"

namespace vdn {
namespace {

constexpr int kC = kDecayC;
constexpr int kThreads = 512;
constexpr uint32_t kPanel = kC * 128;  // 64 tokens x 64 channels
constexpr uint32_t kTmemCols = 512;

template <int DP>  // channels padded to panels
struct Cfg {
  static constexpr int kPanels = DP / 64;
  static constexpr uint32_t kTile = kPanels * kPanel;
  static constexpr uint32_t kStageBytes = 3 * kTile;  // Q, K, V
  static constexpr int kStages = DP == 128 ? 4 : 6;
  // shared memory, from a 1024-byte aligned base; a 128-row operand reads
  // 8 KB past its 64-row tile, which the next tile or P covers
  static constexpr uint32_t kOffP = kStages * kStageBytes;
  static constexpr uint32_t kOffO = kOffP + kPanel;
  static constexpr uint32_t kOffTab = kOffO + kTile;
  static constexpr uint32_t kTabFloats = 2 * 3 * kC + 72 + 4;  // w, c, f per set; l^n; carries
  static constexpr uint32_t kOffBar = kOffTab + 4 * kTabFloats;
  static constexpr uint32_t kBars = 2 * kStages + 11;
  static constexpr size_t kSmem = 1024 + kOffBar + 8 * kBars + 16;
  // TMEM columns
  static constexpr uint32_t kX = 0, kU = DP, kO = 2 * DP, kSC = kO + kC, kVT = kSC + kC;
  static_assert(kVT + 3 * kC / 2 <= kTmemCols, "TMEM");
  static_assert(kOffBar % 8 == 0 && kOffTab % 16 == 0, "alignment");
};

struct DecayMaps {
  CUtensorMap m[kDecayTensors];
};

__device__ __forceinline__ void fail(volatile int *abort, int32_t *info) {
  *abort = 1;
  if (info) atomicExch(info, VDN_INFO_TIMEOUT);
}

// Two values as three bf16 parts each (a in the low halves).
__device__ __forceinline__ void split3(float a, float b, uint32_t &h, uint32_t &m, uint32_t &l) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  const float ra = a - __low2float(x), rb = b - __high2float(x);
  const __nv_bfloat162 y = __floats2bfloat162_rn(ra, rb);
  const __nv_bfloat162 z = __floats2bfloat162_rn(ra - __low2float(y), rb - __high2float(y));
  h = *reinterpret_cast<const uint32_t *>(&x);
  m = *reinterpret_cast<const uint32_t *>(&y);
  l = *reinterpret_cast<const uint32_t *>(&z);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

template <int DP, bool SUMS>
__global__ void __launch_bounds__(kThreads, 1)
    decay_tc_kernel(const __grid_constant__ DecayMaps maps, const __grid_constant__ DecayArgs p) {
  using F = Cfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float *tab = reinterpret_cast<float *>(smem + F::kOffTab);
  float *pw = tab + 2 * 3 * kC;       // l^n, n = 0..64
  float *carry = pw + 72;             // per set: l^n of its valid rows as two floats
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + F::kOffBar);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * F::kStages;
  const uint32_t sc_full = empty0 + 8 * F::kStages, sc_free = sc_full + 8, p_ready = sc_free + 8;
  const uint32_t vt_ready = p_ready + 8, kv_full = vt_ready + 8, u_free = kv_full + 8;
  const uint32_t x_ready = u_free + 8, qx_done = x_ready + 8, pv_done = qx_done + 8, o_free = pv_done + 8;
  const uint32_t drain = o_free + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + F::kBars);
  volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const DecayWork w = decay_work(p, blockIdx.x);
  const DecayOp &op = p.op[w.op];
  const int back = op.back;
  const bool fin = w.seg == decay_final_seg(w, back);
  if (SUMS ? !decay_before_final(w, back) : (w.nch == 0 && !fin)) return;
  const int nch = w.nch, d = p.d;
  const long long DD = (long long)d * d;
  const int tail = w.end - w.begin - (nch - 1) * kC;  // rows of the segment's last chunk
  const float g = p.g[w.h];
  const bool steep = (double)g * kC < -41.588830833596719;  // l^64 < 2^-60
  auto chunk_at = [&](int it) { return back ? nch - 1 - it : it; };
  auto rows_of = [&](int c) { return c == nch - 1 ? tail : kC; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < F::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(sc_full, 1);
    mbar_init(sc_free, 64);
    mbar_init(p_ready, 64);
    mbar_init(vt_ready, DP);
    mbar_init(kv_full, 1);
    mbar_init(u_free, 2 * DP);
    mbar_init(x_ready, 2 * DP);
    mbar_init(qx_done, 1);
    mbar_init(pv_done, 1);
    mbar_init(o_free, DP);
    mbar_init(drain, 1);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 3) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  // the weights of whole chunks (set 0) and of the segment's last one (set 1)
  if (threadIdx.x < 2 * kC) {
    const int set = threadIdx.x / kC, x = threadIdx.x % kC, n = set ? tail : kC;
    float *t = tab + set * 3 * kC;
    const int er = back ? n - 1 - x : x + 1, ew = back ? x + 1 : n - 1 - x;
    t[x] = x < n ? (float)decay_pow(g, ew) : 0.f;
    t[kC + x] = x < n && !steep ? (float)(1.0 / decay_pow(g, er)) : 0.f;
    t[2 * kC + x] = x < n ? fmaxf((float)decay_pow(g, er), 0x1p-60f) : 1.f;
  } else if (threadIdx.x < 2 * kC + kC + 1) {
    pw[threadIdx.x - 2 * kC] = (float)decay_pow(g, threadIdx.x - 2 * kC);
  } else if (threadIdx.x >= 256 && threadIdx.x < 258) {
    const int set = threadIdx.x - 256;
    const double l = decay_pow(g, set ? tail : kC);
    carry[2 * set] = (float)l;
    carry[2 * set + 1] = (float)(l - (double)(float)l);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto set_of = [&](int c) { return c == nch - 1 ? 1 : 0; };

  if (warp == 2) {
    // ------------------------------------------------------------- loads
    if (lane == 0) {
      const CUtensorMap *mq = &maps.m[op.q], *mk = &maps.m[op.k], *mv = &maps.m[op.v];
      if (!SUMS) tma_prefetch_desc(mq);
      tma_prefetch_desc(mk);
      tma_prefetch_desc(mv);
      int it = 0;
      for (; it < nch; ++it) {
        const int s = it % F::kStages;
        if (it >= F::kStages && !mbar_wait(empty0 + 8 * s, (uint32_t)((it / F::kStages - 1) & 1), abort)) {
          fail(abort, p.info);
          break;
        }
        const uint32_t dst = smem_u32(smem) + s * F::kStageBytes, fb = full0 + 8 * s;
        const int t0 = w.begin + chunk_at(it) * kC;
        mbar_arrive_expect_tx(fb, SUMS ? 2 * F::kTile : F::kStageBytes);
#pragma unroll
        for (int x = 0; x < F::kPanels; ++x) {
          if (!SUMS) tma_load_3d(dst + x * kPanel, mq, fb, 64 * x, t0, (int)w.bh);
          tma_load_3d(dst + F::kTile + x * kPanel, mk, fb, 64 * x, t0, (int)w.bh);
          tma_load_3d(dst + 2 * F::kTile + x * kPanel, mv, fb, 64 * x, t0, (int)w.bh);
        }
      }
      // every copy issued lands before the CTA may leave
      volatile int never = 0;
      for (int i = it > F::kStages ? it - F::kStages : 0; i < it; ++i)
        mbar_wait(full0 + 8 * (i % F::kStages), (uint32_t)((i / F::kStages) & 1), &never);
    }
  } else if (warp == 3) {
    // -------------------------------------------------------------- MMAs
    if (lane == 0) {
      constexpr uint32_t id_sc = idesc_bf16_f32(128, kC, false, false);
      constexpr uint32_t id_u = idesc_bf16_f32(128, DP, false, true);
      constexpr uint32_t id_pv = idesc_bf16_f32(128, kC, true, false);
      bool ok = true;
      auto wait = [&](uint32_t bar, int i) {
        if (ok && !mbar_wait(bar, (uint32_t)(i & 1), abort)) ok = false;
        tc_fence_after();
        return ok;
      };
      auto base = [&](int it) { return smem_u32(smem) + (it % F::kStages) * F::kStageBytes; };
      auto wait_full = [&](int it) {
        if (ok && !mbar_wait(full0 + 8 * (it % F::kStages), (uint32_t)((it / F::kStages) & 1), abort)) ok = false;
        return ok;
      };
      auto scores = [&](int it) {
        const uint32_t q = base(it), k = q + F::kTile;
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
          const uint32_t off = (ks >> 2) * kPanel + (ks & 3) * 32;
          tc_mma_bf16(tmem + F::kSC, smem_desc_sw128(q + off, 16, 1024), smem_desc_sw128(k + off, 16, 1024), id_sc,
                      ks > 0 ? 1u : 0u);
        }
        tc_commit(sc_full);
      };
      if (!SUMS && nch > 0 && wait_full(0)) scores(0);
      for (int it = 0; it < nch && ok; ++it) {
        const uint32_t q = base(it), k = q + F::kTile, v = k + F::kTile;
        // U = (w v)^T K, the smallest parts first
        if (SUMS && !wait_full(it)) break;
        if (!wait(vt_ready, it) || (it > 0 && !wait(u_free, it - 1))) break;
#pragma unroll
        for (int part = 2; part >= 0; --part)
#pragma unroll
          for (int ks = 0; ks < kC / 16; ++ks)
            tc_mma_bf16_ts(tmem + F::kU, tmem + F::kVT + part * (kC / 2) + 8 * ks,
                           smem_desc_sw128(k + ks * 2048, kPanel, 1024), id_u, part < 2 || ks > 0 ? 1u : 0u);
        tc_commit(kv_full);
        if (SUMS) {
          tc_commit(empty0 + 8 * (it % F::kStages));
          continue;
        }
        // O = X Q^T
        if (!wait(x_ready, it) || (it > 0 && !wait(o_free, it - 1))) break;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks)
            tc_mma_bf16_ts(tmem + F::kO, tmem + F::kX + part * (DP / 2) + 8 * ks,
                           smem_desc_sw128(q + (ks >> 2) * kPanel + (ks & 3) * 32, 16, 1024), id_sc,
                           part > 0 || ks > 0 ? 1u : 0u);
        tc_commit(qx_done);
        // the next chunk's scores run while this one's P is made
        if (it + 1 < nch) {
          if (!wait_full(it + 1) || !wait(sc_free, it)) break;
          scores(it + 1);
        }
        // O += V^T P^T
        if (!wait(p_ready, it)) break;
#pragma unroll
        for (int ks = 0; ks < kC / 16; ++ks)
          tc_mma_bf16(tmem + F::kO, smem_desc_sw128(v + ks * 2048, kPanel, 1024),
                      smem_desc_sw128(smem_u32(smem + F::kOffP) + ks * 32, 16, 1024), id_pv, 1u);
        tc_commit(pv_done);
        tc_commit(empty0 + 8 * (it % F::kStages));
      }
      if (!ok) fail(abort, p.info);
      volatile int never = 0;
      tc_commit(drain);
      mbar_wait(drain, 0, &never);
    }
  } else if (warp < 2) {
    // ----------------------------------------------- scores -> P (row i)
    if (!SUMS) {
      const int i = warp * 32 + lane;
      const uint32_t at = tmem + F::kSC + ((uint32_t)(warp * 32) << 16);
      uint8_t *row = smem + F::kOffP + i * 128;
      for (int it = 0; it < nch; ++it) {
        const int c = chunk_at(it), n = rows_of(c);
        const float *t = tab + set_of(c) * 3 * kC;
        if (!__all_sync(0xffffffffu, mbar_wait(sc_full, (uint32_t)(it & 1), abort))) {
          fail(abort, p.info);
          break;
        }
        tc_fence_after();
        uint32_t pk[kC / 2];
        const float rf = steep ? 1.f / t[2 * kC + i] : 0.f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float v[32];
          tmem_ld32(at + 32 * b, v);
          if (b == 1) {
            tc_fence_before();
            mbar_arrive(sc_free);
          }
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            const int j = 32 * b + x;
            float cj[4];
            if (steep) {
#pragma unroll
              for (int y = 0; y < 4; ++y) cj[y] = rf * pw[abs(i - j - y)];
            } else {
              const float4 c4 = *reinterpret_cast<const float4 *>(t + kC + j);
              cj[0] = c4.x, cj[1] = c4.y, cj[2] = c4.z, cj[3] = c4.w;
            }
            float r[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const bool in = back ? (j + y >= i && j + y < n) : j + y <= i;
              r[y] = in ? v[x + y] * cj[y] : 0.f;
            }
            pk[j / 2] = pack_bf16(r[0], r[1]);
            pk[j / 2 + 1] = pack_bf16(r[2], r[3]);
          }
        }
        // the previous chunk's product has read P
        if (it > 0 && !__all_sync(0xffffffffu, mbar_wait(pv_done, (uint32_t)((it - 1) & 1), abort))) {
          fail(abort, p.info);
          break;
        }
#pragma unroll
        for (int x = 0; x < 8; ++x)
          *reinterpret_cast<uint4 *>(row + ((x ^ (i & 7)) << 4)) =
              make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
        fence_proxy_async_smem();
        mbar_arrive(p_ready);
      }
    }
  } else if (warp < 12) {
    // --------------------------------------------------------- the state
    const int sub = warp & 3, half = (warp - 4) >> 2;
    const int r = sub * 32 + lane, c0 = half * (DP / 2);  // value channel, first key channel
    const uint32_t lanes = (uint32_t)(sub * 32) << 16;
    if (sub * 32 < DP) {
      float X[DP / 2];
      const float *src = nullptr;
      bool tr = false;
      if (!SUMS) {
        if (p.nseg > 1) {
          src = p.ws + (long long)blockIdx.x * DD;
        } else if (op.s_in) {
          src = op.s_in + w.bh * DD;
          tr = op.s_in_t;
        }
      }
#pragma unroll
      for (int x = 0; x < DP / 2; x += 4) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (src && r < d && c0 + x < d) {
          if (tr) {
            const float *z = src + (c0 + x) * d + r;
            y = make_float4(z[0], z[d], z[2 * d], z[3 * d]);
          } else {
            y = *reinterpret_cast<const float4 *>(src + r * d + c0 + x);
          }
        }
        X[x] = y.x, X[x + 1] = y.y, X[x + 2] = y.z, X[x + 3] = y.w;
      }
      auto publish = [&] {
#pragma unroll
        for (int b = 0; b < DP / 64; ++b) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) split_bf16x2(X[32 * b + 2 * x], X[32 * b + 2 * x + 1], hi[x], lo[x]);
          tmem_st16(tmem + lanes + F::kX + half * (DP / 4) + 16 * b, hi);
          tmem_st16(tmem + lanes + F::kX + DP / 2 + half * (DP / 4) + 16 * b, lo);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(x_ready);
      };
      if (!SUMS && nch > 0) publish();
      bool ok = true;
      for (int it = 0; it < nch; ++it) {
        const float l0 = carry[2 * set_of(chunk_at(it))], l1 = carry[2 * set_of(chunk_at(it)) + 1];
        ok = __all_sync(0xffffffffu, mbar_wait(kv_full, (uint32_t)(it & 1), abort));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < DP / 64; ++b) {
          float u[32];
          tmem_ld32(tmem + lanes + F::kU + c0 + 32 * b, u);
#pragma unroll
          for (int x = 0; x < 32; ++x) X[32 * b + x] = fmaf(X[32 * b + x], l0, fmaf(X[32 * b + x], l1, u[x]));
        }
        tc_fence_before();
        mbar_arrive(u_free);
        if (!SUMS && it + 1 < nch) {
          ok = __all_sync(0xffffffffu, mbar_wait(qx_done, (uint32_t)(it & 1), abort));
          if (!ok) break;
          tc_fence_after();
          publish();
        }
      }
      if (!ok) fail(abort, p.info);
      float *dst = SUMS ? p.ws + (long long)blockIdx.x * DD : (fin && op.s_out ? op.s_out + w.bh * DD : nullptr);
      if (dst && r < d) {
#pragma unroll
        for (int x = 0; x < DP / 2; x += 4)
          if (c0 + x < d)
            *reinterpret_cast<float4 *>(dst + r * d + c0 + x) = make_float4(X[x], X[x + 1], X[x + 2], X[x + 3]);
      }
    }
  } else {
    // ------------------------------------- weighted values, then outputs
    const int sub = warp & 3, r = sub * 32 + lane;  // value channel
    const uint32_t lanes = (uint32_t)(sub * 32) << 16;
    if (sub * 32 < DP) {
      // byte offset of (token x, this channel) in a swizzled tile: col[x & 7] + 128 x
      uint32_t col[8];
#pragma unroll
      for (int x = 0; x < 8; ++x)
        col[x] = (uint32_t)(r >> 6) * kPanel + ((((uint32_t)(r & 63) >> 3) ^ (uint32_t)x) << 4) + (uint32_t)(r & 7) * 2u;
      bool ok = true;
      const int gt = threadIdx.x - 384;
      uint8_t *ob = smem + F::kOffO;
      auto values = [&](int it) {
        const int s = it % F::kStages, c = chunk_at(it), n = rows_of(c);
        uint8_t *v = smem + s * F::kStageBytes + 2 * F::kTile;
        const float *wt = tab + set_of(c) * 3 * kC;
        ok = __all_sync(0xffffffffu, mbar_wait(full0 + 8 * s, (uint32_t)((it / F::kStages) & 1), abort));
        if (!ok) return;
        // the previous chunk's U has read the weighted values
        if (it > 0) ok = __all_sync(0xffffffffu, mbar_wait(kv_full, (uint32_t)((it - 1) & 1), abort));
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t h[16], m[16], l[16];
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            const int j = 32 * b + x;
            const float4 w4 = *reinterpret_cast<const float4 *>(wt + j);
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(v + col[(j + e) & 7] + 128 * (j + e)) << 16);
            y[0] *= w4.x, y[1] *= w4.y, y[2] *= w4.z, y[3] *= w4.w;
            if (n < kC) {
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = j + e < n ? y[e] : 0.f;
            }
            split3(y[0], y[1], h[x / 2], m[x / 2], l[x / 2]);
            split3(y[2], y[3], h[x / 2 + 1], m[x / 2 + 1], l[x / 2 + 1]);
          }
          tmem_st16(tmem + lanes + F::kVT + 16 * b, h);
          tmem_st16(tmem + lanes + F::kVT + kC / 2 + 16 * b, m);
          tmem_st16(tmem + lanes + F::kVT + kC + 16 * b, l);
        }
        if (n < kC) {
          // what lies behind the sequence's end meets zeros in the products:
          // it may be no number, so it is cleared (keys and values)
          for (int x = n; x < kC; ++x) {
            *reinterpret_cast<uint16_t *>(v + col[x & 7] + 128 * x) = 0;
            *reinterpret_cast<uint16_t *>(v - F::kTile + col[x & 7] + 128 * x) = 0;
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(vt_ready);
      };
      auto outputs = [&](int it) {
        const int c = chunk_at(it), n = rows_of(c), t0 = w.begin + c * kC;
        const float *f = tab + set_of(c) * 3 * kC + 2 * kC;
        ok = __all_sync(0xffffffffu, mbar_wait(pv_done, (uint32_t)(it & 1), abort));
        if (!ok) return;
        tc_fence_after();
        uint32_t y[kC / 2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float v[32];
          tmem_ld32(tmem + lanes + F::kO + 32 * b, v);
          if (b == 1) {
            tc_fence_before();
            mbar_arrive(o_free);
          }
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            const float4 f4 = *reinterpret_cast<const float4 *>(f + 32 * b + x);
            y[16 * b + x / 2] = pack_bf16(v[x] * f4.x, v[x + 1] * f4.y);
            y[16 * b + x / 2 + 1] = pack_bf16(v[x + 2] * f4.z, v[x + 3] * f4.w);
          }
        }
        // the last store has read the staging tile
        if (gt == 0) bulk_wait_read<0>();
        asm volatile("bar.sync 1, %0;" ::"n"(DP) : "memory");
#pragma unroll
        for (int x = 0; x < kC; x += 2) {
          *reinterpret_cast<uint16_t *>(ob + col[x & 7] + 128 * x) = (uint16_t)y[x / 2];
          *reinterpret_cast<uint16_t *>(ob + col[(x + 1) & 7] + 128 * (x + 1)) = (uint16_t)(y[x / 2] >> 16);
        }
        if (n == kC) {
          fence_proxy_async_smem();
          asm volatile("bar.sync 1, %0;" ::"n"(DP) : "memory");
          if (gt == 0) {
#pragma unroll
            for (int x = 0; x < F::kPanels; ++x)
              tma_store_3d(&maps.m[op.o], smem_u32(ob) + x * kPanel, 64 * x, t0, (int)w.bh);
            bulk_commit();
          }
        } else {
          // a sequence that ends inside the tile: its rows alone
          asm volatile("bar.sync 1, %0;" ::"n"(DP) : "memory");
          __nv_bfloat16 *out = (__nv_bfloat16 *)p.t[op.o] + (w.bh * (long long)p.N + t0) * d;
          const int per = d / 8;
          for (int e = gt; e < n * per; e += DP) {
            const int row = e / per, ch = e - row * per;
            *reinterpret_cast<uint4 *>(out + (long long)row * d + ch * 8) =
                *reinterpret_cast<const uint4 *>(ob + (ch >> 3) * kPanel + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
          }
        }
      };
      for (int it = 0; it < nch && ok; ++it) {
        values(it);
        if (!SUMS && ok && it > 0) outputs(it - 1);
      }
      if (!SUMS && ok && nch > 0) outputs(nch - 1);
      if (!ok) fail(abort, p.info);
      if (gt == 0) bulk_wait_all();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// [BH][N][d] bf16 in boxes of 64 channels x 64 tokens, 128-byte swizzle;
// channels and tokens outside read as 0 and are not written.
bool make_token_map(CUtensorMap *m, void *base, long long BH, int N, int d) {
  auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)BH};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)N * d * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)kC, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, bool SUMS>
cudaError_t launch_t(const DecayMaps &maps, const DecayArgs &a, cudaStream_t st) {
  constexpr size_t smem = Cfg<DP>::kSmem;
  static_assert(smem <= 232448, "shared memory");
  auto *kern = decay_tc_kernel<DP, SUMS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(a.nops * a.BH * a.nseg), kThreads, smem, st>>>(maps, a);
  return cudaGetLastError();
}

}  // namespace

bool decay_tc_supported(int in_dtype, int out_dtype) { return in_dtype == VDN_BF16 && out_dtype == VDN_BF16; }

cudaError_t launch_decay_tc(const DecayArgs &a, bool sums, cudaStream_t st) {
  DecayMaps maps;
  for (int i = 0; i < kDecayTensors; ++i)
    if (a.t[i] && !make_token_map(&maps.m[i], a.t[i], a.BH, a.N, a.d)) return cudaErrorInvalidValue;
  if (a.d > 64) return sums ? launch_t<128, true>(maps, a, st) : launch_t<128, false>(maps, a, st);
  return sums ? launch_t<64, true>(maps, a, st) : launch_t<64, false>(maps, a, st);
}

}  // namespace vdn
