// Decay attention in chunks on the 5th-generation tensor cores (tcgen05 + TMEM
// + TMA), bf16 in and out, d in {16, 32, 64, 128}; sums and state in float32.
//
// Per chunk of 64 tokens (local indexes i, j; n valid rows; X the state in
// front of it, rows = value channels), with s_ij = q_i . k_j and the weights
// w_j = l^{n-1-j} (back: l^{j+1}) that take a token's write to the chunk's end:
//   X'  = l^n X + sum_j (w_j v_j) k_j^T
//   o_i = 1/w_i (l^n X q_i + sum_j s_ij w_j v_j),   j <= i (back: j >= i),
// since l^{i-j} = w_j / w_i and l^{i+1} = l^n / w_i (back: l^{j-i}, l^{n-1-i}). So the weighted values
// serve both sums, the scores need no weights of their own, and both terms of o_i share one accumulator.
// 1/w_i is at most 1/l^64; values and state carry a factor 2^c, c half of that range (45 at most): sums up to
// 2^(127-c) fit (2^82 = 5e24 in the worst head), and values down to 2^-57 = 7e-18 keep all of their bits under
// the smallest weight. A head that decays by more than 2^-90 over a chunk ("steep") would lose its
// early values to float32's range: with l^{i+1} = 2^{e_i} f_i, 1 <= f_i < 2 (back: l^{n-1-i}), it takes
//   o_i = f_i (X (2^{e_i} q_i) + sum_j c_ij s_ij v_j),   c_ij = l^{|i-j|} / f_i on the scores.
// The power of two goes onto Q's row in shared memory, once the scores have read it: exact, and no
// factor anywhere is above 1, so nothing overflows that the sums do not. Below 2^-126 a row takes
// nothing of the state: |S| |q| 2^-126 is all that it loses.
//
// Four products per chunk, all with 128 TMEM lanes:
//   SC[i][j]  = Q K^T                 A = Q, B = K (K-major tiles as TMA brings them; rows 64.. unused)
//   U[v][k]   = (w V)^T K             A = the weighted values in TMEM, B = K (MN-major)
//   O[v][i]   = X Q^T + (w V)^T P^T   A = l^n X in TMEM, B = Q; A = the weighted values (steep: V,
//                                     MN-major), B = P = the masked SC, in shared memory
// The state stays in registers in float32 and is written to TMEM once per chunk, so it never passes
// through shared memory; the outputs come transposed (lane = channel) and leave through a swizzled
// staging tile by TMA. The weighted values enter U as three bf16 parts (2^-24 together): two would
// leave 3e-6 in the float32 state. P, and the copy of the state that the outputs read, are two bf16 parts
// each (2^-17), the weighted values beside P too, so that a bf16 output is off by its own rounding and
// little else. With one part of P and of the state it was off by 1.41 times that, more in small cases, at 24
// us against 25 (prompts below), 83 against 92 (ragged), 905 against 945 (long), 434 against 470 (gradients).
//
// One CTA of 32 warps walks one segment of one (operator, batch, head):
//   warps 0, 1  : scores SC -> P (TMEM lanes 0..63)
//   warp 2      : TMA loads, the products U
//   warp 3      : TMEM allocation, the products SC and O
//   warps 4..19 : the state: lane = value channel (warp % 4), 32 key channels from 32 ((warp - 4) / 4)
//   warps 20..27: the weighted values: 32 channels (warp % 4), half of them (warp - 20) / 4
//   warps 28..31: the outputs
// Many warps with little each: every role is a chain of dependent steps on the way from one chunk
// to the next, so it is the length of a warp's share that counts.
//
// What bounds it: 10 000 instructions of all warps a chunk, in chains of TMEM reads, waits and products that
// take 2200 to 2900 cycles from one chunk to the next, and the code's size: the loops of the roles together
// are more than the instruction caches hold, so P's blocks are rolled at d = 128 (unrolled 12 % slower in
// long sequences; at d = 64, where half of the warps are idle, unrolled is 4 % faster) and masks are selects
// by bit (as words built for pairs of columns: 9 % slower). Leaving out the second parts' products alone
// changes 0 to 4 %. Measured at d = 128 in bf16: 4 x 24 heads of 512 tokens 25 us (8 chunks each); 24 heads of
// 102 816 tokens 0.77 ms alone (pass for the segments' states 0.22 ms, join 0.01, walk 0.54; 2.5 GB in and
// out, 3.4 GB moved) and 0.82 to 0.95 ms one after another, when they draw 995 W and the clock falls, so that
// it is the energy of a chunk that counts; the gradients of 20 160 tokens 0.39 ms alone, 0.43 to 0.47 in a row. At d = 64, 8 x 16 ragged heads of up to 4099 tokens 92 us, the longest walk's 65 chunks. Steep
// heads throughout: 138 us there, 1.04 ms for the long sequences.
// Tried at equal or less speed: scores and values as tf32 beside P (no splitting, but the values once more
// and one buffer of them: 103 us against 105 at d = 64 then, equal at d = 128); P by the warps of the
// other half of the lanes at d = 64, beside the issuing warps (137 us against 105), or those on the busy half
// (150); two buffers of scores at d = 64 (equal); loads of the scores ahead (12 % slower, code's size); masks
// kept in registers (7 %); the state and the outputs in two TMEM buffers at d = 64 (2 %), with two
// output tiles in shared memory (9 %); outputs by the state's warps (10 %), the scores issued by P's warp,
// one warp for all products in a fixed order (2 %).
// SUMS: only what a segment adds to the state (from zero), for the walk's later segments.
// Every wait is bounded.
#include <cudaTypedefs.h>

#include "common.cuh"
#include "decay.h"
#include "internal.h"

namespace vdn {
namespace {

constexpr int kC = kDecayC;
constexpr int kThreads = 1024;
constexpr uint32_t kPanel = kC * 128;  // 64 tokens x 64 channels
constexpr uint32_t kTmemCols = 512;

template <int DP, bool SUMS>  // channels padded to panels
struct Cfg {
  static constexpr int kPanels = DP / 64;
  static constexpr uint32_t kTile = kPanels * kPanel;
  static constexpr uint32_t kOffK = SUMS ? 0 : kTile, kOffV = kOffK + kTile;  // in a stage, behind Q
  static constexpr uint32_t kStageBytes = kOffV + kTile;
  static constexpr int kStages = !SUMS && DP == 128 ? 3 : 6;
  // shared memory, from a 1024-byte aligned base; a 128-row operand reads
  // 8 KB past its 64-row tile, which the next tile or P covers
  static constexpr uint32_t kOffP = kStages * kStageBytes;
  static constexpr uint32_t kOffO = kOffP + (SUMS ? 0 : 4 * kPanel);  // two P of two parts, an output tile
  // the weighted values' third part lies in shared memory where TMEM has no room for it
  static constexpr bool kLow = !SUMS && DP == 128;
  static constexpr uint32_t kOffLow = kOffO + (SUMS ? 0 : kTile), kLowBytes = 2 * kPanel;
  static constexpr uint32_t kOffTab = kOffLow + (kLow ? 2 * kLowBytes : 0);
  static constexpr uint32_t kTabFloats = 2 * 2 * kC + 72 + 8 + 16;  // w, f per set; l^n; carries and 2^c, 2^-c; l^-n
  static constexpr uint32_t kOffBar = kOffTab + 4 * kTabFloats;
  static constexpr uint32_t kBars = 2 * kStages + 14;
  static_assert(kBars <= 32, "a lane each");
  static constexpr size_t kSmem = 1024 + kOffBar + 8 * kBars + 16;
  static constexpr int kParts = DP / 32;  // of the state, 32 key channels each
  // TMEM columns
  static constexpr uint32_t kX = 0, kXLow = DP / 2, kU = DP, kO = kU + DP, kSC = kO + kC, kVT = kSC + kC;
  static constexpr uint32_t kVTCols = (kLow ? 2 : 3) * kC / 2;  // of each of two buffers
  static_assert(SUMS || kVT + 2 * kVTCols <= kTmemCols, "TMEM");
  // SUMS: two buffers of U as well (from column 0)
  static constexpr uint32_t kVT2 = 2 * DP;
  static_assert(kVT2 + 2 * kVTCols <= kTmemCols, "TMEM");
  static_assert(kOffBar % 8 == 0 && kOffTab % 16 == 0, "alignment");
};

struct DecayMaps {
  CUtensorMap m[kDecayTensors];
};

__device__ __forceinline__ void fail(volatile int *abort, int32_t *info) {
  *abort = 1;
  if (info) atomicExch(info, VDN_INFO_TIMEOUT);
}

// mbar_wait with the suspending test (mbarrier.try_wait): with 32 warps in the
// block, warps that spin take the issue slots of those that work.
__device__ __forceinline__ bool mbar_sleep(uint32_t bar, uint32_t parity, volatile int *abort) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    if (it == 0) t0 = global_ns();
    if (global_ns() - t0 > kWaitLimitNs) return false;
  }
}
// Whether a phase is done now, for all lanes; two at a time, so that their
// latencies (100 cycles and more under load) pass together.
__device__ __forceinline__ bool warp_test(uint32_t a, uint32_t pa, uint32_t b, uint32_t pb) {
  const bool x = mbar_try_wait(a, pa), y = mbar_try_wait(b, pb);
  return __all_sync(0xffffffffu, x && y);
}
// A whole warp waits.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
  return __all_sync(0xffffffffu, mbar_sleep(bar, parity, abort));
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds_f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts_u4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 lds_u4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
// Keeps a value from being computed anew at each of its uses.
__device__ __forceinline__ int pinned(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

__device__ __forceinline__ uint32_t as_u32(const __nv_bfloat162 &x) { return *reinterpret_cast<const uint32_t *>(&x); }
// The largest power of two in x >= 0; 0 below the normal floats.
__device__ __forceinline__ float pow2_in(float x) { return __uint_as_float(__float_as_uint(x) & 0x7F800000u); }
// A bf16 pair as two floats (the low half first).
__device__ __forceinline__ float2 unpack2(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}
// The upper 16 bits of each of x (a bf16 pair); x becomes what they leave. Cut
// off, not rounded: the next part takes up the rest, exactly, and a byte
// permutation is cheaper than a conversion.
__device__ __forceinline__ uint32_t take_bf16(float2 &x) {
  const uint32_t a = __float_as_uint(x.x), b = __float_as_uint(x.y);
  x = __ffma2_rn(make_float2(__uint_as_float(a & 0xFFFF0000u), __uint_as_float(b & 0xFFFF0000u)),
                 make_float2(-1.f, -1.f), x);
  return __byte_perm(a, b, 0x7632);
}

// x as two bf16 parts, 2^-17 of it left over: the first, and the second in `low`.
__device__ __forceinline__ uint32_t split_bf16(float2 x, uint32_t &low) {
  const uint32_t high = as_u32(__floats2bfloat162_rn(x.x, x.y));
  x = __ffma2_rn(unpack2(high), make_float2(-1.f, -1.f), x);
  low = as_u32(__floats2bfloat162_rn(x.x, x.y));
  return high;
}

// Four transposed 8 x 8 bf16 matrices (lane l: the address of row l % 8 of
// matrix l / 8). Lane l holds elements (2 (l % 4), l / 4) and (2 (l % 4) + 1,
// l / 4) of each matrix as it lies in shared memory.
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t &x, uint32_t &y, uint32_t &z, uint32_t &w) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(x), "=r"(y), "=r"(z), "=r"(w)
               : "r"(a)
               : "memory");
}
// The other way round (stsm4t), and rows as they are (stsm4).
__device__ __forceinline__ void stsm4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y),
               "r"(z), "r"(w)
               : "memory");
}
// 16 TMEM lanes x 16 words: register 2 n + e of lane l is lane l / 4 + 8 e,
// column 4 n + l % 4.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 32 TMEM lanes x 16 (8) words: lane l's row.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
// 16 TMEM lanes x 64 words: registers 4 n + 2 e + c of lane l are lane l / 4 +
// 8 e, column 8 n + 2 (l % 4) + c. The values are there after tmem_ld_frag_wait.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_frag_wait(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                 "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}

// A steep head: each valid row of Q (up to `last`) takes the power of two in its decay; `each`
// pieces of 16 bytes a thread. pw: l^n. A call of its own: within the state's loop its registers and instructions cost
// the other heads 3 to 5 % (24 heads of 102 816 tokens, d = 128), by P's warps even the steep ones more
// (8 x 16 heads of 4099 tokens, d = 64: 147 us against 136).
__device__ __noinline__ void scale_q(uint32_t tile, uint32_t pw, int piece, int threads, int each, int last, int back) {
  for (int x = 0; x < each; ++x, piece += threads) {
    const int row = (piece >> 3) & (kC - 1);
    if (row <= last) {
      const uint32_t a = tile + 16 * piece;
      const __nv_bfloat162 p2 = __float2bfloat162_rn(pow2_in(lds_f(pw + 4 * (back ? last - row : row + 1))));
      auto times = [&](uint32_t y) { return as_u32(__hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&y), p2)); };
      const uint4 y = lds_u4(a);
      sts_u4(a, times(y.x), times(y.y), times(y.z), times(y.w));
    }
  }
  fence_proxy_async_smem();
}

template <int DP, bool SUMS>
__global__ void __launch_bounds__(kThreads, 1)
    decay_tc_kernel(const __grid_constant__ DecayMaps maps, const __grid_constant__ DecayArgs p) {
  using F = Cfg<DP, SUMS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float *tab = reinterpret_cast<float *>(smem + F::kOffTab);
  float *pw = tab + 2 * 2 * kC;       // l^n, n = 0..64
  float *carry = pw + 72;             // per set: l^n of its valid rows
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + F::kOffBar);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * F::kStages;
  const uint32_t sc_full = empty0 + 8 * F::kStages, sc_free = sc_full + 8, p_ready = sc_free + 8;  // p, kv: per buffer
  const uint32_t kv_ok = p_ready + 16, kv_full = kv_ok + 16, pv_done = kv_full + 16;
  const uint32_t qx_ok = pv_done + 16, qx_done = qx_ok + 8, drain = qx_done + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + F::kBars);
  volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  constexpr int loads = SUMS ? 3 : 2;  // the warp that loads; it sets up the barriers, one per lane
  if (warp == loads) {
    constexpr int S = F::kStages;
    const int r = lane - 2 * S;
    // p_ready; kv_ok: the values are there, U has been read; qx_ok: the state is there, O has been read
    const int n = r < 0              ? (lane < S || SUMS ? 1 : 2)
                  : r >= 1 && r <= 3 ? 64
                  : r == 4 || r == 5 ? (F::kParts + 2) * DP
                  : r == 10          ? (F::kParts + 1) * DP
                  : r == 12          ? 2
                                     : 1;
    if (lane < 2 * S + 13) mbar_init(full0 + 8 * lane, n);
    if (lane == 0) *abort = 0;
    fence_barrier_init();
    __syncwarp();
  }

  const DecayWork w = decay_work(p, blockIdx.x, SUMS);
  const DecayOp &op = p.op[w.op];
  const int back = pinned(op.back);
  const bool fin = w.seg == decay_final_seg(w, back);
  launch_dependents();
  if (SUMS ? !decay_before_final(w, back) : (w.nch == 0 && !fin)) return;
  const int nch = pinned(w.nch), d = pinned(p.d);
  const int tail = pinned(w.end - w.begin - (nch - 1) * kC);  // rows of the segment's last chunk
  const float g = p.g[w.h];
  const uint32_t smem_a = (uint32_t)pinned((int)smem_u32(smem)), tab_a = smem_a + F::kOffTab;
  auto chunk_at = [&](int it) { return back ? nch - 1 - it : it; };
  auto rows_of = [&](int c) { return c == nch - 1 ? tail : kC; };

  const CUtensorMap *mq = &maps.m[op.q], *mk = &maps.m[op.k], *mv = &maps.m[op.v];
  auto load = [&](int it) {
    const uint32_t dst = smem_a + (it % F::kStages) * F::kStageBytes, fb = full0 + 8 * (it % F::kStages);
    const int t0 = w.begin + chunk_at(it) * kC;
    if (elect_one()) {
      mbar_arrive_expect_tx(fb, F::kStageBytes);
#pragma unroll
      for (int x = 0; x < F::kPanels; ++x) {
        if (!SUMS) tma_load_3d(dst + x * kPanel, mq, fb, 64 * x, t0, (int)w.bh);
        tma_load_3d(dst + F::kOffK + x * kPanel, mk, fb, 64 * x, t0, (int)w.bh);
        tma_load_3d(dst + F::kOffV + x * kPanel, mv, fb, 64 * x, t0, (int)w.bh);
      }
    }
    __syncwarp();
  };
  // it starts on the first tiles before anything else
  if (warp == loads) {
    for (int it = 0; it < nch && it < F::kStages; ++it) load(it);
  }
  if (warp == 3) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  // 0: l^64 >= 2^-90, values and state times 2^c; 1: l^64 >= 2^-126, the weights on the scores as products of
  // two powers; 2: steeper, where one of the two could leave float32's range
  const int steep = pinned((double)g * kC >= -62.383246250395077 ? 0 : (double)g * kC >= -87.3 ? 1 : 2);
  // a sequence without tokens only hands its state on, as it is
  const int c2 = steep || nch == 0 ? 0 : (int)((double)g * kC * -0.72134752044448170);  // 1 / (2 ln 2)
  // the weights of whole chunks (set 0) and of the segment's last one (set 1)
  if (threadIdx.x < 2 * kC) {
    const int set = threadIdx.x / kC, x = threadIdx.x % kC, n = set ? tail : kC;
    float *t = tab + set * 2 * kC;
    const double wx = decay_pow(g, back ? x + 1 : n - 1 - x);
    t[x] = x < n ? (float)scalbn(wx, c2) : 0.f;
    float f = 1.f;
    if (x < n && !steep) f = (float)(1.0 / scalbn(wx, c2));
    if (x < n && steep) {
      const float r = (float)decay_pow(g, back ? n - 1 - x : x + 1), p2 = pow2_in(r);
      f = p2 > 0.f ? r / p2 : 1.f;
    }
    t[kC + x] = f;
  } else if (threadIdx.x < 2 * kC + kC + 1) {
    pw[threadIdx.x - 2 * kC] = (float)decay_pow(g, threadIdx.x - 2 * kC);
  } else if (threadIdx.x >= 224 && threadIdx.x < 240) {
    const int x = threadIdx.x - 224;
    carry[8 + x] = steep == 1 ? (float)(1.0 / decay_pow(g, back ? 15 - x : x)) : 0.f;
  } else if (threadIdx.x >= 256 && threadIdx.x < 258) {
    const int set = threadIdx.x - 256;
    // l^n lies between two neighbouring floats; taking the upper one for this
    // share of the chunks keeps the product over many chunks from drifting
    const double l = decay_pow(g, set ? tail : kC);
    const float lo = __double2float_rd(l), hi = __double2float_ru(l);
    carry[4 * set] = lo;
    carry[4 * set + 3] = (float)scalbn(1.0, set ? -c2 : c2);
    carry[4 * set + 1] = hi;
    carry[4 * set + 2] = __uint_as_float(hi > lo ? __double2uint_rn((l - lo) / ((double)hi - lo) * 4294967295.0) : 0u);
  }
  if (!SUMS)
    for (uint32_t x = threadIdx.x; x < 4 * kPanel / 16; x += kThreads) sts_u4(smem_a + F::kOffP + 16 * x, 0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto set_of = [&](int c) { return c == nch - 1 ? 1 : 0; };
  // two buffers of the weighted values; of U where TMEM has the room
  constexpr int kBufU = SUMS ? 2 : 1;
  auto buf = [](int it) { return it & 1; };
  auto phase = [](int it) { return (uint32_t)((it >> 1) & 1); };
  auto u_at = [&](int it) { return tmem + (SUMS ? (uint32_t)((it & 1) * DP) : F::kU); };
  auto vt_at = [&](int it) { return tmem + (SUMS ? F::kVT2 : F::kVT) + (uint32_t)(it & 1) * F::kVTCols; };

  if (warp == 2 || warp == 3) {
    // ------------------------------------------------- loads and products
    // Two warps issue, so that one's waits pass under the other's products:
    // warp 2 the loads and U, warp 3 the scores and the outputs (with SUMS the
    // loads). A whole warp
    // walks its loop and one elected lane issues: in a branch of one lane each
    // product would first move its operands to uniform registers lane by lane
    // (200 cycles a product instead of 35 to 70).
    constexpr uint32_t id_sc = idesc_bf16_f32(128, kC, false, false);
    constexpr uint32_t id_u = idesc_bf16_f32(128, DP, false, true);
    constexpr uint32_t id_pv = idesc_bf16_f32(128, kC, true, false);
    // descriptors: one per tile and form; an offset of b bytes adds b / 16
    // values that the compiler knows to be the same in all lanes stay in uniform registers
    const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_slot, 0), sm = smem_u32(smem);
    const uint64_t kmaj = smem_desc_sw128(sm, 16, 1024), mnmaj = smem_desc_sw128(sm, kPanel, 1024);
    const uint64_t dp = kmaj + (F::kOffP >> 4);
    auto stage_off = [&](int it) { return (uint64_t)((it % F::kStages) * (F::kStageBytes >> 4)); };
    auto empty = [&](int it) { return empty0 + 8 * (it % F::kStages); };
    auto full = [&](int it) { return full0 + 8 * (it % F::kStages); };
    auto turn_of = [&](int it) { return (uint32_t)((it / F::kStages) & 1); };
    auto vt_of = [&](int it) { return tm + (SUMS ? F::kVT2 : F::kVT) + (uint32_t)(it & 1) * F::kVTCols; };
    bool ok = true;
    // every copy issued lands before the CTA may leave
    auto land = [&](int loaded) {
      volatile int never = 0;
      for (int i = loaded > F::kStages ? loaded - F::kStages : 0; i < loaded; ++i) warp_wait(full(i), turn_of(i), &never);
    };
    if (warp == 2) {
      int loaded = min(nch, F::kStages);
      for (int it = 0; it < nch; ++it) {
        // U = (w v)^T K, the smallest parts first (the values' warps have seen the tile arrive)
        ok = warp_wait(kv_ok + 8 * buf(it), phase(it), abort);
        if (!ok) break;
        tc_fence_after();
        const uint64_t k = mnmaj + stage_off(it) + (F::kOffK >> 4);
        const uint32_t u = tm + (SUMS ? (uint32_t)((it & 1) * DP) : F::kU), vt = vt_of(it);
        const uint64_t low = kmaj + ((F::kOffLow + (it & 1) * F::kLowBytes) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int part = 2; part >= 0; --part)
#pragma unroll
            for (int ks = 0; ks < kC / 16; ++ks) {
              if (F::kLow && part == 2)
                tc_mma_bf16(u, low + ks * (32 >> 4), k + ks * (2048 >> 4), id_u, ks > 0 ? 1u : 0u);
              else
                tc_mma_bf16_ts(u, vt + part * (kC / 2) + 8 * ks, k + ks * (2048 >> 4), id_u, part < 2 || ks > 0 ? 1u : 0u);
            }
          tc_commit(kv_full + 8 * buf(it));
          tc_commit(empty(it));
        }
        __syncwarp();
        // the stage of the chunk before takes the next load
        if (!SUMS && it > 0 && loaded < nch) {
          ok = warp_wait(empty(it - 1), turn_of(it - 1), abort);
          if (!ok) break;
          load(loaded++);
        }
      }
      if (!ok) fail(abort, p.info);
      if (!SUMS) land(loaded);
    } else if (SUMS) {
      int loaded = min(nch, F::kStages);
      for (; loaded < nch && ok; ++loaded) {
        ok = warp_wait(empty(loaded), turn_of(loaded - F::kStages), abort);
        if (!ok) break;
        load(loaded);
      }
      if (!ok) fail(abort, p.info);
      land(loaded);
    } else {
      auto scores = [&](int it) {
        const uint64_t q = kmaj + stage_off(it), k = q + (F::kOffK >> 4);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * kPanel + (ks & 3) * 32) >> 4;
            tc_mma_bf16(tm + F::kSC, q + off, k + off, id_sc, ks > 0 ? 1u : 0u);
          }
          tc_commit(sc_full);
        }
        __syncwarp();
      };
      if (nch > 0) {
        ok = warp_wait(full(0), 0, abort);
        if (ok) scores(0);
      }
      for (int it = 0; it < nch && ok; ++it) {
        // the next chunk's scores, so that its P is made under this one's outputs
        if (it + 1 < nch) {
          if (!warp_test(full(it + 1), turn_of(it + 1), sc_free, (uint32_t)(it & 1)))
            ok = warp_wait(full(it + 1), turn_of(it + 1), abort) && warp_wait(sc_free, (uint32_t)(it & 1), abort);
          if (!ok) break;
          tc_fence_after();
          scores(it + 1);
        }
        // O = X Q^T (a steep head: Q as the state's warps have left it)
        ok = warp_wait(qx_ok, (uint32_t)(it & 1), abort);
        if (!ok) break;
        tc_fence_after();
        const uint64_t q = kmaj + stage_off(it);
        if (elect_one()) {
#pragma unroll
          for (int part = 1; part >= 0; --part)
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks)
              tc_mma_bf16_ts(tm + F::kO, tm + (part ? F::kXLow : F::kX) + 8 * ks,
                             q + (((ks >> 2) * kPanel + (ks & 3) * 32) >> 4), id_sc, part == 0 || ks > 0 ? 1u : 0u);
          tc_commit(qx_done);
        }
        __syncwarp();
        // O += (w V)^T P^T (a steep head: V^T P^T)
        if (!warp_test(p_ready + 8 * (it & 1), phase(it), kv_ok + 8 * (it & 1), phase(it)))
          ok = warp_wait(p_ready + 8 * (it & 1), phase(it), abort) && warp_wait(kv_ok + 8 * (it & 1), phase(it), abort);
        if (!ok) break;
        tc_fence_after();
        const uint64_t pb = dp + (it & 1) * (2 * kPanel >> 4), pl = pb + (kPanel >> 4);
        const uint64_t v = mnmaj + stage_off(it) + (F::kOffV >> 4);
        const uint32_t vt = vt_of(it);
        if (elect_one()) {
          if (steep) {
#pragma unroll
            for (int part = 1; part >= 0; --part)
#pragma unroll
              for (int ks = 0; ks < kC / 16; ++ks)
                tc_mma_bf16(tm + F::kO, v + ks * (2048 >> 4), (part ? pl : pb) + ks * (32 >> 4), id_pv, 1u);
          } else {
            // values and scores in two parts each, but for the product of the second ones
#pragma unroll
            for (int part = 2; part >= 0; --part)
#pragma unroll
              for (int ks = 0; ks < kC / 16; ++ks)
                tc_mma_bf16_ts(tm + F::kO, vt + (part == 1 ? kC / 2 : 0) + 8 * ks, (part == 2 ? pl : pb) + ks * (32 >> 4), id_sc, 1u);
          }
          tc_commit(pv_done + 8 * (it & 1));
          tc_commit(empty(it));
        }
        __syncwarp();
      }
      if (!ok) fail(abort, p.info);
    }
    // every product is done before TMEM is given back
    if (elect_one()) tc_commit(drain);
    __syncwarp();
    volatile int never = 0;
    warp_wait(drain, 0, &never);
  } else if (warp < 2) {
    // ----------------------------------------------- scores -> P (row i)
    if (!SUMS) {
      // of the tile's four 32 x 32 blocks one lies outside of every mask: it
      // was cleared at the start
      const int skip = back ? (warp == 1 ? 0 : -1) : (warp == 0 ? 1 : -1);
      for (int it = 0; it < nch; ++it) {
        const int i = pinned(warp * 32 + lane);  // addresses made here, not kept
        const int c = chunk_at(it), n = rows_of(c);
        const uint32_t t = tab_a + set_of(c) * (2 * kC * 4), pw_a = tab_a + 4 * 2 * 2 * kC;
        const uint32_t row = smem_a + F::kOffP + (it & 1) * 2 * kPanel + i * 128;
        // the columns this row takes
        const uint64_t upto = (2ull << i) - 1, rows = n < kC ? (1ull << n) - 1 : ~0ull;
        const uint64_t mask = back ? rows & ~(upto >> 1) : upto;
        // once these scores are done, so is the product that read this P buffer
        if (!warp_wait(sc_full, (uint32_t)(it & 1), abort)) {
          fail(abort, p.info);
          break;
        }
        tc_fence_after();
#pragma unroll(DP == 128 ? 2 : 4)  // see the code's size above
        for (int b = 0; b < 4; ++b) {  // 16 columns
          if ((b >> 1) == skip) continue;
          float v[16];
          tmem_ld16(tmem + F::kSC + ((uint32_t)(warp * 32) << 16) + 16 * b, v);
          if (b == 3 || (b == 1 && skip == 1)) {
            tc_fence_before();
            mbar_arrive(sc_free);
          }
          if (steep) {
            const int ii = pinned(i);
            const float rf = 1.f / lds_f(t + 4 * (kC + ii));
            // 1: l^|i-j| as a power of the row's way from these 16 columns'
            // first (back: last) one and one of the column's way
            const float r = rf * lds_f(pw_a + 4 * abs(ii - 16 * b - (back ? 15 : 0)));
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const int at = pinned(steep == 2 ? abs(ii - 16 * b - x) : 80 + x);
              v[x] *= (steep == 2 ? rf : r) * lds_f(pw_a + 4 * at);
            }
          }
          const bool all = (b >> 1) != warp && n == kC;  // the block lies within the mask
          const uint32_t m = (uint32_t)(mask >> (16 * b));
          if (!all) {
#pragma unroll
            for (int x = 0; x < 16; ++x) v[x] = m >> x & 1 ? v[x] : 0.f;
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t pk[4], pl[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) pk[e] = split_bf16(make_float2(v[8 * x + 2 * e], v[8 * x + 2 * e + 1]), pl[e]);
            const uint32_t to = row + (((2 * b + x) ^ (i & 7)) << 4);
            sts_u4(to, pk[0], pk[1], pk[2], pk[3]);
            sts_u4(to + kPanel, pl[0], pl[1], pl[2], pl[3]);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(p_ready + 8 * (it & 1));
      }
    }
  } else if (warp < 20) {
    // --------------------------------------------------------- the state
    const int sub = warp & 3, part = (warp - 4) >> 2;
    const int r = sub * 32 + lane, c0 = part * 32;  // value channel, first key channel
    const uint32_t lanes = (uint32_t)(sub * 32) << 16;
    if (sub * 32 < DP && part < F::kParts) {
      float2 X[16];
      const float *src = nullptr;
      bool tr = false;
      if (!SUMS) {
        src = decay_start(p, op, w, tr);
        wait_for_launches();
      }
      const int sr = tr ? 1 : d, sc = tr ? d : 1;  // strides of a state's row and column
      const float up = lds_f(tab_a + 4 * (2 * 2 * kC + 72 + 3));
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        X[x] = make_float2(0.f, 0.f);
        if (src && r < d && c0 + 2 * x < d) {
          const float *y = src + r * sr + (c0 + 2 * x) * sc;
          X[x] = make_float2(up * y[0], up * y[sc]);
        }
      }
      auto publish = [&](int it) {
        const float lx = steep ? 1.f : lds_f(tab_a + 4 * (2 * 2 * kC + 72 + 4 * set_of(chunk_at(it))));
        const float2 sc = make_float2(lx, lx);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint32_t y[4], low[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            float2 z = X[4 * b + x];
            asm volatile("" : "+f"(z.x), "+f"(z.y));  // piece by piece: fewer registers at once
            y[x] = split_bf16(__fmul2_rn(z, sc), low[x]);
          }
          tmem_st4(tmem + lanes + F::kX + part * 16 + 4 * b, y);
          tmem_st4(tmem + lanes + F::kXLow + part * 16 + 4 * b, low);
        }
        tmem_st_wait();
        tc_fence_before();
      };
      for (int i = 0; i < kBufU; ++i) mbar_arrive(kv_ok + 8 * i);  // nothing in U yet
      bool ok = true;
      uint32_t turn = 0x80000000u;
      for (int it = 0; it < nch; ++it) {
        if (!SUMS) {
          if (it > 0) {
            ok = warp_wait(qx_done, (uint32_t)((it - 1) & 1), abort);
            if (!ok) break;
            tc_fence_after();
          }
          publish(it);
          if (steep) {
            // P is there, so the scores have read Q (the tile's own wait shows its bytes to these threads)
            const int s = it % F::kStages;
            ok = warp_wait(p_ready + 8 * buf(it), phase(it), abort) &&
                 warp_wait(full0 + 8 * s, (uint32_t)((it / F::kStages) & 1), abort);
            if (!ok) break;
            scale_q(smem_a + s * F::kStageBytes, tab_a + 4 * (2 * 2 * kC), part * DP + r, F::kParts * DP, 8 / F::kParts,
                    rows_of(chunk_at(it)) - 1, back);
          }
          mbar_arrive(qx_ok);
        }
        const float4 ca = lds_f4(tab_a + 4 * (2 * 2 * kC + 72 + 4 * set_of(chunk_at(it))));
        const uint32_t before = turn;
        turn += __float_as_uint(ca.z);
        const float ll = turn < before ? ca.y : ca.x;
        const float2 l = make_float2(ll, ll);
        ok = warp_wait(kv_full + 8 * buf(it), phase(it), abort);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          float u[8];
          tmem_ld8(u_at(it) + lanes + c0 + 8 * b, u);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            float2 &y = X[4 * b + x];
            y = __ffma2_rn(y, l, make_float2(u[2 * x], u[2 * x + 1]));
          }
        }
        tc_fence_before();
        mbar_arrive(kv_ok + 8 * buf(it + kBufU));
      }
      if (!ok) fail(abort, p.info);
      // where it goes is found anew: kept over the loop, it would cost registers
      const int tid = pinned((int)threadIdx.x), blk = pinned((int)blockIdx.x), r1 = tid & 127, c1 = ((tid >> 7) - 1) * 32;
      const DecayWork w1 = decay_work(p, blk, SUMS);
      const DecayOp &op1 = p.op[w1.op];
      float *dst = nullptr;
      if (SUMS)
        dst = p.ws + (long long)blk * p.d * p.d;
      else if (w1.seg == decay_final_seg(w1, op1.back) && op1.s_out)
        dst = op1.s_out + w1.bh * (long long)p.d * p.d;
      const float down = lds_f(tab_a + 4 * (2 * 2 * kC + 72 + 7));
      if (dst && r1 < p.d) {
#pragma unroll
        for (int x = 0; x < 32; x += 4)
          if (c1 + x < p.d)
            *reinterpret_cast<float4 *>(dst + r1 * p.d + c1 + x) =
                make_float4(down * X[x / 2].x, down * X[x / 2].y, down * X[x / 2 + 1].x, down * X[x / 2 + 1].y);
      }
    }
  } else {
    // -------------------------------------- weighted values and outputs
    // In fragments of 16 channels x 16 tokens: ldmatrix and stmatrix transpose
    // between the tiles (rows = tokens) and TMEM (lanes = channels).
    const int sub = warp & 3;
    if (sub * 32 < DP) {
      bool ok = true;
      const int gt = (int)threadIdx.x - 896;  // thread of the outputs' warps
      const uint32_t ob = smem_a + F::kOffO, lanes = (uint32_t)(sub * 32) << 16;
      // this lane's matrix row: token 8 (lane / 16) + lane % 8 of a pair of
      // token groups, channels 8 ((lane / 8) % 2) .. of a group of 16
      auto row_at = [&](int h) {
        const uint32_t ch = (uint32_t)(sub * 4 + h * 2 + ((lane >> 3) & 1));  // group of 8 channels
        return (ch >> 3) * kPanel + (uint32_t)((lane >> 4) * 8 + (lane & 7)) * 128u + (((ch & 7) ^ (uint32_t)(lane & 7)) << 4);
      };
      const int tok = 2 * (lane & 3);  // this lane's tokens: 8 n + tok, + 1
      auto values = [&](int it, int h, uint32_t at) {
        const int s = it % F::kStages, c = chunk_at(it), n = rows_of(c);
        const uint32_t v = smem_a + s * F::kStageBytes + F::kOffV;
        const uint32_t wt = tab_a + set_of(c) * (2 * kC * 4) + 4 * tok;
        ok = warp_wait(full0 + 8 * s, (uint32_t)((it / F::kStages) & 1), abort);
        if (!ok) return;
        uint32_t x[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) ldsm4t(v + at + e * 2048, x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        if (n < kC) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int j = 8 * (e >> 1) + tok;
            x[e] = j + 1 < n ? x[e] : j < n ? x[e] & 0xFFFFu : 0u;
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t m[8], l[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int g8 = 4 * half + e;  // token group
            const float2 w2 = lds_f2(wt + 32 * g8);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float2 y = __fmul2_rn(unpack2(x[2 * g8 + q]), w2);
              x[2 * g8 + q] = take_bf16(y);
              m[2 * e + q] = take_bf16(y);
              l[2 * e + q] = as_u32(__floats2bfloat162_rn(y.x, y.y));
            }
          }
          // the products of the chunk before in this buffer have read it
          if (half == 0 && it >= 2) {
            if (SUMS)
              ok = warp_wait(kv_full + 8 * buf(it), phase(it - 2), abort);
            else if (!warp_test(kv_full + 8 * buf(it), phase(it - 2), pv_done + 8 * buf(it), phase(it - 2)))
              ok = warp_wait(kv_full + 8 * buf(it), phase(it - 2), abort) &&
                   warp_wait(pv_done + 8 * buf(it), phase(it - 2), abort);
            if (!ok) return;
            tc_fence_after();
          }
          const uint32_t to = vt_at(it) + lanes + ((uint32_t)(16 * h) << 16) + 16 * half;
          tmem_st_frag(to, &x[8 * half]);
          tmem_st_frag(to + kC / 2, m);
          if (F::kLow) {
            // rows of channels, 8 tokens (16 bytes) a piece
            const uint32_t row = smem_a + F::kOffLow + buf(it) * F::kLowBytes +
                                 (uint32_t)(sub * 32 + 16 * h + (lane & 15)) * 128u;
#pragma unroll
            for (int e = 0; e < 2; ++e)
              stsm4(row + (((uint32_t)(4 * half + 2 * e + (lane >> 4)) ^ (uint32_t)(lane & 7)) << 4), l[4 * e], l[4 * e + 1],
                    l[4 * e + 2], l[4 * e + 3]);
          } else {
            tmem_st_frag(to + kC, l);
          }
        }
        if (n < kC) {
          // what lies behind the sequence's end meets zeros in the products:
          // it may be no number, so it is cleared (keys and values; every
          // warp its own 16 channels, 2 of its lanes to a row)
          __syncwarp();
          for (int y = n + (lane >> 1); y < kC; y += 16) {
            const uint32_t ch = (uint32_t)(sub * 4 + h * 2 + (lane & 1));
            const uint32_t a = v + (ch >> 3) * kPanel + y * 128 + (((ch & 7) ^ (uint32_t)(y & 7)) << 4);
            sts_u4(a, 0, 0, 0, 0);
            sts_u4(a - F::kOffV + F::kOffK, 0, 0, 0, 0);
          }
        }
        if (F::kLow || n < kC) fence_proxy_async_smem();
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(kv_ok + 8 * buf(it));
      };
      auto outputs = [&](int it, uint32_t at0, uint32_t at1) {
        const int c = chunk_at(it), n = rows_of(c), t0 = w.begin + c * kC;
        const uint32_t f = tab_a + (set_of(c) * 2 + 1) * kC * 4 + 4 * tok;
        // the last store has read the staging tile
        if (gt == 0) bulk_wait_read<0>();
        asm volatile("bar.sync 1, %0;" ::"n"(DP) : "memory");
        ok = ok && warp_wait(pv_done + 8 * buf(it), phase(it), abort);
        tc_fence_after();
        if (ok) {
          const uint32_t o = tmem + lanes + F::kO;
          float v[32];
          uint32_t y[16];
          auto pack = [&]() {
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              const float2 f2 = lds_f2(f + 32 * m);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const float2 z = __fmul2_rn(make_float2(v[4 * m + 2 * q], v[4 * m + 2 * q + 1]), f2);
                y[2 * m + q] = as_u32(__floats2bfloat162_rn(z.x, z.y));
              }
            }
          };
          auto stage = [&](uint32_t at) {
#pragma unroll
            for (int e = 0; e < 4; ++e) stsm4t(ob + at + e * 2048, y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          };
          tmem_ld_frag(o, v);
          tmem_ld_frag_wait(v);
          pack();
          tmem_ld_frag(o + (16u << 16), v);  // under the first half's way out
          stage(at0);
          tmem_ld_frag_wait(v);
          tc_fence_before();
          mbar_arrive(qx_ok);
          pack();
          stage(at1);
        }
        fence_proxy_async_smem();
        asm volatile("bar.sync 1, %0;" ::"n"(DP) : "memory");
        if (n == kC) {
          if (ok && gt == 0) {
#pragma unroll
            for (int x = 0; x < F::kPanels; ++x)
              tma_store_3d(&maps.m[op.o], ob + x * kPanel, 64 * x, t0, (int)w.bh);
            bulk_commit();
          }
        } else if (ok) {
          // a sequence that ends inside the tile: its rows alone
          __nv_bfloat16 *out = (__nv_bfloat16 *)p.t[op.o] + (w.bh * (long long)p.N + t0) * d;
          const int per = d / 8;
          for (int e = gt; e < n * per; e += DP) {
            const int row = e / per, ch = e - row * per;
            *reinterpret_cast<uint4 *>(out + (long long)row * d + ch * 8) =
                lds_u4(ob + (ch >> 3) * kPanel + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
          }
        }
      };
      if (warp < 28) {
        const int h = (warp - 20) >> 2;
        const uint32_t at = row_at(h);
        for (int it = 0; it < nch && ok; ++it) values(it, h, at);
      } else if (!SUMS) {
        const uint32_t at0 = row_at(0), at1 = row_at(1);
        mbar_arrive(qx_ok);  // nothing in O yet
        // after a failed wait: keep the barriers, skip the work
        for (int it = 0; it < nch; ++it) outputs(it, at0, at1);
      }
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
  constexpr size_t smem = Cfg<DP, SUMS>::kSmem;
  static_assert(smem <= 232448, "shared memory");
  auto *kern = decay_tc_kernel<DP, SUMS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long grid = SUMS ? a.nsums * a.BH * a.nseg * a.nsub : a.nops * a.BH * a.nseg;
  return launch_after(kern, grid, kThreads, smem, st, !SUMS && a.nseg > 1, maps, a);
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
