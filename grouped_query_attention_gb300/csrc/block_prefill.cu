// Tensor-core attention over the block-scaled int8 cache for prompts and long
// chunks (head and group sizes up to 128), fp16 or fp32 queries.
//
// CTA = two 128-row query tiles of one KV head (b, g), rows = (position,
// grouped head), whole positions of a group: of 128 rows a group of 7 heads uses
// 126. Dims behind the head size are zeros (copies past the tensors' ends). The codes of a 128-key tile become fp16 operand tiles (small
// integers, exact); S = Q K^T and O += P V run on tcgen05 with S, P and O in
// tensor memory. Scales are one number for 16 keys (the smallest block):
//   score (log2 domain)  s = S ks k_row,  k_row = scale log2(e) [2^e fp32 row]
//   P' = exp2(s - m + kLift + log2 v'),  v' = vs 2^-w in (0, 1], 2^w above the
//   largest V scale of the CTA's keys: the V scale costs an addend of the
//   exponent instead of a product per key, and l sums P' / v' per 16 keys.
// kLift = 6 keeps P' at most 2^14 (a row's reference maximum may lag by 2^8)
// and its 11 bits down to v' p = 2^-20. fp32 queries and P are split into two
// fp16 parts as in the prefill over per-channel caches: twice the MMAs.
//
// Warps: 0 TMA of the query tiles, then of the code tiles into a two-tile
// ring; 1 MMA issue, tensor memory; 2 the scales of a tile, two tiles ahead;
// 4..11 softmax, one thread per row, epilogue; 12..15 converters: code tile to
// fp16 operand tile (3 idle: register shares go by warpgroup). Converters that
// loaded the next codes themselves waited for them at every proxy fence:
// 2400 cycles a tile pair, which set the pace (4700 against 2400 of MMAs).
// The tensor-memory accumulator rounds towards zero: over thousands of keys its
// error outgrows the other fp32 roundings (2.4e-6 at 1500 keys, 3.3e-6 at
// 4096). With fp32 queries O therefore moves, every 512 keys, into fp32 sums in
// the workspace (one read and write of a row's 512 bytes through L2), and the
// next P V starts from zero.
//
// A step is 64 or 128 keys. S of 64 keys is 64 tensor-memory columns, so each
// query tile has two S buffers beside its O (2 x (2 x 64 + 128) = 512 columns)
// and S of the step after next is issued behind P.V of this one: a softmax
// never waits for its own P.V, but S runs at half the rate (its B operand is
// half as wide). S of 128 keys has one buffer, at the full rate. Every barrier
// wait is bounded.
//
// Bound: without a softcap the chain of a query tile's S, softmax and P V (of
// 3500 clocks 1850 are the softmax, 770 MMAs behind it, the rest the hand-offs
// between the roles; P V of the first 64 keys runs beside the softmax of the
// others). Two fp16 prompts of 4096 tokens, 32 heads over 8 (275 GFLOP): 244
// us, 1.13 PFLOP/s. With one, instructions: the fit, the exponents and the codes'
// conversion take 12 a score. Chunks of 8 x 512 tokens, 64 heads over 8, window
// 4096 (488 GFLOP): 651 us, 0.75 PFLOP/s, FMA pipe 39 % busy, tensor pipe 31 %.
// Two threads per row took 274 and 634 us, loops over 32 columns instead of
// unrolled steps 275 and 688, the second 64 scores kept in registers 272.
#include <cuda_fp16.h>

#include "block_internal.h"
#include "block_tc.cuh"
#include "common.cuh"
#include "tcgen05.cuh"
#include "tma_host.h"

namespace gqa {
namespace {

using namespace tc;

constexpr int kBM = 128;                       // rows per query tile
constexpr int kBN = 128;                       // keys per K/V tile
constexpr int kHD = 128;                       // dims of the operand tiles; those behind the head size are zeros
constexpr int kGroups = kBN / 16;              // 16-key groups of a tile, one scale each
constexpr int kThreads = 512;
constexpr int kSoftWarp0 = 4;
constexpr int kConvWarp0 = 12;
// Registers per thread of each warpgroup after the split (launched with 128):
// TMA + MMA, two softmax groups, converters; the sum is what was launched.
constexpr int kRegsIssue = 80, kRegsSoft = 176, kRegsConv = 80;
static_assert(kRegsIssue + 2 * kRegsSoft + kRegsConv == 4 * 128, "register split");
constexpr int kConvWarps = 4;
constexpr int kConvRows = kBN / kConvWarps;
constexpr int kScStages = 4;                   // scale slots: a tile's are read until both its softmaxes end
constexpr uint32_t kBox = 128u * 128u;         // 128 rows x 128 bytes
constexpr uint32_t kTile = 2u * kBox;          // fp16 operand tile
constexpr float kLazy = 8.0f;                  // log2 growth tolerated before rescaling O
constexpr float kMinNormal = 1.17549435e-38f;
constexpr float kLift = 6.0f;
// Keys whose V scale is below 2^-9 of the largest (kLift + log2 v' at most this)
// enter the sum of the rounded probabilities with the exact ones: theirs may
// round to nothing in fp16, and a block of zero values still has its weight.
constexpr float kRoundedLv = kLift - 9.0f;
constexpr uint32_t kIdO = idesc_f16(128, 128, 0, 1);

// F32: hi and lo query tiles (the raw fp32 tile before) and one operand tile each of K and V; fp16: two each.
template <bool F32>
struct __align__(1024) PfSmem {
  static constexpr uint32_t kQ = F32 ? 4 * kBox : 2 * kBox;
  static constexpr int kNB = F32 ? 1 : 2;
  uint8_t q[2][kQ];
  uint8_t kf[kNB][kTile];
  uint8_t vf[kNB][kTile];
  uint8_t raw[2][kBox];          // code tiles as copied
  float rho[2][kBM];             // fp32 rows: 2^e
  float ks[kScStages][kGroups];  // K scales
  float lv[kScStages][kGroups];  // kLift + log2 v'
  float iv[kScStages][kGroups];  // 2^-kLift / v'
  uint64_t sc_full[kScStages], sc_empty[kScStages];
  uint64_t raw_full[2], raw_empty[2];
  uint64_t q_land[2], q_ready[2];
  uint64_t kf_full[2], kf_empty[2], vf_full[2], vf_empty[2];
  uint64_t s_full[2][2], p_full[2][2], o_done[2];   // [query tile][buffer; P of one buffer: half]
  uint64_t drain;
  uint32_t tmem;
  unsigned vmax;                 // bits of the largest V scale
  int abort;
};
static_assert(sizeof(PfSmem<true>) + 1024 <= 232448 && sizeof(PfSmem<false>) + 1024 <= 232448, "shared memory per CTA");

template <typename SM>
__device__ __forceinline__ bool aborted(const SM& sm) {
  return *reinterpret_cast<const volatile int*>(&sm.abort) != 0;
}
template <typename SM>
__device__ __forceinline__ void set_abort(const BlockParams& p, SM& sm) {
  *reinterpret_cast<volatile int*>(&sm.abort) = 1;
  if (p.status) atomicOr(p.status, GQA_DEVICE_TIMEOUT_BIT);
}

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// a + the two halves of h, in fp32.
__device__ __forceinline__ float2 add_half2(float2 a, uint32_t h) {
  float2 r;
  asm("{ .reg .f16 l, u; mov.b32 {l, u}, %2; add.rn.f32.f16 %0, l, %3; add.rn.f32.f16 %1, u, %4; }"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h), "f"(a.x), "f"(a.y));
  return r;
}

// All bits of `v` over the 128 threads of softmax group q (named barrier 1 + q).
__device__ __forceinline__ bool group_all(bool v, int q) {
  uint32_t r;
  asm volatile("{ .reg .pred p, c; setp.ne.u32 c, %1, 0; bar.red.and.pred p, %2, 128, c; selp.u32 %0, 1, 0, p; }"
               : "=r"(r)
               : "r"((uint32_t)v), "r"(1 + q)
               : "memory");
  return r != 0;
}

// fp32 query tiles, in place, by the 256 softmax threads (wt = 0 .. 255), 8
// lanes per row: brought to [1, 2) by 2^-e (kept in rho) and split into hi
// (boxes 0, 1) and lo (boxes 2, 3) fp16 tiles over the row's own lines.
__device__ void split_rows(const BlockParams& p, PfSmem<true>& sm, int wt, int nq) {
  const int l8 = wt & 7, sub = wt >> 3, lane = wt & 31;
  for (int tile = 0; tile < nq; ++tile) {
    if (!__all_sync(0xffffffffu, mbar_wait(&sm.q_land[tile], 0, p.wait_budget)) && lane == 0) set_abort(p, sm);
    uint8_t* qt = sm.q[tile];
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const int rl = k * 32 + sub;
      float x[2][8];
      float mx = 0.f;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {   // dims 64 hf + 8 l8 ..: box 2 hf + l8 / 4, chunks 2 (l8 % 4), + 1
        const uint8_t* line = qt + (2 * hf + (l8 >> 2)) * kBox;
        const float4 a = *reinterpret_cast<const float4*>(line + sw128_offset(rl, 2 * (l8 & 3)));
        const float4 b = *reinterpret_cast<const float4*>(line + sw128_offset(rl, 2 * (l8 & 3) + 1));
        x[hf][0] = a.x; x[hf][1] = a.y; x[hf][2] = a.z; x[hf][3] = a.w;
        x[hf][4] = b.x; x[hf][5] = b.y; x[hf][6] = b.z; x[hf][7] = b.w;
#pragma unroll
        for (int e = 0; e < 8; e += 2) mx = fmax3(mx, fabsf(x[hf][e]), fabsf(x[hf][e + 1]));
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const int eb = (__float_as_int(mx) >> 23) & 0xff;
      const int e = eb == 0 ? 0 : min(eb, 253) - 127;
      const float down = __int_as_float((127 - e) << 23);
      uint32_t hw[2][4], lw[2][4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[hf][2 * i] * down, b = x[hf][2 * i + 1] * down;
          const __half2 hh = __floats2half2_rn(a, b);
          const float2 f = __half22float2(hh);
          const __half2 ll = __floats2half2_rn(a - f.x, b - f.y);
          hw[hf][i] = *reinterpret_cast<const uint32_t*>(&hh);
          lw[hf][i] = *reinterpret_cast<const uint32_t*>(&ll);
        }
      __syncwarp();   // every lane of the row has read its values
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        *reinterpret_cast<uint4*>(qt + hf * kBox + sw128_offset(rl, l8)) =
            make_uint4(hw[hf][0], hw[hf][1], hw[hf][2], hw[hf][3]);
        *reinterpret_cast<uint4*>(qt + (2 + hf) * kBox + sw128_offset(rl, l8)) =
            make_uint4(lw[hf][0], lw[hf][1], lw[hf][2], lw[hf][3]);
      }
      if (l8 == 0) sm.rho[tile][rl] = __int_as_float((127 + e) << 23);
    }
    fence_async_smem();   // rewritten tile (generic stores) -> async proxy: the S MMAs may read it
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_ready[tile]);
  }
}

// STEP: keys per step, 64 or 128 (see above). RND: the output is divided by the
// sum of the probabilities as P V has them, not by the exact one.
// nq: query tiles of a CTA, one where a KV head has no more rows.
template <bool F32, bool CAP, int STEP, bool RND, int nq>
__global__ void __launch_bounds__(kThreads, 1)
block_prefill_kernel(const BlockParams p, const __grid_constant__ CUtensorMap tmq,
                     const __grid_constant__ CUtensorMap tmo, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv) {
  using SM = PfSmem<F32>;
  using T = typename std::conditional<F32, float, __half>::type;
  constexpr int kNB = SM::kNB;
  constexpr int kSub = kBN / STEP;          // steps of a K/V tile = S buffers of a query tile
  constexpr int kHalves = STEP / 64;        // 64-column pieces of a step
  constexpr uint32_t kIdS = idesc_f16(128, STEP, 0, 0);
  constexpr int kBoxes = F32 ? 4 : 2, kBoxDims = kHD / kBoxes;
  extern __shared__ uint8_t smem_raw[];
  SM& sm = *reinterpret_cast<SM*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nrows = p.S * p.G;
  const int tr = p.tile_rows;
  const int nqb = (nrows + 2 * tr - 1) / (2 * tr);
  const bool qbm = p.qb_major != 0;
  const int qb = nqb - 1 - (int)(qbm ? blockIdx.y : blockIdx.x);   // longest key ranges first
  const int bg = (int)(qbm ? blockIdx.x : blockIdx.y), b = bg / p.Nkv, g = bg % p.Nkv;

  // ---- block-uniform checks before any barrier or tensor memory
  int total, fresh;
  if (!block_lengths(p, b, &total, &fresh)) {
    dep_wait();   // also without work: what follows on the stream waits for this kernel alone
    if (qb == nqb - 1 && g == 0 && tid == 0 && p.status) atomicOr(p.status, GQA_DEVICE_BAD_SEQLEN_BIT);
    return;
  }
  const int past = total - fresh;
  const int r0 = qb * 2 * tr;
  const int i_lo = r0 / p.G;
  const int i_hi = min((min(r0 + 2 * tr, nrows) - 1) / p.G, fresh - 1);
  if (i_lo > i_hi) {   // padding rows only
    dep_wait();
    for (int r = r0 + warp; r < min(r0 + 2 * tr, nrows); r += kThreads / 32) {   // a warp per row
      T* o = static_cast<T*>(p.out) + ((long long)(b * (long long)p.S + r / p.G) * p.N + g * p.G + r % p.G) * p.H;
      for (int x = lane; x < p.H * (int)sizeof(T) / 16; x += 32) reinterpret_cast<uint4*>(o)[x] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  const int kmax = past + i_hi + 1;
  const int kmin = p.window >= 0 ? max(0, past + i_lo - p.window) & ~15 : 0;   // scales change at multiples of 16
  const int nsteps = (kmax - kmin + STEP - 1) / STEP;
  const int ntiles = (nsteps + kSub - 1) / kSub;
  const int flush = F32 && p.o_acc ? kPrefillFlush / STEP : 1 << 30;   // steps between two flushes of O

  if (warp == 1) tmem_alloc(&sm.tmem, 512);
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.q_land[t], 1);
      mbar_init(&sm.q_ready[t], 8);
      for (int u = 0; u < 2; ++u) {
        mbar_init(&sm.s_full[t][u], 1);
        mbar_init(&sm.p_full[t][u], 4);   // warps of a softmax group
      }
      mbar_init(&sm.o_done[t], 1);
      mbar_init(&sm.kf_full[t], kConvWarps);
      mbar_init(&sm.kf_empty[t], 1);
      mbar_init(&sm.vf_full[t], kConvWarps);
      mbar_init(&sm.vf_empty[t], 1);
      mbar_init(&sm.raw_full[t], 1);
      mbar_init(&sm.raw_empty[t], kConvWarps);
    }
    for (int t = 0; t < kScStages; ++t) {
      mbar_init(&sm.sc_full[t], 1);
      mbar_init(&sm.sc_empty[t], 4 * nq);   // softmax warps
    }
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    sm.vmax = 0;
    mbar_fence_init();
  }
  if (tr < kBM) {   // rows of the query tiles that no copy fills
    for (int x = tid; x < 2 * kBoxes * (kBM - tr) * 8; x += kThreads) {
      const int box = x / ((kBM - tr) * 8), at = x % ((kBM - tr) * 8);
      *reinterpret_cast<uint4*>(sm.q[box / kBoxes] + (box % kBoxes) * kBox + tr * 128 + at * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0 && elect_one()) {   // query tiles
    for (int q = 0; q < nq; ++q) {
      mbar_arrive_tx(&sm.q_land[q], (uint32_t)(kBoxes * tr * 128));
      for (int k = 0; k < kBoxes; ++k)
        tma_load_4d(sm.q[q] + k * kBox, &tmq, kBoxDims * k, g * p.G, (r0 + q * tr) / p.G, b, &sm.q_land[q]);
    }
  }
  __syncwarp();
  dep_wait();   // the cache is complete (queries and lengths are older than the kernel ahead)
  dep_launch();
  {   // the largest V scale of the keys
    const float* vs = p.vs + (long long)bg * p.nblk;
    const int b1 = (kmax - 1) >> p.bs_log2;
    float v = 0.f;
    for (int x = (kmin >> p.bs_log2) + tid; x <= b1; x += kThreads) v = fmaxf(v, vs[x]);
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (lane == 0) atomicMax(&sm.vmax, __float_as_uint(v));
  }
  __syncthreads();
  const uint32_t tmem = sm.tmem;
  const int wexp = min(max((int)(sm.vmax >> 23) - 126, -100), 120);
  const int krow0 = bg * p.C + kmin;   // below 2^31 (checked by the host)
  // Order of the code tiles: K(0), then K(t+1) (operand tile free once
  // S_1(t+1 - kNB) is done) and V(t).
  const int nconv = 2 * ntiles;
  auto item = [&](int n, bool& is_k) -> int {
    if (n == 0) {
      is_k = true;
      return 0;
    }
    const int t = (n - 1) >> 1;
    // With one operand tile of each kind V(t) goes first: K(t+1) has to wait for S_1(t).
    const bool first = ((n - 1) & 1) == 0;
    is_k = (kNB == 1 ? !first : first) && t + 1 < ntiles;
    return is_k ? t + 1 : t;
  };

  if (warp < kSoftWarp0) {
  regs_down<kRegsIssue>();
  if (warp == 0) {
    // ================================================================ TMA of the code tiles
    bool ok = true;
    int n = 0;
    for (; n < nconv && ok; ++n) {
      bool is_k;
      const int u = item(n, is_k);
      if (u == p.withhold_tile) break;   // testing: this tile is never copied, the waits for it expire
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.raw_empty[n & 1], ((uint32_t)(n >> 1) & 1u) ^ 1u, p.wait_budget) && !aborted(sm));
      if (ok && elect_one()) {
        mbar_arrive_tx(&sm.raw_full[n & 1], kBox);
        tma_load_2d(sm.raw[n & 1], is_k ? &tmk : &tmv, 0, krow0 + u * kBN, &sm.raw_full[n & 1]);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) set_abort(p, sm);
    if (!ok) --n;
    // No copy of this CTA may still be landing when it exits.
    mbar_wait(&sm.q_land[0], 0, p.wait_budget);
    if (nq == 2) mbar_wait(&sm.q_land[1], 0, p.wait_budget);
    for (int x = n > 2 ? n - 2 : 0; x < n; ++x) mbar_wait(&sm.raw_full[x & 1], (uint32_t)(x >> 1) & 1u, p.wait_budget);
  } else if (warp == 2) {
    // ================================================================ scales
    // Lanes 0..7: K scale of a 16-key group, 8..15: V scale. Keys behind the
    // sequence are masked: any finite scale serves.
    auto load = [&](int u) -> float {
      const int j = kmin + u * kBN + 16 * (lane & (kGroups - 1));
      const float* src = (lane < kGroups ? p.ks : p.vs) + (long long)bg * p.nblk;
      return lane < 2 * kGroups && u < ntiles && j < total ? __ldg(src + (j >> p.bs_log2)) : 1.f;
    };
    float next = load(0), after = load(1);
    bool ok = true;
    for (int u = 0; u < ntiles && ok; ++u) {
      const int slot = u & (kScStages - 1);
      const float scale = next;
      next = after;
      after = load(u + 2);
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.sc_empty[slot], ((uint32_t)(u / kScStages) & 1u) ^ 1u, p.wait_budget) && !aborted(sm));
      if (!ok) break;
      if (lane < kGroups) {
        sm.ks[slot][lane] = scale;
      } else if (lane < 2 * kGroups) {
        // v' at least 2^-60: a zero block's V adds nothing that counts, but its keys' P must reach l
        const float v = fminf(fmaxf(scale * __int_as_float((127 - wexp) << 23), 0x1p-60f), 1.f);
        sm.lv[slot][lane - kGroups] = kLift + log2f(v);
        sm.iv[slot][lane - kGroups] = __fdiv_rn(0x1p-6f, v);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.sc_full[slot]);
    }
    if (!ok && lane == 0) set_abort(p, sm);
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    // Descriptors of buffer 0; a buffer further is a constant away (16-byte units).
    const uint64_t dk0 = desc_kmajor_sw128(smem_addr(sm.kf[0])), dq0 = desc_kmajor_sw128(smem_addr(sm.q[0]));
    const uint64_t dv0 = desc_mnmajor_sw128(smem_addr(sm.vf[0]), kBox, 1024);
    // S_q of step h into buffer h % kSub of query tile q: keys STEP (h % kSub) .. of K tile h / kSub.
    auto issue_s = [&](int q, int h) {
      const int bf = h % kSub, t = h / kSub;
      const uint32_t d = tmem + q * 128 + bf * STEP;
      const uint64_t b0 = dk0 + (uint64_t)((t % kNB) * (int)(kTile >> 4) + bf * (STEP * 128 >> 4));
#pragma unroll
      for (int part = F32 ? 1 : 0; part >= 0; --part) {
        // The lo tile (32 KB behind the hi tile) goes first: the accumulator's
        // roundings are relative to its size, which the hi products bring.
        const uint64_t a0 = dq0 + (uint64_t)(q * (int)(SM::kQ >> 4) + part * (int)((2 * kBox) >> 4));
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint64_t off = (uint64_t)((ks >> 2) * 1024 + (ks & 3) * 2);
          mma_f16_ss(d, a0 + off, b0 + off, kIdS, (F32 && part == 0) || ks > 0);
        }
      }
      mma_commit(&sm.s_full[q][bf]);
    };
    // O_q += P V of step h: keys 64 x .. of it in columns 64 x .. + 31 of the S buffer (lo pairs in the next 32).
    // A step of 128 keys in two halves, as their P is ready.
    auto issue_pv = [&](int q, int h, int half) {
      const int bf = h % kSub, t = h / kSub;
      const uint32_t d = tmem + 256 + q * 128;
      const uint32_t pa = tmem + q * 128 + bf * STEP;
      const uint64_t b0 = dv0 + (uint64_t)((t % kNB) * (int)(kTile >> 4) + bf * (STEP * 128 >> 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ks = 4 * half + i;
        const uint32_t col = (uint32_t)((ks >> 2) * 64 + (ks & 3) * 8);
        const uint64_t bv = b0 + (uint64_t)(ks * 128);
        mma_f16_ts(d, pa + col, bv, kIdO, h % flush > 0 || ks > 0);
        if constexpr (F32) mma_f16_ts(d, pa + col + 32, bv, kIdO, true);
      }
      if (half == kHalves - 1) mma_commit(&sm.o_done[q]);
    };
    auto wait1 = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, mbar_wait(bar, par, p.wait_budget)) != 0;
    };
    // S of step h for query tile q; the K tile is released behind its last use.
    auto next_s = [&](int q, int h) {
      if (elect_one()) {
        issue_s(q, h);
        if (q == nq - 1 && (h % kSub == kSub - 1 || h + 1 == nsteps)) mma_commit(&sm.kf_empty[(h / kSub) % kNB]);
      }
      __syncwarp();
    };
    uint64_t* q_ok = F32 ? sm.q_ready : sm.q_land;
    bool ok = wait1(&sm.kf_full[0], 0);
    for (int q = 0; q < nq && ok; ++q) {
      ok = wait1(&q_ok[q], 0);
      if (!ok) break;
      tc_fence_after();
      next_s(q, 0);
    }
    if (kSub == 2 && nsteps > 1)
      for (int q = 0; q < nq && ok; ++q) next_s(q, 1);
    for (int h = 0; h < nsteps && ok; ++h) {
      const int t = h / kSub, bf = h % kSub;
      if (bf == 0) ok = wait1(&sm.vf_full[t % kNB], (uint32_t)(t / kNB) & 1u);
      for (int q = 0; q < nq && ok; ++q) {
        if constexpr (kHalves == 2) {
          ok = wait1(&sm.p_full[q][0], (uint32_t)t & 1u);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) issue_pv(q, h, 0);
          __syncwarp();
        }
        ok = wait1(&sm.p_full[q][kHalves == 2 ? 1 : bf], (uint32_t)t & 1u);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          issue_pv(q, h, kHalves - 1);
          if (q == nq - 1 && (bf == kSub - 1 || h + 1 == nsteps)) mma_commit(&sm.vf_empty[t % kNB]);
        }
        __syncwarp();
        if (h + kSub < nsteps) {   // the buffer just read: S kSub steps on
          if (q == 0 && bf == 0) {
            ok = wait1(&sm.kf_full[(t + 1) % kNB], (uint32_t)((t + 1) / kNB) & 1u);
            if (!ok) break;
            tc_fence_after();
          }
          next_s(q, h + kSub);
        }
      }
      if (__any_sync(0xffffffffu, aborted(sm))) ok = false;
    }
    if (!ok && lane == 0) set_abort(p, sm);
    // Drain: every MMA this thread issued has finished before tensor memory is freed.
    if (elect_one()) {
      mma_commit(&sm.drain);
      mbar_wait(&sm.drain, 0, p.wait_budget);
    }
    __syncwarp();
  }
  } else if (warp >= kConvWarp0) {
    regs_down<kRegsConv>();
    // ================================================================ converters
    constexpr int kSteps = kConvRows * 8 / 32;
    const int row0 = (warp - kConvWarp0) * kConvRows;
    bool ok = true;
    for (int n = 0; n < nconv && ok; ++n) {
      bool is_k;
      const int u = item(n, is_k);
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.raw_full[n & 1], (uint32_t)(n >> 1) & 1u, p.wait_budget) && !aborted(sm));
      if (!ok) break;
      uint4 w[kSteps];
#pragma unroll
      for (int s = 0; s < kSteps; ++s)   // step s: rows row0 + 4 s .., lane = 16-byte chunk in order
        w[s] = *reinterpret_cast<const uint4*>(sm.raw[n & 1] + row0 * kHD + (s * 32 + lane) * 16);
      ok = __all_sync(0xffffffffu, mbar_wait(is_k ? &sm.kf_empty[u % kNB] : &sm.vf_empty[u % kNB],
                                             ((uint32_t)(u / kNB) & 1u) ^ 1u, p.wait_budget) && !aborted(sm));
      if (!ok) break;
      uint8_t* dst = is_k ? sm.kf[u % kNB] : sm.vf[u % kNB];
      // Chunk j (16 codes) is fp16 chunks 2 (j % 4), + 1 of box j / 4. Eight lanes
      // hold a row: those of box 1 store their odd chunk first, so that a store
      // covers all eight 16-byte bank groups.
      const int j = lane & 7, odd = j >> 2;
      uint8_t* bx = dst + odd * kBox;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int row = row0 + ((s * 32 + lane) >> 3);
        const uint4 v = odd ? make_uint4(w[s].z, w[s].w, w[s].x, w[s].y) : w[s];
        uint32_t h[8];
        codes16(v, h);
        *reinterpret_cast<uint4*>(bx + sw128_offset(row, 2 * (j & 3) + odd)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(bx + sw128_offset(row, 2 * (j & 3) + (odd ^ 1))) = make_uint4(h[4], h[5], h[6], h[7]);
      }
      fence_async_smem();   // fp16 tile (generic stores) -> async proxy: the MMAs may read it
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.raw_empty[n & 1]);
        mbar_arrive(is_k ? &sm.kf_full[u % kNB] : &sm.vf_full[u % kNB]);
      }
    }
    if (!ok && lane == 0) set_abort(p, sm);
  } else {
    // ================================================================ softmax groups
    regs_up<kRegsSoft>();
    const int q = (warp - kSoftWarp0) >> 2;   // query tile of this group
    const int quarter = warp & 3;             // tensor-memory lane quarter of this warp
    const int rl = quarter * 32 + lane;
    // Rows behind the tile's last (zeros) see what that one sees, and are not written.
    const int r = r0 + q * tr + min(rl, tr - 1);
    const bool row_ok = r < nrows;
    const int i = row_ok ? r / p.G : 0;
    const int h = g * p.G + (row_ok ? r % p.G : 0);
    const int pos = past + i;
    const bool seen = row_ok && i < fresh, live = seen && rl < tr;
    const int hi_key = seen ? pos + 1 : 0;    // visible keys [lo_key, hi_key)
    const int lo_key = p.window >= 0 ? max(0, pos - p.window) : 0;
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_addr + q * 128;
    const uint32_t o_addr = tmem + lane_addr + 256 + q * 128;
    const bool idle = q >= nq;                // no rows: the group skips everything below
    bool ok = !idle;
    float rho = 1.f;
    if constexpr (F32) {
      split_rows(p, sm, tid - 32 * kSoftWarp0, nq);
      if (!idle) {
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_ready[q], 0, p.wait_budget));   // rho of every row written
        rho = sm.rho[q][rl];
      }
    }
    const float k_row = rho * p.scale * (CAP ? 1.f / p.softcap : kLog2e);
    const float c2 = p.softcap * kLog2e;
    float m_run = kNegBig, l_run = 0.f, m_acc = kNegBig;
    [[maybe_unused]] float l_rnd = 0.f;
    // This row's sums, four floats at a time, rows of a tile side by side.
    float4* o_acc = F32 && p.o_acc ? reinterpret_cast<float4*>(p.o_acc) + ((long long)(bg * nqb + qb) * 2 + q) * (kHD / 4) * kBM + rl : nullptr;
    for (int st = 0; st < nsteps && ok; ++st) {
      const int t = st / kSub, bf = st % kSub, slot = t & (kScStages - 1);
      bool got = mbar_wait(&sm.s_full[q][bf], (uint32_t)t & 1u, p.wait_budget) && !aborted(sm);
      if (bf == 0) got = got && mbar_wait(&sm.sc_full[slot], (uint32_t)(t / kScStages) & 1u, p.wait_budget);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t s_buf = s_addr + bf * STEP;
      const float* sc_k = &sm.ks[slot][bf * (STEP / 16)];
      const int j0 = kmin + st * STEP;
      const int lo = max(lo_key - j0, 0), hi = min(hi_key - j0, STEP);   // visible columns [lo, hi)
      const bool full = __all_sync(0xffffffffu, lo == 0 && hi == STEP);
      if constexpr (F32) {
        if (st > 0 && st % flush == 0) {   // O of the steps before, complete, into the sums
          if (!__all_sync(0xffffffffu, mbar_wait(&sm.o_done[q], (uint32_t)(st - 1) & 1u, p.wait_budget))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const bool first = st == flush;
          const float f = ex2(m_acc - m_run);
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t raw[16];
            tmem_ld16(o_addr + c * 16, raw);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float4 v = make_float4(__uint_as_float(raw[4 * e]), __uint_as_float(raw[4 * e + 1]),
                                     __uint_as_float(raw[4 * e + 2]), __uint_as_float(raw[4 * e + 3]));
              float4* at = o_acc + (4 * c + e) * kBM;
              if (!first) {
                const float4 a = *at;
                v = make_float4(fmaf(a.x, f, v.x), fmaf(a.y, f, v.y), fmaf(a.z, f, v.z), fmaf(a.w, f, v.w));
              }
              *at = v;
            }
          }
          m_acc = m_run;
        }
      }
      // Row max (a softcap is monotone); a softcap also takes the largest
      // |score|. Masked columns then hold what the exponent turns into -inf:
      // -inf, or +inf under a softcap's fit (its last coefficient is negative,
      // so u Q(u^2) is -inf there).
      uint32_t x[64];
      float mt = -INFINITY, ua = 0.f;
#pragma unroll
      for (int hf = 0; hf < kHalves; ++hf) {
        tmem_ld32(s_buf + hf * 64, x);
        tmem_ld32(s_buf + hf * 64 + 32, x + 32);
        const float4 kg = *reinterpret_cast<const float4*>(sc_k + 4 * hf);
        // (Scale and row factor first: either may be far out of range where their product is not. A group that
        // is masked as a whole gives -inf, or NaN on a scale of 0, which the maximum passes over.)
        const float ksg[4] = {kg.x * k_row, kg.y * k_row, kg.z * k_row, kg.w * k_row};
        tmem_ld_wait();
        if constexpr (CAP) {
          if (!full) {
#pragma unroll
            for (int e = 0; e < 64; ++e) x[e] = (e >= lo - 64 * hf && e < hi - 64 * hf) ? x[e] : 0u;
          }
#pragma unroll
          for (int gi = 0; gi < 4; ++gi) {
            float a = 0.f, c = 0.f;
#pragma unroll
            for (int e = 16 * gi; e < 16 * gi + 16; e += 4) {
              a = fmax3(a, fabsf(__uint_as_float(x[e])), fabsf(__uint_as_float(x[e + 1])));
              c = fmax3(c, fabsf(__uint_as_float(x[e + 2])), fabsf(__uint_as_float(x[e + 3])));
            }
            ua = fmaxf(ua, fmaxf(a, c) * ksg[gi]);
          }
        }
        if (!full) {
#pragma unroll
          for (int e = 0; e < 64; ++e) x[e] = (e >= lo - 64 * hf && e < hi - 64 * hf) ? x[e] : 0xff800000u;   // -inf
        }
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
          float a = __uint_as_float(x[16 * gi]), c = __uint_as_float(x[16 * gi + 1]);
#pragma unroll
          for (int e = 16 * gi + 2; e < 16 * gi + 14; e += 4) {
            a = fmax3(a, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
            c = fmax3(c, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
          }
          a = fmax3(a, __uint_as_float(x[16 * gi + 14]), __uint_as_float(x[16 * gi + 15]));
          mt = fmaxf(mt, fmaxf(a, c) * ksg[gi]);
        }
        if (!full) {
          if constexpr (CAP) {
#pragma unroll
            for (int e = 0; e < 64; ++e) x[e] = x[e] == 0xff800000u ? 0x7f800000u : x[e];   // +inf
          }
          if constexpr (kHalves == 2) {   // read again below
            tmem_st32(s_buf + hf * 64, x);
            tmem_st32(s_buf + hf * 64 + 32, x + 32);
          }
        }
      }
      if (kHalves == 2 && !full) tmem_st_wait();
      if constexpr (CAP) {
        if (mt > kNegBig) mt = cap_far(mt, c2);   // a reference: any rounding serves
      }
      // Lazy rescale: O_q holds P.V up to the last step once that is done.
      const bool grow = mt > m_run + kLazy;
      if (__any_sync(0xffffffffu, grow)) {
        const float m_new = grow ? mt : m_run;
        if (st > 0) {
          if (!__all_sync(0xffffffffu, mbar_wait(&sm.o_done[q], (uint32_t)(st - 1) & 1u, p.wait_budget))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float f = grow ? ex2(m_run - m_new) : 1.0f;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {   // 16 columns at a time: the step's scores stay live
            uint32_t raw[16];
            tmem_ld16(o_addr + c * 16, raw);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) raw[e] = __float_as_uint(__uint_as_float(raw[e]) * f);
            tmem_st16(o_addr + c * 16, raw);
          }
          l_run *= f;
          if constexpr (RND) l_rnd *= f;
        }
        m_run = m_new;
      }
      // P' of the step: per 64 keys hi pairs over the piece's first 32 columns, lo pairs over the next.
      // MODE 0: no softcap; 3, 7: its fit of that degree; 9: any size.
      auto exponents = [&](auto mode) {
        constexpr int MODE = decltype(mode)::value;
#pragma unroll
        for (int hf = 0; hf < kHalves; ++hf) {
          if constexpr (kHalves == 2) {
            tmem_ld32(s_buf + hf * 64, x);
            tmem_ld32(s_buf + hf * 64 + 32, x + 32);
          }
          const float4 kg = *reinterpret_cast<const float4*>(sc_k + 4 * hf);
          const float4 lg = *reinterpret_cast<const float4*>(&sm.lv[slot][bf * (STEP / 16) + 4 * hf]);
          const float4 ig = *reinterpret_cast<const float4*>(&sm.iv[slot][bf * (STEP / 16) + 4 * hf]);
          // At least the smallest normal number: a masked score (-inf) times 0 would be NaN.
          const float kkg[4] = {fmaxf(kg.x * k_row, kMinNormal), fmaxf(kg.y * k_row, kMinNormal),
                                fmaxf(kg.z * k_row, kMinNormal), fmaxf(kg.w * k_row, kMinNormal)};
          const float ccg[4] = {lg.x - m_run, lg.y - m_run, lg.z - m_run, lg.w - m_run}, ivg[4] = {ig.x, ig.y, ig.z, ig.w};
          [[maybe_unused]] const float lvg[4] = {lg.x, lg.y, lg.z, lg.w};
          if constexpr (kHalves == 2) tmem_ld_wait();
#pragma unroll
          for (int qq = 0; qq < 2; ++qq) {
            uint32_t ph[16];
            [[maybe_unused]] uint32_t pl[F32 ? 16 : 1];
#pragma unroll
            for (int gi = 0; gi < 2; ++gi) {
              const int gr = 2 * qq + gi;
              const float2 kk2 = make_float2(kkg[gr], kkg[gr]), cc2 = make_float2(ccg[gr], ccg[gr]);
              float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};   // two chains
              [[maybe_unused]] float2 lr[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int e = 16 * gr + 2 * k;
                const float2 x2 = make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                float2 arg;
                if constexpr (MODE == 0) {
                  arg = ffma2(x2, kk2, cc2);
                } else {
                  const float2 u = ffma2(x2, kk2, make_float2(0.f, 0.f));
                  if constexpr (MODE == 9) {
                    const float2 y = cap_any(u, c2);
                    arg = make_float2(y.x + ccg[gr], y.y + ccg[gr]);
                    if (!full) {
                      arg.x = x[e] == 0x7f800000u ? -INFINITY : arg.x;
                      arg.y = x[e + 1] == 0x7f800000u ? -INFINITY : arg.y;
                    }
                  } else {
                    const float2 z = ffma2(u, u, make_float2(0.f, 0.f));
                    arg = ffma2(u, cap_fit<MODE>(z, c2), cc2);
                  }
                }
                const float pa = ex2(arg.x), pb = ex2(arg.y);
                ls[k & 1] = fadd2(make_float2(pa, pb), ls[k & 1]);
                const __half2 hp = __floats2half2_rn(pa, pb);
                ph[8 * gi + k] = *reinterpret_cast<const uint32_t*>(&hp);
                if constexpr (RND) lr[k & 1] = add_half2(lr[k & 1], ph[8 * gi + k]);
                if constexpr (F32) {
                  const float2 hf2 = __half22float2(hp);
                  const __half2 lp = __floats2half2_rn(pa - hf2.x, pb - hf2.y);
                  pl[8 * gi + k] = *reinterpret_cast<const uint32_t*>(&lp);
                }
              }
              const float2 lt = fadd2(ls[0], ls[1]);
              l_run = fmaf(lt.x + lt.y, ivg[gr], l_run);
              if constexpr (RND) {
                const float2 rt = fadd2(lr[0], lr[1]);
                l_rnd = fmaf(lvg[gr] > kRoundedLv ? rt.x + rt.y : lt.x + lt.y, ivg[gr], l_rnd);
              }
            }
            tmem_st16(s_buf + hf * 64 + 16 * qq, ph);
            if constexpr (F32) tmem_st16(s_buf + hf * 64 + 32 + 16 * qq, pl);
          }
          if (hf == 0 && kHalves == 2) {   // P V of the first half may start
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[q][0]);
          }
        }
      };
      if constexpr (CAP) {
        const unsigned um = __reduce_max_sync(0xffffffffu, __float_as_uint(ua));   // ua >= 0: ordered as integers
        if (um <= __float_as_uint(kCapLow))
          exponents(std::integral_constant<int, 3>());
        else if (um <= __float_as_uint(kCapHigh))
          exponents(std::integral_constant<int, 7>());
        else
          exponents(std::integral_constant<int, 9>());
      } else {
        exponents(std::integral_constant<int, 0>());
      }
      tmem_st_wait();
      // The epilogue waits for the last P.V by its phase parity: the one before
      // must be over by then (it may still run here).
      if (st > 0 && st + 1 == nsteps &&
          !__all_sync(0xffffffffu, mbar_wait(&sm.o_done[q], (uint32_t)(st - 1) & 1u, p.wait_budget))) {
        ok = false;
        break;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.p_full[q][kHalves == 2 ? 1 : bf]);
        if (bf == kSub - 1 || st + 1 == nsteps) mbar_arrive(&sm.sc_empty[slot]);
      }
    }
    // ---- epilogue: O / l (+ sink) in units of 2^(wexp - kLift), staged in the
    // group's query tile (free once its last P.V is done) and written with
    // tensor stores (rows past S are skipped).
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_done[q], (uint32_t)(nsteps - 1) & 1u, p.wait_budget) && !aborted(sm));
    if (ok) {
      tc_fence_after();
      float mf = m_run, extra = 0.f;
      if (p.sink || p.smooth) {
        const float sg = (p.sink ? (F32 ? reinterpret_cast<const float*>(p.sink)[h] : __half2float(reinterpret_cast<const __half*>(p.sink)[h])) : 0.f) * kLog2e;
        mf = fmaxf(m_run, sg);
        extra = ex2(sg - mf);
      }
      const float f = ex2(m_run - mf);
      const float den = l_run * f + extra;
      const float div = RND ? l_rnd * f + extra : den;
      const float so = (live && div > 0.f) ? f / div * __int_as_float((127 + wexp - (int)kLift) << 23) : 0.f;
      if (p.lse && live) p.lse[(long long)bg * nrows + r] = mf + log2f(den);
      uint8_t* stage = sm.q[q];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t raw[32];
        tmem_ld32(o_addr + c * 32, raw);
        tmem_ld_wait();
        if constexpr (F32) {   // box c: dims 32 c ..
          if (nsteps > flush) {
            const float fa = ex2(m_acc - m_run);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 a = o_acc[(8 * c + e) * kBM];
              raw[4 * e] = __float_as_uint(fmaf(a.x, fa, __uint_as_float(raw[4 * e])));
              raw[4 * e + 1] = __float_as_uint(fmaf(a.y, fa, __uint_as_float(raw[4 * e + 1])));
              raw[4 * e + 2] = __float_as_uint(fmaf(a.z, fa, __uint_as_float(raw[4 * e + 2])));
              raw[4 * e + 3] = __float_as_uint(fmaf(a.w, fa, __uint_as_float(raw[4 * e + 3])));
            }
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(stage + c * kBox + sw128_offset(rl, e >> 2)) =
                make_float4(__uint_as_float(raw[e]) * so, __uint_as_float(raw[e + 1]) * so,
                            __uint_as_float(raw[e + 2]) * so, __uint_as_float(raw[e + 3]) * so);
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {   // dims d ..: box d / 64, chunk (d % 64) / 8
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __half2 h2 = __floats2half2_rn(__uint_as_float(raw[e + 2 * k]) * so, __uint_as_float(raw[e + 2 * k + 1]) * so);
              u[k] = *reinterpret_cast<const uint32_t*>(&h2);
            }
            const int d = c * 32 + e;
            *reinterpret_cast<uint4*>(stage + (d >> 6) * kBox + sw128_offset(rl, (d & 63) >> 3)) = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
      }
      fence_async_smem();   // staged rows (generic stores) -> async proxy: the tensor stores read them
    }
    if (idle) {
      // nothing to write
    } else if (!group_all(ok, q)) {
      if (lane == 0) set_abort(p, sm);
    } else if (quarter == 0 && elect_one()) {   // one thread of the group
      for (int k = 0; k < kBoxes && kBoxDims * k < p.H; ++k)
        tma_store_4d(&tmo, sm.q[q] + k * kBox, kBoxDims * k, g * p.G, (r0 + q * tr) / p.G, b);
      bulk_commit();
      bulk_wait_read();   // the staged tile is read before the CTA may exit
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

constexpr int kMaxDevices = 64;

template <bool F32, bool CAP, int STEP, bool RND, int nq>
cudaError_t launch_nq(const BlockParams& p, cudaStream_t st) {
  static bool done[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  const int smem = (int)sizeof(PfSmem<F32>) + 1024;
  auto kern = block_prefill_kernel<F32, CAP, STEP, RND, nq>;
  if (!done[dev]) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    done[dev] = true;
  }
  CUtensorMap mq, mo, mk, mv;
  const uint64_t crows = (uint64_t)p.B * p.Nkv * p.C;
  if ((e = encode_u8_2d(&mk, p.kc, crows, p.H, p.H, kHD, kBN)) != cudaSuccess) return e;
  if ((e = encode_u8_2d(&mv, p.vc, crows, p.H, p.H, kHD, kBN)) != cudaSuccess) return e;
  auto encode = [&](CUtensorMap* m, const void* base) {
    return F32 ? encode_f32_query_sw128(m, base, p.B, p.S, p.N, (uint32_t)p.G, (uint64_t)p.H)
               : encode_fp16_query_sw128(m, base, p.B, p.S, p.N, (uint32_t)p.G, kBM, (uint64_t)p.H);
  };
  if ((e = encode(&mq, p.q)) != cudaSuccess) return e;
  if ((e = encode(&mo, p.out)) != cudaSuccess) return e;
  const unsigned nqb = (unsigned)((p.S * p.G + 2 * p.tile_rows - 1) / (2 * p.tile_rows)), nbg = (unsigned)(p.B * p.Nkv);
  return launch_dependent(p.k != nullptr, kern, p.qb_major ? dim3(nbg, nqb) : dim3(nqb, nbg), kThreads, (size_t)smem, st,
                          p, mq, mo, mk, mv);
}

// 8 sequences of 32 new tokens, 32 heads over 8, on 1024 keys: one tile 24 us, two (one of them empty) 33; fp32 33, 39.
template <bool F32, bool CAP, int STEP, bool RND = false>
cudaError_t launch_one(const BlockParams& p, cudaStream_t st) {
  return p.S * p.G <= p.tile_rows ? launch_nq<F32, CAP, STEP, RND, 1>(p, st) : launch_nq<F32, CAP, STEP, RND, 2>(p, st);
}

}  // namespace

cudaError_t launch_block_prefill(const BlockParams& p, cudaStream_t st) {
  const bool cap = p.softcap > 0.f;
  // With a softcap the softmax sets the pace and two S buffers hide its waits
  // (64 keys a step: 0.65 against 0.86 ms on 512-token chunks of 8 sequences);
  // without, the MMAs do, and a 64-key S takes as long as a 128-key one (0.30
  // against 0.26 ms on two 4096-token prompts). fp32: equal.
  if (p.t_type == kF32) return cap ? launch_one<true, true, 64>(p, st) : launch_one<true, false, 128>(p, st);
  // fp16 probabilities: with few keys their roundings have no company to cancel
  // in, so ranges up to 1024 keys are divided by what was added up (100 keys:
  // 2.3e-4 off instead of 4.1e-4, one rounding of the output 2.1e-4). On longer
  // ones the difference falls below 1e-4 and the second sum costs 12 % of the time.
  // The rule is the call's bound, not what a row sees, so the first rows of a long
  // prompt keep the 4.1e-4: a choice per CTA put two forms of the softmax into one
  // kernel and took 4 to 6 % more also where no CTA rounds (664 -> 687 to 708 us,
  // 394 -> 405 to 412 with 4096-token prompts), inside the steps or around them.
  if (p.T <= 1024) return cap ? launch_one<false, true, 64, true>(p, st) : launch_one<false, false, 128, true>(p, st);
  return cap ? launch_one<false, true, 64>(p, st) : launch_one<false, false, 128>(p, st);
}

}  // namespace gqa
