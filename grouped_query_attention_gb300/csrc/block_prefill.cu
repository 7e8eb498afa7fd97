// Tensor-core attention over the block-scaled int8 cache for prompts and long
// chunks (head size 128, group size dividing 128), fp16 or fp32 queries.
//
// CTA = two 128-row query tiles of one KV head (b, g), rows = (position,
// grouped head). The codes of a 128-key tile become fp16 operand tiles (small
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
// Warps: 0 TMA of the query tiles; 1 MMA issue, tensor memory; 2..9 softmax,
// one thread per row, epilogue; 10..13 converters: codes of the next K or V
// tile from global memory into registers while the current one is converted.
// S0 | S1 | O0 | O1 in tensor memory; the order of the MMAs is the other
// prefills'. Every barrier wait is bounded.
#include <cuda_fp16.h>

#include "block_internal.h"
#include "common.cuh"
#include "tcgen05.cuh"
#include "tma_host.h"

namespace gqa {
namespace {

using namespace tc;

constexpr int kBM = 128;                       // rows per query tile
constexpr int kBN = 128;                       // keys per K/V tile
constexpr int kHD = 128;                       // head size
constexpr int kGroups = kBN / 16;              // 16-key groups of a tile, one scale each
constexpr int kThreads = 448;
constexpr int kConvWarp0 = 10;
constexpr int kConvWarps = 4;
constexpr int kConvRows = kBN / kConvWarps;
constexpr int kScStages = 4;                   // scale slots: a tile's are read until both its softmaxes end
constexpr uint32_t kBox = 128u * 128u;         // 128 rows x 128 bytes
constexpr uint32_t kTile = 2u * kBox;          // fp16 operand tile
constexpr float kLazy = 8.0f;                  // log2 growth tolerated before rescaling O
constexpr float kLift = 6.0f;
constexpr uint32_t kIdS = idesc_f16(128, 128, 0, 0);
constexpr uint32_t kIdO = idesc_f16(128, 128, 0, 1);

// F32: hi and lo query tiles (the raw fp32 tile before), one V buffer; fp16: one tile, two V buffers.
template <bool F32>
struct __align__(1024) PfSmem {
  static constexpr uint32_t kQ = F32 ? 4 * kBox : 2 * kBox;
  static constexpr int kVB = F32 ? 1 : 2;
  uint8_t q[2][kQ];
  uint8_t kf[2][kTile];
  uint8_t vf[kVB][kTile];
  float rho[2][kBM];             // fp32 rows: 2^e
  float ks[kScStages][kGroups];  // K scales
  float lv[kScStages][kGroups];  // kLift + log2 v'
  float iv[kScStages][kGroups];  // 2^-kLift / v'
  uint64_t q_land[2], q_ready[2];
  uint64_t kf_full[2], kf_empty[2], vf_full[2], vf_empty[2];
  uint64_t s_full[2], p_full[2], o_done[2];
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

// Sixteen codes as fp16: byte x ^ 0x80 under the exponent of 1024, less 1152.
__device__ __forceinline__ void codes16(uint4 w, uint32_t* h) {
  const __half2 bias = __floats2half2_rn(1152.f, 1152.f);
  const uint32_t wv[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t p01 = __byte_perm(wv[k], 0x64646464u, 0x4140u);
    const uint32_t p23 = __byte_perm(wv[k], 0x64646464u, 0x4342u);
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&p01), bias);
    const __half2 c = __hsub2(*reinterpret_cast<const __half2*>(&p23), bias);
    h[2 * k] = *reinterpret_cast<const uint32_t*>(&a);
    h[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&c);
  }
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

// c tanh(u) log2(e) on |u| <= 5/8 as u Q(u^2), Q the degree-5 least-squares fit
// of tanh(u) / u in u^2 (relative error 5e-8 in fp32 Horner); a warp's half
// with a larger |u| takes c (1 - 2 / (e^2u + 1)) for those values, whose own
// size keeps the cancellation harmless. As packed pairs: 8 instructions for
// two scores against four special-function ones.
constexpr float kCapZ = 0.625f * 0.625f;
__device__ __forceinline__ float2 cap_poly(float2 u, float2 z, const float* q) {
  float2 y = make_float2(q[5], q[5]);
#pragma unroll
  for (int i = 4; i >= 0; --i) y = ffma2(y, z, make_float2(q[i], q[i]));
  return ffma2(u, y, make_float2(0.f, 0.f));
}
__device__ __forceinline__ float cap_exp(float u, float c2) {
  return fmaf(__frcp_rn(ex2(u * (2.f * kLog2e)) + 1.f), -2.f * c2, c2);
}

// fp32 query tiles, in place, by the 256 softmax threads (wt = 0 .. 255), 8
// lanes per row: brought to [1, 2) by 2^-e (kept in rho) and split into hi
// (boxes 0, 1) and lo (boxes 2, 3) fp16 tiles over the row's own lines.
__device__ void split_rows(const BlockParams& p, PfSmem<true>& sm, int wt) {
  const int l8 = wt & 7, sub = wt >> 3, lane = wt & 31;
  for (int tile = 0; tile < 2; ++tile) {
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

template <bool F32, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
block_prefill_kernel(const BlockParams p, const __grid_constant__ CUtensorMap tmq,
                     const __grid_constant__ CUtensorMap tmo) {
  using SM = PfSmem<F32>;
  using T = typename std::conditional<F32, float, __half>::type;
  constexpr int kVB = SM::kVB;
  constexpr int kBoxes = F32 ? 4 : 2, kBoxDims = kHD / kBoxes;
  extern __shared__ uint8_t smem_raw[];
  SM& sm = *reinterpret_cast<SM*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nrows = p.S * p.G;
  const int nqb = (nrows + 2 * kBM - 1) / (2 * kBM);
  const bool qbm = p.qb_major != 0;
  const int qb = nqb - 1 - (int)(qbm ? blockIdx.y : blockIdx.x);   // longest key ranges first
  const int bg = (int)(qbm ? blockIdx.x : blockIdx.y), b = bg / p.Nkv, g = bg % p.Nkv;

  // ---- block-uniform checks before any barrier or tensor memory
  int total, fresh;
  if (!block_lengths(p, b, &total, &fresh)) {
    if (qb == nqb - 1 && g == 0 && tid == 0 && p.status) atomicOr(p.status, GQA_DEVICE_BAD_SEQLEN_BIT);
    return;
  }
  const int past = total - fresh;
  const int r0 = qb * 2 * kBM;
  const int i_lo = r0 / p.G;
  const int i_hi = min((min(r0 + 2 * kBM, nrows) - 1) / p.G, fresh - 1);
  if (i_lo > i_hi) {   // padding rows only
    for (int x = tid; x < 2 * kBM * kHD; x += kThreads) {
      const int r = r0 + x / kHD, d = x % kHD;
      if (r < nrows)
        static_cast<T*>(p.out)[((long long)(b * (long long)p.S + r / p.G) * p.N + g * p.G + r % p.G) * kHD + d] = T(0.f);
    }
    return;
  }
  const int kmax = past + i_hi + 1;
  const int kmin = p.window >= 0 ? max(0, past + i_lo - p.window) & ~15 : 0;   // scales change at multiples of 16
  const int ntiles = (kmax - kmin + kBN - 1) / kBN;

  if (warp == 1) tmem_alloc(&sm.tmem, 512);
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.q_land[t], 1);
      mbar_init(&sm.q_ready[t], 8);
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.p_full[t], kBM);
      mbar_init(&sm.o_done[t], 1);
      mbar_init(&sm.kf_full[t], kConvWarps);
      mbar_init(&sm.kf_empty[t], 1);
      mbar_init(&sm.vf_full[t], kConvWarps);
      mbar_init(&sm.vf_empty[t], 1);
    }
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    sm.vmax = 0;
    mbar_fence_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0 && elect_one()) {   // query tiles
    for (int q = 0; q < 2; ++q) {
      mbar_arrive_tx(&sm.q_land[q], SM::kQ);
      for (int k = 0; k < kBoxes; ++k)
        tma_load_4d(sm.q[q] + k * kBox, &tmq, kBoxDims * k, g * p.G, (r0 + q * kBM) / p.G, b, &sm.q_land[q]);
    }
  }
  __syncwarp();
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
  const long long krow0 = (long long)bg * p.C + kmin;

  if (warp == 0) {
    // No copy of this CTA may still be landing when it exits.
    mbar_wait(&sm.q_land[0], 0, p.wait_budget);
    mbar_wait(&sm.q_land[1], 0, p.wait_budget);
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    uint64_t dk[2], dq[2], dv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      dk[i] = desc_kmajor_sw128(smem_addr(sm.kf[i]));
      dq[i] = desc_kmajor_sw128(smem_addr(sm.q[i]));
      dv[i] = desc_mnmajor_sw128(smem_addr(sm.vf[i % kVB]), kBox, 1024);
    }
    auto issue_s = [&](int q, int kb) {
      const uint32_t d = tmem + q * 128;
#pragma unroll
      for (int part = 0; part < (F32 ? 2 : 1); ++part) {   // the lo tile starts 32 KB after the hi tile
        const uint64_t a0 = dq[q] + (uint64_t)(part * (int)((2 * kBox) >> 4));
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint64_t off = (uint64_t)((ks >> 2) * 1024 + (ks & 3) * 2);
          mma_f16_ss(d, a0 + off, dk[kb] + off, kIdS, part > 0 || ks > 0);
        }
      }
      mma_commit(&sm.s_full[q]);
    };
    // Keys 64 h .. of P: hi pairs in columns 64 h .. + 31 of S_q (lo pairs in the next 32).
    auto issue_pv = [&](int q, int vb, bool acc) {
      const uint32_t d = tmem + 256 + q * 128;
      const uint32_t pa = tmem + q * 128;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint32_t col = (uint32_t)((ks >> 2) * 64 + (ks & 3) * 8);
        const uint64_t bv = dv[vb] + (uint64_t)(ks * 128);
        mma_f16_ts(d, pa + col, bv, kIdO, acc || ks > 0);
        if constexpr (F32) mma_f16_ts(d, pa + col + 32, bv, kIdO, true);
      }
      mma_commit(&sm.o_done[q]);
    };
    auto wait1 = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, mbar_wait(bar, par, p.wait_budget)) != 0;
    };
    uint64_t* q_ok = F32 ? sm.q_ready : sm.q_land;
    bool ok = wait1(&q_ok[0], 0) && wait1(&sm.kf_full[0], 0);
    if (ok && elect_one()) {
      tc_fence_after();
      issue_s(0, 0);
    }
    __syncwarp();
    if (ok) ok = wait1(&q_ok[1], 0);
    if (ok && elect_one()) {
      tc_fence_after();
      issue_s(1, 0);
      mma_commit(&sm.kf_empty[0]);
    }
    __syncwarp();
    for (int t = 0; t < ntiles && ok; ++t) {
      const uint32_t tp = (uint32_t)t & 1u;
      const bool more = t + 1 < ntiles;
      const int kb1 = (t + 1) & 1, vb = t % kVB;
      if (!wait1(&sm.vf_full[vb], (uint32_t)(t / kVB) & 1u) || !wait1(&sm.p_full[0], tp)) {
        ok = false;
        break;
      }
      if (elect_one()) {
        tc_fence_after();
        issue_pv(0, vb, t > 0);
      }
      __syncwarp();
      if (more && !wait1(&sm.kf_full[kb1], (uint32_t)((t + 1) >> 1) & 1u)) {
        ok = false;
        break;
      }
      if (more && elect_one()) {
        tc_fence_after();
        issue_s(0, kb1);
      }
      __syncwarp();
      if (!wait1(&sm.p_full[1], tp)) {
        ok = false;
        break;
      }
      if (elect_one()) {
        tc_fence_after();
        issue_pv(1, vb, t > 0);
        mma_commit(&sm.vf_empty[vb]);
        if (more) {
          issue_s(1, kb1);
          mma_commit(&sm.kf_empty[kb1]);
        }
      }
      __syncwarp();
      if (__any_sync(0xffffffffu, aborted(sm))) ok = false;
    }
    if (!ok && lane == 0) set_abort(p, sm);
    // Drain: every MMA this thread issued has finished before tensor memory is freed.
    if (elect_one()) {
      mma_commit(&sm.drain);
      mbar_wait(&sm.drain, 0, p.wait_budget);
    }
    __syncwarp();
  } else if (warp >= kConvWarp0) {
    // ================================================================ converters
    // Order: K(0), then K(t+1) (its buffer is free once S_1(t-1) is done) and
    // V(t). The scales of a tile (both kinds) go out with its K.
    constexpr int kSteps = kConvRows * 8 / 32;
    const int row0 = (warp - kConvWarp0) * kConvRows;
    const long long ncache = (long long)p.B * p.Nkv * p.C;
    const int nconv = 2 * ntiles;
    auto item = [&](int n, bool& is_k) -> int {
      if (n == 0) {
        is_k = true;
        return 0;
      }
      const int t = (n - 1) >> 1;
      is_k = ((n - 1) & 1) == 0 && t + 1 < ntiles;
      return is_k ? t + 1 : t;
    };
    auto load = [&](int n, uint4* w, float& scale) {
      bool is_k;
      const int u = item(n, is_k);
      const int8_t* cache = is_k ? p.kc : p.vc;
      const long long grow0 = krow0 + (long long)u * kBN + row0;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int x = s * 32 + lane;
        const long long gr = grow0 + (x >> 3);
        w[s] = gr < ncache ? __ldg(reinterpret_cast<const uint4*>(cache + gr * kHD + (x & 7) * 16)) : make_uint4(0u, 0u, 0u, 0u);
      }
      if (is_k && warp == kConvWarp0 && lane < 2 * kGroups) {
        const int j = kmin + u * kBN + 16 * (lane & (kGroups - 1));
        const float* src = (lane < kGroups ? p.ks : p.vs) + (long long)bg * p.nblk;
        scale = j < total ? __ldg(src + (j >> p.bs_log2)) : 1.f;   // masked keys: any finite scale
      }
    };
    bool withheld = false;
    auto convert = [&](int n, const uint4* w, float scale) -> bool {
      bool is_k;
      const int u = item(n, is_k);
      if (u == p.withhold_tile) {   // testing: this tile is never converted, the waits for it expire
        withheld = true;
        return false;
      }
      uint64_t* empty = is_k ? &sm.kf_empty[u & 1] : &sm.vf_empty[u % kVB];
      const uint32_t pe = (is_k ? (uint32_t)(u >> 1) : (uint32_t)(u / kVB)) & 1u;
      if (!__all_sync(0xffffffffu, mbar_wait(empty, pe ^ 1u, p.wait_budget)) || aborted(sm)) return false;
      uint8_t* dst = is_k ? sm.kf[u & 1] : sm.vf[u % kVB];
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int x = s * 32 + lane, row = row0 + (x >> 3), j = x & 7;
        uint32_t h[8];
        codes16(w[s], h);
        uint8_t* bx = dst + (j >> 2) * kBox;
        *reinterpret_cast<uint4*>(bx + sw128_offset(row, 2 * (j & 3))) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(bx + sw128_offset(row, 2 * (j & 3) + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
      }
      if (is_k && warp == kConvWarp0 && lane < 2 * kGroups) {
        const int slot = u & (kScStages - 1), grp = lane & (kGroups - 1);
        if (lane < kGroups) {
          sm.ks[slot][grp] = fmaxf(scale, 1e-30f);   // positive: a mask of -inf stays -inf
        } else {
          // v' at least 2^-60: a zero block's V adds nothing that counts, but its keys' P must reach l
          const float v = fminf(fmaxf(scale * __int_as_float((127 - wexp) << 23), 0x1p-60f), 1.f);
          sm.lv[slot][grp] = kLift + log2f(v);
          sm.iv[slot][grp] = __fdiv_rn(0x1p-6f, v);
        }
      }
      fence_async_smem();   // fp16 tile (generic stores) -> async proxy: the MMAs may read it
      __syncwarp();
      if (lane == 0) mbar_arrive(is_k ? &sm.kf_full[u & 1] : &sm.vf_full[u % kVB]);
      return true;
    };
    uint4 wa[kSteps], wb[kSteps];
    float sa = 1.f, sb = 1.f;
    bool ok = true;
    load(0, wa, sa);
    for (int n = 0; n < nconv && ok; n += 2) {
      if (n + 1 < nconv) load(n + 1, wb, sb);
      ok = convert(n, wa, sa);
      if (!ok || n + 1 >= nconv) break;
      if (n + 2 < nconv) load(n + 2, wa, sa);
      ok = convert(n + 1, wb, sb);
    }
    if (!ok && !withheld && lane == 0) set_abort(p, sm);
  } else {
    // ================================================================ softmax groups
    const int q = (warp - 2) >> 2;            // query tile of this group
    const int quarter = warp & 3;             // tensor-memory lane quarter of this warp
    const int rl = quarter * 32 + lane;
    const int r = r0 + q * kBM + rl;
    const bool row_ok = r < nrows;
    const int i = row_ok ? r / p.G : 0;
    const int h = g * p.G + (row_ok ? r % p.G : 0);
    const int pos = past + i;
    const bool live = row_ok && i < fresh;
    const int hi_key = live ? pos + 1 : 0;    // visible keys [lo_key, hi_key)
    const int lo_key = p.window >= 0 ? max(0, pos - p.window) : 0;
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_addr + q * 128;
    const uint32_t o_addr = tmem + lane_addr + 256 + q * 128;
    bool ok = true;
    float rho = 1.f;
    if constexpr (F32) {
      split_rows(p, sm, tid - 64);
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_ready[q], 0, p.wait_budget));   // rho of every row written
      rho = sm.rho[q][rl];
    }
    const float k_row = rho * p.scale * (CAP ? 1.f / p.softcap : kLog2e);
    float cq[6];
    const float c2 = p.softcap * kLog2e;
    if constexpr (CAP) {
      const float fit[6] = {1.0f, -0.3333325982093811f, 0.13331091403961182f, -0.053718484938144684f,
                            0.020583488047122955f, -0.005652355030179024f};
#pragma unroll
      for (int e = 0; e < 6; ++e) cq[e] = fit[e] * c2;
    }
    float m_run = kNegBig, l_run = 0.f;
    for (int t = 0; t < ntiles && ok; ++t) {
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.s_full[q], (uint32_t)t & 1u, p.wait_budget) && !aborted(sm))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int slot = t & (kScStages - 1);
      const int j0 = kmin + t * kBN;
      const int lo = max(lo_key - j0, 0), hi = min(hi_key - j0, kBN);   // visible columns [lo, hi)
      const bool full = __all_sync(0xffffffffu, lo == 0 && hi == kBN);
      // Pass 1: row max, 64 columns at a time; masked (and softcapped) scores are written back.
      float mt = kNegBig;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t x[64];
        tmem_ld32(s_addr + hf * 64, x);
        tmem_ld32(s_addr + hf * 64 + 32, x + 32);
        tmem_ld_wait();
        const float4 kg = *reinterpret_cast<const float4*>(&sm.ks[slot][4 * hf]);
        const float ksg[4] = {kg.x, kg.y, kg.z, kg.w};
        if constexpr (CAP) {
          float zmax = 0.f;
#pragma unroll
          for (int gi = 0; gi < 4; ++gi) {
            const float f = ksg[gi] * k_row;
            const float2 f2 = make_float2(f, f);
#pragma unroll
            for (int e = 16 * gi; e < 16 * gi + 16; e += 2) {
              const float2 u = ffma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), f2, make_float2(0.f, 0.f));
              const float2 z = ffma2(u, u, make_float2(0.f, 0.f));
              zmax = fmax3(zmax, z.x, z.y);
              const float2 y = cap_poly(u, z, cq);
              x[e] = __float_as_uint(y.x);
              x[e + 1] = __float_as_uint(y.y);
            }
          }
          if (__any_sync(0xffffffffu, !(zmax <= kCapZ))) {   // large scores: the raw products once more
#pragma unroll 1
            for (int gi = 0; gi < 4; ++gi) {
              const float f = sm.ks[slot][4 * hf + gi] * k_row;
              uint32_t raw[16];
              tmem_ld16(s_addr + hf * 64 + 16 * gi, raw);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const float2 u = make_float2(__uint_as_float(raw[e]) * f, __uint_as_float(raw[e + 1]) * f);
                const float2 z = make_float2(u.x * u.x, u.y * u.y);
                const float2 y = cap_poly(u, z, cq);
                raw[e] = __float_as_uint(z.x <= kCapZ ? y.x : cap_exp(u.x, c2));
                raw[e + 1] = __float_as_uint(z.y <= kCapZ ? y.y : cap_exp(u.y, c2));
              }
              tmem_st16(s_addr + hf * 64 + 16 * gi, raw);
            }
            tmem_st_wait();
            tmem_ld32(s_addr + hf * 64, x);
            tmem_ld32(s_addr + hf * 64 + 32, x + 32);
            tmem_ld_wait();
          }
        }
        if (CAP || !full) {
          if (!full) {
#pragma unroll
            for (int e = 0; e < 64; ++e) {
              const int col = hf * 64 + e;
              x[e] = (col >= lo && col < hi) ? x[e] : 0xff800000u;   // -inf
            }
          }
          tmem_st32(s_addr + hf * 64, x);
          tmem_st32(s_addr + hf * 64 + 32, x + 32);
        }
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
          float a = fmax3(__uint_as_float(x[16 * gi]), __uint_as_float(x[16 * gi + 1]), __uint_as_float(x[16 * gi + 2]));
          float c = fmax3(__uint_as_float(x[16 * gi + 3]), __uint_as_float(x[16 * gi + 4]), __uint_as_float(x[16 * gi + 5]));
#pragma unroll
          for (int e = 6; e < 16; e += 4) {
            a = fmax3(a, __uint_as_float(x[16 * gi + e]), __uint_as_float(x[16 * gi + e + 1]));
            if (e + 2 < 16) c = fmax3(c, __uint_as_float(x[16 * gi + e + 2]), __uint_as_float(x[16 * gi + e + 3]));
          }
          const float mg = fmaxf(a, c);
          mt = fmaxf(mt, CAP ? mg : mg * (ksg[gi] * k_row));
        }
      }
      if (CAP || !full) tmem_st_wait();
      // Lazy rescale: O_q is complete up to tile t-1 (its MMAs precede S_q(t)).
      const bool grow = mt > m_run + kLazy;
      const float m_new = grow ? mt : m_run;
      if (t > 0 && __any_sync(0xffffffffu, grow)) {
        const float f = grow ? ex2(m_run - m_new) : 1.0f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t raw[32];
          tmem_ld32(o_addr + c * 32, raw);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) raw[e] = __float_as_uint(__uint_as_float(raw[e]) * f);
          tmem_st32(o_addr + c * 32, raw);
        }
        l_run *= f;
      }
      m_run = m_new;
      // Pass 2: P' per 16 keys; keys 64 hf ..: hi pairs over columns 64 hf ..
      // + 31, lo pairs over the next 32 (only columns of the half just read).
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t x[64];
        tmem_ld32(s_addr + hf * 64, x);
        tmem_ld32(s_addr + hf * 64 + 32, x + 32);
        const float4 kg = *reinterpret_cast<const float4*>(&sm.ks[slot][4 * hf]);
        const float4 lg = *reinterpret_cast<const float4*>(&sm.lv[slot][4 * hf]);
        const float4 ig = *reinterpret_cast<const float4*>(&sm.iv[slot][4 * hf]);
        const float ksg[4] = {kg.x, kg.y, kg.z, kg.w}, lvg[4] = {lg.x, lg.y, lg.z, lg.w}, ivg[4] = {ig.x, ig.y, ig.z, ig.w};
        tmem_ld_wait();
#pragma unroll
        for (int qq = 0; qq < 2; ++qq) {
          uint32_t ph[16], pl[F32 ? 16 : 1];
#pragma unroll
          for (int gi = 0; gi < 2; ++gi) {
            const int gr = 2 * qq + gi;
            const float kk = CAP ? 1.f : ksg[gr] * k_row, cc = lvg[gr] - m_run;
            const float2 kk2 = make_float2(kk, kk), cc2 = make_float2(cc, cc);
            float2 ls = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int e = 16 * gr + 2 * k;
              const float2 arg = ffma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), kk2, cc2);
              const float pa = ex2(arg.x), pb = ex2(arg.y);
              ls = ffma2(make_float2(pa, pb), make_float2(1.f, 1.f), ls);
              const __half2 hp = __floats2half2_rn(pa, pb);
              ph[8 * gi + k] = *reinterpret_cast<const uint32_t*>(&hp);
              if constexpr (F32) {
                const float2 hf2 = __half22float2(hp);
                const __half2 lp = __floats2half2_rn(pa - hf2.x, pb - hf2.y);
                pl[8 * gi + k] = *reinterpret_cast<const uint32_t*>(&lp);
              }
            }
            l_run = fmaf(ls.x + ls.y, ivg[gr], l_run);
          }
          tmem_st16(s_addr + hf * 64 + 16 * qq, ph);
          if constexpr (F32) tmem_st16(s_addr + hf * 64 + 32 + 16 * qq, pl);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&sm.p_full[q]);
    }
    // ---- epilogue: O / l (+ sink) in units of 2^(wexp - kLift), staged in the
    // group's query tile (free once its last P.V is done) and written with
    // tensor stores (rows past S are skipped).
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_done[q], (uint32_t)(ntiles - 1) & 1u, p.wait_budget) && !aborted(sm));
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
      const float so = (live && den > 0.f) ? f / den * __int_as_float((127 + wexp - (int)kLift) << 23) : 0.f;
      if (p.lse && live) p.lse[(long long)bg * nrows + r] = mf + log2f(den);
      uint8_t* stage = sm.q[q];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t raw[32];
        tmem_ld32(o_addr + c * 32, raw);
        tmem_ld_wait();
        if constexpr (F32) {   // box c: dims 32 c ..
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
    if (!group_all(ok, q)) {
      if (lane == 0) set_abort(p, sm);
    } else if (quarter == 2 && elect_one()) {   // warp 2 (group 0) or 6 (group 1)
      for (int k = 0; k < kBoxes; ++k)
        tma_store_4d(&tmo, sm.q[q] + k * kBox, kBoxDims * k, g * p.G, (r0 + q * kBM) / p.G, b);
      bulk_commit();
      bulk_wait_read();   // the staged tile is read before the CTA may exit
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

constexpr int kMaxDevices = 64;

template <bool F32, bool CAP>
cudaError_t launch_one(const BlockParams& p, cudaStream_t st) {
  static bool done[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  const int smem = (int)sizeof(PfSmem<F32>) + 1024;
  auto kern = block_prefill_kernel<F32, CAP>;
  if (!done[dev]) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    done[dev] = true;
  }
  CUtensorMap mq, mo;
  auto encode = F32 ? encode_f32_query_sw128 : encode_fp16_query_sw128;
  if ((e = encode(&mq, p.q, p.B, p.S, p.N, (uint32_t)p.G)) != cudaSuccess) return e;
  if ((e = encode(&mo, p.out, p.B, p.S, p.N, (uint32_t)p.G)) != cudaSuccess) return e;
  const unsigned nqb = (unsigned)((p.S * p.G + 2 * kBM - 1) / (2 * kBM)), nbg = (unsigned)(p.B * p.Nkv);
  kern<<<p.qb_major ? dim3(nbg, nqb) : dim3(nqb, nbg), kThreads, smem, st>>>(p, mq, mo);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_prefill(const BlockParams& p, cudaStream_t st) {
  const bool cap = p.softcap > 0.f;
  if (p.t_type == kF32) return cap ? launch_one<true, true>(p, st) : launch_one<true, false>(p, st);
  return cap ? launch_one<false, true>(p, st) : launch_one<false, false>(p, st);
}

}  // namespace gqa
