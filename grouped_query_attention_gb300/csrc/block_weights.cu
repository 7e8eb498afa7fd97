// Attention weights of the cache rows after a tensor-core prefill (fp16, head
// size up to 128, group size up to 64 or 128): w[j] = sum over the query rows r that
// see key j of exp2(s_rj - lse_r), lse_r the row's log-sum-exp that the
// prefill left in the workspace (log2 domain).
//
// CTA = 128 keys of one KV head. Keys are the M side of S^T = K Q^T (128 keys
// x 64 query rows a tile), so a key is a tensor-memory lane and its sum stays
// in one thread: no reduction across threads, no atomics, and the K scale is
// one number per thread. The key tile is the A operand and stays in tensor
// memory (64 columns, beside three S buffers of 64), so that a tile's products
// read the query rows alone from shared memory. Query tiles arrive by TMA (four
// stages); two softmax groups take alternate tiles. Two CTAs share an SM.
//
// Bound: exp2 (one per visible pair, 32 a clock and SM) and the MMAs, 512
// clocks each per 128 x 128 pairs. Two prompts of 4096 tokens, 32 heads over 8
// (537 M pairs): 133 us, either pipe 45 % busy, 2.3 instructions a clock; the
// rest waits for S. With the key tile in shared memory, where the MMAs fetch
// both operands (twice the bytes a clock can bring), it took 175 us; with whole
// and masked tiles in one unrolled loop, whose instructions had to be fetched
// anew every tile, 150.
// Causal: key tile 0 meets every query row, the last few; the longest start first.
#include <cuda_fp16.h>

#include "block_internal.h"
#include "block_tc.cuh"
#include "common.cuh"
#include "tcgen05.cuh"
#include "tma_host.h"

namespace gqa {
namespace {

using namespace tc;

constexpr int kKeys = 128;                     // keys of a CTA
constexpr int kRows = 64;                      // query rows of a tile
constexpr int kStages = 4;                     // query tiles in shared memory
constexpr int kBufs = 3;                       // S buffers in tensor memory
constexpr int kThreads = 384;
constexpr int kSoftWarp0 = 4;
constexpr uint32_t kBox = kRows * 128u;        // 64 rows x 128 bytes
constexpr uint32_t kTile = 2u * kBox;
constexpr uint32_t kIdS = idesc_f16(kKeys, kRows, 0, 0);

struct __align__(1024) WtSmem {
  uint8_t q[kStages][kTile];
  float nl[kBufs][kRows];                      // -lse of the tile's rows
  float part[kKeys];                           // the second group's sums
  uint64_t q_full[kStages], q_empty[kStages];
  uint64_t nl_full[kBufs], s_full[kBufs], s_empty[kBufs];
  uint64_t drain;
  uint32_t tmem;
  int abort;
};
static_assert(2 * (sizeof(WtSmem) + 1024 + 1024) <= 233472, "two CTAs per SM");

__device__ __forceinline__ bool aborted(const WtSmem& sm) {
  return *reinterpret_cast<const volatile int*>(&sm.abort) != 0;
}
__device__ __forceinline__ void set_abort(const BlockParams& p, WtSmem& sm) {
  *reinterpret_cast<volatile int*>(&sm.abort) = 1;
  if (p.status) atomicOr(p.status, GQA_DEVICE_TIMEOUT_BIT);
}

template <bool CAP>
__global__ void __launch_bounds__(kThreads, 2)
block_weights_tc_kernel(const BlockParams p, const __grid_constant__ CUtensorMap tmq) {
  extern __shared__ uint8_t smem_raw[];
  WtSmem& sm = *reinterpret_cast<WtSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bg = blockIdx.x, b = bg / p.Nkv, g = bg % p.Nkv;
  int total, fresh;
  dep_wait();   // every block: what follows on the stream waits for this kernel alone
  if (!block_lengths(p, b, &total, &fresh)) return;
  const int j0 = (int)blockIdx.y * kKeys;
  if (j0 >= total) return;
  const int past = total - fresh;
  // Positions of the step that see a key of this block, and their rows in tiles of 128.
  const int i_lo = max(0, j0 - past);
  const int i_hi = p.window >= 0 ? min(fresh, j0 + kKeys + p.window - past) : fresh;
  const int rows0 = i_lo * p.G, rows1 = i_hi * p.G;
  const int tr = p.G < kRows ? kRows / p.G * p.G : kRows;   // rows of a tile in use: whole positions, or a part of one
  const int ntiles = rows1 > rows0 ? (rows1 - rows0 + tr - 1) / tr : 0;

  if (warp == 1) tmem_alloc(&sm.tmem, 256);
  if (tid == 0) {
    for (int t = 0; t < kStages; ++t) {
      mbar_init(&sm.q_full[t], 1);
      mbar_init(&sm.q_empty[t], 1);
    }
    for (int t = 0; t < kBufs; ++t) {
      mbar_init(&sm.nl_full[t], 1);
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.s_empty[t], 4);
    }
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    mbar_fence_init();
  }
  if (tr < kRows) {   // rows of the query tiles that no copy fills
    for (int x = tid; x < 2 * kStages * (kRows - tr) * 8; x += kThreads) {
      const int box = x / ((kRows - tr) * 8), at = x % ((kRows - tr) * 8);
      *reinterpret_cast<uint4*>(sm.q[box / 2] + (box & 1) * kBox + tr * 128 + at * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem, tmem_k = tmem + kBufs * kRows;
  // The key tile as fp16 pairs, a key per lane; rows behind the sequence are zeros.
  if (warp >= kSoftWarp0) {
    const int row = j0 + (warp & 3) * 32 + lane, half = (warp - kSoftWarp0) >> 2;
    const uint4* src = reinterpret_cast<const uint4*>(p.kc + ((long long)bg * p.C + row) * p.H) + 4 * half;
    uint32_t h[32];
#pragma unroll
    for (int k = 0; k < 4; ++k) codes16(row < total && 64 * half + 16 * k < p.H ? src[k] : make_uint4(0u, 0u, 0u, 0u), h + 8 * k);
    tmem_st32(tmem_k + ((uint32_t)((warp & 3) * 32) << 16) + 32 * half, h);
    tmem_st_wait();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp == 0) {
    // ================================================================ TMA: query tiles
    bool ok = true;
    int n = 0;
    for (; n < ntiles && ok; ++n) {
      if (n == p.withhold_tile) break;   // testing: this tile is never copied, the waits for it expire
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_empty[n % kStages], ((uint32_t)(n / kStages) & 1u) ^ 1u, p.wait_budget) && !aborted(sm));
      if (ok && elect_one()) {
        mbar_arrive_tx(&sm.q_full[n % kStages], (uint32_t)(2 * tr * 128));
        for (int k = 0; k < 2; ++k)
          tma_load_4d(sm.q[n % kStages] + k * kBox, &tmq, 64 * k, g * p.G + n * tr % p.G, i_lo + n * tr / p.G, b,
                      &sm.q_full[n % kStages]);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) set_abort(p, sm);
    if (!ok) --n;
    // No copy of this CTA may still be landing when it exits.
    for (int x = n > kStages ? n - kStages : 0; x < n; ++x)
      mbar_wait(&sm.q_full[x % kStages], (uint32_t)(x / kStages) & 1u, p.wait_budget);
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    const uint64_t dq = desc_kmajor_sw128(smem_addr(sm.q[0]));
    bool ok = true;
    for (int n = 0; n < ntiles && ok; ++n) {
      const int st = n % kStages, bf = n % kBufs;
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_full[st], (uint32_t)(n / kStages) & 1u, p.wait_budget) &&
                                       mbar_wait(&sm.s_empty[bf], ((uint32_t)(n / kBufs) & 1u) ^ 1u, p.wait_budget) &&
                                       !aborted(sm));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t b0 = dq + (uint64_t)(st * (int)(kTile >> 4));
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_f16_ts(tmem + bf * kRows, tmem_k + ks * 8, b0 + (uint64_t)((ks >> 2) * (int)(kBox >> 4) + (ks & 3) * 2), kIdS,
                     ks > 0);
        mma_commit(&sm.q_empty[st]);
        mma_commit(&sm.s_full[bf]);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) set_abort(p, sm);
    if (elect_one()) {   // every MMA has finished before tensor memory is freed
      mma_commit(&sm.drain);
      mbar_wait(&sm.drain, 0, p.wait_budget);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ================================================================ -lse of the rows, a tile ahead
    const float* lse = p.lse + (long long)bg * p.S * p.G;
    auto load = [&](int n) -> float2 {   // rows behind the tile's or the last one add nothing
      const int r = rows0 + n * tr + 2 * lane, end = min(rows1, rows0 + (n + 1) * tr);
      return make_float2(r < end ? -lse[r] : -INFINITY, r + 1 < end ? -lse[r + 1] : -INFINITY);
    };
    float2 next = load(0);
    bool ok = true;
    for (int n = 0; n < ntiles && ok; ++n) {
      const float2 v = next;
      if (n + 1 < ntiles) next = load(n + 1);
      // The buffer's last readers are those of its S.
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.s_empty[n % kBufs], ((uint32_t)(n / kBufs) & 1u) ^ 1u, p.wait_budget) && !aborted(sm));
      if (!ok) break;
      *reinterpret_cast<float2*>(&sm.nl[n % kBufs][2 * lane]) = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.nl_full[n % kBufs]);
    }
    if (!ok && lane == 0) set_abort(p, sm);
  }
  float sum = 0.f;
  const int key = (warp & 3) * 32 + lane, j = j0 + key;   // softmax threads: tensor-memory lane = key
  if (warp >= kSoftWarp0) {
    // ================================================================ sums of one key
    const int grp = (warp - kSoftWarp0) >> 2;
    const float ks = j < total ? p.ks[(long long)bg * p.nblk + (j >> p.bs_log2)] : 0.f;
    const float kk = ks * p.scale * (CAP ? 1.f / p.softcap : kLog2e), c2 = p.softcap * kLog2e;
    const float2 kk2 = make_float2(kk, kk);
    // Rows [r_lo, r_hi) see the key.
    const int r_lo = max(0, j - past) * p.G;
    const int r_hi = j < total ? (p.window >= 0 ? min(rows1, (int)min((long long)(j - past) + p.window + 1, (long long)fresh) * p.G) : rows1) : 0;
    bool ok = true;
    for (int n = grp; n < ntiles && ok; n += 2) {
      const int bf = n % kBufs;
      const uint32_t par = (uint32_t)(n / kBufs) & 1u, s_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16) + bf * kRows;
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.s_full[bf], par, p.wait_budget) &&
                                       mbar_wait(&sm.nl_full[bf], par, p.wait_budget) && !aborted(sm));
      if (!ok) break;
      tc_fence_after();
      const int r0 = rows0 + n * tr;
      const int lo = r_lo - r0, hi = r_hi - r0;   // visible columns [lo, hi)
      const bool full = __all_sync(0xffffffffu, lo <= 0 && hi >= tr);
      float2 acc = make_float2(0.f, 0.f), acc2 = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int c = 0; c < kRows; c += 32) {
        uint32_t x[32];
        tmem_ld32(s_addr + c, x);
        tmem_ld_wait();
        int mode = 0;
        if constexpr (CAP) {
          float a = 0.f;
#pragma unroll
          for (int e = 0; e < 32; e += 2) a = fmax3(a, fabsf(__uint_as_float(x[e])), fabsf(__uint_as_float(x[e + 1])));
          a *= kk;
          mode = __all_sync(0xffffffffu, !(a > kCapLow)) ? 3 : __all_sync(0xffffffffu, !(a > kCapHigh)) ? 7 : 9;
        }
        auto add = [&](auto m, auto whole) {
          constexpr int MODE = decltype(m)::value;
#pragma unroll
          for (int e4 = 0; e4 < 32; e4 += 4) {
            const float4 nl = *reinterpret_cast<const float4*>(&sm.nl[bf][c + e4]);
            const float nv[4] = {nl.x, nl.y, nl.z, nl.w};
#pragma unroll
            for (int e = e4; e < e4 + 4; e += 2) {
              const float2 x2 = make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
              const float2 n2 = make_float2(nv[e - e4], nv[e - e4 + 1]);
              float2 arg;
              if constexpr (MODE == 0) {
                arg = ffma2(x2, kk2, n2);
              } else {
                const float2 u = ffma2(x2, kk2, make_float2(0.f, 0.f));
                if constexpr (MODE == 9) {
                  const float2 y = cap_any(u, c2);
                  arg = make_float2(y.x + n2.x, y.y + n2.y);
                } else {
                  const float2 z = ffma2(u, u, make_float2(0.f, 0.f));
                  arg = ffma2(u, cap_fit<MODE>(z, c2), n2);
                }
              }
              if constexpr (!decltype(whole)::value) {
                arg.x = c + e >= lo && c + e < hi ? arg.x : -INFINITY;
                arg.y = c + e + 1 >= lo && c + e + 1 < hi ? arg.y : -INFINITY;
              }
              const float2 w = make_float2(ex2(arg.x), ex2(arg.y));
              if (e & 2) acc2 = fadd2(acc2, w);
              else acc = fadd2(acc, w);
            }
          }
        };
        auto pick = [&](auto whole) {
          if constexpr (CAP) {
            if (mode == 3) add(std::integral_constant<int, 3>(), whole);
            else if (mode == 7) add(std::integral_constant<int, 7>(), whole);
            else add(std::integral_constant<int, 9>(), whole);
          } else {
            add(std::integral_constant<int, 0>(), whole);
          }
        };
        if (full) pick(std::true_type());
        else pick(std::false_type());
      }
      acc = fadd2(acc, acc2);
      sum += acc.x + acc.y;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.s_empty[bf]);
    }
    if (!ok && lane == 0) set_abort(p, sm);
    if (grp == 1) sm.part[key] = sum;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 256);
  if (warp >= kSoftWarp0 && warp < kSoftWarp0 + 4 && j < total && !aborted(sm)) {
    const long long at = (long long)bg * p.C + j;
    p.present_w[at] = sum + sm.part[key] + (p.past_w && j < past ? p.past_w[at] : 0.f);
  }
}

constexpr int kMaxDevices = 64;

template <bool CAP>
cudaError_t launch_one(const BlockParams& p, cudaStream_t st) {
  static bool done[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  const int smem = (int)sizeof(WtSmem) + 1024;
  if (!done[dev]) {
    if ((e = cudaFuncSetAttribute(block_weights_tc_kernel<CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
      return e;
    done[dev] = true;
  }
  CUtensorMap mq;
  if ((e = encode_fp16_query_sw128(&mq, p.q, p.B, p.S, p.N, (uint32_t)p.G, kRows, (uint64_t)p.H)) != cudaSuccess) return e;
  const dim3 grid((unsigned)(p.B * p.Nkv), (unsigned)((p.T + kKeys - 1) / kKeys));
  return launch_dependent(true, block_weights_tc_kernel<CAP>, grid, kThreads, (size_t)smem, st, p, mq);
}

}  // namespace

cudaError_t launch_block_weights_tc(const BlockParams& p, cudaStream_t st) {
  return p.softcap > 0.f ? launch_one<true>(p, st) : launch_one<false>(p, st);
}

}  // namespace gqa
