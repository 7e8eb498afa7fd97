// Attention over the block-scaled int8 cache by a split over the keys (decode
// steps, short chunks, and every shape the tensor-core prefill does not take).
//
// Rows of a KV head (b, g): query rows (position, grouped head), in row tiles
// of 8 or 16. A decode step has a few rows against many keys, so the keys are
// the M side of the warp MMA (m16n8k16, fp16 in, fp32 sums): S^T = K Q^T takes
// 16 keys against 8 rows, O^T += V^T P^T 16 coordinates against 8 rows, and a
// row tile of 8 leaves nothing idle. P^T leaves the first product with keys
// along the lanes and enters the second with rows along them: one 8 x 8
// transpose (movmatrix) per 8 keys. The codes are small integers, exact in
// fp16; the block's K scale multiplies the scores, its V scale the
// probabilities (both are one number for 16 keys). fp32 queries and
// probabilities keep their precision as two fp16 parts, hi = fp16(x) and
// lo = fp16(x - hi) (queries brought to [1, 2) by a power of two per row).
//
// Bound: HBM, 2 H bytes per cache row; the instructions that turn codes into
// fp16 fragments (11 per 4-code word of K and of V) come next. Every warp is a
// worker of its own: the 32-key units of all ranges (b, g, row tile) are laid
// end to end, a worker takes an equal share, copies its units by TMA through a
// private ring (128-byte swizzle, so the fragment reads do not conflict), and
// nothing waits for another warp. A worker's piece of a range ends as a
// partial (m, l, O) in the workspace; a second launch merges the pieces of
// each row and adds the attention weights of the cache rows.
//
// Measured: fp16, 16 sequences of 1025 to 8192 keys, 8 KV heads of 128 (151
// MB): 31 us, 4.9 TB/s (DRAM 58 % busy, 2.2 instructions a clock), merge 7 us.
// fp32, 32 sequences of 4097 to 16384 keys with weights (672 MB of codes and
// scores): 117 us, 5.7 TB/s; merge and weights 17 us.
#include <cuda_fp16.h>

#include "block_internal.h"
#include "common.cuh"
#include "tcgen05.cuh"
#include "tma_host.h"

namespace gqa {
namespace {

// Warps of a CTA. Three CTAs of four share an SM up to a head size of 128; behind
// it a warp's ring takes 32 KB and one CTA of seven fills the shared memory.
constexpr int warps_of(int H) { return H > 128 ? 7 : 4; }

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of fp16 pairs held by a warp (row lane / 4, columns 2 (lane % 4), + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four bytes, or zeros when !on.
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool on) {
  const int n = on ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Bytes 0, 1 (lo) or 2, 3 (hi) of x (codes ^ 0x80) as two fp16 values: under
// the exponent of 1024 a byte u reads 1024 + u; 1152 = 1024 + 128 comes off.
__device__ __forceinline__ uint32_t codes_lo(uint32_t x) {
  const uint32_t h = __byte_perm(x, 0x64646464u, 0x4140u);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), __floats2half2_rn(1152.f, 1152.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t x) {
  const uint32_t h = __byte_perm(x, 0x64646464u, 0x4342u);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), __floats2half2_rn(1152.f, 1152.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }

// 16-byte chunk `c` of row `r` of a 32-row tile as TMA lands it: rows of 64
// bytes (64-byte swizzle) or boxes of 128-byte rows (128-byte swizzle).
template <int HP>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if constexpr (HP == 64) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  return (uint32_t)((c >> 3) * (kBlockUnit * 128) + r * 128 + (((c ^ r) & 7) << 4));
}

// Key range of sequence b shared by its row tiles: units [t0, t0 + nt).
__device__ __forceinline__ void units_of(const BlockParams& p, int total, int fresh, int* t0, int* nt) {
  *t0 = 0;
  *nt = 0;
  if (fresh <= 0) return;
  const int kmin = p.window >= 0 ? max(0, total - fresh - p.window) : 0;
  *t0 = kmin / kBlockUnit;
  *nt = (total + kBlockUnit - 1) / kBlockUnit - *t0;
}

// Units [lo, hi) (of the nt above) that row tile rt sees a key of.
__device__ __forceinline__ void tile_units(const BlockParams& p, int total, int fresh, int t0, int nt, int rt,
                                           int* lo, int* hi) {
  const int r0 = rt * p.rt_rows, r1 = min(r0 + p.rt_rows, p.S * p.G) - 1;
  const int i0 = r0 / p.G, i1 = min(r1 / p.G, fresh - 1);
  if (i0 > i1) {   // padding rows only
    *lo = *hi = 0;
    return;
  }
  const int past = total - fresh;
  const int kmin = p.window >= 0 ? max(0, past + i0 - p.window) : 0;
  *lo = kmin / kBlockUnit - t0;
  *hi = (past + i1) / kBlockUnit + 1 - t0;
}

// Units of sequence b counting every range's extra cost; 0 when nothing is to do.
__device__ __forceinline__ long long seq_units(const BlockParams& p, int b, int* total, int* fresh, int* t0, int* nt) {
  if (!block_lengths(p, b, total, fresh)) *fresh = 0;
  units_of(p, *total, *fresh, t0, nt);
  return *nt > 0 ? (long long)p.Nkv * p.nrt * (*nt + kBlockRangeCost) : 0;
}

// Sum of seq_units over the batch, by one warp.
__device__ long long all_units(const BlockParams& p) {
  const int lane = threadIdx.x & 31;
  long long sum = 0;
  for (int b = lane; b < p.B; b += 32) {
    int a, f, t0, nt;
    sum += seq_units(p, b, &a, &f, &t0, &nt);
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Workers that share the units out: the grid's, which the host sized for
// total_sequence_length, unless the lengths leave fewer units. Each then owns
// one unit at least, so that every piece the merge counts has been written.
// (16 steps of 200 keys for a bound of 8192: 12.3 us; two units a worker 12.4,
// four 15.9. 8 of 40 keys, bound 4096: 9.2, 10.4, 10.8.)
__device__ __forceinline__ long long live_workers(const BlockParams& p, long long units) {
  return max(1LL, min((long long)p.workers, units));
}

// Walk over a worker's units: range (b, g, rt) and unit `off` of the sequence's
// units; `left` units of the share remain. Divisions only where a range begins.
struct Walk {
  int b, g, rt, bg, off, nt, t0, total, fresh, hi;
  long long left;

  __device__ void enter_seq(const BlockParams& p) {
    while (b < p.B && seq_units(p, b, &total, &fresh, &t0, &nt) == 0) ++b;
    if (b >= p.B) left = 0;
  }
  // Skip the units no row of the tile sees, and the ends of ranges.
  __device__ void settle(const BlockParams& p) {
    while (left > 0) {
      int lo;
      tile_units(p, total, fresh, t0, nt, rt, &lo, &hi);
      if (off < lo) {
        left -= lo - off;
        off = lo;
        if (left <= 0) break;
      }
      if (off < hi) break;
      left -= nt + kBlockRangeCost - off;
      off = 0;
      if (++rt == p.nrt) {
        rt = 0;
        if (++g == p.Nkv) {
          g = 0;
          ++b;
          if (left > 0) enter_seq(p);
        }
      }
    }
    bg = b * p.Nkv + g;
  }
  // A share of n units from unit u on (u below the sum of all); one warp.
  __device__ void start(const BlockParams& p, long long u, long long n) {
    left = n;
    const int lane = threadIdx.x & 31;
    for (b = 0; b < p.B; b += 32) {   // the sequence that holds unit u, 32 at a time
      long long s = b + lane < p.B ? seq_units(p, b + lane, &total, &fresh, &t0, &nt) : 0;
      const long long own = s;
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
      }
      const unsigned past_u = __ballot_sync(0xffffffffu, s > u);
      if (past_u) {
        const int at = __ffs(past_u) - 1;
        u -= __shfl_sync(0xffffffffu, s - own, at);
        b += at;
        break;
      }
      u -= __shfl_sync(0xffffffffu, s, 31);
    }
    seq_units(p, b, &total, &fresh, &t0, &nt);
    const int gr = (int)(u / (nt + kBlockRangeCost));
    off = (int)(u - (long long)gr * (nt + kBlockRangeCost));
    g = gr / p.nrt;
    rt = gr - g * p.nrt;
    settle(p);
  }
  // The next unit; true when it is not of the same range (or there is none).
  __device__ bool next(const BlockParams& p) {
    --left;
    ++off;
    if (off < hi && left > 0) return false;
    const bool ends = off >= hi || left <= 0;
    settle(p);
    return ends;
  }
};

constexpr int kStages = 2;   // units in the ring: one being read, one landing

template <int HP>
struct __align__(1024) WarpSmem {
  uint8_t ring[kStages][2 * kBlockUnit * HP];   // K tile, V tile
};
struct WarpCtl {
  float sc[kStages][4];    // K scales of the unit's two 16-key groups, V scales
  uint64_t full[kStages];
};

// CTAs per SM the registers and the ring leave room for.
template <int HP, int NT, bool FLUSH>
constexpr int ctas_per_sm() {
  return HP > 128 ? 1 : NT > 1 || FLUSH ? 2 : 3;
}

// Query fragments of a row tile: thread t of a quad holds coordinates t HP/4
// .. of row gq of every 8-row tile (the order of the contraction is free as
// long as the keys use the same), four per MMA step. up[n]: the power of two
// an fp32 row was divided by.
template <typename T, int HP, int NT>
__device__ void load_queries(const BlockParams& p, int b, int g, int rt, uint2 (*qf)[HP / 16], float* up) {
  constexpr bool kHalf = sizeof(T) == 2;
  const int lane = threadIdx.x & 31, gq = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = rt * p.rt_rows + 8 * n + gq;
    const T* row = r < p.S * p.G ? static_cast<const T*>(p.q) +
                                       ((b * (long long)p.S + r / p.G) * p.N + g * p.G + r % p.G) * p.H
                                 : nullptr;
    if constexpr (kHalf) {
      up[n] = 1.f;
#pragma unroll
      for (int ks = 0; ks < HP / 16; ++ks) {
        const int d = t * (HP / 4) + 4 * ks;
        qf[n][ks] = row && d < p.H ? *reinterpret_cast<const uint2*>(row + d) : make_uint2(0u, 0u);
      }
    } else {
      float4 v[HP / 16];
      float mx = 0.f;
#pragma unroll
      for (int ks = 0; ks < HP / 16; ++ks) {
        const int d = t * (HP / 4) + 4 * ks;
        v[ks] = row && d < p.H ? *reinterpret_cast<const float4*>(row + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        mx = fmax3(mx, fabsf(v[ks].x), fabsf(v[ks].y));
        mx = fmax3(mx, fabsf(v[ks].z), fabsf(v[ks].w));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int ex = (__float_as_int(mx) >> 23) & 0xff;
      const int e = ex == 0 ? 0 : min(ex, 253) - 127;
      const float down = __int_as_float((127 - e) << 23);
      up[n] = __int_as_float((127 + e) << 23);
#pragma unroll
      for (int ks = 0; ks < HP / 16; ++ks) {   // hi parts in tile n, lo parts in tile NT + n
        const float4 x = make_float4(v[ks].x * down, v[ks].y * down, v[ks].z * down, v[ks].w * down);
        const uint2 hi = make_uint2(pack(x.x, x.y), pack(x.z, x.w));
        const float2 h0 = unpack(hi.x), h1 = unpack(hi.y);
        qf[n][ks] = hi;
        qf[NT + n][ks] = make_uint2(pack(x.x - h0.x, x.y - h0.y), pack(x.z - h1.x, x.w - h1.y));
      }
    }
  }
}

// NT: 8-row tiles of a row tile. PLAIN: no softcap and no score stash. FLUSH:
// the MMA accumulator drops what does not fit (it rounds towards zero), so over
// a thousand keys its error grows past the other fp32 roundings; every 8 units
// O moves into sums that round to nearest. For fp32 prompts, where a worker
// meets whole ranges (1.8e-6 against 0.6e-6 at 1500 keys); a decode step's
// pieces are short and its registers go to a third CTA.
template <typename T, int HP, int NT, bool PLAIN, bool FLUSH>
__global__ void __launch_bounds__(warps_of(HP) * 32, ctas_per_sm<HP, NT, FLUSH>())
block_attn_kernel(const BlockParams p, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  constexpr bool kHalf = sizeof(T) == 2;
  constexpr int kParts = kHalf ? 1 : 2;     // fp16 parts of queries and probabilities
  constexpr int kTileBytes = kBlockUnit * HP;
  constexpr int kSteps = HP / 16;           // MMA steps over the coordinates; output tiles of 16 coordinates
  constexpr float kGrow = 4.f;              // log2 growth of a maximum tolerated before rescaling
  extern __shared__ uint8_t smem_raw[];
  WarpSmem<HP>* rings = reinterpret_cast<WarpSmem<HP>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ WarpCtl ctls[warps_of(HP)];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, t = lane & 3;
  WarpSmem<HP>& sm = rings[warp];
  WarpCtl& ctl = ctls[warp];
  const long long worker = (long long)blockIdx.x * warps_of(HP) + warp;

  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) tc::mbar_init(&ctl.full[s], 1);
    tc::mbar_fence_init();
  }
  __syncwarp();
  if (blockIdx.x == 0 && warp == 0 && p.status) {   // lengths out of range
    bool bad = false;
    for (int b = lane; b < p.B; b += 32) {
      int a, f;
      bad |= !block_lengths(p, b, &a, &f);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.status, GQA_DEVICE_BAD_SEQLEN_BIT);
  }
  const long long units = all_units(p);   // lengths are older than the kernel ahead
  dep_launch();
  const long long live = live_workers(p, units);
  const long long u0 = units * worker / live, u1 = units * (worker + 1) / live;
  if (worker >= live || u0 >= u1) {   // (no units at all)
    dep_wait();
    return;
  }
  Walk ld, cp;
  ld.start(p, u0, u1 - u0);
  cp = ld;

  // The append kernel writes the blocks from the first new row's on and no
  // other: units before them are copied while it may still run.
  bool waited = false;
  int fetched = 0;
  // Start the copies of the unit at `ld` into stage s and move on.
  auto fetch = [&](int s) {
    if (ld.left > 0 && (p.withhold_tile < 0 || fetched != p.withhold_tile)) {
      ++fetched;
      const int j0 = (ld.t0 + ld.off) * kBlockUnit;
      if (!waited && j0 + kBlockUnit > ((ld.total - ld.fresh) >> p.bs_log2 << p.bs_log2)) {
        dep_wait();
        waited = true;
      }
      if (lane == 0) {
        const int row = ld.bg * p.C + j0;   // below 2^31 (checked by the host)
        tc::mbar_arrive_tx(&ctl.full[s], 2 * kTileBytes);
#pragma unroll
        for (int x = 0; x < (HP > 128 ? 2 : 1); ++x) {
          tc::tma_load_2d(sm.ring[s] + x * kBlockUnit * 128, &tmk, 128 * x, row, &ctl.full[s]);
          tc::tma_load_2d(sm.ring[s] + kTileBytes + x * kBlockUnit * 128, &tmv, 128 * x, row, &ctl.full[s]);
        }
      }
      if (lane < 4) {   // scales of the two 16-key groups; 0 behind the last row
        const int j = j0 + 16 * (lane & 1);
        const float* src = (lane < 2 ? p.ks : p.vs) + (long long)ld.bg * p.nblk;
        const bool on = j < ld.total;
        cp4((uint32_t)__cvta_generic_to_shared(&ctl.sc[s][lane]), src + (on ? j >> p.bs_log2 : 0), on);
      }
      ld.next(p);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(s);

  uint2 qf[NT * kParts][kSteps];
  float o[kSteps][NT][4];       // O^T: coordinates gq HP/8 + 2 i (0, 1) and + 1 (2, 3), rows 2 t (0, 2) and + 1 (1, 3)
  float m[NT][2], l[NT][2], mul[NT][2];   // of rows 8 n + 2 t, + 1
  float acc[FLUSH ? kSteps : 1][NT][4];
  int held = 0;                 // FLUSH: units in o
  float lr[kHalf ? NT : 1][2];            // fp16: the sum of the probabilities as the product with V has them
  int wexp = -200;              // the V scales enter as vs 2^-wexp
  bool fresh_piece = true;
  int r0 = 0, past = 0, pos_lo = 0, pos_hi = 0;   // of the piece: first row, cached rows, positions of its first and last row
  int stage = 0;
  uint32_t parity = 0;
  while (cp.left > 0) {
    const int j0 = (cp.t0 + cp.off) * kBlockUnit;
    __syncwarp();                                  // the other stage has been read by every lane
    fetch(stage ^ 1);
    if (fresh_piece) {
      fresh_piece = false;
      float up[NT];
      load_queries<T, HP, NT>(p, cp.b, cp.g, cp.rt, qf, up);
      r0 = cp.rt * p.rt_rows;
      past = cp.total - cp.fresh;
      pos_lo = past + r0 / p.G;
      pos_hi = past + (r0 + 8 * NT - 1) / p.G;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float f = __shfl_sync(0xffffffffu, up[n], 4 * (2 * t + h)) * p.scale;
          mul[n][h] = p.softcap > 0.f ? f : f * kLog2e;
          m[n][h] = kNegBig;
          l[n][h] = 0.f;
          if (kHalf) lr[n][h] = 0.f;
        }
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
          if constexpr (FLUSH) acc[i][n][0] = acc[i][n][1] = acc[i][n][2] = acc[i][n][3] = 0.f;
        }
      held = 0;
      wexp = -200;
    }
    cp_wait<kStages - 1>();
    if (!__all_sync(0xffffffffu, tc::mbar_wait(&ctl.full[stage], parity, p.wait_budget))) {
      if (lane == 0 && p.status) atomicOr(p.status, GQA_DEVICE_TIMEOUT_BIT);
      tc::mbar_wait(&ctl.full[stage ^ 1], stage == 0 ? parity : parity ^ 1u, p.wait_budget);   // a copy still landing
      break;
    }
    const uint8_t* kt = sm.ring[stage];
    const uint8_t* vt = kt + kTileBytes;

    // ---- scores: s[kk][n] holds keys 16 kk + gq (0, 1) and + 8 (2, 3), rows 2 t (0, 2) and + 1 (1, 3)
    float s[2][NT][4];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      uint32_t kw[2][kSteps];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kSteps / 4; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(kt + chunk_at<HP>(16 * kk + 8 * h + gq, t * (HP / 64) + i));
          kw[h][4 * i] = v.x ^ 0x80808080u;
          kw[h][4 * i + 1] = v.y ^ 0x80808080u;
          kw[h][4 * i + 2] = v.z ^ 0x80808080u;
          kw[h][4 * i + 3] = v.w ^ 0x80808080u;
        }
      float c[NT * kParts][4];
#pragma unroll
      for (int n = 0; n < NT * kParts; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        const uint32_t a[4] = {codes_lo(kw[0][ks]), codes_lo(kw[1][ks]), codes_hi(kw[0][ks]), codes_hi(kw[1][ks])};
#pragma unroll
        for (int n = 0; n < NT * kParts; ++n) mma16816(c[n], a, qf[n][ks].x, qf[n][ks].y);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[kk][n][e] = kHalf ? c[n][e] : c[n][e] + c[NT * (kParts - 1) + n][e];
    }
    const float4 sc = *reinterpret_cast<const float4*>(ctl.sc[stage]);
    const float ksc[2] = {sc.x, sc.y}, vsc[2] = {sc.z, sc.w};
    // Log2-domain scores.
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float f[2] = {mul[n][0] * ksc[kk], mul[n][1] * ksc[kk]};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[kk][n][e] *= f[e & 1];
          if (!PLAIN && p.softcap > 0.f) s[kk][n][e] = p.softcap * kLog2e * tanhf(s[kk][n][e] / p.softcap);
        }
      }
    if (j0 + kBlockUnit - 1 > pos_lo || (p.window >= 0 && j0 < pos_hi - p.window)) {   // a mask border crosses the unit
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int pos = past + (r0 + 8 * n + 2 * t + h) / p.G;
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int j = j0 + 16 * kk + 8 * x + gq;
              if (j > pos || (p.window >= 0 && j < pos - p.window)) s[kk][n][2 * x + h] = -INFINITY;
            }
        }
    }
    if (!PLAIN && p.stash) {
      float* dst = p.stash + ((long long)cp.bg * p.stash_ld + j0 + gq) * p.stash_rows + 2 * t;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (8 * n + 2 * t < p.stash_rows) {
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              *reinterpret_cast<float2*>(dst + (16 * kk + 8 * x) * p.stash_rows + 8 * n) =
                  make_float2(s[kk][n][2 * x], s[kk][n][2 * x + 1]);
        }
    }
    // ---- running maximum; O is rescaled only when one grows by more than 2^4
    // or the V scales outgrow their reference.
    float mx[NT][2];
    bool grow = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = fmaxf(fmax3(s[0][n][h], s[0][n][2 + h], s[1][n][h]), s[1][n][2 + h]);
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        mx[n][h] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        grow |= mx[n][h] > m[n][h] + kGrow;
      }
    // P enters the MMA as p vs 2^-wexp, at most 2^14: vs 2^-wexp in [2^9, 2^10)
    // for the block that set it, and fp16 keeps its 11 bits down to 2^-14.
    const int vexp = (__float_as_int(fmaxf(vsc[0], vsc[1])) >> 23) - 127 - 9;
    if (__any_sync(0xffffffffu, grow) || vexp > wexp) {
      const int dw = vexp > wexp ? max(wexp - vexp, -126) : 0;
      if (vexp > wexp) wexp = max(vexp, -110);
      const float fw = __int_as_float((127 + dw) << 23);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = mx[n][h] > m[n][h] + kGrow ? mx[n][h] : m[n][h];
          const float e = ex2(m[n][h] - mn);
          m[n][h] = mn;
          l[n][h] *= e;
          if (kHalf) lr[n][h] *= e;
          f[h] = e * fw;
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          o[i][n][0] *= f[0];
          o[i][n][1] *= f[1];
          o[i][n][2] *= f[0];
          o[i][n][3] *= f[1];
          if constexpr (FLUSH) {
            acc[i][n][0] *= f[0];
            acc[i][n][1] *= f[1];
            acc[i][n][2] *= f[0];
            acc[i][n][3] *= f[1];
          }
        }
      }
    }
    const float down = __int_as_float((127 - wexp) << 23);   // wexp is in [-110, 119] here
    // ---- P, and O^T += V^T P^T, 16 keys per step
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const float vm = vsc[kk] * down;
      // fp16: dividing the output by the sum of the rounded probabilities takes
      // the common part of their roundings out (the dominant key's own most of
      // all). Blocks of far smaller values keep the exact ones: theirs may
      // round to nothing.
      const bool rounded = kHalf && vm > 0.125f;
      const float ivm = rounded ? __frcp_rn(vm) : 1.f;
      uint32_t pb[NT * kParts][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float p0 = ex2(s[kk][n][2 * x] - m[n][0]), p1 = ex2(s[kk][n][2 * x + 1] - m[n][1]);
          l[n][0] += p0;
          l[n][1] += p1;
          const float x0 = p0 * vm, x1 = p1 * vm;
          const uint32_t hi = pack(x0, x1);
          pb[n][x] = transpose8(hi);
          if constexpr (kHalf) {
            const float2 r = unpack(hi);
            lr[n][0] = fmaf(rounded ? r.x : p0, ivm, lr[n][0]);
            lr[n][1] = fmaf(rounded ? r.y : p1, ivm, lr[n][1]);
          } else {
            const float2 h2 = unpack(hi);
            pb[NT + n][x] = transpose8(pack(x0 - h2.x, x1 - h2.y));
          }
        }
      // Keys 16 kk + 2 t, + 1, + 8, + 9 of thread t; coordinates gq HP/8 .. of quad gq.
      constexpr int kWords = HP / 32 < 4 ? HP / 32 : 4;   // 4-coordinate words per pass
#pragma unroll
      for (int hf = 0; hf < HP / 32 / kWords; ++hf) {
        uint32_t w[4][kWords];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = 16 * kk + 2 * t + (x & 1) + 8 * (x >> 1);
          const int byte = gq * (HP / 8) + 16 * hf;
          const uint8_t* src = vt + chunk_at<HP>(r, byte >> 4) + (byte & 15);
          if constexpr (kWords == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(src);
            w[x][0] = v.x ^ 0x80808080u;
            w[x][1] = v.y ^ 0x80808080u;
            w[x][2] = v.z ^ 0x80808080u;
            w[x][3] = v.w ^ 0x80808080u;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(src);
            w[x][0] = v.x ^ 0x80808080u;
            w[x][1] = v.y ^ 0x80808080u;
          }
        }
#pragma unroll
        for (int y = 0; y < kWords; ++y) {
          const uint32_t alo = __byte_perm(w[0][y], w[1][y], 0x5140u), ahi = __byte_perm(w[0][y], w[1][y], 0x7362u);
          const uint32_t blo = __byte_perm(w[2][y], w[3][y], 0x5140u), bhi = __byte_perm(w[2][y], w[3][y], 0x7362u);
          const uint32_t a0[4] = {codes_lo(alo), codes_hi(alo), codes_lo(blo), codes_hi(blo)};
          const uint32_t a1[4] = {codes_lo(ahi), codes_hi(ahi), codes_lo(bhi), codes_hi(bhi)};
          const int i = 8 * hf + 2 * y;
#pragma unroll
          for (int n = 0; n < NT * kParts; ++n) {
            mma16816(o[i][n % NT], a0, pb[n][0], pb[n][1]);
            mma16816(o[i + 1][n % NT], a1, pb[n][0], pb[n][1]);
          }
        }
      }
    }
    if constexpr (FLUSH) {
      if (++held == 8) {
        held = 0;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              acc[i][n][e] += o[i][n][e];
              o[i][n][e] = 0.f;
            }
      }
    }
    stage ^= 1;
    if (stage == 0) parity ^= 1;
    const long long slot = worker + (long long)cp.bg * p.nrt + cp.rt;
    if (!cp.next(p)) continue;

    // ---- the piece ends: (m, l) and O of its rows into slot worker + range
    fresh_piece = true;
    const float upw = __int_as_float((127 + wexp) << 23);   // O is in units of 2^wexp
    if constexpr (FLUSH) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][n][e] += acc[i][n][e];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float sum = l[n][h], sr = kHalf ? lr[n][h] : 0.f;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, x);
          if (kHalf) sr += __shfl_xor_sync(0xffffffffu, sr, x);
        }
        const int row = 8 * n + 2 * t + h;
        if (r0 + row >= p.S * p.G) continue;
        if (gq == 0)
          *reinterpret_cast<float4*>(p.part_ml + (slot * p.rt_rows + row) * 4) = make_float4(m[n][h], sum, kHalf ? sr : sum, 0.f);
        float* dst = p.part_o + (slot * p.rt_rows + row) * p.H;
#pragma unroll
        for (int i = 0; i < kSteps; i += 2) {
          const int d = gq * (HP / 8) + 2 * i;
          if (d < p.H)
            *reinterpret_cast<float4*>(dst + d) = make_float4(o[i][n][h] * upw, o[i][n][2 + h] * upw,
                                                              o[i + 1][n][h] * upw, o[i + 1][n][2 + h] * upw);
        }
      }
  }
  cp_wait<0>();
  if (!waited) dep_wait();   // also without need: what follows on the stream waits for this kernel alone
}

// ------------------------------------------------------------------ merge

// Slots of the pieces of range (b, g, rt) in the split above: [first, first + n).
__device__ __forceinline__ int pieces_of(const BlockParams& p, long long units, int b, int gr, int total, int fresh,
                                         int t0, int nt, long long before, long long* first) {
  int lo, hi;
  tile_units(p, total, fresh, t0, nt, gr % p.nrt, &lo, &hi);
  if (nt <= 0 || lo >= hi) return 0;
  const long long base = before + (long long)gr * (nt + kBlockRangeCost);
  const long long live = live_workers(p, units);
  const long long w0 = ((base + lo + 1) * live - 1) / units, w1 = ((base + hi) * live - 1) / units;
  *first = w0 + (long long)b * p.Nkv * p.nrt + gr;
  return (int)(w1 - w0) + 1;
}

struct RangeInfo {
  long long slot0;
  int n, total, fresh;
};

// All of the block: the batch's units and the pieces of range (b, gr).
__device__ RangeInfo range_info(const BlockParams& p, int b, int gr) {
  const int lane = threadIdx.x & 31;
  long long units = 0, before = 0;
  for (int x = lane; x < p.B; x += 32) {
    int a, f, t0, nt;
    const long long u = seq_units(p, x, &a, &f, &t0, &nt);
    units += u;
    if (x < b) before += u;
  }
  for (int o = 16; o; o >>= 1) {
    units += __shfl_xor_sync(0xffffffffu, units, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  RangeInfo r;
  int t0, nt;
  r.slot0 = 0;
  seq_units(p, b, &r.total, &r.fresh, &t0, &nt);
  r.n = pieces_of(p, units, b, gr, r.total, r.fresh, t0, nt, before, &r.slot0);
  return r;
}

constexpr int kMaxPieces = 152 * warps_of(128) * 3 + 1;   // workers, at most

// Maximum / sum of v over the THREADS threads of the block.
template <int THREADS, bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, x) : v + x;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < THREADS / 32; ++i) v = MAX ? fmaxf(v, red[i]) : v + red[i];
  return v;
}

// Blocks [0, row_blocks) merge one query row each, the others add the weights
// of `keys` cache rows of one (b, g).
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS)
block_merge_kernel(const BlockParams p, long long row_blocks, int weight_chunks, int keys) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ float red[THREADS / 32];
  __shared__ float fac[kMaxPieces];
  __shared__ float4 acc[THREADS];
  // Every block waits for the attention kernel, also one without work: what
  // follows on the stream waits for this kernel alone.
  if (blockIdx.x < row_blocks) {
    const int nrows = p.S * p.G;
    const int bg = (int)(blockIdx.x / nrows), r = (int)(blockIdx.x % nrows), b = bg / p.Nkv, g = bg % p.Nkv;
    int total, fresh;
    if (!block_lengths(p, b, &total, &fresh)) {
      dep_wait();
      return;
    }
    const int i = r / p.G, h = g * p.G + r % p.G, rt = r / p.rt_rows, row = r % p.rt_rows;
    T* out = static_cast<T*>(p.out) + (((long long)b * p.S + i) * p.N + h) * p.H;
    const int q4 = p.H / 4;            // float4 columns, 4 .. 64
    if (i >= fresh) {
      dep_wait();
      for (int d = tid; d < p.H; d += THREADS) out[d] = T(0.f);
      return;
    }
    const RangeInfo ri = range_info(p, b, g * p.nrt + rt);
    const bool has_sink = p.sink || p.smooth;
    const float sink = has_sink ? (p.sink ? load_t(p.sink, h, p.t_type) : 0.f) * kLog2e : kNegBig;
    const int groups = THREADS / q4, grp = tid / q4, c = tid % q4;
    const float* src = p.part_o + (ri.slot0 * p.rt_rows + row) * p.H + 4 * c;
    const long long ld = (long long)p.rt_rows * p.H;
    dep_wait();
    constexpr int kAhead = 8;   // pieces of a thread under way while their factors are worked out
    float4 ahead[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (grp < groups && grp + k * groups < ri.n) ahead[k] = *reinterpret_cast<const float4*>(src + (grp + k * groups) * ld);
    float m = sink;
    for (int x = tid; x < ri.n; x += THREADS) {
      fac[x] = p.part_ml[((ri.slot0 + x) * p.rt_rows + row) * 4];
      m = fmaxf(m, fac[x]);
    }
    m = block_reduce<THREADS, true>(m, red);
    float l = 0.f, lr = 0.f;
    for (int x = tid; x < ri.n; x += THREADS) {
      const float f = ex2(fac[x] - m);
      fac[x] = f;
      const float4 v = *reinterpret_cast<const float4*>(p.part_ml + ((ri.slot0 + x) * p.rt_rows + row) * 4);
      l = fmaf(v.y, f, l);
      lr = fmaf(v.z, f, lr);
    }
    const float extra = has_sink ? ex2(sink - m) : 0.f;
    if (p.lse) {
      l = block_reduce<THREADS, false>(l, red) + extra;
      if (tid == 0) p.lse[(long long)bg * nrows + r] = l > 0.f ? m + log2f(l) : INFINITY;
    }
    l = block_reduce<THREADS, false>(lr, red) + extra;   // (fac is complete behind it)
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float4 v, float f) {
      a.x = fmaf(v.x, f, a.x);
      a.y = fmaf(v.y, f, a.y);
      a.z = fmaf(v.z, f, a.z);
      a.w = fmaf(v.w, f, a.w);
    };
    if (grp < groups) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (grp + k * groups < ri.n) add(ahead[k], fac[grp + k * groups]);
#pragma unroll 4
      for (int x = grp + kAhead * groups; x < ri.n; x += groups) add(*reinterpret_cast<const float4*>(src + x * ld), fac[x]);
    }
    acc[tid] = a;
    __syncthreads();
    if (tid < q4) {
      for (int x = 1; x < groups; ++x) {
        const float4 v = acc[x * q4 + tid];
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
      const float f = l > 0.f ? 1.f / l : 0.f;
      if constexpr (sizeof(T) == 2) {
        const uint2 v = make_uint2(pack(a.x * f, a.y * f), pack(a.z * f, a.w * f));
        *reinterpret_cast<uint2*>(out + 4 * tid) = v;
      } else {
        *reinterpret_cast<float4*>(out + 4 * tid) = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
      }
    }
    return;
  }
  // ---- weights (one row tile: p.stash holds every row's scores)
  const long long x = blockIdx.x - row_blocks;
  const int bg = (int)(x / weight_chunks), chunk = (int)(x % weight_chunks), b = bg / p.Nkv, g = bg % p.Nkv;
  int total, fresh;
  const int j0 = chunk * keys;
  if (!block_lengths(p, b, &total, &fresh) || j0 >= total) {
    dep_wait();
    return;
  }
  __shared__ float nl[16];                       // -lse of the rows
  const int nrows = fresh * p.G, rs = p.stash_rows;   // live rows (at most one row tile)
  const RangeInfo ri = range_info(p, b, g);
  int t0, nt;
  units_of(p, total, fresh, &t0, &nt);
  const long long at0 = (long long)bg * p.C;
  const float* st = p.stash + (long long)bg * p.stash_ld * rs;
  const int jend = min(total, j0 + keys), seen = t0 * kBlockUnit;   // keys before `seen`: no scores
  dep_wait();
  // A thread's keys, kAhead at a time: their loads are under way together, the
  // first ones while the rows' sums are worked out.
  constexpr int kAhead = 8;
  const bool quads = (rs & 3) == 0 && nrows >= 4;
  float w[kAhead];
  float4 v[kAhead];
  auto scored = [&](int j) { return j < jend && j >= seen; };
  auto fetch = [&](int j) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int ju = j + u * THREADS;
      w[u] = p.past_w && ju < min(jend, total - fresh) ? p.past_w[at0 + ju] : 0.f;
      if (quads && scored(ju)) v[u] = *reinterpret_cast<const float4*>(st + (long long)ju * rs);
    }
  };
  fetch(j0 + tid);
  for (int r = warp; r < nrows; r += THREADS / 32) {   // a warp per row, lanes over the pieces
    const float4* ml = reinterpret_cast<const float4*>(p.part_ml) + ri.slot0 * p.rt_rows + r;   // (m, l, ..)
    const bool has_sink = p.sink || p.smooth;
    const float sink = has_sink ? (p.sink ? load_t(p.sink, g * p.G + r % p.G, p.t_type) : 0.f) * kLog2e : kNegBig;
    float m = sink, l = 0.f;
    for (int i = lane; i < ri.n; i += 32) m = fmaxf(m, ml[(long long)i * p.rt_rows].x);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int i = lane; i < ri.n; i += 32) {
      const float4 x4 = ml[(long long)i * p.rt_rows];
      l = fmaf(x4.y, ex2(x4.x - m), l);
    }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (has_sink) l += ex2(sink - m);
    if (lane == 0) nl[r] = -(m + log2f(l));
  }
  __syncthreads();
  for (int j = j0 + tid; j < jend; j += kAhead * THREADS) {
    if (j != j0 + tid) fetch(j);
    int r = 0;
    if (quads) {
      for (; r + 4 <= nrows; r += 4) {
        if (r > 0) {
#pragma unroll
          for (int u = 0; u < kAhead; ++u)
            if (scored(j + u * THREADS)) v[u] = *reinterpret_cast<const float4*>(st + (long long)(j + u * THREADS) * rs + r);
        }
        const float4 n = make_float4(nl[r], nl[r + 1], nl[r + 2], nl[r + 3]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (scored(j + u * THREADS))
            w[u] += (ex2(v[u].x + n.x) + ex2(v[u].y + n.y)) + (ex2(v[u].z + n.z) + ex2(v[u].w + n.w));
      }
    }
    for (; r < nrows; ++r) {
      float s1[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (scored(j + u * THREADS)) s1[u] = st[(long long)(j + u * THREADS) * rs + r];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (scored(j + u * THREADS)) w[u] += ex2(s1[u] + nl[r]);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (j + u * THREADS < jend) p.present_w[at0 + j + u * THREADS] = w[u];
  }
}

// ------------------------------------------------------------------ weights of long chunks

constexpr int kWKeys = 64;       // cache rows per block, 16 per warp
constexpr int kWRows = 64;       // query rows staged at a time

// present_weights from the rows' log-sum-exp: a warp holds 16 keys as the A
// operand and runs over the query rows (B operand, staged in shared memory in
// fragment order, hi and lo parts for fp32).
template <typename T, int HP>
__global__ void __launch_bounds__(128)
block_weights_kernel(const BlockParams p) {
  constexpr bool kHalf = sizeof(T) == 2;
  constexpr int kSteps = HP / 16;
  constexpr int kParts = kHalf ? 1 : 2;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint2* qs = reinterpret_cast<uint2*>(smem_raw);              // [row tile of 8][step][part][lane]
  float4* rp = reinterpret_cast<float4*>(smem_raw + kWRows * HP * 2 * kParts);  // per row: -, lse, position
  float* up = reinterpret_cast<float*>(rp + kWRows);                              // per row: 2^e of an fp32 row
  const int bg = blockIdx.y, b = bg / p.Nkv, g = bg % p.Nkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, t = lane & 3;
  int total, fresh;
  if (!block_lengths(p, b, &total, &fresh)) return;
  const int j0 = blockIdx.x * kWKeys;
  if (j0 >= total) return;
  const int past = total - fresh, jw = j0 + 16 * warp;
  const float ks = jw < total ? p.ks[(long long)bg * p.nblk + (jw >> p.bs_log2)] : 0.f;
  uint32_t a[kSteps][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = jw + gq + 8 * h;
    const int8_t* row = p.kc + ((long long)bg * p.C + j) * p.H;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int d = t * (HP / 4) + 4 * i;
      const uint32_t w = (j < total && d < p.H ? *reinterpret_cast<const uint32_t*>(row + d) : 0u) ^ 0x80808080u;
      a[i][h] = codes_lo(w);
      a[i][2 + h] = codes_hi(w);
    }
  }
  float sum[2] = {0.f, 0.f};
  // Query rows that see a key of this block: positions j0 .. j0 + 63 + W.
  const int i_lo = max(0, j0 - past);
  const int i_hi = p.window >= 0 ? min(fresh, j0 + kWKeys + p.window - past) : fresh;
  for (int r0 = i_lo * p.G; r0 < i_hi * p.G; r0 += kWRows) {
    __syncthreads();
    for (int x = tid; x < kWRows; x += 128) {
      const int r = r0 + x;
      float4 v = make_float4(0.f, INFINITY, 0.f, 0.f);   // a row that does not count: exp2(0 - inf) = 0
      if (r < i_hi * p.G) {
        v.y = p.lse[(long long)bg * p.S * p.G + r];
        v.z = __int_as_float(past + r / p.G);
      }
      rp[x] = v;
    }
    for (int x = warp; x < kWRows / 8; x += 4) {
      const int r = r0 + 8 * x + gq;
      const T* q = r < i_hi * p.G ? static_cast<const T*>(p.q) +
                                        (((long long)b * p.S + r / p.G) * p.N + g * p.G + r % p.G) * p.H
                                  : nullptr;
      float down = 1.f;
      if constexpr (!kHalf) {
        float mx = 0.f;
        for (int i = 0; i < kSteps; ++i) {
          const int d = t * (HP / 4) + 4 * i;
          if (q && d < p.H) {
            const float4 v = *reinterpret_cast<const float4*>(q + d);
            mx = fmax3(mx, fabsf(v.x), fabsf(v.y));
            mx = fmax3(mx, fabsf(v.z), fabsf(v.w));
          }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int ex = (__float_as_int(mx) >> 23) & 0xff;
        const int e = ex == 0 ? 0 : min(ex, 253) - 127;
        down = __int_as_float((127 - e) << 23);
        if (t == 0) up[8 * x + gq] = __int_as_float((127 + e) << 23);
      }
      for (int i = 0; i < kSteps; ++i) {
        const int d = t * (HP / 4) + 4 * i;
        uint2 hi = make_uint2(0u, 0u), lo = hi;
        if (q && d < p.H) {
          if constexpr (kHalf) {
            hi = *reinterpret_cast<const uint2*>(q + d);
          } else {
            float4 v = *reinterpret_cast<const float4*>(q + d);
            v.x *= down;
            v.y *= down;
            v.z *= down;
            v.w *= down;
            hi = make_uint2(pack(v.x, v.y), pack(v.z, v.w));
            const float2 h0 = unpack(hi.x), h1 = unpack(hi.y);
            lo = make_uint2(pack(v.x - h0.x, v.y - h0.y), pack(v.z - h1.x, v.w - h1.y));
          }
        }
        qs[((x * kSteps + i) * kParts) * 32 + lane] = hi;
        if constexpr (!kHalf) qs[((x * kSteps + i) * kParts + 1) * 32 + lane] = lo;
      }
    }
    __syncthreads();
    if (jw < total) {
      for (int x = 0; x < kWRows / 8; ++x) {
        // The attention kernel's scores bit for bit (same products, order and
        // factors): their own error then cancels against the log-sum-exp's.
        float c2[kParts][4] = {};
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            const uint2 q = qs[((x * kSteps + i) * kParts + part) * 32 + lane];
            mma16816(c2[part], a[i], q.x, q.y);
          }
        float c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = kHalf ? c2[0][e] : c2[0][e] + c2[kParts - 1][e];
#pragma unroll
        for (int u = 0; u < 2; ++u) {   // rows 8 x + 2 t + u
          const float4 v = rp[8 * x + 2 * t + u];
          const int pos = __float_as_int(v.z);
          const float us = (kHalf ? 1.f : up[8 * x + 2 * t + u]) * p.scale;
          const float f = (p.softcap > 0.f ? us : us * kLog2e) * ks;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int j = jw + gq + 8 * h;
            float z = c[2 * h + u] * f;
            if (p.softcap > 0.f) z = p.softcap * kLog2e * tanhf(z / p.softcap);
            const bool see = j <= pos && (p.window < 0 || j >= pos - p.window);
            sum[h] += see ? ex2(z - v.y) : 0.f;
          }
        }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
    const int j = jw + gq + 8 * h;
    if (t == 0 && j < total) {
      const long long at = (long long)bg * p.C + j;
      p.present_w[at] = sum[h] + (p.past_w && j < past ? p.past_w[at] : 0.f);
    }
  }
}

// ------------------------------------------------------------------ launches

constexpr int kMaxDevices = 64;

// Dynamic shared memory above 48 KB is allowed once per kernel and device.
template <typename K>
cudaError_t allow_smem(K kern, int bytes, bool* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
    done[dev] = true;
  }
  return cudaSuccess;
}

template <typename T, int HP, int NT, bool PLAIN, bool FLUSH>
cudaError_t attn_one(const BlockParams& p, cudaStream_t st) {
  static bool done[kMaxDevices];
  constexpr int kWarps = warps_of(HP), smem = kWarps * (int)sizeof(WarpSmem<HP>) + 1024;
  static_assert(smem + kWarps * sizeof(WarpCtl) <= 232448, "shared memory per CTA");
  cudaError_t e = allow_smem(block_attn_kernel<T, HP, NT, PLAIN, FLUSH>, smem, done);
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  const uint64_t rows = (uint64_t)p.B * p.Nkv * p.C;
  if ((e = encode_codes(&mk, p.kc, rows, p.H, HP, kBlockUnit)) != cudaSuccess) return e;
  if ((e = encode_codes(&mv, p.vc, rows, p.H, HP, kBlockUnit)) != cudaSuccess) return e;
  return launch_dependent(p.k != nullptr, block_attn_kernel<T, HP, NT, PLAIN, FLUSH>, dim3((unsigned)(p.workers / kWarps)),
                          kWarps * 32, (size_t)smem, st, p, mk, mv);
}

template <typename T, int HP, int NT>
cudaError_t attn_nt(const BlockParams& p, cudaStream_t st) {
  const bool plain = !(p.softcap > 0.f || p.stash);
  if constexpr (sizeof(T) == 4) {
    if (p.flush) return plain ? attn_one<T, HP, NT, true, true>(p, st) : attn_one<T, HP, NT, false, true>(p, st);
  }
  return plain ? attn_one<T, HP, NT, true, false>(p, st) : attn_one<T, HP, NT, false, false>(p, st);
}

template <int HP>
cudaError_t attn_hp(const BlockParams& p, cudaStream_t st) {
  if (p.t_type == kF32) return attn_nt<float, HP, 1>(p, st);
  if constexpr (HP <= 128) {
    if (p.rt_rows == 16) return attn_nt<__half, HP, 2>(p, st);
  }
  return attn_nt<__half, HP, 1>(p, st);
}

template <typename T, int HP>
cudaError_t weights_one(const BlockParams& p, cudaStream_t st) {
  static bool done[kMaxDevices];
  const int smem = kWRows * HP * 2 * (sizeof(T) == 2 ? 1 : 2) + kWRows * 20;
  cudaError_t e = allow_smem(block_weights_kernel<T, HP>, smem, done);
  if (e != cudaSuccess) return e;
  block_weights_kernel<T, HP><<<dim3((unsigned)((p.T + kWKeys - 1) / kWKeys), (unsigned)(p.B * p.Nkv)), 128, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

// fp32 rows come as two fp16 parts: a tile of 8 rows is two MMA tiles. Up to 8
// fp16 rows take one, more take tiles of 16 (the codes are converted half as
// often), but for head sizes above 128, whose output tiles fill the registers.
int block_row_tile(int t_type, int H, long long rows) { return t_type == kF16 && H <= 128 && rows > 8 ? 16 : 8; }

// One worker per warp, as many CTAs of four as an SM holds; fewer when there
// are not four units for each.
int block_workers(const BlockParams& p) {
  const int kWarps = warps_of(p.H);
  const long long most = 152LL * kWarps * (p.H > 128 ? 1 : p.rt_rows > 8 || p.flush ? 2 : 3);
  const int keys = p.window >= 0 && (long long)p.window + p.S < p.T ? p.window + p.S + kBlockUnit : p.T;
  const long long units =
      (long long)p.B * p.Nkv * p.nrt * ((keys + kBlockUnit - 1) / kBlockUnit + kBlockRangeCost);
  long long w = (units + 3) / 4;
  w = (w + kWarps - 1) / kWarps * kWarps;
  return (int)(w < most ? w : most);
}

cudaError_t launch_block_attn(const BlockParams& p, cudaStream_t st) {
  return p.H <= 64 ? attn_hp<64>(p, st) : p.H <= 128 ? attn_hp<128>(p, st) : attn_hp<256>(p, st);
}

cudaError_t launch_block_merge(const BlockParams& p, cudaStream_t st) {
  const long long rows = (long long)p.B * p.Nkv * p.S * p.G;
  // Cache rows of a weight block: every block first adds up the rows' sums, so
  // 2048 where that still leaves the SMs several blocks each, else 512.
  const int keys = (long long)p.B * p.Nkv * p.T >= 152LL * 4 * 2048 ? 2048 : 512;
  const int chunks = p.stash ? (p.T + keys - 1) / keys : 0;
  const long long blocks = rows + (long long)p.B * p.Nkv * chunks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  // A row of a long split has many pieces: more threads read them at once.
  const bool many = p.workers / ((long long)p.B * p.Nkv * p.nrt) >= 64;
  const dim3 grid((unsigned)blocks);
  if (p.t_type == kF16)
    return many ? launch_dependent(true, block_merge_kernel<__half, 512>, grid, 512, 0, st, p, rows, chunks, keys)
                : launch_dependent(true, block_merge_kernel<__half, 128>, grid, 128, 0, st, p, rows, chunks, keys);
  return many ? launch_dependent(true, block_merge_kernel<float, 512>, grid, 512, 0, st, p, rows, chunks, keys)
              : launch_dependent(true, block_merge_kernel<float, 128>, grid, 128, 0, st, p, rows, chunks, keys);
}

cudaError_t launch_block_weights(const BlockParams& p, cudaStream_t st) {
  if (p.t_type == kF16)
    return p.H <= 64 ? weights_one<__half, 64>(p, st) : p.H <= 128 ? weights_one<__half, 128>(p, st) : weights_one<__half, 256>(p, st);
  return p.H <= 64 ? weights_one<float, 64>(p, st) : p.H <= 128 ? weights_one<float, 128>(p, st) : weights_one<float, 256>(p, st);
}

}  // namespace gqa
