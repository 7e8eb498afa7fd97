// Attention of drafted nodes on the tensor cores: fp16, head sizes up to 128,
// positive scales.
//
// Rows are (node, grouped head) of a KV head (b, g), 128 in a row tile; keys
// come in units of 128, the cached rows first, then the nodes, whose keys and
// values are read from the call's own tensors (nothing waits for the append,
// which the same launch does). All units are laid end to end and every SM takes
// an equal share (tree_internal.h): one long sequence fills the GPU.
//
// S = Q K^T and O += P V run on tcgen05 with S, P and O in tensor memory, two
// softmax groups of 128 threads (a thread a row) beside them. A row tile of up
// to 128 rows (NQ = 1) gives each group every second unit of keys, with an O and
// running maximum of its own, joined when a range ends (a thread reads both O of
// its row: tensor memory is shared by lane, not by group); more rows (NQ = 2)
// give each group a row tile, so a unit is read once for 256 rows.
//
// Warps: 0 TMA into a ring of K and V tiles, across the ends of ranges; 1 MMA
// issue, tensor memory; 2, 3 clean V tiles that some rows see in part (rows
// behind the last are zeroed, and what is not finite, which would reach the
// rows that do not see it as 0 x inf, goes to the epilogue); 4..11 softmax,
// queries, epilogue. Every wait is bounded.
//
// P enters as 2^6 p of a reference maximum that may lag by 2^8; the output is
// divided by the sum of the rounded P, which takes the common part of their
// roundings out.
//
// What bounds it. Few rows: HBM. 16 sequences of 1024..8176 rows, 16 nodes, 32
// heads over 8: 60 us (ncu) for 310 MB, 5.2 TB/s (0.76 of the measured copy); the rest
// are the starts and ends of ranges, which the ring runs across. More rows: the
// chain S, maximum, exponents, P V of two groups, with two softmax warps a
// scheduler (1.5 to 1.7 instructions a clock; the MMA pipe is busy 26 % of the
// time, the exponents' 27 %). 208 rows of 64 dims: 1.8 us a unit of 256 rows (200k
// keys: 42 us, ncu); 256 rows of 128 dims with a softcap 3.5 us, 0.69 PFLOP/s (without
// one 83 us where it takes 101). Measured by events around single cold launches: steps
// of 64 keys with two S tiles a group 126 against 105 us (softcap) and 50 against 44
// (200k keys); scores kept in registers between maximum and exponents spilled (107 to
// 115, 44 to 52).
#include <cuda_fp16.h>

#include "block_tc.cuh"
#include "common.cuh"
#include "tcgen05.cuh"
#include "tma_host.h"
#include "tree_internal.h"

namespace gqa {
namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kSoftWarp0 = 4;
constexpr int kKeys = 128;                     // keys of a unit
constexpr uint32_t kBox = 128u * 128u;         // 128 rows x 64 dims
constexpr float kLazy = 8.0f;                  // log2 growth of a maximum tolerated before rescaling O
constexpr float kLift = 6.0f;
constexpr int kOddNodes = kTreeNodes / 32;     // words of a piece's odd keys: nodes, then
constexpr int kOddEdge = 21;                   // cached rows from the first on that a window hides from some nodes
constexpr int kOddSets = 8;                    // pieces the cleaners may be ahead of the epilogue, and more
constexpr uint32_t kIdS = idesc_f16(128, 128, 0, 0);

// HB: 64-dim boxes of a row. NQ: row tiles of a piece.
template <int HB, int NQ>
struct __align__(1024) TcSmem {
  static constexpr uint32_t kTile = HB * kBox;
  static constexpr int kRing = HB == 1 ? 8 : 4;   // (3 to 5 tiles of 32 KB: within 2 %)
  uint8_t q[NQ][kTile];
  uint8_t ring[kRing][kTile];
  float2 ml[2][128];             // m, l of a group's rows (NQ = 1)
  // A slot's copy has landed; the cleaners are through with it (every item, so that its phase is the slot's); it may be
  // written again: the MMAs that read it are done, and the cleaners have seen it (they never fall a phase behind).
  uint64_t full[kRing], clean[kRing], empty[kRing];
  uint64_t q_ready, q_free;
  uint64_t s_full[2], p_full[2][2], o_done[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
  unsigned odd[kOddSets][kOddNodes + kOddEdge + 1];   // last word: any
  short par[kTreeNodes];
};

template <typename SM>
__device__ __forceinline__ bool aborted(const SM& sm) {
  return *reinterpret_cast<const volatile int*>(&sm.abort) != 0;
}
template <typename SM>
__device__ __forceinline__ void set_abort(const TreeParams& p, SM& sm) {
  *reinterpret_cast<volatile int*>(&sm.abort) = 1;
  if (p.status) atomicOr(p.status, GQA_DEVICE_TIMEOUT_BIT);
}

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// AND over the 256 softmax threads.
__device__ __forceinline__ bool soft_all(bool v) {
  uint32_t r;
  asm volatile("{ .reg .pred p, c; setp.ne.u32 c, %1, 0; bar.red.and.pred p, 1, 256, c; selp.u32 %0, 1, 0, p; }"
               : "=r"(r)
               : "r"((uint32_t)v)
               : "memory");
  return r != 0;
}

// a + the two halves of h, in fp32.
__device__ __forceinline__ float2 add_half2(float2 a, uint32_t h) {
  float2 r;
  asm("{ .reg .f16 l, u; mov.b32 {l, u}, %2; add.rn.f32.f16 %0, l, %3; add.rn.f32.f16 %1, u, %4; }"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h), "f"(a.x), "f"(a.y));
  return r;
}

// A unit of keys of a range: first row (of the cache, or node), and whether some rows see it in part.
struct Unit {
  bool cached;
  int first, n;      // valid rows
  bool edge;         // a window hides some of it from some nodes
  bool partial;      // its V tile needs the cleaners
};
__device__ __forceinline__ Unit unit_of(const TreeParams& p, const TreeSeq& s, int u) {
  Unit x;
  x.cached = u < s.np;
  x.first = x.cached ? s.k0 + u * kKeys : (u - s.np) * kKeys;
  x.n = min(kKeys, x.cached ? s.past - x.first : s.fresh - x.first);
  x.edge = x.cached && p.window >= 0 && x.first < s.past - p.window + s.fresh;
  x.partial = !x.cached || x.n < kKeys || x.edge;
  return x;
}

template <bool CAP, int HB, int NQ>
__global__ void __launch_bounds__(kThreads, 1)
tree_tc_kernel(const TreeParams p, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
               const __grid_constant__ CUtensorMap tmnk, const __grid_constant__ CUtensorMap tmnv) {
  using SM = TcSmem<HB, NQ>;
  constexpr int R = SM::kRing, L = NQ == 1 ? 2 : 1;   // L: units whose S is issued ahead of the first P V
  constexpr int kRows = 128 * NQ;
  constexpr uint32_t kIdO = idesc_f16(128, 64 * HB, 0, 1);
  extern __shared__ uint8_t smem_raw[];
  SM& sm = *reinterpret_cast<SM*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const long long units = tree_units(p);
  const long long live = tree_live(p, units);
  const long long u0 = units * blockIdx.x / live, u1 = units * (blockIdx.x + 1) / live;
  const bool work = blockIdx.x < live && u0 < u1;   // uniform over the CTA

  if (warp == 1) tmem_alloc(&sm.tmem, 512);
  for (int x = tid; x < kOddSets * (kOddNodes + kOddEdge + 1); x += kThreads) sm.odd[0][x] = 0u;
  if (tid == 0) {
    for (int i = 0; i < R; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.clean[i], 2);
      mbar_init(&sm.empty[i], 3);
    }
    mbar_init(&sm.q_ready, 8);
    mbar_init(&sm.q_free, 1);
    for (int q = 0; q < 2; ++q) {
      mbar_init(&sm.s_full[q], 1);
      mbar_init(&sm.p_full[q][0], 4);
      mbar_init(&sm.p_full[q][1], 4);
      mbar_init(&sm.o_done[q], 1);
    }
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    mbar_fence_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  dep_launch();
  const uint32_t tmem = sm.tmem;
  TreeWalk w;
  w.left = 0;
  if (work) w.start(p, u0, u1 - u0);

  if (warp == 0) {
    // ================================================================ TMA of the key and value tiles
    bool ok = true;
    int it = 0, copied = 0;   // items of the ring; units begun (testing)
    for (; w.left > 0 && ok; w.next(p, w.piece())) {
      const int n = w.piece();
      const long long bg = (long long)w.b * p.Nkv + w.g;
      auto item = [&](int j, bool is_k) {
        if (!ok) return;
        if (is_k && copied++ == p.withhold_tile) {   // testing: never copied, the waits for it expire
          ok = false;
          return;
        }
        const int slot = it % R;
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.empty[slot], ((uint32_t)(it / R) & 1u) ^ 1u, p.wait_budget) && !aborted(sm));
        if (!ok) {
          if (lane == 0) set_abort(p, sm);
          return;
        }
        const Unit x = unit_of(p, w.s, w.off + j);
        if (elect_one()) {
          mbar_arrive_tx(&sm.full[slot], SM::kTile);
#pragma unroll
          for (int h = 0; h < HB; ++h) {
            if (x.cached)
              tma_load_2d(sm.ring[slot] + h * kBox, is_k ? &tmk : &tmv, 64 * h, (int)(bg * p.C) + x.first, &sm.full[slot]);
            else
              tma_load_4d(sm.ring[slot] + h * kBox, is_k ? &tmnk : &tmnv, 64 * h, w.g, x.first, w.b, &sm.full[slot]);
          }
        }
        __syncwarp();
        ++it;
      };
      for (int j = 0; j < min(L, n); ++j) item(j, true);
      for (int j = 0; j < n; ++j) {
        item(j, false);
        if (j + L < n) item(j + L, true);
      }
    }
    // No copy of this CTA may still be landing when it exits.
    for (int x = it > R ? it - R : 0; x < it; ++x) mbar_wait(&sm.full[x % R], (uint32_t)(x / R) & 1u, p.wait_budget);
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    const uint64_t dr0 = desc_kmajor_sw128(smem_addr(sm.ring[0])), dq0 = desc_kmajor_sw128(smem_addr(sm.q[0]));
    const uint64_t dv0 = desc_mnmajor_sw128(smem_addr(sm.ring[0]), kBox, 1024);
    bool ok = true;
    int it = 0, piece = 0, jobs[2] = {0, 0};   // jobs: (unit, group) pairs whose P V is issued
    auto wait1 = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, mbar_wait(bar, par, p.wait_budget) && !aborted(sm)) != 0;
    };
    auto issue_s = [&](int q, int slot) {
      const uint64_t a0 = dq0 + (uint64_t)((NQ == 2 ? q : 0) * (int)(SM::kTile >> 4));
      const uint64_t b0 = dr0 + (uint64_t)(slot * (int)(SM::kTile >> 4));
#pragma unroll
      for (int ks = 0; ks < 4 * HB; ++ks) {
        const uint64_t off = (uint64_t)((ks >> 2) * (int)(kBox >> 4) + (ks & 3) * 2);
        mma_f16_ss(tmem + q * 128, a0 + off, b0 + off, kIdS, ks > 0);
      }
      mma_commit(&sm.s_full[q]);
    };
    // O_q += P V of 64 keys, whose P is in columns 64 half .. + 31 of the group's S.
    auto issue_pv = [&](int q, int slot, int half, bool first) {
      const uint64_t b0 = dv0 + (uint64_t)(slot * (int)(SM::kTile >> 4));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mma_f16_ts(tmem + 256 + q * 128, tmem + q * 128 + half * 64 + i * 8, b0 + (uint64_t)((4 * half + i) * 128), kIdO,
                   !first || half > 0 || i > 0);
    };
    for (; w.left > 0 && ok; w.next(p, w.piece()), ++piece) {
      const int n = w.piece();
      ok = wait1(&sm.q_ready, (uint32_t)piece & 1u);
      // S of unit j for group q; K's tile is free behind its last use, the queries' behind the piece's last S.
      auto next_s = [&](int j, int q, int slot, bool last_use) {
        if (elect_one()) {
          issue_s(q, slot);
          if (last_use) mma_commit(&sm.empty[slot]);
          if (last_use && j == n - 1) mma_commit(&sm.q_free);
        }
        __syncwarp();
      };
      for (int j = 0; j < min(L, n) && ok; ++j, ++it) {
        ok = wait1(&sm.full[it % R], (uint32_t)(it / R) & 1u);
        if (!ok) break;
        tc_fence_after();
        if (NQ == 2) {
          next_s(j, 0, it % R, false);
          next_s(j, 1, it % R, true);
        } else {
          next_s(j, j & 1, it % R, true);
        }
      }
      for (int j = 0; j < n && ok; ++j) {
        const int vs = it % R;
        ok = wait1(unit_of(p, w.s, w.off + j).partial ? &sm.clean[vs] : &sm.full[vs], (uint32_t)(it / R) & 1u);
        if (!ok) break;
        ++it;
        const bool more = j + L < n;
        const int ks = it % R;
        const uint32_t kpar = (uint32_t)(it / R) & 1u;
        if (more) ++it;
#pragma unroll
        for (int y = 0; y < NQ; ++y) {
          const int q = NQ == 2 ? y : j & 1;
          const uint32_t par = (uint32_t)jobs[q] & 1u;
          for (int half = 0; half < 2 && ok; ++half) {
            ok = wait1(&sm.p_full[q][half], par);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              issue_pv(q, vs, half, j < L);
              if (half == 1) {
                mma_commit(&sm.o_done[q]);
                if (y == NQ - 1) mma_commit(&sm.empty[vs]);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          ++jobs[q];
          if (more) {
            if (y == 0) {
              ok = wait1(&sm.full[ks], kpar);
              if (!ok) break;
              tc_fence_after();
            }
            next_s(j + L, q, ks, y == NQ - 1);
          }
        }
      }
    }
    if (!ok && lane == 0) set_abort(p, sm);
    // Drain: every MMA this thread issued has finished before tensor memory is freed.
    if (elect_one()) {
      mma_commit(&sm.drain);
      mbar_wait(&sm.drain, 0, p.wait_budget);
    }
    __syncwarp();
  } else if (warp < kSoftWarp0) {
    // ================================================================ cleaners; lengths and trees out of range
    const int ct = tid - 64;
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
      int past, fresh;
      bool bad_tree = false;
      const bool good = tree_lengths(p, b, &past, &fresh);
      if (good)
        for (int i = ct; i < fresh; i += 64) tree_parent(p.parents[(long long)b * p.parents_ld + i], i, &bad_tree);
      if (bad_tree && p.status) atomicOr(p.status, GQA_DEVICE_BAD_TREE_BIT);
      if (!good && ct == 0 && p.status) atomicOr(p.status, GQA_DEVICE_BAD_SEQLEN_BIT);
    }
    bool ok = true;
    int it = 0;
    for (int piece = 0; w.left > 0 && ok; w.next(p, w.piece()), ++piece) {
      const int n = w.piece();
      unsigned* odd = sm.odd[piece % kOddSets];
      for (int k = 0; k < 2 * n; ++k, ++it) {   // items in the ring's order
        const int slot = it % R;
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[slot], (uint32_t)(it / R) & 1u, p.wait_budget) && !aborted(sm));
        if (!ok) break;
        // The item: keys of the first L units, then values and keys in turn until the keys run out.
        const int y = k - min(L, n), keys = n - min(L, n);
        const bool is_v = y >= 0 && (y >= 2 * keys || (y & 1) == 0);
        const int j = y < 2 * keys ? y >> 1 : y - keys;
        const Unit x = unit_of(p, w.s, w.off + max(j, 0));
        uint8_t* v = sm.ring[slot];
        if (is_v && x.partial) {
          const bool scan = !x.cached || x.edge;
          for (int e = ct + (scan ? 0 : x.n * 8 * HB); e < 128 * 8 * HB; e += 64) {
            const int r = e / (8 * HB), c = e % (8 * HB);
            uint4* at = reinterpret_cast<uint4*>(v + (c >> 3) * kBox + sw128_offset((uint32_t)r, (uint32_t)(c & 7)));
            if (r >= x.n) {
              *at = make_uint4(0u, 0u, 0u, 0u);
              continue;
            }
            const uint4 q4 = *at;
            uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
            bool any = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // an exponent of all ones: the carry of one more reaches the sign's place
              const uint32_t hit = ((q[k] & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
              if (hit) {
                any = true;
                q[k] &= ~((hit >> 15) * 0xffffu);
              }
            }
            if (any) {
              *at = make_uint4(q[0], q[1], q[2], q[3]);
              const int key = x.cached ? x.first - w.s.k0 + r : x.first + r;
              if (!x.cached || key < 32 * kOddEdge) {
                atomicOr(&odd[(x.cached ? kOddNodes : 0) + (key >> 5)], 1u << (key & 31));
                odd[kOddNodes + kOddEdge] = 1u;
              }
            }
          }
          fence_async_smem();   // cleaned tile (generic stores) -> async proxy: the P V MMAs read it
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.clean[slot]);
          mbar_arrive(&sm.empty[slot]);
        }
      }
    }
    if (!ok && lane == 0) set_abort(p, sm);
  } else {
    // ================================================================ softmax groups
    const int q = (warp - kSoftWarp0) >> 2;   // group
    const int quarter = warp & 3;             // tensor-memory lane quarter of this warp
    const int rl = quarter * 32 + lane;
    const int st = tid - 32 * kSoftWarp0;
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_addr + q * 128;
    const uint32_t o_addr = tmem + lane_addr + 256;
    // (At least the smallest normal number: a hidden score times 0 would be NaN.)
    const float mul = fmaxf(p.scale * (CAP ? 1.f / p.softcap : kLog2e), 1.17549435e-38f);
    const float c2 = p.softcap * kLog2e;
    const __half* qsrc = static_cast<const __half*>(p.q);
    bool ok = true, appended = false;
    int job = 0;                              // S tiles of this group so far
    auto append = [&]() {   // padding rows and the nodes' cache rows, a part each
      const int kv = p.Nkv * p.H / 8, qh = p.N * p.H / 8, rc = p.H / 8;   // 16-byte chunks of a node
      for (long long x = blockIdx.x; x < (long long)p.B * p.S; x += gridDim.x) {
        const int b = (int)(x / p.S), i = (int)(x % p.S);
        int past, fresh;
        if (!tree_lengths(p, b, &past, &fresh)) continue;
        if (i >= fresh) {
          uint4* o = reinterpret_cast<uint4*>(p.out) + x * qh;
          for (int c = st; c < qh; c += 256) o[c] = make_uint4(0u, 0u, 0u, 0u);
          continue;
        }
        for (int c = st; c < 2 * kv; c += 256) {
          const bool is_v = c >= kv;
          const int d = is_v ? c - kv : c, g = d / rc;
          const uint4 v = reinterpret_cast<const uint4*>(is_v ? p.v : p.k)[x * kv + d];
          reinterpret_cast<uint4*>(is_v ? p.vc : p.kc)[(((long long)b * p.Nkv + g) * p.C + past + i) * rc + d % rc] = v;
        }
      }
    };
    for (int piece = 0; w.left > 0; ++piece) {
      const int n = w.piece();
      const TreeSeq s = w.s;
      const int nrows = s.fresh * p.G;
      const int r = w.rt * kRows + (NQ == 2 ? q * 128 : 0) + rl;
      const bool live_row = r < nrows;
      const int i = live_row ? r / p.G : 0, hd = w.g * p.G + (live_row ? r % p.G : 0);
      // ---- queries: a thread its row (NQ = 1: the groups half of it each)
      if (piece > 0 && ok)
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_free, (uint32_t)(piece - 1) & 1u, p.wait_budget) && !aborted(sm));
      {
        const uint4* src = reinterpret_cast<const uint4*>(qsrc + (((long long)w.b * p.S + i) * p.N + hd) * p.H);
        constexpr int kC = NQ == 2 ? 8 * HB : 4 * HB;
        const int c0 = NQ == 2 ? 0 : q * kC;
        uint4 x[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) x[c] = live_row && (c0 + c) * 8 < p.H ? src[c0 + c] : make_uint4(0u, 0u, 0u, 0u);
        uint8_t* dst = sm.q[NQ == 2 ? q : 0];
#pragma unroll
        for (int c = 0; c < kC; ++c)
          *reinterpret_cast<uint4*>(dst + ((c0 + c) >> 3) * kBox + sw128_offset((uint32_t)rl, (uint32_t)((c0 + c) & 7))) = x[c];
        fence_async_smem();   // query rows (generic stores) -> async proxy: the S MMAs read them
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_ready);
      }
      // ---- the tree, where the piece meets its nodes or a window needs the depths
      const bool tree = w.off + n > s.np || p.window >= 0;
      if (tree) {
        soft_sync();   // nobody reads the piece before's
        bool bad = false;
        for (int x = st; x < s.fresh; x += 256)
          sm.par[x] = (short)tree_parent(p.parents[(long long)w.b * p.parents_ld + x], x, &bad);
        soft_sync();
      }
      if (!appended) {
        append();
        appended = true;
      }
      int lo_key = 0;
      if (p.window >= 0) {
        int d = 0;
        for (int a = sm.par[i]; a >= 0; a = sm.par[a]) ++d;
        lo_key = s.past + d - p.window;
      }
      float m_run = kNegBig, l_run = 0.f;
      // Exponents are s mul + base, the product exact (fma). base less kLift is -m_run but for roundings, which `far` takes
      // out where scores are so large (2^23) that they matter.
      [[maybe_unused]] float base = kLift - kNegBig, far = 0.f;
      int mine = 0;   // units of this group in the piece
      for (int j = NQ == 2 ? 0 : q; j < n && ok; j += NQ == 2 ? 1 : 2, ++job, ++mine) {
        const Unit x = unit_of(p, s, w.off + j);
        // ---- visible columns: all, or four words of them
        unsigned vis[4] = {~0u, ~0u, ~0u, ~0u};
        bool full = x.cached && x.n == kKeys && lo_key <= x.first;
        full = __all_sync(0xffffffffu, full);
        if (!full) {
          if (x.cached) {
            const int lo = max(lo_key - x.first, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int a = min(max(lo - 32 * k, 0), 32), z = min(max(x.n - 32 * k, 0), 32);   // columns [a, z)
              vis[k] = a < z ? (z == 32 ? ~0u : (1u << z) - 1u) & ~((1u << a) - 1u) : 0u;
            }
          } else {
            vis[0] = vis[1] = vis[2] = vis[3] = 0u;
            int d = 0;
            for (int a = live_row ? i : -1; a >= x.first && (p.window < 0 || d <= p.window); a = sm.par[a], ++d) {
              const int c = a - x.first;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (c >> 5 == k) vis[k] |= 1u << (c & 31);
            }
          }
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.s_full[q], (uint32_t)job & 1u, p.wait_budget) && !aborted(sm))) {
          ok = false;
          break;
        }
        tc_fence_after();
        // ---- row maximum (a softcap is monotone; it takes the largest |score| too). Hidden columns become -inf, or
        // +inf under a softcap's fit, whose last coefficient turns it into -inf.
        uint32_t v[64];
        float mt = -INFINITY, ua = 0.f;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          tmem_ld32(s_addr + hf * 64, v);
          tmem_ld32(s_addr + hf * 64 + 32, v + 32);
          tmem_ld_wait();
          if (CAP && !full) {
#pragma unroll
            for (int e = 0; e < 64; ++e) v[e] = (vis[2 * hf + (e >> 5)] >> (e & 31)) & 1u ? v[e] : 0u;
          }
          if constexpr (CAP) {
            float a = 0.f, c = 0.f;
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
              a = fmax3(a, fabsf(__uint_as_float(v[e])), fabsf(__uint_as_float(v[e + 1])));
              c = fmax3(c, fabsf(__uint_as_float(v[e + 2])), fabsf(__uint_as_float(v[e + 3])));
            }
            ua = fmaxf(ua, fmaxf(a, c));
          }
          if (!full) {
#pragma unroll
            for (int e = 0; e < 64; ++e) v[e] = (vis[2 * hf + (e >> 5)] >> (e & 31)) & 1u ? v[e] : 0xff800000u;
          }
          float a = -INFINITY, c = -INFINITY;
#pragma unroll
          for (int e = 0; e < 64; e += 4) {
            a = fmax3(a, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
            c = fmax3(c, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
          }
          mt = fmax3(mt, a, c);
          if (!full) {
            if constexpr (CAP) {
#pragma unroll
              for (int e = 0; e < 64; ++e) v[e] = (vis[2 * hf + (e >> 5)] >> (e & 31)) & 1u ? v[e] : 0x7f800000u;
            }
            tmem_st32(s_addr + hf * 64, v);
            tmem_st32(s_addr + hf * 64 + 32, v + 32);
          }
        }
        if (!full) tmem_st_wait();
        // The largest exponent's growth over the reference, by the steps of the exponents: none can pass it.
        [[maybe_unused]] const float top = mt, over = fmaf(mt, mul, base) - far - kLift;
        mt *= mul;
        if constexpr (CAP) {
          ua *= mul;
          if (mt > kNegBig) mt = cap_far(mt, c2);   // a reference: any rounding serves (softcap_fits)
        }
        // ---- rescale O when a maximum outgrew its reference (P V of the unit before is over: S came behind it)
        const bool grow = CAP ? mt > m_run + kLazy : over > kLazy;
        if (__any_sync(0xffffffffu, grow)) {
          const float m_new = grow ? mt : m_run;
          if (mine > 0) {
            const float f = grow ? ex2(m_run - m_new) : 1.0f;
#pragma unroll 1
            for (int c = 0; c < 4 * HB; ++c) {
              uint32_t raw[16];
              tmem_ld16(o_addr + q * 128 + c * 16, raw);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) raw[e] = __float_as_uint(__uint_as_float(raw[e]) * f);
              tmem_st16(o_addr + q * 128 + c * 16, raw);
            }
            l_run *= f;
          }
          m_run = m_new;
          if (!CAP && grow) {
            base = kLift - m_run;
            far = fmaf(top, mul, base) - kLift;
            if (fabsf(far) < 2.f) far = 0.f;
          }
        }
        // ---- P, 64 columns at a time. MODE 0, 1: no softcap (1: with far); 3, 7: its fit of that degree; 9: any size.
        auto exponents = [&](auto mode) {
          constexpr int MODE = decltype(mode)::value;
          const float c0 = CAP ? kLift - m_run : base;
          const float2 kk = make_float2(mul, mul), cc = make_float2(c0, c0);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            tmem_ld32(s_addr + hf * 64, v);
            tmem_ld32(s_addr + hf * 64 + 32, v + 32);
            tmem_ld_wait();
            float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              const float2 x2 = make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              float2 arg;
              if constexpr (MODE <= 1) {
                arg = ffma2(x2, kk, cc);
                if constexpr (MODE == 1) arg = fadd2(arg, make_float2(-far, -far));
              } else {
                const float2 u = ffma2(x2, kk, make_float2(0.f, 0.f));
                if constexpr (MODE == 9) {
                  const float2 y = cap_any(u, c2);
                  arg = make_float2(y.x + cc.x, y.y + cc.x);
                  if (!full) {
                    const unsigned word = vis[2 * hf + (e >> 5)] >> (e & 31);
                    arg.x = word & 1u ? arg.x : -INFINITY;
                    arg.y = word & 2u ? arg.y : -INFINITY;
                  }
                } else {
                  const float2 z = ffma2(u, u, make_float2(0.f, 0.f));
                  arg = ffma2(u, cap_fit<MODE>(z, c2), cc);
                }
              }
              const __half2 hp = __floats2half2_rn(ex2(arg.x), ex2(arg.y));
              v[e >> 1] = *reinterpret_cast<const uint32_t*>(&hp);
              ls[(e >> 1) & 1] = add_half2(ls[(e >> 1) & 1], v[e >> 1]);
            }
            const float2 lt = fadd2(ls[0], ls[1]);
            l_run += lt.x + lt.y;
            tmem_st32(s_addr + hf * 64, v);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[q][hf]);   // P V of these keys may start
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
        } else if (__builtin_expect(__all_sync(0xffffffffu, far == 0.f), 1)) {
          exponents(std::integral_constant<int, 0>());
        } else {
          exponents(std::integral_constant<int, 1>());
        }
      }
      // ---- the piece ends: O / l to the output, or m, l and O to the workspace
      if (ok && mine > 0)
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_done[q], (uint32_t)(job - 1) & 1u, p.wait_budget) && !aborted(sm));
      float m = m_run, l = l_run, f[2] = {1.f, 1.f};
      if constexpr (NQ == 1) {   // join the groups: each takes half of the columns of both O
        sm.ml[q][rl] = make_float2(m_run, l_run);
        ok = soft_all(ok);
        const float2 o = sm.ml[q ^ 1][rl];
        m = fmaxf(m_run, o.x);
        f[q] = ex2(m_run - m);
        f[q ^ 1] = ex2(o.x - m);
        l = fmaf(l_run, f[q], o.y * f[q ^ 1]);
      }
      tc_fence_after();
      if (ok) {
        const bool whole = n == s.work;
        float so = 1.f;
        if (whole) {
          float extra = 0.f, fm = 1.f;
          if (p.sink || p.smooth) {
            const float sg = (p.sink ? __half2float(reinterpret_cast<const __half*>(p.sink)[hd]) : 0.f) * kLog2e;
            const float mf = fmaxf(m, sg);
            fm = ex2(m - mf);
            extra = ex2(sg - mf + kLift);
          }
          const float den = fmaf(l, fm, extra);
          so = den == 0.f ? 0.f : fm / den;
        }
        const int rl_tile = (NQ == 2 ? q * 128 : 0) + rl;
        const long long row = tree_slot(blockIdx.x, w.off == 0) * kRows + rl_tile;
        if (!whole && live_row && (NQ == 2 || q == 0)) *reinterpret_cast<float2*>(p.part_ml + row * 2) = make_float2(m, l);
        const volatile unsigned* odd = sm.odd[piece % kOddSets];   // (written before the P V that o_done stands for)
        const bool any_odd = odd[kOddNodes + kOddEdge] != 0u;
        constexpr int kPer = NQ == 2 ? 2 * HB : HB;   // 32-column pieces of a thread
#pragma unroll 1
        for (int c = 0; c < kPer; ++c) {
          const int d0 = 32 * ((NQ == 2 ? 0 : q * kPer) + c);
          uint32_t raw[32];
          float o[32];
          if constexpr (NQ == 2) {
            tmem_ld32(o_addr + q * 128 + d0, raw);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(raw[e]);
          } else {
            tmem_ld32(o_addr + d0, raw);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(raw[e]) * f[0];
            if (n > 1) {   // (one unit: the second group has no O)
              tmem_ld32(o_addr + 128 + d0, raw);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(raw[e]), f[1], o[e]);
            }
          }
          if (!live_row || d0 >= p.H) continue;
          if (any_odd) {   // values that are not finite, for the rows that see them
            for (int x = 0; x < 32 * (kOddNodes + kOddEdge); ++x) {
              if (!(odd[x >> 5] >> (x & 31) & 1u)) continue;
              const bool node = x < kTreeNodes;
              const int key = node ? x : s.k0 + x - kTreeNodes;
              if (key >= (node ? s.fresh : s.past)) continue;
              if (node) {
                int a = i, d = 0;
                for (; a > key; a = sm.par[a]) ++d;
                if (a != key || (p.window >= 0 && d > p.window)) continue;
              } else if (key < lo_key) {
                continue;
              }
              const __half* src = node ? static_cast<const __half*>(p.v) + (((long long)w.b * p.S + key) * p.Nkv + w.g) * p.H
                                       : static_cast<const __half*>(p.vc) + (((long long)w.b * p.Nkv + w.g) * p.C + key) * p.H;
              for (int e = 0; e < 32; ++e) {
                const float y = d0 + e < p.H ? __half2float(src[d0 + e]) : 0.f;
                if (!(fabsf(y) < INFINITY))
#pragma unroll
                  for (int z = 0; z < 32; ++z)
                    if (z == e) o[z] += y;
              }
            }
          }
          if (whole) {
            __half* dst = static_cast<__half*>(p.out) + (((long long)w.b * p.S + i) * p.N + hd) * p.H + d0;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t u[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __half2 h2 = __floats2half2_rn(o[e + 2 * k] * so, o[e + 2 * k + 1] * so);
                u[k] = *reinterpret_cast<const uint32_t*>(&h2);
              }
              if (d0 + e < p.H) *reinterpret_cast<uint4*>(dst + e) = make_uint4(u[0], u[1], u[2], u[3]);
            }
          } else {
            // a slot's rows side by side: a warp writes 512 bytes in a row
            float* dst = p.part_o + (row - rl_tile) * p.H + 4 * rl_tile;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              if (d0 + e < p.H) *reinterpret_cast<float4*>(dst + (d0 + e) * kRows) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
      }
      tc_fence_before();
      ok = soft_all(ok);   // every O is read: the next piece may overwrite it; all go on, or none
      if (!ok) {
        if (lane == 0) set_abort(p, sm);
        break;
      }
      // (the cleaners come back to this set when these threads are pieces further)
      if (st < kOddNodes + kOddEdge + 1) sm.odd[piece % kOddSets][st] = 0u;
      w.next(p, n);
    }
    if (!appended) append();   // (a share of range ends only, or none)
  }
  dep_wait();   // what follows on the stream waits for this kernel alone
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

constexpr int kMaxDevices = 64;

template <bool CAP, int HB, int NQ>
cudaError_t launch_one(const TreeParams& p, cudaStream_t st) {
  static bool done[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  constexpr int smem = (int)sizeof(TcSmem<HB, NQ>) + 1024;
  static_assert(smem <= 232448, "shared memory per CTA");
  auto kern = tree_tc_kernel<CAP, HB, NQ>;
  if (!done[dev]) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    done[dev] = true;
  }
  CUtensorMap mk, mv, nk, nv;
  const uint64_t rows = (uint64_t)p.B * p.Nkv * p.C, row_bytes = (uint64_t)p.H * 2;
  if ((e = encode_fp16_2d_sw128(&mk, p.kc, rows, (uint64_t)p.H, row_bytes, 64, kKeys)) != cudaSuccess) return e;
  if ((e = encode_fp16_2d_sw128(&mv, p.vc, rows, (uint64_t)p.H, row_bytes, 64, kKeys)) != cudaSuccess) return e;
  // Nodes of one KV head: a box of 64 dims x 1 head x 128 nodes.
  if ((e = encode_fp16_query_sw128(&nk, p.k, p.B, p.S, p.Nkv, 1, kKeys, (uint64_t)p.H)) != cudaSuccess) return e;
  if ((e = encode_fp16_query_sw128(&nv, p.v, p.B, p.S, p.Nkv, 1, kKeys, (uint64_t)p.H)) != cudaSuccess) return e;
  return launch_dependent(false, kern, dim3((unsigned)p.workers), kThreads, (size_t)smem, st, p, mk, mv, nk, nv);
}

template <bool CAP, int HB>
cudaError_t launch_nq(const TreeParams& p, cudaStream_t st) {
  return p.rt_log2 == 7 ? launch_one<CAP, HB, 1>(p, st) : launch_one<CAP, HB, 2>(p, st);
}

}  // namespace

cudaError_t launch_tree_tc(const TreeParams& p, cudaStream_t st) {
  const bool cap = p.softcap > 0.f;
  if (p.H <= 64) return cap ? launch_nq<true, 1>(p, st) : launch_nq<false, 1>(p, st);
  return cap ? launch_nq<true, 2>(p, st) : launch_nq<false, 2>(p, st);
}

}  // namespace gqa
