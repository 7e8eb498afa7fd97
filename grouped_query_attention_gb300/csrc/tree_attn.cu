// Attention of drafted nodes over a float cache on warp MMAs: every type, head
// size, group size and scale (fp32, and what the tensor-core pipeline does not
// take), and the merge of both.
//
// Rows of a KV head (b, g): query rows (node, grouped head), in row tiles of 16,
// 32 or 64. The keys of a row tile are the cached rows and the nodes themselves,
// in units of 64 (fp16) or 32 (fp32); all units are laid end to end and a CTA
// takes an equal share, so a single long sequence fills the GPU as well as many
// short ones. A CTA streams its units through shared memory (cp.async, two
// stages). Its warps hold 16 rows each; those left over share the keys of a unit
// and join their results at the end. The nodes' keys and values come from the
// call's own key and value tensors, so nothing waits for the append, which the
// same launch does.
//
// fp16: m16n8k16, fp32 sums; probabilities enter as 2^15 p (the row maximum is
// exact, so 2^15 p <= 2^15, and p keeps 11 bits down to 2^-29), and the output is
// divided by the sum of the rounded ones, which takes the common part of their
// roundings out. fp32: m16n8k8 on tf32 parts, x = hi + lo with 11 bits each,
// hi hi + hi lo + lo hi (2^-20 of a product is lost at most). The MMA accumulators
// round towards zero, so O of every unit moves into fp32 sums that round to
// nearest.
//
// What bounds it. fp32: three MMAs for one, and the splitting of both operands: 8
// sequences of 4096..16384 rows, 8 nodes, 32 heads over 8: 236 us for 674 MB (2.9
// TB/s); the MMA pipe is busy 38 % of the time (the MMAs alone take 110 us), and two
// warps a scheduler (255 registers) cannot hide the chains around them. Measured
// there (events around single cold launches): eight warps of 16 rows 275 us, 32 rows a warp 265, units of 16 keys and
// three CTAs an SM 255, queries split ahead in shared memory 263, rows brought by
// bulk copies 359. fp16 heads of 256, 32 rows: 64 us for 101 MB, 256 rows 117.
#include <cuda_fp16.h>

#include "block_tc.cuh"
#include "common.cuh"
#include "tree_internal.h"

namespace gqa {
namespace {

constexpr float kLiftHalf = 15.f;   // log2 of what fp16 probabilities are multiplied by

template <typename T, int HP, int RW>
struct Cfg {
  static constexpr bool kHalf = sizeof(T) == 2;
  // Four warps; eight where shared memory leaves an SM room for one CTA anyway (heads of 256: fp32 199 -> 156 us).
  static constexpr int kWarps = HP > 128 && RW > 1 ? 8 : 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int KW = kWarps / RW;                 // warps that share a unit's keys
  static constexpr int RT = 16 * RW;
  static constexpr int KT = kHalf ? 64 : 32;             // keys of a unit
  static constexpr int WK = KT / KW;                     // ... of a warp
  // Row strides: fp16 ldmatrix reads 8 rows of 16 bytes (16 bytes apart mod 128). fp32 keys are read as four
  // coordinates by 8 rows x 4 lanes (64 bytes apart mod 128), values as four coordinates of rows 2t, 2t + 1
  // (16 bytes apart).
  static constexpr int QS = HP + (kHalf ? 8 : 16);
  static constexpr int KS = HP + (kHalf ? 8 : 16);
  static constexpr int VS = HP + (kHalf ? 8 : 4);
  static constexpr int kStage = KT * (KS + VS) * (int)sizeof(T);
  static constexpr int kStages = 2;
  static constexpr int kJoin = KW > 1 ? (KW - 1) * RW * (16 * HP + 64) * 4 : 0;   // other key warps' O, m, l
  static constexpr int kRing = kStages * kStage > kJoin ? kStages * kStage : kJoin;
  static constexpr int kSmem = RT * QS * (int)sizeof(T) + kRing;
};

__device__ __forceinline__ uint32_t saddr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// 16 bytes, or zeros when !on (the source is not read).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  const int n = on ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float* c, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// x = hi + lo + what is lost: hi the nearest of 11 bits, lo 11 bits of the rest. (lo is cut off: a NaN stays one
// there, while the sum in hi wraps it to zero.)
__device__ __forceinline__ void split_tf32(float x, uint32_t* hi, uint32_t* lo) {
  *hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  *lo = __float_as_uint(x - __uint_as_float(*hi)) & 0xffffe000u;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }

// Softcap of a score in the log2 domain.
__device__ __forceinline__ float capped(float s, float softcap) { return softcap * kLog2e * tanhf(s / softcap); }

template <typename T, int HP, int RW>
__global__ void __launch_bounds__(Cfg<T, HP, RW>::kThreads)
tree_attn_kernel(const TreeParams p) {
  using K = Cfg<T, HP, RW>;
  constexpr bool kHalf = K::kHalf;
  constexpr int kThreads = K::kThreads;
  constexpr int KT = K::KT, WK = K::WK, NT = WK / 8, ND = HP / 8;
  constexpr int kE = 16 / (int)sizeof(T);              // elements of a 16-byte chunk
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t anc[K::RT][kTreeNodes / 32];     // ancestors of the tile's positions, as bits
  __shared__ short par[kTreeNodes];
  __shared__ short depth[K::RT];
  __shared__ unsigned odd[KT / 32];                    // keys of a unit whose values are not all finite
  T* qs = reinterpret_cast<T*>(smem);
  T* ring = qs + K::RT * K::QS;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, t = lane & 3;
  const int rw = warp % RW, kw = warp / RW;
  constexpr int kFetchRows = kThreads / (HP / kE);     // of a unit that the CTA copies at a time: this thread's, its chunk
  const int fr = tid / (HP / kE), fc = tid % (HP / kE);

  // ---- status, padding rows, the append: every CTA a part
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    int past, fresh;
    bool bad_tree = false;
    const bool ok = tree_lengths(p, b, &past, &fresh);
    if (ok)
      for (int i = tid; i < fresh; i += kThreads) tree_parent(p.parents[(long long)b * p.parents_ld + i], i, &bad_tree);
    if (__syncthreads_or(bad_tree) && tid == 0 && p.status) atomicOr(p.status, GQA_DEVICE_BAD_TREE_BIT);
    if (!ok && tid == 0 && p.status) atomicOr(p.status, GQA_DEVICE_BAD_SEQLEN_BIT);
  }
  const long long units = tree_units(p);
  dep_launch();
  auto append = [&]() {
    const int kv = p.Nkv * p.H / kE, qh = p.N * p.H / kE, rc = p.H / kE;   // chunks of a node
    for (long long x = blockIdx.x; x < (long long)p.B * p.S; x += gridDim.x) {
      const int b = (int)(x / p.S), i = (int)(x % p.S);
      int past, fresh;
      if (!tree_lengths(p, b, &past, &fresh)) continue;
      if (i >= fresh) {
        uint4* o = reinterpret_cast<uint4*>(p.out) + x * qh;
        for (int c = tid; c < qh; c += kThreads) o[c] = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      for (int c = tid; c < 2 * kv; c += kThreads) {
        const bool is_v = c >= kv;
        const int d = is_v ? c - kv : c, g = d / rc;
        const uint4 w = reinterpret_cast<const uint4*>(is_v ? p.v : p.k)[x * kv + d];
        reinterpret_cast<uint4*>(is_v ? p.vc : p.kc)[(((long long)b * p.Nkv + g) * p.C + past + i) * rc + d % rc] = w;
      }
    }
  };
  const long long live = tree_live(p, units);
  const long long u0 = units * blockIdx.x / live, u1 = units * (blockIdx.x + 1) / live;
  if (blockIdx.x >= live || u0 >= u1) {
    append();
    dep_wait();
    return;
  }
  TreeWalk w;
  w.start(p, u0, u1 - u0);
  bool appended = false;

  while (w.left > 0) {
    const int n_units = w.piece();
    const TreeSeq s = w.s;
    const int r0 = w.rt * K::RT, nrows = s.fresh * p.G;
    const int i0 = r0 / p.G, i1 = (min(r0 + K::RT, nrows) - 1) / p.G;   // positions of the tile
    const long long bg = (long long)w.b * p.Nkv + w.g;
    __syncthreads();   // shared memory of the piece before is free
    // ---- queries; the first units on their way
    for (int x = tid; x < K::RT * (HP / kE); x += kThreads) {
      const int r = x / (HP / kE), c = x % (HP / kE), row = r0 + r;
      const bool on = row < nrows && c * kE < p.H;
      const T* src = static_cast<const T*>(p.q) +
                     (on ? (((long long)w.b * p.S + row / p.G) * p.N + w.g * p.G + row % p.G) * p.H + c * kE : 0);
      cp16(saddr(qs + r * K::QS + c * kE), src, on);
    }
    // Copies of unit u (of the range) into stage st: rows [0, n) of a cached or drafted run of keys, zeros behind.
    auto fetch = [&](int u, int st) {
      const bool cached = u < s.np;
      const int first = cached ? s.k0 + u * KT : (u - s.np) * KT;
      const int n = min(KT, cached ? s.past - first : s.fresh - first);
      const long long ld = cached ? p.H : (long long)p.Nkv * p.H;
      const long long at = cached ? (bg * p.C + first) * p.H : (((long long)w.b * p.S + first) * p.Nkv + w.g) * p.H;
      const T* ksrc = static_cast<const T*>(cached ? p.kc : p.k) + at + fr * ld + fc * kE;
      const T* vsrc = static_cast<const T*>(cached ? p.vc : p.v) + at + fr * ld + fc * kE;
      const uint32_t kd = saddr(ring) + st * K::kStage + (fr * K::KS + fc * kE) * (uint32_t)sizeof(T);
      const uint32_t vd = saddr(ring) + st * K::kStage + (KT * K::KS + fr * K::VS + fc * kE) * (uint32_t)sizeof(T);
#pragma unroll
      for (int i = 0; i < KT; i += kFetchRows) {
        const bool on = fr + i < n && fc * kE < p.H;
        cp16(kd + i * K::KS * (uint32_t)sizeof(T), ksrc, on);
        cp16(vd + i * K::VS * (uint32_t)sizeof(T), vsrc, on);
        ksrc += kFetchRows * ld;
        vsrc += kFetchRows * ld;
      }
    };
    fetch(w.off, 0);
    cp_commit();
    if (tid < KT / 32) odd[tid] = 0u;
    // ---- ancestors (a window ends them and needs the depths)
    const bool nodes = w.off + n_units > s.np;
    if (nodes || p.window >= 0) {
      bool bad = false;
      for (int i = tid; i <= i1; i += kThreads)
        par[i] = (short)tree_parent(p.parents[(long long)w.b * p.parents_ld + i], i, &bad);
      __syncthreads();
      const int words = (i1 >> 5) + 1;
      for (int x = tid; x <= i1 - i0; x += kThreads) {
        for (int c = 0; c < kTreeNodes / 32; ++c)
          if (c < words) anc[x][c] = 0u;
        int d = 0;
        for (int a = i0 + x; a >= 0; a = par[a], ++d)
          if (p.window < 0 || d <= p.window) anc[x][a >> 5] |= 1u << (a & 31);
        depth[x] = (short)(d - 1);
      }
      __syncthreads();
    }
    if (!appended) {
      append();
      appended = true;
    }

    float o[ND][4], m[2] = {kNegBig, kNegBig}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    int lo_key[2] = {0, 0};        // first visible cached row of rows gq, gq + 8 of the warp
    const int pos0 = min(r0 + 16 * rw + gq, nrows - 1) / p.G - i0, pos1 = min(r0 + 16 * rw + gq + 8, nrows - 1) / p.G - i0;
    if (p.window >= 0) {
      lo_key[0] = s.past + depth[pos0] - p.window;
      lo_key[1] = s.past + depth[pos1] - p.window;
    }
    const float mul = p.softcap > 0.f ? p.scale : p.scale * kLog2e;

    for (int x = 0; x < n_units; ++x) {
      const int u = w.off + x, st = x & 1;
      if (x + 1 < n_units) fetch(u + 1, st ^ 1);
      cp_commit();
      cp_wait<1>();
      __syncthreads();
      T* kt = ring + st * (K::kStage / (int)sizeof(T));
      T* vt = kt + KT * K::KS;
      const bool cached = u < s.np;
      const int first = cached ? s.k0 + u * KT : (u - s.np) * KT;
      // A unit that some rows see in part: what is not finite among its values would reach the others as 0 x it. It
      // leaves the tile and comes back row by row, below.
      const bool partial = !cached || (p.window >= 0 && first < s.past - p.window + i1);
      if (partial) {
        for (int y = tid; y < KT * (HP / kE); y += kThreads) {
          const int r = y / (HP / kE);
          T* e = vt + r * K::VS + y % (HP / kE) * kE;
          bool any = false;
#pragma unroll
          for (int z = 0; z < kE; ++z) {
            const float f = (float)e[z];
            if (!(fabsf(f) < INFINITY)) {
              e[z] = T(0.f);
              any = true;
            }
          }
          if (any) atomicOr(&odd[r >> 5], 1u << (r & 31));
        }
        __syncthreads();
      }
      // ---- scores: keys kw WK + 8 n + 2 t, + 1 (n < NT), rows 16 rw + gq (0, 1) and + 8 (2, 3)
      float sc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
      if constexpr (kHalf) {
        const uint32_t qa = saddr(qs + (16 * rw + (lane & 15)) * K::QS + (lane >> 4) * 8);
        const uint32_t ka = saddr(kt + (kw * WK + (lane & 7) + ((lane >> 4) << 3)) * K::KS + ((lane >> 3) & 1) * 8);
#pragma unroll
        for (int ks = 0; ks < HP / 16; ++ks) {
          uint32_t a[4];
          ldsm4(a, qa + ks * 32);
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            uint32_t b[4];
            ldsm4(b, ka + n * 8 * K::KS * 2 + ks * 32);
            mma_f16(sc[n], a, b[0], b[1]);
            mma_f16(sc[n + 1], a, b[2], b[3]);
          }
        }
      } else {
        const T* q0 = qs + (16 * rw + gq) * K::QS + 4 * t;
        const T* k0 = kt + (kw * WK + gq) * K::KS + 4 * t;
        // The products with a lo part add up on their own, hi ones over 16 coordinates at a time: short chains of MMAs
        // (one of 6 for 16 coordinates: 279 us, this 240), whose rounding towards zero stays small (a single one of 48
        // was 3.1e-6 off).
        float cl[2][NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) cl[0][n][e] = cl[1][n][e] = 0.f;
#pragma unroll 4
        for (int j = 0; j < (HP > 64 ? p.H / 16 : HP / 16); ++j) {   // coordinates 16 j + 4 t ..: two MMA steps
          const float4 x0 = *reinterpret_cast<const float4*>(q0 + 16 * j);
          const float4 x1 = *reinterpret_cast<const float4*>(q0 + 8 * K::QS + 16 * j);
          uint32_t ah[2][4], al[2][4];
          split_tf32(x0.x, &ah[0][0], &al[0][0]);
          split_tf32(x1.x, &ah[0][1], &al[0][1]);
          split_tf32(x0.y, &ah[0][2], &al[0][2]);
          split_tf32(x1.y, &ah[0][3], &al[0][3]);
          split_tf32(x0.z, &ah[1][0], &al[1][0]);
          split_tf32(x1.z, &ah[1][1], &al[1][1]);
          split_tf32(x0.w, &ah[1][2], &al[1][2]);
          split_tf32(x1.w, &ah[1][3], &al[1][3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float4 y = *reinterpret_cast<const float4*>(k0 + n * 8 * K::KS + 16 * j);
            uint32_t bh[2][2], bl[2][2];
            split_tf32(y.x, &bh[0][0], &bl[0][0]);
            split_tf32(y.y, &bh[0][1], &bl[0][1]);
            split_tf32(y.z, &bh[1][0], &bl[1][0]);
            split_tf32(y.w, &bh[1][1], &bl[1][1]);
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              mma_tf32(c, ah[h], bh[h]);
              mma_tf32(cl[0][n], al[h], bh[h]);
              mma_tf32(cl[1][n], ah[h], bl[h]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][e] += c[e];
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] += cl[0][n][e] + cl[1][n][e];
      }
      // ---- log2 domain, masks
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[n][e] *= mul;
          if (p.softcap > 0.f) sc[n][e] = capped(sc[n][e], p.softcap);
        }
      if (cached) {
        if (first + KT > s.past || p.window >= 0) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = first + kw * WK + 8 * n + 2 * t + (e & 1);
              if (j >= s.past || j < lo_key[e >> 1]) sc[n][e] = -INFINITY;
            }
        }
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int a = first + kw * WK + 8 * n + 2 * t;   // even: both keys in one word
          const uint32_t w0 = a <= i1 ? anc[pos0][a >> 5] >> (a & 31) : 0u, w1 = a <= i1 ? anc[pos1][a >> 5] >> (a & 31) : 0u;
          if (!(w0 & 1u)) sc[n][0] = -INFINITY;
          if (!(w0 & 2u)) sc[n][1] = -INFINITY;
          if (!(w1 & 1u)) sc[n][2] = -INFINITY;
          if (!(w1 & 2u)) sc[n][3] = -INFINITY;
        }
      }
      // ---- running maximum, probabilities
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = m[h];
#pragma unroll
        for (int n = 0; n < NT; ++n) mx = fmax3(mx, sc[n][2 * h], sc[n][2 * h + 1]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        f[h] = ex2(m[h] - mx);
        m[h] = mx;
        l[h] *= f[h];
      }
      // (Rounded up: of a maximum from 2^24 on, m - 15 could be m - 16, and 2^16 is no fp16 number.)
      const float ref[2] = {kHalf ? __fsub_ru(m[0], kLiftHalf) : m[0], kHalf ? __fsub_ru(m[1], kLiftHalf) : m[1]};
      if constexpr (kHalf) {
        uint32_t pa[NT][2];   // rows gq, gq + 8
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            pa[n][h] = pack2(ex2(sc[n][2 * h] - ref[h]), ex2(sc[n][2 * h + 1] - ref[h]));
            const float2 r = unpack2(pa[n][h]);
            l[h] += r.x + r.y;
          }
        const uint32_t va = saddr(vt + (kw * WK + (lane & 15)) * K::VS + (lane >> 4) * 8);
#pragma unroll
        for (int d = 0; d < ND; d += 2) {
          if (HP > 64 && 8 * d >= p.H) break;
          float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            uint32_t b[4];
            ldsm4t(b, va + n * 8 * K::VS * 2 + d * 16);
            const uint32_t a[4] = {pa[n][0], pa[n][1], pa[n + 1][0], pa[n + 1][1]};
            mma_f16(c[0], a, b[0], b[1]);
            mma_f16(c[1], a, b[2], b[3]);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d + y][e] = fmaf(o[d + y][e], f[e >> 1], c[y][e]);
        }
      } else {
        uint32_t ph[NT][4], pl[NT][4];   // A operand: key 2 t is k = t, key 2 t + 1 k = t + 4
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x1 = ex2(sc[n][e] - ref[e >> 1]);
            l[e >> 1] += x1;
            const int at = (e >> 1) + 2 * (e & 1);
            split_tf32(x1, &ph[n][at], &pl[n][at]);
          }
        const T* v0 = vt + (kw * WK + 2 * t) * K::VS + 4 * gq;
#pragma unroll
        for (int d = 0; d < ND; d += 4) {   // coordinates 8 d + 4 gq + e of MMA d + e
          if (HP > 64 && 8 * d >= p.H) break;
          float c[4][4];
#pragma unroll
          for (int y = 0; y < 4; ++y) c[y][0] = c[y][1] = c[y][2] = c[y][3] = 0.f;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float4 y0 = *reinterpret_cast<const float4*>(v0 + n * 8 * K::VS + 8 * d);
            const float4 y1 = *reinterpret_cast<const float4*>(v0 + (n * 8 + 1) * K::VS + 8 * d);
            const float a0[4] = {y0.x, y0.y, y0.z, y0.w}, a1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t bh[2], bl[2];
              split_tf32(a0[y], &bh[0], &bl[0]);
              split_tf32(a1[y], &bh[1], &bl[1]);
              mma_tf32(c[y], pl[n], bh);
              mma_tf32(c[y], ph[n], bl);
              mma_tf32(c[y], ph[n], bh);
            }
          }
#pragma unroll
          for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d + y][e] = fmaf(o[d + y][e], f[e >> 1], c[y][e]);
        }
      }
      if (partial) {
#pragma unroll 1
        for (int kk = kw * WK; kk < kw * WK + WK; ++kk) {
          if (!(odd[kk >> 5] >> (kk & 31) & 1u)) continue;
          const int own = (lane & ~3) | ((kk & 7) >> 1);     // lane of the key's scores
          const T* src = cached ? static_cast<const T*>(p.vc) + (bg * p.C + first + kk) * p.H
                                : static_cast<const T*>(p.v) + (((long long)w.b * p.S + first + kk) * p.Nkv + w.g) * p.H;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x1 = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
              if (n == (kk - kw * WK) >> 3) x1 = kk & 1 ? sc[n][2 * h + 1] : sc[n][2 * h];
            x1 = __shfl_sync(0xffffffffu, x1, own);
            if (x1 == -INFINITY) continue;   // a row that does not see it (the quad shares the row)
            // (a weight too small for a float counts: what it weighs is not finite)
            const float pr = fmaxf(ex2(x1 - ref[h]), 0x1p-126f);
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int c = kHalf ? 8 * d + 2 * t + e : 32 * (d >> 2) + 8 * t + 4 * e + (d & 3);
                const float f = c < p.H ? (float)src[c] : 0.f;
                if (!(fabsf(f) < INFINITY)) o[d][2 * h + e] = fmaf(pr, f, o[d][2 * h + e]);
              }
          }
        }
      }
      __syncthreads();   // every warp is through with the stage
      if (partial && tid < KT / 32) odd[tid] = 0u;   // (written again behind the next copy's barrier)
    }
    cp_wait<0>();
    // ---- the piece ends: rows' sums over the quad, then over the key warps
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    if constexpr (K::KW > 1) {
      float* jo = reinterpret_cast<float*>(ring);                                  // [KW - 1][RW][ND * 4][32]
      float* jm = jo + (K::KW - 1) * RW * 16 * HP;                                 // [KW - 1][RW][64]: m, l of 16 rows (twice)
      if (kw > 0) {
        const int at = (kw - 1) * RW + rw;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) jo[(at * ND * 4 + 4 * d + e) * 32 + lane] = o[d][e];
        if (t == 0) {
          jm[at * 64 + gq] = m[0];
          jm[at * 64 + 8 + gq] = m[1];
          jm[at * 64 + 16 + gq] = l[0];
          jm[at * 64 + 24 + gq] = l[1];
        }
      }
      __syncthreads();
      if (kw == 0) {
        float f[K::KW][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = m[h];
#pragma unroll
          for (int x = 0; x < K::KW - 1; ++x) mx = fmaxf(mx, jm[(x * RW + rw) * 64 + 8 * h + gq]);
          f[0][h] = ex2(m[h] - mx);
          l[h] *= f[0][h];
#pragma unroll
          for (int x = 0; x < K::KW - 1; ++x) {
            f[x + 1][h] = ex2(jm[(x * RW + rw) * 64 + 8 * h + gq] - mx);
            l[h] = fmaf(jm[(x * RW + rw) * 64 + 16 + 8 * h + gq], f[x + 1][h], l[h]);
          }
          m[h] = mx;
        }
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[d][e] *= f[0][e >> 1];
#pragma unroll
            for (int x = 0; x < K::KW - 1; ++x)
              o[d][e] = fmaf(jo[((x * RW + rw) * ND * 4 + 4 * d + e) * 32 + lane], f[x + 1][e >> 1], o[d][e]);
          }
      }
    }
    // ---- write: all of a range to the output, a part of it to the workspace
    const bool whole = n_units == s.work;
    if (kw == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int rl = 16 * rw + gq + 8 * h, r = r0 + rl;
        if (r >= nrows) continue;
        float so = 1.f;
        const int i = r / p.G, hd = w.g * p.G + r % p.G;
        const long long slot = tree_slot(blockIdx.x, w.off == 0);
        if (whole) {
          float extra = 0.f, fm = 1.f;
          if (p.sink || p.smooth) {
            const float sg = (p.sink ? load_t(p.sink, hd, p.t_type) : 0.f) * kLog2e;
            const float mf = fmaxf(m[h], sg);
            fm = ex2(m[h] - mf);
            extra = ex2(sg - mf + (kHalf ? kLiftHalf : 0.f));
          }
          const float den = fmaf(l[h], fm, extra);
          so = den == 0.f ? 0.f : fm / den;
        } else if (t == 0) {
          *reinterpret_cast<float2*>(p.part_ml + (slot * K::RT + rl) * 2) = make_float2(m[h], l[h]);
        }
        T* dst = static_cast<T*>(p.out) + (((long long)w.b * p.S + i) * p.N + hd) * p.H;
        float* part = p.part_o + (slot * K::RT + rl) * p.H;
        if constexpr (kHalf) {
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            const int c = 8 * d + 2 * t;
            if (c >= p.H) continue;
            if (whole)
              *reinterpret_cast<uint32_t*>(dst + c) = pack2(o[d][2 * h] * so, o[d][2 * h + 1] * so);
            else
              *reinterpret_cast<float2*>(part + c) = make_float2(o[d][2 * h], o[d][2 * h + 1]);
          }
        } else {
#pragma unroll
          for (int d = 0; d < ND; d += 4)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int c = 8 * d + 8 * t + 4 * y;
              if (c >= p.H) continue;
              *reinterpret_cast<float4*>((whole ? reinterpret_cast<float*>(dst) : part) + c) =
                  make_float4(o[d][2 * h + y] * so, o[d + 1][2 * h + y] * so, o[d + 2][2 * h + y] * so, o[d + 3][2 * h + y] * so);
            }
        }
      }
    }
    w.next(p, n_units);
  }
  if (!appended) append();   // (a share of range ends only)
  dep_wait();   // what follows on the stream waits for this kernel alone
}

// ------------------------------------------------------------------ merge

constexpr int kMergeWarps = 8;

// Rows of ranges that several workers share, four at a time: W warps take their
// pieces in turn, a lane four (H / 32) groups of four coordinates of one row. A
// piece's O is in units of its own maximum. A block stays within a (b, g), rows
// [rows blockIdx.x, + rows). HG: 32-coordinate groups of a row.
template <typename T, int W, int HG>
__global__ void __launch_bounds__(32 * kMergeWarps)
tree_merge_kernel(const TreeParams p, int rows) {
  constexpr int kTeams = kMergeWarps / W;
  constexpr int kAhead = HG > 4 ? 2 : 4;        // pieces of a warp under way
  __shared__ float4 join[W > 1 ? kMergeWarps : 1][HG][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, team = warp / W, sub = warp % W;
  const int ri = lane & 3, c8 = lane >> 2;      // row of the four; coordinates 4 (c8 + 8 k) ..
  const int b = blockIdx.y / p.Nkv, g = blockIdx.y % p.Nkv;
  long long units = 0, base = 0;
  TreeSeq s;
  for (int x = lane; x < p.B; x += 32) {
    if (!tree_seq(p, x, &s)) continue;
    const long long n = (long long)p.Nkv * s.nrt * s.units;
    units += n;
    if (x < b) base += n;
  }
  for (int o = 16; o; o >>= 1) {
    units += __shfl_xor_sync(0xffffffffu, units, o);
    base += __shfl_xor_sync(0xffffffffu, base, o);
  }
  const int nrows = tree_seq(p, b, &s) ? s.fresh * p.G : 0;
  const long long live = tree_live(p, units);
  const int tile = 1 << p.rt_log2;
  // Rows of a slot's O side by side (the pipeline's threads hold one each), or its coordinates.
  const int row_ld = p.tc ? 4 : p.H, col_ld = p.tc ? 4 * tile : 4;
  long long w0 = 0, w1 = 0;
  int rt = -1;
  dep_wait();
  for (int r0 = blockIdx.x * rows; r0 < min((int)(blockIdx.x + 1) * rows, nrows); r0 += 4 * kTeams) {
    // (A row behind the last, and a team without rows, does the last one's work once more. Four rows share a tile.)
    const int r = min(r0 + 4 * team + ri, nrows - 1), first = min(r0 + 4 * team, nrows - 1);
    if (first >> p.rt_log2 != rt) {
      rt = first >> p.rt_log2;
      tree_pieces(base + (long long)(g * s.nrt + rt) * s.units, s.work, live, units, &w0, &w1);
    }
    const int n = (int)(w1 - w0) + 1, hd = g * p.G + r % p.G, row = r & (tile - 1);
    float4 a[HG];
#pragma unroll
    for (int k = 0; k < HG; ++k) a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    if (n > 1) {                                // (else one worker wrote the output)
      const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + row;
      const bool has_sink = p.sink || p.smooth;
      const float sg = has_sink ? (p.sink ? load_t(p.sink, hd, p.t_type) : 0.f) * kLog2e : kNegBig;
      const float* src = p.part_o + (long long)row * row_ld + c8 * col_ld;
      float4 o[kAhead][HG];
      float f[kAhead];
      auto load = [&](int x) {   // pieces x, x + W, ..: O and maximum
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
          const int at = min(x + y * W, n - 1);
          const long long slot = tree_slot(w0 + at, at == 0) * tile;
          f[y] = x + y * W < n ? ml[slot].x : INFINITY;
#pragma unroll
          for (int k = 0; k < HG; ++k)
            if (4 * (c8 + 8 * k) < p.H) o[y][k] = *reinterpret_cast<const float4*>(src + slot * p.H + 8 * k * col_ld);
        }
      };
      load(sub);   // on their way while the row's maximum and sum are worked out, by the eight lanes that share it
      const float2 own = c8 < n ? ml[tree_slot(w0 + c8, c8 == 0) * tile] : make_float2(kNegBig, 0.f);
      float m = fmaxf(sg, own.x);
      for (int x = c8 + 8; x < n; x += 8) m = fmaxf(m, ml[tree_slot(w0 + x, false) * tile].x);
#pragma unroll
      for (int z = 4; z < 32; z <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, z));
      l = own.y * ex2(own.x - m);
      for (int x = c8 + 8; x < n; x += 8) {
        const float2 v = ml[tree_slot(w0 + x, false) * tile];
        l = fmaf(v.y, ex2(v.x - m), l);
      }
#pragma unroll
      for (int z = 4; z < 32; z <<= 1) l += __shfl_xor_sync(0xffffffffu, l, z);
      if (has_sink) l += ex2(sg - m + p.lift);
      for (int x = sub; x < n; x += W * kAhead) {
        if (x != sub) load(x);
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
          if (f[y] == INFINITY) continue;       // (counted already)
          const float fy = ex2(f[y] - m);       // (0 too: what is not finite in its O goes on)
#pragma unroll
          for (int k = 0; k < HG; ++k) {
            if (4 * (c8 + 8 * k) >= p.H) continue;
            a[k].x = fmaf(o[y][k].x, fy, a[k].x);
            a[k].y = fmaf(o[y][k].y, fy, a[k].y);
            a[k].z = fmaf(o[y][k].z, fy, a[k].z);
            a[k].w = fmaf(o[y][k].w, fy, a[k].w);
          }
        }
      }
    }
    if constexpr (W > 1) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < HG; ++k) join[warp][k][lane] = a[k];
      __syncthreads();
      if (sub > 0) continue;
#pragma unroll
      for (int x = 1; x < W; ++x)
#pragma unroll
        for (int k = 0; k < HG; ++k) {
          const float4 v = join[warp + x][k][lane];
          a[k] = make_float4(a[k].x + v.x, a[k].y + v.y, a[k].z + v.z, a[k].w + v.w);
        }
    }
    if (n == 1 || r0 + 4 * team + ri >= nrows) continue;
    const float inv = l == 0.f ? 0.f : 1.f / l;   // (a NaN goes on, also from a piece without weight)
    T* dst = static_cast<T*>(p.out) + (((long long)b * p.S + r / p.G) * p.N + hd) * p.H;
#pragma unroll
    for (int k = 0; k < HG; ++k) {
      const int c = 4 * (c8 + 8 * k);
      if (c >= p.H) continue;
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2*>(dst + c) = make_uint2(pack2(a[k].x * inv, a[k].y * inv), pack2(a[k].z * inv, a[k].w * inv));
      else
        *reinterpret_cast<float4*>(dst + c) = make_float4(a[k].x * inv, a[k].y * inv, a[k].z * inv, a[k].w * inv);
    }
  }
}

template <typename T, int W, int HG>
cudaError_t merge_hg(const TreeParams& p, cudaStream_t st) {
  constexpr int kStep = 4 * kMergeWarps / W;   // rows of a turn
  // Rows of a block: so many that the blocks fit the GPU about once beside the attention.
  const long long per_head = ((long long)p.S * p.G + kStep - 1) / kStep, all = per_head * p.B * p.Nkv;
  const int rows = (int)((all + 911) / 912) * kStep;
  const dim3 grid((unsigned)((p.S * p.G + rows - 1) / rows), (unsigned)(p.B * p.Nkv));
  return launch_dependent(true, tree_merge_kernel<T, W, HG>, grid, 32 * kMergeWarps, 0, st, p, rows);
}

template <typename T, int W>
cudaError_t merge_w(const TreeParams& p, cudaStream_t st) {
  return p.H <= 64 ? merge_hg<T, W, 2>(p, st) : p.H <= 128 ? merge_hg<T, W, 4>(p, st) : merge_hg<T, W, 8>(p, st);
}

template <typename T>
cudaError_t merge_t(const TreeParams& p, cudaStream_t st) {
  const long long pieces = p.workers / ((long long)p.B * p.Nkv * p.nrt) + 2;   // of a range, about
  return pieces <= 4 ? merge_w<T, 1>(p, st) : pieces <= 16 ? merge_w<T, 2>(p, st) : merge_w<T, 8>(p, st);
}

constexpr int kMaxDevices = 64;

template <typename T, int HP, int RW>
cudaError_t launch_rw(const TreeParams& p, cudaStream_t st) {
  static bool done[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  constexpr int smem = Cfg<T, HP, RW>::kSmem;
  auto kern = tree_attn_kernel<T, HP, RW>;
  if (!done[dev]) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    done[dev] = true;
  }
  return launch_dependent(false, kern, dim3((unsigned)p.workers), Cfg<T, HP, RW>::kThreads, (size_t)smem, st, p);
}

template <typename T, int HP>
cudaError_t launch_hp(const TreeParams& p, cudaStream_t st) {
  return p.rt_log2 == 4 ? launch_rw<T, HP, 1>(p, st) : p.rt_log2 == 5 ? launch_rw<T, HP, 2>(p, st) : launch_rw<T, HP, 4>(p, st);
}

template <typename T>
cudaError_t launch_t(const TreeParams& p, cudaStream_t st) {
  return p.H <= 64 ? launch_hp<T, 64>(p, st) : p.H <= 128 ? launch_hp<T, 128>(p, st) : launch_hp<T, 256>(p, st);
}

}  // namespace

// The tensor-core pipeline where it can: it holds 128 rows as cheaply as 16, and its copies run across the ends of
// ranges (16 sequences of 1k to 8k rows, 16 query rows: 74 us, the warp MMAs 80; 32 rows 76, 89; 5 nodes on 1030 rows
// 15, 17; events around single cold launches). It takes row maxima before the scale, which a negative one would turn,
// and softcaps of a range (softcap_fits; scale / softcap far from the ends of the floats).
bool use_tc(const TreeParams& p) {
  if (p.t_type != kF16 || p.H > 128 || !(p.scale > 0.f) || !softcap_fits(p.softcap)) return false;
  return p.softcap == 0.f || (p.scale > 0x1p-40f && p.scale < 0x1p40f);
}

void tree_attn_plan(TreeParams* p) {
  const int rows = p->S * p->G;
  p->tc = use_tc(*p);
  p->lift = p->tc ? 6.f : p->t_type == kF16 ? kLiftHalf : 0.f;
  // CTAs an SM holds: one of the pipeline; of the warp MMAs by their registers and shared memory (two stages of 64 KB
  // above a head size of 128).
  long long most = 152;
  if (p->tc) {
    p->cost = 4;   // (16 sequences of 1k to 8k rows with a softcap: 85 us, 91 with 2)
    p->rt_log2 = rows <= 128 ? 7 : 8;
    p->unit_log2 = 7;
  } else {
    p->cost = 2;
    p->rt_log2 = rows <= 16 ? 4 : rows <= 32 ? 5 : 6;
    p->unit_log2 = p->t_type == kF16 ? 6 : 5;
    most *= p->H <= 128 ? 2 : 1;
  }
  p->nrt = (rows + (1 << p->rt_log2) - 1) >> p->rt_log2;
  const int u = (1 << p->unit_log2) - 1;
  const int keys = p->window >= 0 && p->window < p->T - p->S ? p->window + 16 : p->T;
  const long long ranges = (long long)p->B * p->Nkv * p->nrt;
  const long long units = ranges * (((keys + u) >> p->unit_log2) + ((p->S + u) >> p->unit_log2) + p->cost);
  p->workers = (int)(units < most ? units : most);
}

cudaError_t launch_tree_attn(const TreeParams& p, cudaStream_t st) {
  if (p.tc) return launch_tree_tc(p, st);
  return p.t_type == kF16 ? launch_t<__half>(p, st) : launch_t<float>(p, st);
}

cudaError_t launch_tree_merge(const TreeParams& p, cudaStream_t st) {
  return p.t_type == kF16 ? merge_t<__half>(p, st) : merge_t<float>(p, st);
}

}  // namespace gqa
