// The block-scaled int8 cache: storing new rows, and eviction by accumulated
// attention weight (selection of the rows that stay, then their copy).
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "../../include/gqa.h"
#include "block_internal.h"
#include "common.cuh"

namespace gqa {
namespace {

// ------------------------------------------------------------------ codes

constexpr float kMagic = 12582912.f;   // 1.5 2^23: x + kMagic rounds |x| < 2^22 to an integer, held in the low bits

// c + the step towards the integer nearest to the exact quotient (hi + lo) / s,
// c within one of it and |lo| at most half a last place of hi. Beside a border
// hi - c s is exact in fp32 (multiples of the last place of s or, for |hi| < s,
// the difference of numbers within a factor of two), and so is 2 |rem| - s; lo
// only decides its sign. Ties go to the even integer.
__device__ __forceinline__ float nearest_step(float hi, float lo, float s, float c) {
  const float rem = fmaf(-c, s, hi);
  const float d = (2.f * fabsf(rem) - s) + (rem < 0.f ? -2.f * lo : 2.f * lo);
  return d > 0.f || (d == 0.f && ((int)c & 1)) ? c + copysignf(1.f, rem) : c;
}

// The integer nearest to the exact quotient x / s, within +-127; NaN gives 0.
__device__ __forceinline__ int code_slow(float x, float s, float inv) {
  if (x != x) return 0;
  const float q = inv < 3.0e38f ? x * inv : __fdiv_rn(x, s);   // 1/s overflows for a subnormal s
  const float c = fminf(fmaxf(rintf(q), -127.f), 127.f);
  if (fabsf(x) > 3.402823466e38f) return (int)c;
  return (int)fminf(fmaxf(nearest_step(x, 0.f, s, c), -127.f), 127.f);
}

// The larger of two values, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(float a, float b, float c, float d) {
  const uint32_t lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040u);
  const uint32_t hi = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040u);
  return __byte_perm(lo, hi, 0x5410u);
}

// Eight codes of x[0..7] by scale s > 0, inv = 1/s. c = rint(x inv) is off by
// at most one and only beside a border. There the remainder x - c s is exact
// in fp32 (both are multiples of the smaller operand's last place, and it is
// about s / 2), so 2 |x - c s| < s proves c. What it does not prove (a border,
// a tie, infinities, NaN) is settled one value at a time.
__device__ __forceinline__ uint2 codes8(const float* x, float s, float inv) {
  float2 r[4];
  float worst = 0.f;
  const float2 inv2 = make_float2(inv, inv), magic = make_float2(kMagic, kMagic), neg = make_float2(-kMagic, -kMagic);
  const float2 s2 = make_float2(-s, -s);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = make_float2(x[2 * i], x[2 * i + 1]);
    r[i] = ffma2(v, inv2, magic);
    const float2 rem = ffma2(fadd2(r[i], neg), s2, v);
    worst = max_nan(worst, max_nan(fabsf(rem.x), fabsf(rem.y)));
  }
  uint2 w = make_uint2(low_bytes(r[0].x, r[0].y, r[1].x, r[1].y), low_bytes(r[2].x, r[2].y, r[3].x, r[3].y));
  if (!(2.f * worst < s)) {
    w = make_uint2(0u, 0u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w.x |= (uint32_t)(code_slow(x[e], s, inv) & 0xff) << (8 * e);
      w.y |= (uint32_t)(code_slow(x[4 + e], s, inv) & 0xff) << (8 * e);
    }
  }
  return w;
}

// Four codes as the integers nearest to code * from / to (ties to even), from
// <= to. ratio is fp32(from / to): code * ratio is within 2e-5 of its quotient,
// so only one that close to a border needs the exact comparison.
__device__ __forceinline__ uint32_t recode4(uint32_t w, float from, float to, float ratio) {
  const uint32_t u = w ^ 0x80808080u;   // code + 128 in each byte
  const float2 ratio2 = make_float2(ratio, ratio), magic = make_float2(kMagic, kMagic);
  const float2 base = make_float2(-8388736.f, -8388736.f), minus = make_float2(-1.f, -1.f);
  float2 r[2];
  float near = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // a byte under the exponent of 2^23, less 2^23 + 128
    const float2 v = fadd2(make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440u | (2 * i))),
                                       __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440u | (2 * i + 1)))), base);
    r[i] = ffma2(v, ratio2, magic);
    // v ratio - c, rounded once
    const float2 d = ffma2(v, ratio2, ffma2(r[i], minus, magic));
    near = fmax3(near, fabsf(d.x), fabsf(d.y));
  }
  uint32_t out = low_bytes(r[0].x, r[0].y, r[1].x, r[1].y);
  if (near > 0.5f - 4e-5f) {
    out = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float c0 = (float)(int)(int8_t)(w >> (8 * e)), hi = c0 * from;
      out |= (uint32_t)((int)nearest_step(hi, fmaf(c0, from, -hi), to, rintf(c0 * ratio)) & 0xff) << (8 * e);
    }
  }
  return out;
}

// Eight values of a row as loaded.
template <typename T>
struct Raw8;
template <>
struct Raw8<__half> {
  static constexpr unsigned kInfinity = 0x7c00u;
  uint32_t w[4];
  __device__ __forceinline__ void load(const __half* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = a.x;
      f[2 * i + 1] = a.y;
    }
  }
  // The larger of m and the bits of every |x| (ordered as the values are), two halves side by side.
  __device__ __forceinline__ unsigned top(unsigned m) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    return m;
  }
  static __device__ __forceinline__ unsigned fold(unsigned m) { return max(m & 0xffffu, m >> 16); }
  static __device__ __forceinline__ float value(unsigned bits) { return __half2float(__ushort_as_half((unsigned short)bits)); }
};
template <>
struct Raw8<float> {
  static constexpr unsigned kInfinity = 0x7f800000u;
  uint32_t w[8];
  __device__ __forceinline__ void load(const float* p) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  }
  __device__ __forceinline__ unsigned top(unsigned m) const {
#pragma unroll
    for (int i = 0; i < 8; i += 2) m = max(max(m, w[i] & 0x7fffffffu), w[i + 1] & 0x7fffffffu);
    return m;
  }
  static __device__ __forceinline__ unsigned fold(unsigned m) { return m; }
  static __device__ __forceinline__ float value(unsigned bits) { return __uint_as_float(bits); }
};

// ------------------------------------------------------------------ append

constexpr int kAppendThreads = 128;

// i / d for i < 8192, d <= 32 as a product (the rounding of 2^20 / d adds less than 1 / d).
struct SmallDiv {
  unsigned m, d;
  __device__ explicit SmallDiv(int div) : m((1u << 20) / (unsigned)div + 1u), d((unsigned)div) {}
  __device__ __forceinline__ int quot(int i) const { return (int)(((unsigned)i * m) >> 20); }
};

// One block of tokens of one (b, g), K (z = 0) or V (z = 1): the largest |x|
// of its new rows, the scale, the codes. The rows are read twice, the second
// time out of the L1 / L2 cache; HBM sees sizeof(T) + 1 bytes per element.
// Bound: a decode step the latency of its loads, one behind the other (4.7 us);
// a prompt the instructions (2 x 4096 tokens, 8 heads of 128, fp16: 20 us, 2.3
// a clock). Rows kept in registers for the second pass took 2 us off the prompt
// and put 8 on the decode step: the larger blocks left the attention kernel
// that starts beside them an uneven share of the SMs.
template <typename T>
__global__ void __launch_bounds__(kAppendThreads)
block_append_kernel(const BlockParams p) {
  dep_launch();   // the attention kernel may set itself up meanwhile
  const int bg = blockIdx.y, b = bg / p.Nkv, g = bg % p.Nkv, tid = threadIdx.x;
  int total, fresh;
  if (!block_lengths(p, b, &total, &fresh)) {
    if (blockIdx.x == 0 && g == 0 && tid == 0 && p.status) atomicOr(p.status, GQA_DEVICE_BAD_SEQLEN_BIT);
    return;
  }
  if (fresh == 0) return;
  const int past = total - fresh;
  const int blk = (past >> p.bs_log2) + (int)blockIdx.x;
  const int first = blk << p.bs_log2;
  if (first >= total) return;
  const int lo = max(first, past), hi = min(first + (1 << p.bs_log2), total);   // new rows of this block
  const T* x = static_cast<const T*>(blockIdx.z == 0 ? p.k : p.v);
  int8_t* codes = (blockIdx.z == 0 ? p.kc : p.vc) + (long long)bg * p.C * p.H;
  float* scale = (blockIdx.z == 0 ? p.ks : p.vs) + (long long)bg * p.nblk + blk;
  const int chunks = p.H / 8, n = (hi - lo) * chunks;
  const SmallDiv div(chunks);
  const long long ld = (long long)p.Nkv * p.H;                                   // elements between tokens
  const T* src = x + ((long long)b * p.S + (lo - past)) * ld + (long long)g * p.H;

  auto load = [&](int i) {
    const int r = div.quot(i);
    Raw8<T> v;
    v.load(src + r * ld + 8 * (i - r * chunks));
    return v;
  };
  __shared__ unsigned red[kAppendThreads / 32];
  auto block_max = [&](unsigned m) {
    m = __reduce_max_sync(0xffffffffu, m);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int i = 1; i < kAppendThreads / 32; ++i) m = max(m, red[i]);
    return m;
  };
  unsigned mx = 0;
#pragma unroll 4
  for (int i = tid; i < n; i += kAppendThreads) mx = load(i).top(mx);
  mx = block_max(Raw8<T>::fold(mx));
  float amax = Raw8<T>::value(mx);
  if (mx >= Raw8<T>::kInfinity) {   // infinities and NaN do not enter a scale: once more without them
    amax = 0.f;
    for (int i = tid; i < n; i += kAppendThreads) {
      float f[8];
      load(i).get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]) <= 3.402823466e38f ? fabsf(f[e]) : 0.f);
    }
    amax = __uint_as_float(block_max(__float_as_uint(amax)));
  }

  float s = __fmul_rn(amax, 1.0f / 127.0f);
  if (first < past) {   // the block holds rows already
    const float s0 = *scale;
    if (s > s0) {
      const float ratio = __fdiv_rn(s0, s);
      uint32_t* old = reinterpret_cast<uint32_t*>(codes + (long long)first * p.H);
      for (int i = tid; i < (past - first) * p.H / 4; i += kAppendThreads) old[i] = recode4(old[i], s0, s, ratio);
    } else {
      s = s0;
    }
    __syncthreads();   // every thread has read the old scale
  }
  if (tid == 0) *scale = s;
  const float inv = __fdiv_rn(1.f, s);
  int8_t* dst = codes + (long long)lo * p.H;
#pragma unroll 2
  for (int i = tid; i < n; i += kAppendThreads) {
    float f[8];
    load(i).get(f);
    *reinterpret_cast<uint2*>(dst + (long long)i * 8) = s > 0.f ? codes8(f, s, inv) : make_uint2(0u, 0u);
  }
}

// ------------------------------------------------------------------ eviction: which rows stay

constexpr int kSelThreads = 1024;

// Weights as unsigned keys in their order (a larger weight is a larger key);
// -0 equals +0, NaN is the lowest.
__device__ __forceinline__ unsigned weight_key(float w) {
  if (w != w) return 0u;
  const unsigned u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelKeys = 16;                        // consecutive rows a thread holds in registers
constexpr int kSelRows = kSelThreads * kSelKeys;    // rows of a CTA at a time

constexpr int kSelCluster = 8;                      // CTAs of a cluster, at most
constexpr int kSelBins = 2048;                      // 11 bits a pass
constexpr int kSelList = 512;                       // keys ranked by comparing each with each

// One (b, g) per cluster of CL CTAs, each with an equal slice of the rows
// between `first` and `recent`. A radix selection, 11 bits at a time from the
// top, finds the key of the last row that stays and how many rows with exactly
// that key do: counts in shared memory (the CTAs' added over distributed
// shared memory), a scan over the bins. It ends once every row with the digits
// found so far stays, or once at most 512 rows have them: those are ranked by
// comparison. Threads hold consecutive rows in registers, so one scan places
// the rows that stay in order. Bound: latency, 4 bytes a row. (Eight-bit
// passes with a scan by one warp took 21 us on 8192 rows, four-bit passes with
// counters in registers as much: their reductions cost what the atomics did.)
// 128 (b, g) of 8192 rows: 12 us; 8 of 131072 rows, clusters of 8: 23 us.
__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const EvictParams p, int CL) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = CL > 1 ? (int)cluster.block_rank() : 0;
  const int bg = blockIdx.x / CL, b = bg / p.Nkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int total = p.seqlens[b] + 1;
  dep_launch();
  int* kept = p.kept + (long long)bg * p.keep;
  const int step = CL * kSelThreads, at = rank * kSelThreads + tid;
  if (total < 0 || total > p.C || total > p.T) {   // every CTA of the cluster leaves
    if (bg % p.Nkv == 0 && rank == 0 && tid == 0) {
      if (p.status) atomicOr(p.status, GQA_DEVICE_BAD_SEQLEN_BIT);
      if (p.fill & GQA_FILL_SEQLENS) p.seqlens_to[b] = -1;
    }
    if (p.fill & GQA_FILL_KEPT)
      for (int i = at; i < p.keep; i += step) kept[i] = -1;
    return;
  }
  if (bg % p.Nkv == 0 && rank == 0 && tid == 0) p.seqlens_to[b] = min(total, p.keep) - 1;
  if (total <= p.keep) {
    for (int i = at; i < p.keep; i += step) kept[i] = i < total ? i : -1;
    return;
  }
  const int lo = p.first, hi = total - p.recent;
  for (int i = at; i < p.first; i += step) kept[i] = i;
  for (int i = at; i < p.recent; i += step) kept[p.keep - p.recent + i] = hi + i;
  int need = p.keep - p.first - p.recent;   // of the rows [lo, hi); need < hi - lo
  if (need == 0) return;
  const int per = (hi - lo + CL - 1) / CL;                       // rows of a CTA
  const int a = min(lo + rank * per, hi), n = min(per, hi - a);  // its own
  const float* w = p.w + (long long)bg * p.C + a;
  const int rounds = (n + kSelRows - 1) / kSelRows;              // 1 unless the slice exceeds the registers
  const int kpt = min((n + kSelThreads - 1) / kSelThreads, kSelKeys);   // rows of a thread in a round
  unsigned key[kSelKeys];
  int mine = 0;                                                  // keys held
  auto load = [&](int round) {
    const int base = round * kSelRows + tid * kpt;
    mine = max(0, min(kpt, n - base));
#pragma unroll
    for (int k = 0; k < kSelKeys; ++k)
      if (k < mine) key[k] = weight_key(w[base + k]);
  };
  if (rounds <= 1) load(0);

  __shared__ __align__(8) int hist[2][kSelBins];    // the CTA's counts, by pass parity
  __shared__ unsigned list[kSelList], all_list[kSelList];
  __shared__ int wsum[kSelThreads / 32], s_count[2], s_list, s_need, s_bin_count;
  __shared__ unsigned s_key;
  auto group_sync = [&] {
    if (CL > 1) cluster.sync(); else __syncthreads();
  };
  unsigned prefix = 0, mask = 0;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kSelBins;
    int* h = hist[pass & 1];
    for (int i = tid; i < kSelBins; i += kSelThreads) h[i] = 0;
    if (tid == 0) s_list = 0;
    __syncthreads();
    for (int round = 0; round < max(rounds, 1); ++round) {
      if (rounds > 1) load(round);
#pragma unroll
      for (int k = 0; k < kSelKeys; ++k) {
        if (k >= kpt) continue;        // uniform
        const bool in = k < mine && (key[k] & mask) == prefix;
        const unsigned ins = __ballot_sync(0xffffffffu, in);
        if (ins == 0) continue;
        const unsigned digit = (key[k] >> shift) & (unsigned)(bins - 1);
        const unsigned one = __shfl_sync(0xffffffffu, digit, __ffs(ins) - 1);
        if (__all_sync(0xffffffffu, !in || digit == one)) {   // ties: one count for the warp
          if (lane == 0) atomicAdd(&h[one], __popc(ins));
        } else if (in) {
          atomicAdd(&h[digit], 1);
        }
      }
    }
    group_sync();
    // Thread t: bins - 1 - 2 t and the one below it; an inclusive scan from the top.
    int c[2] = {0, 0};
    const int top = bins - 1 - 2 * tid;
    if (top > 0) {
      const int2* at = reinterpret_cast<const int2*>(h + top - 1);
      if (CL == 1) {
        c[0] = at->y;
        c[1] = at->x;
      } else {
#pragma unroll 8
        for (int r = 0; r < CL; ++r) {
          const int2 v = *cluster.map_shared_rank(at, r);
          c[0] += v.y;
          c[1] += v.x;
        }
      }
    }
    int incl = c[0] + c[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int wv = wsum[lane], wincl = wv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, wincl, o);
      if (lane >= o) wincl += v;
    }
    incl += __shfl_sync(0xffffffffu, wincl - wv, warp);
    const int before = incl - c[0] - c[1];
    if (before < need && need <= incl) {   // one thread
      const int second = need > before + c[0];
      s_key = (unsigned)(top - second);
      s_need = need - before - (second ? c[0] : 0);
      s_bin_count = c[second];
    }
    __syncthreads();
    prefix |= s_key << shift;
    mask |= (unsigned)(bins - 1) << shift;
    need = s_need;
    const int count = s_bin_count;
    __syncthreads();
    if (need == count) break;          // all rows with this prefix stay
    if (count <= kSelList && pass < 2) {
      for (int round = 0; round < max(rounds, 1); ++round) {
        if (rounds > 1) load(round);
#pragma unroll
        for (int k = 0; k < kSelKeys; ++k)
          if (k < mine && (key[k] & mask) == prefix) list[atomicAdd(&s_list, 1)] = key[k];   // any order serves
      }
      group_sync();
      int m = 0;                       // every CTA takes all the cluster's keys (at most kSelList), one a thread
      if (CL == 1) {
        m = s_list;
        if (tid < m) all_list[tid] = list[tid];
      } else {
        int at_r = 0, at_i = 0, cnt[kSelCluster];
#pragma unroll
        for (int r = 0; r < kSelCluster; ++r) cnt[r] = r < CL ? *cluster.map_shared_rank(&s_list, r) : 0;
#pragma unroll
        for (int r = 0; r < kSelCluster; ++r) {
          if (tid >= m && tid < m + cnt[r]) at_r = r, at_i = tid - m;
          m += cnt[r];
        }
        if (tid < m) all_list[tid] = cluster.map_shared_rank(list, at_r)[at_i];
      }
      __syncthreads();
      if (tid < m) {
        const unsigned v = all_list[tid];
        int greater = 0, equal = 0;
        for (int i = 0; i < m; ++i) {
          greater += all_list[i] > v;
          equal += all_list[i] == v;
        }
        if (greater < need && need <= greater + equal) {   // equal keys write equal values
          s_key = v;
          s_need = need - greater;
        }
      }
      group_sync();                    // (no CTA reuses its list while it is read)
      prefix = s_key;
      mask = 0xffffffffu;
      need = s_need;
      __syncthreads();
      break;
    }
  }
  // Rows above the prefix stay, and the first `need` with it. A thread's counts
  // of both in one word, scanned over the warp, the CTA and the CTAs before.
  int out = p.first, ties = 0;
  for (int round = 0; round < max(rounds, 1); ++round) {
    if (rounds > 1) load(round);
    unsigned own = 0;                  // above | ties << 16 (a round has at most 16384 rows)
#pragma unroll
    for (int k = 0; k < kSelKeys; ++k)
      if (k < mine) own += (key[k] & mask) > prefix ? 1u : (key[k] & mask) == prefix ? 0x10000u : 0u;
    unsigned incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();                   // the warp sums of the round before have been read
    if (lane == 31) wsum[warp] = (int)incl;
    __syncthreads();
    const unsigned wv = (unsigned)wsum[lane];
    unsigned wincl = wv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xffffffffu, wincl, o);
      if (lane >= o) wincl += v;
    }
    const unsigned all = __shfl_sync(0xffffffffu, wincl, 31);
    const unsigned before = incl - own + __shfl_sync(0xffffffffu, wincl - wv, warp);
    if (CL > 1 && round == 0) {        // totals of the CTAs before this one
      int above_n = (int)(all & 0xffffu), tie_n = (int)(all >> 16);
      for (int r2 = 1; r2 < rounds; ++r2) {   // a slice of several rounds counts them first
        load(r2);
        unsigned o2 = 0;
#pragma unroll
        for (int k = 0; k < kSelKeys; ++k)
          if (k < mine) o2 += (key[k] & mask) > prefix ? 1u : (key[k] & mask) == prefix ? 0x10000u : 0u;
        o2 = __reduce_add_sync(0xffffffffu, o2);
        __syncthreads();
        if (lane == 0) wsum[warp] = (int)o2;
        __syncthreads();
        const unsigned sum = __reduce_add_sync(0xffffffffu, (unsigned)wsum[lane]);
        above_n += (int)(sum & 0xffffu);
        tie_n += (int)(sum >> 16);
      }
      if (rounds > 1) load(0);
      if (tid == 0) {
        s_count[0] = above_n;
        s_count[1] = tie_n;
      }
      cluster.sync();
#pragma unroll
      for (int r = 0; r < kSelCluster - 1; ++r) {
        if (r < rank) {
          const int* cnt = cluster.map_shared_rank(s_count, r);
          out += cnt[0];
          ties += cnt[1];
        }
      }
      out += min(ties, need);
    }
    int above_at = out + (int)(before & 0xffffu), tie_at = ties + (int)(before >> 16);
    const int base = a + round * kSelRows + tid * kpt;
#pragma unroll
    for (int k = 0; k < kSelKeys; ++k) {
      if (k >= mine) continue;
      const unsigned v = key[k] & mask;
      if (v > prefix || (v == prefix && tie_at < need))
        kept[above_at + min(tie_at, need) - min(ties, need)] = base + k;
      above_at += v > prefix;
      tie_at += v == prefix;
    }
    const int tie_all = (int)(all >> 16);
    out += (int)(all & 0xffffu) + min(ties + tie_all, need) - min(ties, need);
    ties += tie_all;
  }
  if (CL > 1) cluster.sync();   // no CTA leaves while its counts may be read
}

// ------------------------------------------------------------------ eviction: the copy

constexpr int kGatherThreads = 128;
constexpr int kGatherAhead = 4;   // 16-byte chunks a thread has in flight before the scales are known

// One block of tokens of one (b, g) of the new cache, K (z = 0) or V (z = 1):
// the largest source scale of its rows, then every row's codes, 16 at a time,
// rounded anew where the row's own scale is smaller. One read and one write of
// each kept row; the bound is HBM, latency first: a thread's first code chunks
// are requested together with the scales, not behind them. 128 (b, g) of 2048
// rows of 128 kept (134 MB moved): 27 us, 5.0 TB/s.
__global__ void __launch_bounds__(kGatherThreads)
evict_gather_kernel(const EvictParams p) {
  const int bg = blockIdx.y, b = bg / p.Nkv, tid = threadIdx.x;
  const int total = p.seqlens[b] + 1;
  dep_wait();   // also without work: what follows on the stream waits for this kernel alone
  if (total < 0 || total > p.C || total > p.T) return;
  const int stay = min(total, p.keep), bs = 1 << p.bs_log2;
  const int first = (int)blockIdx.x << p.bs_log2, n = min(bs, stay - first);
  if (n <= 0) return;
  const bool isv = blockIdx.z == 1;
  const int8_t* from = (isv ? p.vc : p.kc) + (long long)bg * p.C * p.H;
  const float* sc = (isv ? p.vs : p.ks) + (long long)bg * p.nblk;
  int8_t* to = (isv ? p.vc_to : p.kc_to) + ((long long)bg * p.Cto + first) * p.H;
  __shared__ float2 rs[256];       // scale of a row, and its ratio to the block's
  __shared__ float red[kGatherThreads / 32];
  const int* rows = p.kept + (long long)bg * p.keep + first;
  const int chunks = p.H / 16;
  const SmallDiv div(chunks);
  uint4 ahead[kGatherAhead];
#pragma unroll
  for (int k = 0; k < kGatherAhead; ++k) {
    const int i = k * kGatherThreads + tid;
    const int r = div.quot(i);
    if (i < n * chunks)
      ahead[k] = *reinterpret_cast<const uint4*>(from + (long long)rows[r] * p.H + 16 * (i - r * chunks));
  }
  float top = 0.f;
  for (int i = tid; i < n; i += kGatherThreads) {
    const int r = rows[i];
    rs[i].x = sc[r >> p.bs_log2];
    top = fmaxf(top, rs[i].x);
    if (!isv && p.w_to) p.w_to[(long long)bg * p.Cto + first + i] = p.w[(long long)bg * p.C + r];
  }
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) red[tid >> 5] = top;
  __syncthreads();
  top = red[0];
  for (int i = 1; i < kGatherThreads / 32; ++i) top = fmaxf(top, red[i]);
  if (tid == 0) (isv ? p.vs_to : p.ks_to)[(long long)bg * p.nblk_to + blockIdx.x] = top;
  for (int i = tid; i < n; i += kGatherThreads) rs[i].y = top > 0.f ? __fdiv_rn(rs[i].x, top) : 0.f;   // a thread's own rows
  __syncthreads();
  auto put = [&](int i, uint4 w) {
    const int r = div.quot(i), c = i - r * chunks;
    const float s = rs[r].x, ratio = rs[r].y;
    if (s != top) {
      w = make_uint4(recode4(w.x, s, top, ratio), recode4(w.y, s, top, ratio), recode4(w.z, s, top, ratio),
                     recode4(w.w, s, top, ratio));
    }
    *reinterpret_cast<uint4*>(to + (long long)r * p.H + 16 * c) = w;
  };
#pragma unroll
  for (int k = 0; k < kGatherAhead; ++k) {
    const int i = k * kGatherThreads + tid;
    if (i < n * chunks) put(i, ahead[k]);
  }
  for (int i = kGatherAhead * kGatherThreads + tid; i < n * chunks; i += kGatherThreads)
    put(i, *reinterpret_cast<const uint4*>(from + (long long)rows[div.quot(i)] * p.H + 16 * (i - div.quot(i) * chunks)));
}

}  // namespace

cudaError_t launch_block_append(const BlockParams& p, cudaStream_t st) {
  const int bs = 1 << p.bs_log2;
  const dim3 grid((unsigned)((p.S + bs - 2) / bs + 1), (unsigned)(p.B * p.Nkv), 2);
  if (p.t_type == kF16)
    block_append_kernel<__half><<<grid, kAppendThreads, 0, st>>>(p);
  else
    block_append_kernel<float><<<grid, kAppendThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t st) {
  // A CTA for every kSelRows rows, up to the portable cluster size (clusters of
  // 16 took 53 us where 8 take 33, on 8 (b, g) of 131072 rows).
  int CL = 1;
  while (CL < kSelCluster && (long long)CL * kSelRows < p.T) CL *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * p.Nkv * CL));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)CL;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, p, CL);
}

cudaError_t launch_evict_gather(const EvictParams& p, cudaStream_t st) {
  const int rows = p.keep < p.T ? p.keep : p.T, bs = 1 << p.bs_log2;
  return launch_dependent(true, evict_gather_kernel, dim3((unsigned)((rows + bs - 1) / bs), (unsigned)(p.B * p.Nkv), 2),
                          kGatherThreads, 0, st, p);
}

}  // namespace gqa
