// The block-scaled int8 cache: storing new rows, and eviction by accumulated
// attention weight (selection of the rows that stay, then their copy).
#include <cooperative_groups.h>
#include <cuda_fp16.h>

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

// c = rint(x * (1/s)) is off by at most one and only beside a border. There
// the remainder x - c s is exact in fp32 (both are multiples of the smaller
// operand's last place, and it is about s / 2), so 2 |x - c s| < s proves c.
// What it does not prove (a border, a tie, infinities, NaN) is `unsure`.
__device__ __forceinline__ uint32_t code_bits(float x, float s, float inv, bool* unsure) {
  const float r = fmaf(x, inv, kMagic);
  const float rem = fmaf(-(r - kMagic), s, x);
  *unsure |= !(2.f * fabsf(rem) < s);
  return __float_as_uint(r) & 0xffu;
}

// Four codes as the integers nearest to code * from / to (ties to even), from
// <= to. ratio is fp32(from / to): a product is within 2e-5 of its quotient,
// so only one that close to a border needs the exact comparison.
__device__ __forceinline__ uint32_t recode4(uint32_t w, float from, float to, float ratio) {
  const uint32_t u = w ^ 0x80808080u;   // code + 128 in each byte
  uint32_t out = 0;
  float near = 0.f;
  float q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // the byte under the exponent of 2^23, less 2^23 + 128
    q[e] = (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440u | e)) - 8388736.f) * ratio;
    const float r = q[e] + kMagic;
    near = fmaxf(near, fabsf(q[e] - (r - kMagic)));
    out |= (__float_as_uint(r) & 0xffu) << (8 * e);
  }
  if (near > 0.5f - 4e-5f) {
    out = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float c0 = (float)(int)(int8_t)(w >> (8 * e)), hi = c0 * from;
      out |= (uint32_t)((int)nearest_step(hi, fmaf(c0, from, -hi), to, rintf(q[e])) & 0xff) << (8 * e);
    }
  }
  return out;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* f);
template <>
__device__ __forceinline__ void load8<__half>(const __half* p, float* f) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
    f[2 * i] = a.x;
    f[2 * i + 1] = a.y;
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* f) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;   // infinities and NaN do not enter a scale
}

// ------------------------------------------------------------------ append

constexpr int kAppendThreads = 128;

// One block of tokens of one (b, g), K (z = 0) or V (z = 1): the largest |x|
// of its new rows, the scale, the codes. The rows are read twice, the second
// time out of the L1 / L2 cache; HBM sees sizeof(T) + 1 bytes per element.
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
  const long long ld = (long long)p.Nkv * p.H;                                   // elements between tokens
  const T* src = x + ((long long)b * p.S + (lo - past)) * ld + (long long)g * p.H;

  float amax = 0.f;
  for (int i = tid; i < n; i += kAppendThreads) {
    const int r = i / chunks, c = i - r * chunks;
    float f[8];
    load8<T>(src + r * ld + 8 * c, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, finite_abs(f[e]));
  }
  __shared__ float red[kAppendThreads / 32];
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((tid & 31) == 0) red[tid >> 5] = amax;
  __syncthreads();
  amax = red[0];
  for (int i = 1; i < kAppendThreads / 32; ++i) amax = fmaxf(amax, red[i]);

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
  for (int i = tid; i < n; i += kAppendThreads) {
    const int r = i / chunks, c = i - r * chunks;
    float f[8];
    load8<T>(src + r * ld + 8 * c, f);
    uint32_t w[2] = {0u, 0u};
    if (s > 0.f) {
      bool unsure = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e >> 2] |= code_bits(f[e], s, inv, &unsure) << (8 * (e & 3));
      if (unsure) {
        w[0] = w[1] = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e >> 2] |= (uint32_t)(code_slow(f[e], s, inv) & 0xff) << (8 * (e & 3));
      }
    }
    *reinterpret_cast<uint2*>(dst + (long long)i * 8) = make_uint2(w[0], w[1]);
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

constexpr int kSelCache = 16384;   // rows of a CTA whose keys stay in shared memory
constexpr int kSelRows = 4096;     // rows a CTA is given before the cluster grows

// One (b, g) per cluster of CL CTAs, each with an equal slice of the rows
// between `first` and `recent`. A radix selection (four passes of eight bits
// from the top, the CTAs' histograms added over distributed shared memory)
// finds the key of the last row that stays and how many rows with exactly that
// key do; a scan in row order then writes the indices. Bound: latency, 4 bytes
// a row; one CTA of 131072 rows took 250 us, a cluster of eight 30.
__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const EvictParams p, int CL) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = CL > 1 ? (int)cluster.block_rank() : 0;
  const int bg = blockIdx.x / CL, b = bg / p.Nkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int total = p.seqlens[b] + 1;
  dep_launch();
  if (total < 0 || total > p.C || total > p.T) {   // every CTA of the cluster leaves
    if (bg % p.Nkv == 0 && rank == 0 && tid == 0 && p.status) atomicOr(p.status, GQA_DEVICE_BAD_SEQLEN_BIT);
    return;
  }
  int* kept = p.kept + (long long)bg * p.keep;
  if (bg % p.Nkv == 0 && rank == 0 && tid == 0) p.seqlens_to[b] = min(total, p.keep) - 1;
  const int step = CL * kSelThreads, at = rank * kSelThreads + tid;
  if (total <= p.keep) {
    for (int i = at; i < p.keep; i += step) kept[i] = i < total ? i : -1;
    return;
  }
  const int lo = p.first, hi = total - p.recent;
  for (int i = at; i < p.first; i += step) kept[i] = i;
  for (int i = at; i < p.recent; i += step) kept[p.keep - p.recent + i] = hi + i;
  int need = p.keep - p.first - p.recent;   // of the rows [lo, hi); need < hi - lo
  if (need == 0) return;
  const float* w = p.w + (long long)bg * p.C;
  const int per = ((hi - lo + CL - 1) / CL + 31) & ~31;          // rows of a CTA
  const int a = min(lo + rank * per, hi), n = min(per, hi - a);
  extern __shared__ unsigned keys[];
  const bool cached = n <= kSelCache;
  if (cached)
    for (int i = tid; i < n; i += kSelThreads) keys[i] = weight_key(w[a + i]);
  auto key_at = [&](int i) { return cached ? keys[i] : weight_key(w[a + i]); };
  __shared__ int hist[256];    // this CTA's counts
  __shared__ int sum[256];     // the cluster's
  __shared__ unsigned s_digit;
  __shared__ int s_need, s_count[2];
  __shared__ int wsum[2][kSelThreads / 32];
  unsigned prefix = 0, mask = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += kSelThreads) {
      const int i = i0 + tid;
      const unsigned key = i < n ? key_at(i) : 0u;
      const bool in = i < n && (key & mask) == prefix;
      const unsigned digit = (key >> shift) & 255u;
      const unsigned ins = __ballot_sync(0xffffffffu, in);
      if (ins == 0) continue;
      // a warp whose digits are all the same (top digits, ties) counts them as one
      const unsigned first = __shfl_sync(0xffffffffu, digit, __ffs(ins) - 1);
      if (__all_sync(0xffffffffu, !in || digit == first)) {
        if (lane == 0) atomicAdd(&hist[first], __popc(ins));
      } else if (in) {
        atomicAdd(&hist[digit], 1);
      }
    }
    if (CL > 1) cluster.sync(); else __syncthreads();
    if (tid < 256) {
      int c = 0;
      for (int r = 0; r < CL; ++r) c += CL > 1 ? cluster.map_shared_rank(hist, r)[tid] : hist[tid];
      sum[tid] = c;
    }
    __syncthreads();
    if (warp == 0) {   // from the top digit down: the one at which `need` rows are reached
      int n8 = 0;
      for (int i = 0; i < 8; ++i) n8 += sum[255 - (8 * lane + i)];
      int incl = n8;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      int before = incl - n8;
      if (before < need && incl >= need) {
        for (int i = 0; i < 8; ++i) {
          const int d = 255 - (8 * lane + i), c = sum[d];
          if (before + c >= need) {
            s_digit = (unsigned)d;
            s_need = need - before;
            break;
          }
          before += c;
        }
      }
    }
    if (CL > 1) cluster.sync(); else __syncthreads();   // the histograms have been read, the digit is there
    prefix |= s_digit << shift;
    mask |= 255u << shift;
    need = s_need;
  }
  // `need` rows with key == prefix stay (the lowest), and all above it. Rows
  // and ties of the CTAs before this one:
  int above_n = 0, tie_n = 0;
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    const unsigned key = i < n ? key_at(i) : 0u;
    above_n += i < n && key > prefix;
    tie_n += i < n && key == prefix;
  }
  for (int o = 16; o; o >>= 1) {
    above_n += __shfl_xor_sync(0xffffffffu, above_n, o);
    tie_n += __shfl_xor_sync(0xffffffffu, tie_n, o);
  }
  if (lane == 0) {
    wsum[0][warp] = above_n;
    wsum[1][warp] = tie_n;
  }
  __syncthreads();
  if (tid < 2) {
    int c = 0;
    for (int i = 0; i < kSelThreads / 32; ++i) c += wsum[tid][i];
    s_count[tid] = c;
  }
  if (CL > 1) cluster.sync(); else __syncthreads();
  int out = p.first, ties = 0;
  for (int r = 0; r < rank; ++r) {
    const int* c = cluster.map_shared_rank(s_count, r);
    out += c[0];
    ties += c[1];
  }
  out += min(ties, need);
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    const unsigned key = i < n ? key_at(i) : 0u;
    const bool above = i < n && key > prefix, tie = i < n && key == prefix;
    const unsigned ma = __ballot_sync(0xffffffffu, above), mt = __ballot_sync(0xffffffffu, tie);
    __syncthreads();   // the counts of the round before have been read
    if (lane == 0) {
      wsum[0][warp] = __popc(ma);
      wsum[1][warp] = __popc(mt);
    }
    __syncthreads();
    // every warp scans the 32 warp counts
    const int va = wsum[0][lane], vt = wsum[1][lane];
    int ia = va, it = vt;
    for (int o = 1; o < 32; o <<= 1) {
      const int xa = __shfl_up_sync(0xffffffffu, ia, o), xt = __shfl_up_sync(0xffffffffu, it, o);
      if (lane >= o) {
        ia += xa;
        it += xt;
      }
    }
    const int a_before = __shfl_sync(0xffffffffu, ia - va, warp), t_before = __shfl_sync(0xffffffffu, it - vt, warp);
    const int a_all = __shfl_sync(0xffffffffu, ia, 31), t_all = __shfl_sync(0xffffffffu, it, 31);
    const unsigned below = (1u << lane) - 1u;
    const int t_rank = ties + t_before + __popc(mt & below);
    const int t_taken = min(t_rank, need) - min(ties, need);   // border rows of this round before this one that stay
    if (above || (tie && t_rank < need)) kept[out + a_before + __popc(ma & below) + t_taken] = a + i;
    out += a_all + min(ties + t_all, need) - min(ties, need);
    ties += t_all;
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
// are requested together with the scales, not behind them.
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
  __shared__ float rs[256];
  __shared__ float red[kGatherThreads / 32];
  const int* rows = p.kept + (long long)bg * p.keep + first;
  const int chunks = p.H / 16;
  uint4 ahead[kGatherAhead];
#pragma unroll
  for (int k = 0; k < kGatherAhead; ++k) {
    const int i = k * kGatherThreads + tid;
    if (i < n * chunks)
      ahead[k] = *reinterpret_cast<const uint4*>(from + (long long)rows[i / chunks] * p.H + 16 * (i % chunks));
  }
  float top = 0.f;
  for (int i = tid; i < n; i += kGatherThreads) {
    const int r = rows[i];
    rs[i] = sc[r >> p.bs_log2];
    top = fmaxf(top, rs[i]);
    if (!isv && p.w_to) p.w_to[(long long)bg * p.Cto + first + i] = p.w[(long long)bg * p.C + r];
  }
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) red[tid >> 5] = top;
  __syncthreads();
  top = red[0];
  for (int i = 1; i < kGatherThreads / 32; ++i) top = fmaxf(top, red[i]);
  if (tid == 0) (isv ? p.vs_to : p.ks_to)[(long long)bg * p.nblk_to + blockIdx.x] = top;
  auto put = [&](int i, uint4 w) {
    const int r = i / chunks, c = i - r * chunks;
    const float s = rs[r];
    if (s != top) {
      const float ratio = top > 0.f ? __fdiv_rn(s, top) : 0.f;
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
    put(i, *reinterpret_cast<const uint4*>(from + (long long)rows[i / chunks] * p.H + 16 * (i % chunks)));
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
  // A CTA for every kSelRows rows, up to the portable cluster size.
  int CL = 1;
  while (CL < 8 && (long long)CL * kSelRows < p.T) CL *= 2;
  const long long per = ((p.T + CL - 1) / CL + 31) & ~31LL;
  const size_t smem = (size_t)(per < kSelCache ? per : kSelCache) * sizeof(unsigned);
  static bool done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelCache * (int)sizeof(unsigned));
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * p.Nkv * CL));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
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
