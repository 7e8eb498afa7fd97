// The block-scaled int8 cache: storing new rows, and eviction by accumulated
// attention weight (selection of the rows that stay, then their copy).
#include <cuda_fp16.h>

#include "block_internal.h"
#include "common.cuh"

namespace gqa {
namespace {

// ------------------------------------------------------------------ codes

// The integer nearest to the exact quotient x / s (ties to even), within
// +-127; NaN gives 0. c = rint(x * (1/s)) is off by at most one and only
// beside a border; the remainder x - c s is exact in fp32 there (both are
// multiples of the smaller operand's last place, and it is at most about
// s / 2), so comparing it with s / 2 decides.
__device__ __forceinline__ int code_of(float x, float s, float inv) {
  if (x != x) return 0;
  const float q = inv < 3.0e38f ? x * inv : __fdiv_rn(x, s);   // 1/s overflows for a subnormal s
  float c = fminf(fmaxf(rintf(q), -127.f), 127.f);
  const float rem = fmaf(-c, s, x), two = 2.f * fabsf(rem);
  if (two > s || (two == s && ((int)c & 1))) c += copysignf(1.f, rem);
  return (int)fminf(fmaxf(c, -127.f), 127.f);
}

// The integer nearest to the exact code * from / to (ties to even), from <=
// to. ratio is fp32(from / to): the product is within 2e-5 of the quotient, so
// only one that close to a border needs the 64-bit quotient (exact enough:
// a quotient that is no tie misses the border by more than 2^-34).
__device__ __forceinline__ int recode(int code, float from, float to, float ratio) {
  const float q = (float)code * ratio;
  const float c = rintf(q);
  if (fabsf(fabsf(q - c) - 0.5f) > 4e-5f) return (int)c;
  return (int)rint((double)code * (double)from / (double)to);
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
      char4* old = reinterpret_cast<char4*>(codes + (long long)first * p.H);
      for (int i = tid; i < (past - first) * p.H / 4; i += kAppendThreads) {
        char4 c = old[i];
        c.x = (signed char)recode(c.x, s0, s, ratio);
        c.y = (signed char)recode(c.y, s0, s, ratio);
        c.z = (signed char)recode(c.z, s0, s, ratio);
        c.w = (signed char)recode(c.w, s0, s, ratio);
        old[i] = c;
      }
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
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e >> 2] |= (uint32_t)(code_of(f[e], s, inv) & 0xff) << (8 * (e & 3));
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

// One (b, g) per CTA. A radix selection (four passes of eight bits from the
// top) finds the key of the last row that stays and how many rows with
// exactly that key do; a scan in row order then writes the indices.
__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const EvictParams p) {
  const int bg = blockIdx.x, b = bg / p.Nkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int total = p.seqlens[b] + 1;
  if (total < 0 || total > p.C || total > p.T) {
    if (bg % p.Nkv == 0 && tid == 0 && p.status) atomicOr(p.status, GQA_DEVICE_BAD_SEQLEN_BIT);
    return;
  }
  int* kept = p.kept + (long long)bg * p.keep;
  const int stay = min(total, p.keep);
  if (bg % p.Nkv == 0 && tid == 0) p.seqlens_to[b] = stay - 1;
  if (total <= p.keep) {
    for (int i = tid; i < p.keep; i += kSelThreads) kept[i] = i < total ? i : -1;
    return;
  }
  const float* w = p.w + (long long)bg * p.C;
  const int lo = p.first, hi = total - p.recent;
  int need = p.keep - p.first - p.recent;   // of the rows [lo, hi); need < hi - lo
  __shared__ int hist[256];
  __shared__ unsigned s_digit;
  __shared__ int s_need;
  unsigned prefix = 0, mask = 0;
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int j0 = lo; j0 < hi; j0 += kSelThreads) {
        const int j = j0 + tid;
        unsigned key = 0;
        bool in = j < hi;
        if (in) {
          key = weight_key(w[j]);
          in = (key & mask) == prefix;
        }
        // lanes with the same digit count as one (the top digits of attention weights hardly differ)
        const unsigned digit = in ? (key >> shift) & 255u : 256u;
        const unsigned same = __match_any_sync(0xffffffffu, digit);
        if (in && lane == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
      }
      __syncthreads();
      if (warp == 0) {   // from the top digit down: the one at which `need` rows are reached
        int n8 = 0;
        for (int i = 0; i < 8; ++i) n8 += hist[255 - (8 * lane + i)];
        int incl = n8;
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        int before = incl - n8;
        if (before < need && incl >= need) {
          for (int i = 0; i < 8; ++i) {
            const int d = 255 - (8 * lane + i), c = hist[d];
            if (before + c >= need) {
              s_digit = (unsigned)d;
              s_need = need - before;
              break;
            }
            before += c;
          }
        }
      }
      __syncthreads();
      prefix |= s_digit << shift;
      mask |= 255u << shift;
      need = s_need;
      __syncthreads();
    }
  }
  // need rows with key == prefix stay (the lowest indices), and all above it.
  for (int i = tid; i < p.first; i += kSelThreads) kept[i] = i;
  for (int i = tid; i < p.recent; i += kSelThreads) kept[p.keep - p.recent + i] = hi + i;
  if (p.keep == p.first + p.recent) return;
  __shared__ int wsum[2][kSelThreads / 32];
  int out = p.first, ties = 0;   // rows written, rows of the border key seen
  for (int j0 = lo; j0 < hi; j0 += kSelThreads) {
    const int j = j0 + tid;
    const unsigned key = j < hi ? weight_key(w[j]) : 0u;
    const bool above = j < hi && key > prefix, tie = j < hi && key == prefix;
    const unsigned ma = __ballot_sync(0xffffffffu, above), mt = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) {
      wsum[0][warp] = __popc(ma);
      wsum[1][warp] = __popc(mt);
    }
    __syncthreads();
    int a_before = 0, t_before = 0, a_all = 0, t_all = 0;
    {   // every warp scans the 32 warp counts
      const int va = wsum[0][lane], vt = wsum[1][lane];
      int ia = va, it = vt;
      for (int o = 1; o < 32; o <<= 1) {
        const int xa = __shfl_up_sync(0xffffffffu, ia, o), xt = __shfl_up_sync(0xffffffffu, it, o);
        if (lane >= o) {
          ia += xa;
          it += xt;
        }
      }
      a_before = __shfl_sync(0xffffffffu, ia - va, warp);
      t_before = __shfl_sync(0xffffffffu, it - vt, warp);
      a_all = __shfl_sync(0xffffffffu, ia, 31);
      t_all = __shfl_sync(0xffffffffu, it, 31);
    }
    const unsigned below = (1u << lane) - 1u;
    const int t_rank = ties + t_before + __popc(mt & below);
    const int t_taken = min(t_rank, need);               // border rows before this one that stay
    if (above || (tie && t_rank < need))
      kept[out + a_before + __popc(ma & below) + t_taken - min(ties, need)] = j;
    out += a_all + min(ties + t_all, need) - min(ties, need);
    ties += t_all;
    __syncthreads();
  }
}

// ------------------------------------------------------------------ eviction: the copy

constexpr int kGatherThreads = 256;

// One block of tokens of one (b, g) of the new cache, K (z = 0) or V (z = 1):
// the largest source scale of its rows, then every row's codes, 16 at a time,
// rounded anew where the row's own scale is smaller. One read and one write of
// each kept row; the bound is HBM.
__global__ void __launch_bounds__(kGatherThreads)
evict_gather_kernel(const EvictParams p) {
  const int bg = blockIdx.y, b = bg / p.Nkv, tid = threadIdx.x;
  const int total = p.seqlens[b] + 1;
  if (total < 0 || total > p.C || total > p.T) return;
  const int stay = min(total, p.keep), bs = 1 << p.bs_log2;
  const int first = (int)blockIdx.x << p.bs_log2, n = min(bs, stay - first);
  if (n <= 0) return;
  const bool isv = blockIdx.z == 1;
  const int8_t* from = (isv ? p.vc : p.kc) + (long long)bg * p.C * p.H;
  const float* sc = (isv ? p.vs : p.ks) + (long long)bg * p.nblk;
  int8_t* to = (isv ? p.vc_to : p.kc_to) + ((long long)bg * p.Cto + first) * p.H;
  __shared__ int row[256];
  __shared__ float rs[256];
  __shared__ float red[kGatherThreads / 32];
  float top = 0.f;
  if (tid < n) {
    const int r = p.kept[(long long)bg * p.keep + first + tid];
    row[tid] = r;
    rs[tid] = top = sc[r >> p.bs_log2];
    if (!isv && p.w_to) p.w_to[(long long)bg * p.Cto + first + tid] = p.w[(long long)bg * p.C + r];
  }
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) red[tid >> 5] = top;
  __syncthreads();
  top = red[0];
  for (int i = 1; i < kGatherThreads / 32; ++i) top = fmaxf(top, red[i]);
  if (tid == 0) (isv ? p.vs_to : p.ks_to)[(long long)bg * p.nblk_to + blockIdx.x] = top;
  const int chunks = p.H / 16;
  for (int i = tid; i < n * chunks; i += kGatherThreads) {
    const int r = i / chunks, c = i - r * chunks;
    uint4 w = *reinterpret_cast<const uint4*>(from + (long long)row[r] * p.H + 16 * c);
    const float s = rs[r];
    if (s != top) {
      const float ratio = top > 0.f ? __fdiv_rn(s, top) : 0.f;
      uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t o = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o |= (uint32_t)(recode((int)(int8_t)(v[k] >> (8 * e)), s, top, ratio) & 0xff) << (8 * e);
        v[k] = o;
      }
      w = make_uint4(v[0], v[1], v[2], v[3]);
    }
    *reinterpret_cast<uint4*>(to + (long long)r * p.H + 16 * c) = w;
  }
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
  evict_select_kernel<<<(unsigned)(p.B * p.Nkv), kSelThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_evict_gather(const EvictParams& p, cudaStream_t st) {
  const int rows = p.keep < p.T ? p.keep : p.T, bs = 1 << p.bs_log2;
  evict_gather_kernel<<<dim3((unsigned)((rows + bs - 1) / bs), (unsigned)(p.B * p.Nkv), 2), kGatherThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace gqa
