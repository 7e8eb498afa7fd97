// Rotary embedding whose pairs take their angles from several position axes,
// with the optional RMS norm of the query and key rows before it.
//
//   y[d] = x[d] c - x[d+D] s,  y[d+D] = x[d+D] c + x[d] s,
//   c, s = cos / sin table [positions[axis(d)][token]][d],  d < D <= H/2.
//
// Every row is read and written once, so the bound is HBM. A group of
// LPR = H/16 lanes (rounded up to a power of two) holds one row, lane l the
// pairs 8 l .. 8 l + 7 (both halves, so a pair never leaves its lane) or 16
// coordinates behind the rotated part. The angles depend on the token alone:
// a warp loads its eight cosines and sines per lane once and runs over heads
// of that token with them in registers. 4 x 4096 tokens of 32 + 8 heads of 128,
// fp16 with norm (340 MB): 65 us, 5.2 TB/s; with three blocks an SM instead of
// four 70, with one coordinate an instruction 72. fp32 rows need the registers
// of three (12 + 4 heads of 96, 3 x 1025 tokens: 13 to 14 us against 15.7).
#include <cuda_fp16.h>

#include "block_internal.h"
#include "common.cuh"

namespace gqa {
namespace {

template <typename T>
struct Vec8;  // eight consecutive T values as raw 16-byte words
template <>
struct Vec8<__half> {
  uint4 w;
  __device__ void load(const __half* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ void get(float* f) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
      f[2 * i] = a.x;
      f[2 * i + 1] = a.y;
    }
  }
  static __device__ void store(__half* p, const float* f) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      v[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ void store(float* p, const float* f) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// Packed product, each lane rounded as __fmul_rn does.
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  unsigned long long av = *reinterpret_cast<unsigned long long*>(&a);
  unsigned long long bv = *reinterpret_cast<unsigned long long*>(&b);
  unsigned long long dv;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(dv) : "l"(av), "l"(bv));
  return *reinterpret_cast<float2*>(&dv);
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// Eight table values of this lane's pairs for one token.
template <typename TT>
__device__ __forceinline__ void load_table(const RotaryAxesParams& p, const void* table, int l, const int* row,
                                           float* out) {
  const TT* t = static_cast<const TT*>(table);
  if (p.chunk_uniform[l]) {
    Vec8<TT> v;
    v.load(t + (long long)row[0] * p.pairs + 8 * l);
    v.get(out);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = to_f(t[(long long)row[e] * p.pairs + 8 * l + e]);
  }
}

// LPR lanes per row; the warp's rows are consecutive heads (queries first,
// then keys) of one token, `per_item` passes of them.
template <typename T, int LPR>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 3)
rotary_axes_kernel(const RotaryAxesParams p, int per_item, int items_per_token, long long items) {
  constexpr int kRows = 32 / LPR;
  const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (item >= items) return;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const long long tok = item / items_per_token;
  const int h0 = (int)(item % items_per_token) * per_item * kRows;
  const int heads = p.N + (p.k ? p.Nkv : 0);
  const bool lane_on = l < p.H / 16, rot = l < p.pairs / 8;

  float c[8], s[8];
  bool bad = false;
  if (rot) {
    int row[8];
    const unsigned ax = p.axis_nibbles[l];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      row[e] = p.pos[(long long)((ax >> (4 * e)) & 15u) * p.tokens + tok];
      bad |= row[e] < 0 || row[e] >= p.table_rows;
      if (bad) row[e] = 0;
    }
    if (p.table_f32) {
      load_table<float>(p, p.cos_c, l, row, c);
      load_table<float>(p, p.sin_c, l, row, s);
    } else {
      load_table<T>(p, p.cos_c, l, row, c);
      load_table<T>(p, p.sin_c, l, row, s);
    }
  }
  if (__any_sync(0xffffffffu, bad)) {   // the token is left unwritten
    if (lane == 0 && p.status) atomicOr(p.status, GQA_DEVICE_BAD_ROTARY_BIT);
    return;
  }
  // Coordinates of this lane: lo.. and hi.. (the two halves of its pairs).
  const int lo = rot ? 8 * l : 2 * p.pairs + 16 * (l - p.pairs / 8);
  const int hi = rot ? lo + p.pairs : lo + 8;

  // Rows of this token: head hh of the queries, hh - N of the keys.
  const long long q_at = tok * p.N * p.H, k_at = (tok * p.Nkv - p.N) * p.H;
  const T* q_in = static_cast<const T*>(p.q) + q_at;
  const T* k_in = static_cast<const T*>(p.k) + k_at;
  T* q_out = static_cast<T*>(p.qo) + q_at;
  T* k_out = static_cast<T*>(p.ko) + k_at;
  auto row_in = [&](int hh) { return (hh < p.N ? q_in : k_in) + hh * p.H; };
  Vec8<T> va, vb;
  int hh = h0 + sub;
  bool on = lane_on && hh < heads;
  if (on) {
    va.load(row_in(hh) + lo);
    vb.load(row_in(hh) + hi);
  }
  for (int it = 0; it < per_item; ++it) {
    if (h0 + it * kRows >= heads) break;   // uniform: the warp's rows are all past the last head
    float a[8], b[8];
    if (on) {
      va.get(a);
      vb.get(b);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = b[e] = 0.f;
    }
    const int cur = hh;
    const bool cur_on = on;
    hh += kRows;
    on = lane_on && it + 1 < per_item && hh < heads;
    if (on) {   // the next row's loads run while this one is computed
      va.load(row_in(hh) + lo);
      vb.load(row_in(hh) + hi);
    }
    float2 a2[4], b2[4];   // two coordinates an instruction; every lane rounds as the scalar forms do
    if (p.qw) {
      const T* w = static_cast<const T*>(cur < p.N ? p.qw : p.kw);
      float sa = sumsq8_rn(a), sb = sumsq8_rn(b);
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) {
        sa = __fadd_rn(sa, __shfl_xor_sync(0xffffffffu, sa, o));
        sb = __fadd_rn(sb, __shfl_xor_sync(0xffffffffu, sb, o));
      }
      const float rn = rms_inv_rn(__fadd_rn(sa, sb), p.H, p.eps);
      if (!cur_on) continue;
      Vec8<T> wa, wb;
      float fa[8], fb[8];
      wa.load(w + lo);
      wb.load(w + hi);
      wa.get(fa);
      wb.get(fb);
      const float2 rn2 = make_float2(rn, rn);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a2[e] = fmul2(fmul2(make_float2(a[2 * e], a[2 * e + 1]), rn2), make_float2(fa[2 * e], fa[2 * e + 1]));
        b2[e] = fmul2(fmul2(make_float2(b[2 * e], b[2 * e + 1]), rn2), make_float2(fb[2 * e], fb[2 * e + 1]));
      }
    } else {
      if (!cur_on) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a2[e] = make_float2(a[2 * e], a[2 * e + 1]);
        b2[e] = make_float2(b[2 * e], b[2 * e + 1]);
      }
    }
    if (rot) {
      const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 c2 = make_float2(c[2 * e], c[2 * e + 1]), s2 = make_float2(s[2 * e], s[2 * e + 1]);
        const float2 x = a2[e], y = b2[e];
        a2[e] = ffma2(fmul2(y, s2), minus, fmul2(x, c2));   // x c - y s: three roundings
        b2[e] = fadd2(fmul2(y, c2), fmul2(x, s2));
      }
    }
    T* o = (cur < p.N ? q_out : k_out) + cur * p.H;
    Vec8<T>::store(o + lo, reinterpret_cast<const float*>(a2));
    Vec8<T>::store(o + hi, reinterpret_cast<const float*>(b2));
  }
}

template <typename T, int LPR>
cudaError_t launch_one(const RotaryAxesParams& p, cudaStream_t st) {
  const int rows = 32 / LPR, heads = p.N + (p.k ? p.Nkv : 0);
  const int passes = (heads + rows - 1) / rows;
  // Few tokens: one pass per warp, so that a decode step's rows spread over
  // the SMs; many: all heads of a token in one warp, its angles loaded once.
  long long split = (152LL * 32 + p.tokens - 1) / p.tokens;
  if (split > passes) split = passes;
  const int per_item = (int)((passes + split - 1) / split);
  const int items_per_token = (passes + per_item - 1) / per_item;
  const long long items = p.tokens * items_per_token;
  const long long blocks = (items + 7) / 8;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  rotary_axes_kernel<T, LPR><<<(unsigned)blocks, 256, 0, st>>>(p, per_item, items_per_token, items);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RotaryAxesParams& p, cudaStream_t st) {
  const int lanes = p.H / 16;
  if (lanes <= 1) return launch_one<T, 1>(p, st);
  if (lanes <= 2) return launch_one<T, 2>(p, st);
  if (lanes <= 4) return launch_one<T, 4>(p, st);
  if (lanes <= 8) return launch_one<T, 8>(p, st);
  return launch_one<T, 16>(p, st);
}

}  // namespace

cudaError_t launch_rotary_axes(const RotaryAxesParams& p, int t_type, cudaStream_t st) {
  return t_type == kF16 ? launch_t<__half>(p, st) : launch_t<float>(p, st);
}

}  // namespace gqa
