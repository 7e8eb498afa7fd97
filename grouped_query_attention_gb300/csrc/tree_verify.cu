// Verification of drafted tokens, and the move of the accepted cache rows.
//
// Verification. A node's tests need single probabilities only, and the tokens
// that were turned down leave the target's row as max(a p - b q, 0) with two
// scalars, a = 1 / (Z_1 .. Z_k), b = sum of the products that scale each q: no
// row is ever stored. What has to be read is the row of the node where the path
// ends (and one row more for every test that failed on the way): the sum of it,
// and the place where the running sum passes u sum. A cluster of CTAs takes a
// sequence, each warp an equal run of the vocabulary; the warps' sums travel
// through distributed shared memory, every CTA adds them in the same order and
// takes the same decisions, and the warp that holds the place looks it up.
// Without draft probabilities r is p without the tokens turned down.
//
// The token has to be exact, so the sums may not move the place: values and sums
// are pairs of floats (48 bits; the difference of two floats is exact), as 64-bit
// arithmetic runs at 1/64 of the rate here; single values use 64 bits.
//
// Bound: latency (a few dependent loads, one pass over a row, two cluster
// barriers).
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "tree_internal.h"

namespace gqa {
namespace {

namespace cg = cooperative_groups;

constexpr int kVThreads = 512, kVWarps = kVThreads / 32;
constexpr int kVMaxCluster = 8;

// A sum of floats as a pair: hi + lo, |lo| at most half a step of hi.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), x = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, x)), __fsub_rn(b, x))};
}
__device__ __forceinline__ Pair quick(float a, float b) {   // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair s = two_sum(a.hi, b.hi);
  const Pair e = two_sum(a.lo, b.lo);
  s = quick(s.hi, __fadd_rn(s.lo, e.hi));
  return quick(s.hi, __fadd_rn(s.lo, e.lo));
}
__device__ __forceinline__ Pair mul(Pair a, float b) {
  const float h = __fmul_rn(a.hi, b);
  return quick(h, __fmaf_rn(a.lo, b, __fmaf_rn(a.hi, b, -h)));
}
__device__ __forceinline__ double value(Pair a) { return (double)a.hi + (double)a.lo; }
__device__ __forceinline__ Pair pair_of(double x) {
  const float h = (float)x;
  return {h, (float)(x - (double)h)};
}
__device__ __forceinline__ Pair shfl_xor(Pair a, int o) {
  return {__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
}
__device__ __forceinline__ Pair shfl_up(Pair a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
}
// a > b
__device__ __forceinline__ bool above(Pair a, Pair b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }

// Probabilities as the definition reads them.
__device__ __forceinline__ float proper(float p) { return p > 0.f && p < INFINITY ? p : 0.f; }
template <bool HALF>
__device__ __forceinline__ float prob(const void* base, long long i) {
  if constexpr (HALF) return proper(__half2float(static_cast<const __half*>(base)[i]));
  return proper(static_cast<const float*>(base)[i]);
}

// What is left of a row: max(a p - b q, 0), or p without `n` tokens.
struct Left {
  int node, round;   // round 0: p itself
  double a, b;
  int turned;        // tokens of Ctl::gone (no draft probabilities)
};

template <bool HALF>
struct Row {
  const void *p, *q;   // tensors; q null: no draft probabilities
  long long at;        // of the row's first element
  long long V;
  int off;             // of it in its group of four
  // Elements 4 k - off .. of the row; those outside it read 0.
  __device__ __forceinline__ static float4 four(const void* base, long long at, long long V, int off, long long k) {
    const long long v = 4 * k - off;
    if (v >= 0 && v + 4 <= V) {
      if constexpr (HALF) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __half*>(base) + at + v);
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
        return make_float4(proper(x.x), proper(x.y), proper(y.x), proper(y.y));
      } else {
        const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at + v);
        return make_float4(proper(w.x), proper(w.y), proper(w.z), proper(w.w));
      }
    }
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = v + e >= 0 && v + e < V ? prob<HALF>(base, at + v + e) : 0.f;
    return make_float4(x[0], x[1], x[2], x[3]);
  }
};

struct Ctl {
  int parent[kTreeNodes];
  int token[kTreeNodes];
  float p[kTreeNodes], q[kTreeNodes], u[kTreeNodes];   // of the node's token in its parent's rows; its uniform
  int path[kTreeNodes];
  int gone[kTreeNodes];              // tokens turned down at the current node
  Pair warp_sum[kVWarps];            // of this CTA (read by the cluster)
  Pair all_sum[kVWarps * kVMaxCluster];
  Left left;
  double z;
  int command, path_len, last;
};
enum { kSum = 1, kDraw = 2 };

// Four elements of what is left, from v = 4 k - off on.
template <bool HALF>
__device__ __forceinline__ void left_of(const Row<HALF>& row, const Left& f, Pair a, Pair b, const int* gone, long long k,
                                        Pair* r) {
  const float4 p4 = Row<HALF>::four(row.p, row.at, row.V, row.off, k);
  const float pv[4] = {p4.x, p4.y, p4.z, p4.w};
  if (f.round == 0 || !row.q) {
    const int v = (int)(4 * k - row.off);
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = {pv[e], 0.f};
    for (int x = 0; x < f.turned; ++x) {
      const int d = gone[x] - v;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (d == e) r[e].hi = 0.f;
    }
    return;
  }
  const float4 q4 = Row<HALF>::four(row.q, row.at, row.V, row.off, k);
  const float qv[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    Pair d;
    if (f.round == 1) {   // a = b = 1: exact
      d = two_sum(pv[e], -qv[e]);
    } else {
      const Pair x = mul(a, pv[e]), y = mul(b, qv[e]);
      d = add(x, {-y.hi, -y.lo});
    }
    r[e] = d.hi > 0.f ? d : Pair{0.f, 0.f};
  }
}

template <bool HALF>
__global__ void __launch_bounds__(kVThreads)
tree_verify_kernel(const VerifyParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ Ctl c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int b = blockIdx.x / ranks;
  const int n = p.new_lens ? p.new_lens[b] : p.S;
  int* path = p.path + (long long)b * p.S;
  if (n <= 0 || n > p.S) {   // the whole cluster
    if (rank == 0) {
      for (int i = tid; i < p.S; i += kVThreads) path[i] = -1;
      if (tid == 0) {
        p.path_lens[b] = 0;
        p.next[b] = -1;
        if (n != 0 && p.status) atomicOr(p.status, GQA_DEVICE_BAD_SEQLEN_BIT);
      }
    }
    return;
  }
  // ---- every node's single values
  bool bad = false;
  for (int i = tid; i < n; i += kVThreads) {
    const int par = tree_parent(p.parents[(long long)b * p.parents_ld + i], i, &bad);
    const int tok = p.tokens[(long long)b * p.S + i];
    const bool on = par >= 0 && tok >= 0 && tok < p.V;
    const long long at = on ? ((long long)b * p.S + par) * p.V + tok : 0;
    c.parent[i] = i == 0 ? -1 : par;
    c.token[i] = tok;
    c.p[i] = on ? prob<HALF>(p.target, at) : 0.f;
    c.q[i] = !p.draft ? 1.f : on ? prob<HALF>(p.draft, at) : 0.f;
    c.u[i] = p.accept_u[(long long)b * p.S + i];
  }
  if (__syncthreads_or(bad) && tid == 0 && rank == 0 && p.status) atomicOr(p.status, GQA_DEVICE_BAD_TREE_BIT);
  if (tid == 0) {
    c.left = {0, 0, 1.0, 0.0, 0};
    c.z = 1.0;
    c.path[0] = 0;
    c.path_len = 1;
    c.last = 0;
  }
  bool summed = false;   // warp sums of what is left are at hand
  __syncthreads();
  while (true) {
    // ---- tests, until one fails or no child is left (warp 0)
    if (warp == 0) {
      Left f = c.left;
      double z = c.z;
      int last = c.last, len = c.path_len, command = kDraw;
      while (true) {
        int next = n;   // the next child of f.node behind node `last`
        for (int i = last + 1; i < n; i += 32) {
          const unsigned m = __ballot_sync(0xffffffffu, i + lane < n && c.parent[i + lane] == f.node);
          if (m) {
            next = i + __ffs(m) - 1;
            break;
          }
        }
        if (next >= n) break;
        last = next;
        const double pv = c.p[next], qv = c.q[next], uv = c.u[next];
        double r = pv;
        if (f.round > 0) {
          if (p.draft) {
            r = f.a * pv - f.b * qv;
          } else {
            bool dup = false;
            for (int x = lane; x < f.turned; x += 32) dup |= c.gone[x] == c.token[next];
            if (__any_sync(0xffffffffu, dup)) r = 0.0;
          }
        }
        if (z > 0.0 && uv * qv * z < r) {
          f = {next, 0, 1.0, 0.0, 0};
          z = 1.0;
          if (lane == 0) c.path[len] = next;
          ++len;
          summed = false;
          continue;
        }
        // turned down: r <- max(r / z - q, 0), whose sum is due
        if (p.draft) {
          if (z > 0.0) {   // (nothing left: it stays so)
            f.a = f.a / z;
            f.b = f.b / z + 1.0;
          }
        } else {
          if (lane == 0) c.gone[f.turned] = c.token[next];
          ++f.turned;
        }
        ++f.round;
        command = kSum;
        break;
      }
      if (lane == 0) {
        c.left = f;
        c.z = z;
        c.last = last;
        c.path_len = len;
        // (2: what warp 0 knows about the sums, for everybody)
        c.command = command | (summed ? 4 : 0);
      }
    }
    __syncthreads();
    const int command = c.command & 3;
    summed = (c.command & 4) != 0;
    Left f = c.left;
    if (command == kDraw && summed && !(c.z > 0.0)) {   // nothing left: the target's own row
      f.round = 0;
      f.turned = 0;
      summed = false;
    }
    const long long row_at = ((long long)b * p.S + f.node) * p.V;
    const Row<HALF> row = {p.target, p.draft, row_at, p.V, (int)(row_at & 3)};
    const long long groups = (p.V + row.off + 3) >> 2;          // of four elements
    const int warps = ranks * kVWarps;
    const long long run = ((groups + warps - 1) / warps + 31) / 32 * 32;   // of a warp
    const long long g0 = (rank * kVWarps + warp) * run;
    const Pair a = pair_of(f.a), bb = pair_of(f.b);
    if (command == kSum || !summed) {
      // ---- the sum of what is left, and every warp's part of it
      Pair s = {0.f, 0.f};
      for (long long k = g0 + lane; k < min(g0 + run, groups); k += 32) {
        Pair r[4];
        left_of<HALF>(row, f, a, bb, c.gone, k, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) s = add(s, r[e]);
      }
      for (int o = 16; o; o >>= 1) s = add(s, shfl_xor(s, o));
      if (lane == 0) c.warp_sum[warp] = s;
      cluster.sync();
      if (tid < warps) c.all_sum[tid] = *cluster.map_shared_rank(&c.warp_sum[tid % kVWarps], tid / kVWarps);
      cluster.sync();   // nobody writes the next sums, or leaves, before these are read
      if (warp == 0) {
        Pair z = {0.f, 0.f};
        for (int x = lane; x < warps; x += 32) z = add(z, c.all_sum[x]);
        for (int o = 16; o; o >>= 1) z = add(z, shfl_xor(z, o));
        if (lane == 0) c.z = value(z);
      }
      summed = true;
      __syncthreads();
      if (command == kSum) continue;
    }
    // ---- the draw
    const double z = c.z;
    if (!(z > 0.0)) {
      if (rank == 0 && tid == 0) {
        p.next[b] = -1;
        if (p.status) atomicOr(p.status, GQA_DEVICE_BAD_PROBS_BIT);
      }
    } else {
      // The warp's run that holds the place, by every warp 0 alike.
      if (warp == 0) {
        const Pair goal = pair_of((double)p.sample_u[b] * z);
        Pair before = {0.f, 0.f};
        int at = -1, filled = -1;
        Pair start = before;
        for (int x0 = 0; x0 < warps && at < 0; x0 += 32) {
          const Pair own = x0 + lane < warps ? c.all_sum[x0 + lane] : Pair{0.f, 0.f};
          Pair s = own;
          for (int o = 1; o < 32; o <<= 1) {
            const Pair v = shfl_up(s, o);
            if (lane >= o) s = add(v, s);
          }
          s = add(before, s);
          const unsigned hit = __ballot_sync(0xffffffffu, own.hi > 0.f && above(s, goal));
          const unsigned any = __ballot_sync(0xffffffffu, own.hi > 0.f);
          // sums before each run
          Pair prev = shfl_up(s, 1);
          if (lane == 0) prev = before;
          const int pick = hit ? __ffs(hit) - 1 : any ? 31 - __clz(any) : 0;
          if (hit || any) {
            filled = x0 + pick;
            start.hi = __shfl_sync(0xffffffffu, prev.hi, pick);
            start.lo = __shfl_sync(0xffffffffu, prev.lo, pick);
          }
          if (hit) at = x0 + pick;
          before.hi = __shfl_sync(0xffffffffu, s.hi, 31);
          before.lo = __shfl_sync(0xffffffffu, s.lo, 31);
        }
        if (at < 0) at = filled;   // a number of 1 or more, or a rounding at the very end
        if (at / kVWarps == rank) {
          const long long b0 = (long long)at * run;
          int token = -1, spare = -1;
          Pair sum = start;
          for (long long k0 = b0; k0 < min(b0 + run, groups) && token < 0; k0 += 32) {
            Pair r[4];
            const bool on = k0 + lane < groups;
            if (on) left_of<HALF>(row, f, a, bb, c.gone, k0 + lane, r);
            else r[0] = r[1] = r[2] = r[3] = {0.f, 0.f};
            Pair s = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 4; ++e) s = add(s, r[e]);
            const Pair own = s;
            for (int o = 1; o < 32; o <<= 1) {
              const Pair v = shfl_up(s, o);
              if (lane >= o) s = add(v, s);
            }
            const Pair incl = add(sum, s);
            const unsigned hit = __ballot_sync(0xffffffffu, own.hi > 0.f && above(incl, goal));
            const unsigned any = __ballot_sync(0xffffffffu, own.hi > 0.f);
            Pair prev = shfl_up(incl, 1);
            if (lane == 0) prev = sum;
            const int pick = hit ? __ffs(hit) - 1 : any ? 31 - __clz(any) : -1;
            int found = -1, positive = -1;
            if (lane == pick) {   // the element within the four
              Pair run_sum = prev;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                run_sum = add(run_sum, r[e]);
                if (r[e].hi > 0.f) {
                  const int v = (int)(4 * (k0 + lane) - row.off) + e;
                  positive = v;
                  if (found < 0 && above(run_sum, goal)) found = v;
                }
              }
            }
            if (pick >= 0) {
              found = __shfl_sync(0xffffffffu, found, pick);
              positive = __shfl_sync(0xffffffffu, positive, pick);
              spare = positive;
              if (hit) token = found >= 0 ? found : positive;
            }
            sum.hi = __shfl_sync(0xffffffffu, incl.hi, 31);
            sum.lo = __shfl_sync(0xffffffffu, incl.lo, 31);
          }
          if (lane == 0) p.next[b] = token >= 0 ? token : spare;
        }
      }
    }
    break;
  }
  if (rank == 0) {
    const int len = c.path_len;
    for (int i = tid; i < p.S; i += kVThreads) path[i] = i < len ? c.path[i] : -1;
    if (tid == 0) p.path_lens[b] = len;
  }
}

// ------------------------------------------------------------------ accepted rows

constexpr int kAThreads = 128;
constexpr int kAhead = 8;   // rows of a thread under way

// A thread owns one 16-byte column of a (cache, sequence, KV head) and moves its
// rows in order. A path increases, so row path[i] >= i, and what a group of rows
// writes lies below everything later groups read.
__global__ void __launch_bounds__(kAThreads)
tree_accept_kernel(const AcceptParams p) {
  __shared__ short path[kTreeNodes];
  const int b = blockIdx.y, tid = threadIdx.x;
  const int n = p.new_lens ? p.new_lens[b] : p.S, total = p.seqlens[b] + 1, len = p.path_lens[b];
  const bool lengths = n >= 0 && n <= p.S && total >= n && total <= p.C && len >= 0 && len <= n;
  bool bad = false;
  if (lengths)
    for (int i = tid; i < len; i += kAThreads) {
      const int x = p.path[(long long)b * p.S + i], before = i > 0 ? p.path[(long long)b * p.S + i - 1] : -1;
      bad |= x <= before || x >= n || x < 0;
      path[i] = (short)x;
    }
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && tid == 0) {
    p.into_seqlens[b] = lengths && !bad ? total - n + len - 1 : -1;
    if (p.status && (!lengths || bad)) atomicOr(p.status, lengths ? GQA_DEVICE_BAD_TREE_BIT : GQA_DEVICE_BAD_SEQLEN_BIT);
  }
  if (!lengths || bad) return;
  const int cols = p.row_bytes / 16;
  const int x = blockIdx.x * kAThreads + tid;          // column, KV head, cache
  const int col = x % cols, g = x / cols % p.Nkv, cache = x / cols / p.Nkv;
  if (cache >= 2 * p.layers) return;
  uint4* rows = static_cast<uint4*>(p.cache[cache]) + (((long long)b * p.Nkv + g) * p.C + (total - n)) * cols + col;
  for (int i0 = 0; i0 < len; i0 += kAhead) {
    uint4 w[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k < len && path[i0 + k] != i0 + k) w[k] = rows[(long long)path[i0 + k] * cols];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k < len && path[i0 + k] != i0 + k) rows[(long long)(i0 + k) * cols] = w[k];
  }
}

template <bool HALF>
cudaError_t launch_verify(const VerifyParams& p, int ranks, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * ranks));
  cfg.blockDim = dim3(kVThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_verify_kernel<HALF>, p);
}

}  // namespace

cudaError_t launch_tree_verify(const VerifyParams& p, cudaStream_t st) {
  const int ranks = p.V <= 4096 ? 1 : p.V <= 16384 ? 4 : kVMaxCluster;
  return p.half ? launch_verify<true>(p, ranks, st) : launch_verify<false>(p, ranks, st);
}

cudaError_t launch_tree_accept(const AcceptParams& p, cudaStream_t st) {
  const long long columns = 2LL * p.layers * p.Nkv * (p.row_bytes / 16);
  const dim3 grid((unsigned)((columns + kAThreads - 1) / kAThreads), (unsigned)p.B);
  tree_accept_kernel<<<grid, kAThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace gqa
