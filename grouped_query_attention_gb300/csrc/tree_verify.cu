// Verification of drafted tokens, and the move of the accepted cache rows.
//
// Verification. A node's tests need single probabilities only, and the tokens
// that were turned down leave the target's row as max(a p - b q, 0) with two
// scalars: no row is ever stored. What has to be read is the row of the node
// where the path ends, and once more for every test that failed on the way (from
// L1 then): the sum of what is left, and the place where the running sum passes
// u sum. A cluster of CTAs takes a sequence, each warp an equal run of the
// vocabulary; the warps write their sums to every CTA of the cluster, all of
// them add the sums in one order and take the same decisions, and the warp whose
// run holds the place looks it up, in three levels. Without draft probabilities
// r is p without the tokens turned down, whose sum needs no new pass.
//
// The token has to be exact, so the sums may not move the place: values and sums
// are pairs of floats (48 bits; the difference of two floats is exact), as 64-bit
// arithmetic runs at 1/64 of the rate here. a p - b q gives some of those bits away
// to the difference; a node where that comes to more than 8 (close drafts, turned
// down one behind the other) is worked out anew by the definition's own steps, from
// the sums of all rounds. It costs the passes once more and a step a round in
// each (16 sequences over 100003 tokens, nine drafts turned down: 61 us as usual,
// 174 where the target is certain of a token and the draft almost), at few nodes:
// drafts with logits 0.7 off stay below 5 bits for 12 rounds.
//
// What bounds it: the steps one behind the other. A pass over a row is loads, two
// dozen operations a pair of probabilities, a cluster barrier; every token turned
// down is one more pass, and the draw reads a warp's run again. 16 chains of 8 over
// 131072 tokens: 19 us for 14 MB (ncu); 16 trees of 64 nodes over 100003 37 us (in a
// graph). Clusters of 8 CTAs of 512 threads were the fastest (256 and 1024 threads, one CTA an SM,
// at most 152 or 608 CTAs: slower or the same).
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "tree_internal.h"

namespace gqa {
namespace {

namespace cg = cooperative_groups;

constexpr int kVThreads = 512, kVWarps = kVThreads / 32;
constexpr int kVMaxCluster = 8;
constexpr int kVMaxWarps = kVWarps * kVMaxCluster;

// A sum of floats as a pair: hi + lo, |lo| at most half a step of hi. (Knuth's sum of two numbers and its error, Dekker's
// for ordered ones and his double-length operations, products and their errors by fma.)
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
// (what the low parts' sum loses is 2^-48 of the whole)
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return quick(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Pair neg(Pair a) { return {-a.hi, -a.lo}; }
__device__ __forceinline__ Pair product(float a, float b) {   // exact
  const float h = __fmul_rn(a, b);
  return {h, __fmaf_rn(a, b, -h)};
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  const Pair h = product(a.hi, b.hi);
  return quick(h.hi, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, h.lo)));
}
__device__ __forceinline__ Pair reciprocal(Pair a) {
  const float x = __frcp_rn(a.hi);
  const float rest = __fmaf_rn(-x, a.lo, __fmaf_rn(-x, a.hi, 1.f));   // 1 - x a
  return quick(x, __fmul_rn(rest, x));
}
__device__ __forceinline__ Pair shfl_xor(Pair a, int o) {
  return {__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
}
__device__ __forceinline__ Pair shfl_up(Pair a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
}
// a > b
__device__ __forceinline__ bool above(Pair a, Pair b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }

// Probabilities as the definition reads them: numbers from 2^40 on are none, so that no sum of theirs overflows.
// (The bits of negative, infinite and NaN values lie above those of the positive ones.)
__device__ __forceinline__ float proper(float p) { return __float_as_uint(p) < 0x53800000u ? p : 0.f; }
template <bool HALF>
__device__ __forceinline__ float prob(const void* base, long long i) {
  if constexpr (HALF) return proper(__half2float(static_cast<const __half*>(base)[i]));
  return proper(static_cast<const float*>(base)[i]);
}

// What is left of a row behind `round` tokens turned down: max(a p - b q, 0), or by the definition's own steps, the
// sums of which are in Ctl::over (fine); without draft probabilities p without the tokens of Ctl::gone.
struct Left {
  int node, round, turned, fine;
  Pair a, b;
};
// a p - b q loses log2(a) bits to the difference, a = 1 / (Z_1 .. Z_k-1), and as many as the sum Z_k lies below 1. Where
// both come to more than 8 the definition's own steps take over: they divide every element by the sum of those very
// elements, so that what the row leaves, however little of it, goes on with its bits.
constexpr float kCoarse = 0x1p-8f;
// Products of numbers near the smallest float have no room for their low parts. All sums are of values times kUp: the
// smallest float is 2^-93 there, and a row's sum far below the largest. So are fine values.
constexpr float kUp = 0x1p56f;
__device__ __forceinline__ Pair raised(Pair a) { return {a.hi * kUp, a.lo * kUp}; }

template <bool HALF>
struct Row {
  const void *p, *q;   // tensors; q null: no draft probabilities
  long long at;        // of the row's first element
  long long V;
  int off;             // of it in its group of four
  // Groups 4 k - off .. of four elements; only those [first(), end()) lie within the row.
  __device__ __forceinline__ int first() const { return off > 0 ? 1 : 0; }
  __device__ __forceinline__ int end() const { return (int)((V + off) >> 2); }
  using Raw = typename std::conditional<HALF, uint2, float4>::type;
  __device__ __forceinline__ Raw raw(const void* base, int k) const {
    const long long v = at - off + 4LL * k;
    if constexpr (HALF) return *reinterpret_cast<const uint2*>(static_cast<const __half*>(base) + v);
    else return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + v);
  }
  __device__ __forceinline__ static float4 values(Raw w) {
    if constexpr (HALF) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
      return make_float4(proper(x.x), proper(x.y), proper(y.x), proper(y.y));
    } else {
      return make_float4(proper(w.x), proper(w.y), proper(w.z), proper(w.w));
    }
  }
  // The loads of group k (of its neighbour within the row, where it reaches over an end), and its values; elements
  // outside the row are 0.
  struct Loaded {
    Raw p, q;
  };
  __device__ __forceinline__ Loaded load(int k) const {
    Loaded x = {};
    if (end() > first()) {
      const int kk = min(max(k, first()), end() - 1);
      x.p = raw(p, kk);
      if (q) x.q = raw(q, kk);
    }
    return x;
  }
  __device__ __forceinline__ float4 four(const void* base, Raw w, int k) const {
    if (k >= first() && k < end()) return values(w);
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const long long v = 4LL * k - off + e;
      x[e] = prob<HALF>(base, at + min(max(v, 0LL), V - 1));
      if (v < 0 || v >= V) x[e] = 0.f;
    }
    return make_float4(x[0], x[1], x[2], x[3]);
  }
};

struct Ctl {
  int parent[kTreeNodes];
  int token[kTreeNodes];
  float p[kTreeNodes], q[kTreeNodes], u[kTreeNodes];   // of the node's token in its parent's rows; its uniform
  int path[kTreeNodes];
  int gone[kTreeNodes];              // tokens turned down at the current node
  Pair over[kTreeNodes];             // 1 / (Z kUp) of every round there (Left::fine); 0: nothing was left
  Pair sums[2][kVMaxWarps];          // of every warp of the cluster, two passes in turn
  Left left;
  int command, path_len;
  // the draw: the warp that holds the place (-1: no token), the sum before its run, what the running sum has to pass
  int at;
  Pair before, edge;
  Pair part[kVWarps];                // of the run's sixteenths
};
// What warp 0 asks for: the sum of the node's row as it is (no draft
// probabilities), the sum of what is left, or the draw from it; + 4: the sums
// of what is left are at hand.
enum { kWhole = 0, kSum = 1, kDraw = 2, kSummed = 4 };

// s += d (a value and what rounding left of it), as the sum and its error.
__device__ __forceinline__ void gather(Pair& s, Pair d) {
  const Pair t = two_sum(s.hi, d.hi);
  s.hi = t.hi;
  s.lo = __fadd_rn(s.lo, __fadd_rn(t.lo, d.lo));
}

// What is left of one element, a p - b q (exact for a = b = 1), as a value and what rounding left of it.
__device__ __forceinline__ Pair left_of(float p, float q, Pair a, Pair b) {
  const float x = __fmul_rn(a.hi, p), y = __fmul_rn(b.hi, q);
  const float xl = __fmaf_rn(a.lo, p, __fmaf_rn(a.hi, p, -x));
  const float yl = __fmaf_rn(b.lo, q, __fmaf_rn(b.hi, q, -y));
  Pair d = two_sum(x, -y);
  d.lo = __fadd_rn(d.lo, __fsub_rn(xl, yl));
  return __fadd_rn(d.hi, d.lo) > 0.f ? d : Pair{0.f, 0.f};
}

// ... by the definition's steps, r <- max(r / Z - q, 0), of a p and a q times kUp.
__device__ __noinline__ Pair left_fine(float p, float q, const Pair* over, int round) {
  Pair r = two_sum(p, -q);
  for (int j = 0; j + 1 < round && r.hi > 0.f; ++j) {
    const Pair t = raised(mul(r, over[j]));
    r = two_sum(t.hi, -q);
    r = two_sum(r.hi, __fadd_rn(r.lo, t.lo));
  }
  return r.hi > 0.f ? r : Pair{0.f, 0.f};
}

// ... of group k.
// (Not inlined, like the searches below: a call runs each place once, from cold instruction memory.)
template <bool HALF>
__device__ __noinline__ void left_of4(const Row<HALF>& row, typename Row<HALF>::Loaded in, const Left& f, const int* gone,
                                         int turned, int k, Pair* r) {
  const float4 p4 = row.four(row.p, in.p, k);
  const float pv[4] = {p4.x, p4.y, p4.z, p4.w};
  if (f.round == 0 || !row.q) {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = {pv[e], 0.f};
    for (int x = 0; x < turned; ++x) {
      const int d = gone[x] - (4 * k - row.off);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (d == e) r[e].hi = 0.f;
    }
    return;
  }
  const float4 q4 = row.four(row.q, in.q, k);
  const float qv[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    r[e] = left_of(pv[e], qv[e], f.a, f.b);
    r[e] = quick(r[e].hi, r[e].lo);
  }
}
// ... by the definition's steps. (On its own: few calls come here, and the one above stays without calls.)
template <bool HALF>
__device__ __noinline__ void left_fine4(const Row<HALF>& row, typename Row<HALF>::Loaded in, const Left& f, const Ctl& c, int k,
                                        Pair* r) {
  const float4 p4 = row.four(row.p, in.p, k), q4 = row.four(row.q, in.q, k);
  const float pv[4] = {p4.x, p4.y, p4.z, p4.w}, qv[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll 1
  for (int e = 0; e < 4; ++e) r[e] = left_fine(pv[e] * kUp, qv[e] * kUp, c.over, f.round);
}

// Sum of what is left of groups g0 + lane, + 32, .. within [first, k1), in four
// chains, without the turns in `skip` (a bit stands for 2^fold of them). A turn's loads are all under way before the
// first is looked at (with a condition around each they came one by one).
template <bool HALF, bool DRAFT>
__device__ __forceinline__ void sum_run(const Row<HALF>& row, const Left& f, int g0, int first, int k1, unsigned long long skip, int fold,
                                        Pair* s) {
  constexpr int kGroups = 2;   // (3 or 4: the same or slower, as more instructions come from cold memory)
  if (first >= k1) return;
  for (int k = g0 + (threadIdx.x & 31); k < k1; k += 32 * kGroups) {
    typename Row<HALF>::Raw pr[kGroups], qr[kGroups];
#pragma unroll
    for (int x = 0; x < kGroups; ++x) {
      const int kx = min(max(k + 32 * x, first), k1 - 1);
      pr[x] = row.raw(row.p, kx);
      if constexpr (DRAFT) qr[x] = row.raw(row.q, kx);
    }
#pragma unroll
    for (int x = 0; x < kGroups; ++x) {
      const float4 pv = Row<HALF>::values(pr[x]);
      float4 qv = pv;
      if constexpr (DRAFT) qv = Row<HALF>::values(qr[x]);
      const int kx = k + 32 * x;
      bool on = kx >= first && kx < k1;
      if constexpr (!DRAFT) on = on && !(skip >> ((kx - g0) >> fold & 63) & 1u);
      const float pe[4] = {pv.x, pv.y, pv.z, pv.w}, qe[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p1 = on ? pe[e] : 0.f;
        if constexpr (DRAFT) gather(s[e], left_of(p1, qe[e], f.a, f.b));
        else gather(s[e], {p1, 0.f});
      }
    }
    // (A low part that grew with the run would round ever more of itself away.)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = quick(s[e].hi, s[e].lo);
  }
}

// ... of groups g0 + lane, + 32, .. below k1 one by one, the row's ends among them (Left::fine).
template <bool HALF>
__device__ __noinline__ Pair sum_fine(const Row<HALF>& row, const Left& f, const Ctl& c, int g0, int k1) {
  Pair s = {0.f, 0.f};
  for (int k = g0 + (threadIdx.x & 31); k < k1; k += 32) {
    Pair r[4];
    left_fine4<HALF>(row, row.load(k), f, c, k, r);
    s = add(s, add(add(r[0], r[1]), add(r[2], r[3])));
  }
  return s;
}

__device__ __forceinline__ Pair warp_sum(Pair s) {
#pragma unroll
  for (int o = 16; o; o >>= 1) s = add(s, shfl_xor(s, o));
  return s;
}
// Sum over the lanes up to this one.
__device__ __forceinline__ Pair warp_scan(Pair s) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair v = shfl_up(s, o);
    if (lane >= o) s = add(v, s);
  }
  return s;
}

// One level of the search for the place where the running sum passes `goal`:
// the first lane whose part does (*before becomes the sum before it), or, if
// none does, the last lane with something (*spare) and -1. All of a warp.
__device__ __noinline__ int find_lane(Pair own, Pair goal, Pair* before, int* spare) {
  const Pair upto = add(*before, warp_scan(own));
  const unsigned some = __ballot_sync(0xffffffffu, own.hi > 0.f);
  const unsigned hit = __ballot_sync(0xffffffffu, own.hi > 0.f && above(upto, goal));
  *spare = some ? 31 - __clz(some) : -1;
  const int at = hit ? __ffs(hit) - 1 : -1;
  const int take = hit ? at : 31;   // without a hit: all of it
  Pair prev = shfl_up(upto, 1);
  if ((threadIdx.x & 31) == 0) prev = *before;
  const Pair x = hit ? prev : upto;
  before->hi = __shfl_sync(0xffffffffu, x.hi, take);
  before->lo = __shfl_sync(0xffffffffu, x.lo, take);
  return at;
}

template <bool HALF>
__global__ void __launch_bounds__(kVThreads, 2)
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
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  // ---- every node's single values
  bool bad = false;
  for (int i = tid; i < n; i += kVThreads) {
    const int par = tree_parent(p.parents[(long long)b * p.parents_ld + i], i, &bad);
    const int tok = p.tokens[(long long)b * p.S + i];
    const float u = p.accept_u[(long long)b * p.S + i];
    const bool on = par >= 0 && tok >= 0 && tok < p.V;
    const long long at = on ? ((long long)b * p.S + par) * p.V + tok : 0;
    c.parent[i] = i == 0 ? -1 : par;
    c.token[i] = tok;
    c.p[i] = on ? prob<HALF>(p.target, at) : 0.f;
    c.q[i] = !p.draft ? 1.f : on ? prob<HALF>(p.draft, at) : 0.f;
    c.u[i] = u;
  }
  if (__syncthreads_or(bad) && tid == 0 && rank == 0 && p.status) atomicOr(p.status, GQA_DEVICE_BAD_TREE_BIT);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // every CTA has begun: its memory may be written

  const int warps = ranks * kVWarps;
  // Warp 0's state: what is left at the path's last node, its sum z, the node tested last. (What does not fit beside a
  // pass's registers is kept in shared memory: a, b of Left and the sums of Ctl::over.)
  int node = 0, round = 0, turned_down = 0;
  int fine = 0;                             // Left::fine: the rounds began anew, up to this one
  const Pair one = {1.f, 0.f};
  Pair z = raised(one), whole = {-1.f, 0.f};        // whole (no draft probabilities): the node's last sum that was added up
  int last = 0, len = 1, pass = 0, spare;
  bool summed = false;
  if (tid == 0) c.path[0] = 0;
  while (true) {
    // ---- tests, until a sum is needed or no child is left
    if (warp == 0) {
      int command = kDraw;
      bool again = false;        // behind a sum of the rounds that began anew: the next of them
      if (summed && p.draft) {   // (z is from the last pass)
        if (!fine && round > 1 && !(z.hi >= kCoarse * kUp * c.left.a.hi)) {   // (p - q of the first round is exact)
          fine = round;
          round = 1;
          summed = false;
          command = kSum;
        } else {
          again = round < fine;
        }
      }
      while (command == kDraw) {
        float pv = 0.f;
        bool dup = false;
        if (!again) {
          int next = n;   // the next child of `node` behind node `last`
          for (int i = last + 1; i < n; i += 32) {
            const unsigned m = __ballot_sync(0xffffffffu, i + lane < n && c.parent[i + lane] == node);
            if (m) {
              next = i + __ffs(m) - 1;
              break;
            }
          }
          if (next >= n) break;
          pv = c.p[next];
          const float up = fmaxf(pv, c.q[next]) < 1.f ? kUp : 1.f;   // (numbers far above 1 have no room for it)
          const float ps = pv * up, qv = c.q[next] * up;
          Pair r = {ps, 0.f};
          if (round > 0) {
            if (p.draft) {
              if (fine) {
                r = left_fine(pv * kUp, c.q[next] * kUp, c.over, round);
                r = {r.hi * (up / kUp), r.lo * (up / kUp)};
              } else {
                r = round == 1 ? two_sum(ps, -qv) : add(mul(c.left.a, {ps, 0.f}), neg(mul(c.left.b, {qv, 0.f})));
              }
            } else {
              for (int x = lane; x < turned_down; x += 32) dup |= c.gone[x] == c.token[next];
              dup = __any_sync(0xffffffffu, dup);
              if (dup) r = {0.f, 0.f};
            }
          }
          if (z.hi > 0.f && above(raised(r), mul(product(c.u[next], qv), z))) {
            node = next;
            round = turned_down = 0;
            z = raised(one);
            whole.hi = -1.f;
            if (lane == 0) c.path[len] = next;
            ++len;
            last = next;
            summed = false;
            fine = 0;
            continue;
          }
          if (!p.draft && whole.hi < 0.f) {   // (the test stands: come back with the sum)
            command = kWhole;
            break;
          }
          last = next;
        }
        // turned down: r <- max(r / z - q, 0), or r without the token
        summed = false;
        if (p.draft) {
          if (lane == 0) {
            if (round == 0) {
              c.left.a = c.left.b = one;
            } else if (fine) {
              c.over[round - 1] = z.hi > 0.f ? reciprocal(z) : Pair{0.f, 0.f};
            } else if (z.hi > 0.f) {   // (nothing left: it stays so)
              const Pair over = raised(reciprocal(z));
              c.left.a = mul(c.left.a, over);
              c.left.b = add(mul(c.left.b, over), one);
            }
          }
          __syncwarp();
          ++round;
          command = kSum;
          break;
        }
        ++round;
        if (lane == 0) c.gone[turned_down] = c.token[last];
        __syncwarp();
        ++turned_down;
        z = turned_down == 1 ? add(whole, {-pv * kUp, 0.f}) : dup ? z : add(z, {-pv * kUp, 0.f});
        if (!(z.hi > whole.hi * kCoarse)) {   // too little of that sum for a difference to hold: add it up
          command = kSum;
          break;
        }
      }
      if (command == kDraw && summed && !(z.hi > 0.f)) {   // nothing left: the target's own row
        round = turned_down = fine = 0;
        summed = false;
      }
      if (lane == 0) {
        c.left.node = node;
        c.left.round = round;
        c.left.turned = turned_down;
        c.left.fine = fine > 0;
        c.path_len = len;
        c.command = command | (summed ? kSummed : 0);
      }
    }
    __syncthreads();
    const int command = c.command & 3;
    const Left f = c.left;
    const int turned = command == kWhole ? 0 : f.turned;
    const long long row_at = ((long long)b * p.S + f.node) * p.V;
    const Row<HALF> row = {p.target, p.draft, row_at, p.V, (int)(row_at & 3)};
    const int groups = (int)((p.V + row.off + 3) >> 2);          // of four elements
    const int run = (((groups + warps - 1) / warps) + 31) & ~31; // of a warp
    const int g0 = (rank * kVWarps + warp) * run;
    if (!(c.command & kSummed)) {
      // ---- the sum of what is left, and every warp's part of it
      Pair s[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
      const int k0 = max(g0, row.first()), k1 = min(g0 + run, row.end());
      if (f.fine) {
        s[0] = sum_fine<HALF>(row, f, c, g0, min(g0 + run, groups));
      } else if (f.round > 0 && row.q) {
        sum_run<HALF, true>(row, f, g0, k0, k1, 0, 5, s);
      } else {
        // Groups of this lane with a token turned down, and those that share a bit of the mask with one: one by one.
        const int fold = run > 32 * 64 ? 32 - __clz((run - 1) >> 6) : 5;   // run <= 64 << fold
        unsigned long long skip = 0ull;
        for (int x = 0; x < turned; ++x) {
          const long long k = (((long long)c.gone[x] + row.off) >> 2) - g0;
          if (k >= 0 && k < run && (k & 31) == lane) skip |= 1ull << (k >> fold);
        }
        sum_run<HALF, false>(row, f, g0, k0, k1, skip, fold, s);
        if (skip)
          for (int k = g0 + lane; k < k1; k += 32) {
            if (k < k0 || !(skip >> ((k - g0) >> fold) & 1u)) continue;
            Pair r[4];
            left_of4<HALF>(row, row.load(k), f, c.gone, turned, k, r);
#pragma unroll
            for (int e = 0; e < 4; ++e) gather(s[e], r[e]);
          }
      }
      // Elements of the groups that reach over the row's ends, a lane each: those before the first whole group (lanes
      // 0..), those behind the last (16..).
      if (!f.fine && (g0 == 0 || (g0 < groups && g0 + run >= groups))) {
        const long long head = min((long long)((4 - row.off) & 3), p.V);
        const long long tail = max(4LL * row.end() - row.off, head);
        const long long v = lane < 16 ? lane : tail + lane - 16;
        const bool on = lane < 16 ? g0 == 0 && v < head : g0 + run >= groups && v < p.V;
        if (on) {
          const float pe = prob<HALF>(row.p, row.at + v), qe = row.q ? prob<HALF>(row.q, row.at + v) : 0.f;
          Pair r = f.round == 0 || !row.q ? Pair{pe, 0.f} : left_of(pe, qe, f.a, f.b);
          for (int x = 0; x < turned; ++x)
            if (c.gone[x] == v) r.hi = 0.f;
          gather(s[0], r);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = quick(s[e].hi, s[e].lo);
      Pair t = warp_sum(add(add(s[0], s[1]), add(s[2], s[3])));
      if (!f.fine) t = raised(t);
      Pair* dst = &c.sums[pass & 1][rank * kVWarps + warp];
      if (lane < ranks) *cluster.map_shared_rank(dst, lane) = t;
      cluster.sync();   // (two sets: the next pass writes the other one, and its barrier comes before this one's turn)
      if (warp == 0) {
        Pair w = {0.f, 0.f};
        for (int x = lane; x < warps; x += 32) w = add(w, c.sums[pass & 1][x]);
        const Pair sum = warp_sum(w);
        whole = sum;
        if (command != kWhole) {
          z = sum;
          summed = true;
        }
      }
      ++pass;
      if (command != kDraw) continue;
    }
    // ---- the draw: every warp 0 finds the warp whose run holds the place
    if (warp == 0) {
      int at = -1;
      Pair before = {0.f, 0.f}, edge = {INFINITY, 0.f};   // nothing passes the edge: the last element with something
      if (z.hi > 0.f) {
        const Pair* sums = c.sums[(pass - 1) & 1];
        const Pair goal = mul({p.sample_u[b], 0.f}, z);
        // Four warps a lane, then the one of the four.
        constexpr int kPer = kVMaxWarps / 32;
        Pair part[kPer], own = {0.f, 0.f};
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
          const int w = lane * kPer + x;
          part[x] = w < warps ? sums[w] : Pair{0.f, 0.f};
          own = add(own, part[x]);
        }
        int l0 = find_lane(own, goal, &before, &spare);
        const bool beyond = l0 < 0;   // a number of 1 or more, or a rounding at the very end
        if (beyond) l0 = spare;
        int in = -1, filled = 0;
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
          Pair v;
          v.hi = __shfl_sync(0xffffffffu, part[x].hi, l0);
          v.lo = __shfl_sync(0xffffffffu, part[x].lo, l0);
          if (in >= 0 || !(v.hi > 0.f)) continue;
          filled = x;
          const Pair upto = add(before, v);
          if (!beyond && above(upto, goal)) in = x;
          else before = upto;
        }
        if (in >= 0) edge = goal;
        at = l0 * kPer + (in >= 0 ? in : filled);
      } else if (rank == 0 && lane == 0 && p.status) {
        atomicOr(p.status, GQA_DEVICE_BAD_PROBS_BIT);
      }
      if (lane == 0) {
        c.at = at;
        c.before = before;
        c.edge = edge;
        if (at < 0 && rank == 0) p.next[b] = -1;
      }
    }
    __syncthreads();
    if (c.at >= 0 && c.at / kVWarps == rank) {
      // ---- its run again, a sixteenth of it a warp (the row is in L1 or L2 by now)
      const int sub = run / kVWarps;
      const int b0 = c.at * run + warp * sub, b1 = min(b0 + sub, groups);
      Pair sum = {0.f, 0.f};
      for (int k = b0 + lane; k < b1; k += 32) {
        Pair r[4];
        if (f.fine) left_fine4<HALF>(row, row.load(k), f, c, k, r);
        else left_of4<HALF>(row, row.load(k), f, c.gone, turned, k, r);
        sum = add(sum, add(add(r[0], r[1]), add(r[2], r[3])));
      }
      sum = warp_sum(sum);
      if (lane == 0) c.part[warp] = f.fine ? sum : raised(sum);
      __syncthreads();
      Pair before = c.before, edge = c.edge;
      int mine = find_lane(lane < kVWarps ? c.part[lane] : Pair{0.f, 0.f}, edge, &before, &spare);
      if (mine < 0) {
        mine = spare;
        edge = {INFINITY, 0.f};
      }
      if (warp == mine) {
        int token = -1, behind = -1;   // behind: the last element with something so far
        for (int k0 = b0; k0 < b1 && token < 0; k0 += 32) {
          const int k = k0 + lane;
          Pair r[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
          if (k < b1) {
            if (f.fine) left_fine4<HALF>(row, row.load(k), f, c, k, r);
            else left_of4<HALF>(row, row.load(k), f, c.gone, turned, k, r);
          }
          if (!f.fine) {
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] = raised(r[e]);
          }
          Pair upto = before;
          const int hit = find_lane(add(add(r[0], r[1]), add(r[2], r[3])), edge, &upto, &spare);
          const int pick = hit >= 0 ? hit : spare;
          before = upto;
          if (pick < 0) continue;
          // The element of the four: where it passes, else the last one with something.
          int found = -1, positive = -1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            upto = add(upto, r[e]);
            if (r[e].hi > 0.f) {
              positive = 4 * k - row.off + e;
              if (found < 0 && above(upto, edge)) found = positive;
            }
          }
          found = __shfl_sync(0xffffffffu, found, pick);
          positive = __shfl_sync(0xffffffffu, positive, pick);
          behind = hit >= 0 && found >= 0 ? found : positive;
          if (hit >= 0) token = behind;
        }
        if (lane == 0) p.next[b] = behind;
      }
    }
    break;
  }
  if (rank == 0) {
    const int path_len = c.path_len;
    for (int i = tid; i < p.S; i += kVThreads) path[i] = i < path_len ? c.path[i] : -1;
    if (tid == 0) p.path_lens[b] = path_len;
  }
  cluster.sync();   // nobody leaves while its sums may still be written
}

// ------------------------------------------------------------------ accepted rows

constexpr int kAThreads = 128;
constexpr int kAhead = 8;   // rows of a thread under way

// A thread owns one 16-byte column of a (cache, sequence, KV head) and moves its
// rows in order. A path increases, so row path[i] >= i, and what a group of rows
// writes lies below everything later groups read. Rows that stay are not read.
// Bound: the two dependent loads, of the path and of the rows (16 layers of 16
// sequences, trees of 64 nodes: 10.5 us for 12 MB).
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
  // CTAs of a sequence: as many as have 4096 elements each and find room at once (two an SM).
  int ranks = kVMaxCluster;
  while (ranks > 1 && (p.V / ranks < 4096 || (long long)p.B * ranks > 304)) ranks /= 2;
  return p.half ? launch_verify<true>(p, ranks, st) : launch_verify<false>(p, ranks, st);
}

cudaError_t launch_tree_accept(const AcceptParams& p, cudaStream_t st) {
  const long long columns = 2LL * p.layers * p.Nkv * (p.row_bytes / 16);
  const dim3 grid((unsigned)((columns + kAThreads - 1) / kAThreads), (unsigned)p.B);
  tree_accept_kernel<<<grid, kAThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace gqa
