// Internal interface of the drafted-token operators: parameter blocks and
// launchers (tree_api.cu fills them in).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "block_internal.h"
#include "gqa_internal.h"

namespace gqa {

constexpr int kTreeNodes = 512;    // GQA_MAX_TREE_NODES
constexpr int kTreeLayers = 128;   // GQA_MAX_TREE_LAYERS
#define GQA_DEVICE_BAD_TREE_BIT 8u
#define GQA_DEVICE_BAD_PROBS_BIT 16u

struct TreeParams {
  int B, S, N, Nkv, G, H;
  int C, T;              // cache capacity, total_sequence_length
  int t_type;
  int window;            // -1: none
  float scale, softcap;
  int smooth;
  const void *q, *k, *v;
  void *out, *kc, *vc;   // output; present_key / present_value
  const int *seqlens, *new_lens, *parents;
  int parents_ld;        // S, or 0: one tree for all sequences
  const void* sink;
  uint32_t* status;
  int tc;                // on the tensor-core pipeline
  long long wait_budget;
  int withhold_tile;
  float lift;            // log2 of what the workspace's probabilities (l and O) are multiplied by
  // split over the keys
  int rt_log2, unit_log2;   // query rows of a row tile, keys of a unit: powers of two
  int cost;              // units that the start and the end of a range count as
  int nrt;               // row tiles of S nodes
  int workers;           // shares of the units
  float *part_o, *part_ml;
};

// Lengths of one sequence; false when they break the contract.
__host__ __device__ inline bool tree_lengths(const TreeParams& p, int b, int* past, int* fresh) {
  const int total = p.seqlens[b] + 1;
  *fresh = p.new_lens ? p.new_lens[b] : p.S;
  *past = total - *fresh;
  return total >= 0 && total <= p.T && *fresh >= 0 && *fresh <= p.S && *fresh <= total;
}

// Parent of node i as the operators read it, -1 for one out of range (*bad).
__device__ __forceinline__ int tree_parent(int a, int i, bool* bad) {
  if (a >= -1 && a < i) return a;
  *bad = true;
  return -1;
}

// ---- the units of all ranges (sequence b, KV head g, row tile rt), laid end
// to end: a range has the cached rows' units from the first a row sees on, the
// nodes' units, and `cost` more for its start and end.

struct TreeSeq {
  int past, fresh;   // cached rows, nodes
  int k0;            // first cached row of the first unit
  int np, work, units;   // units of cached rows; of all a range's keys; and with the cost of its ends
  int nrt;           // row tiles
};

// False when nothing is to do for the sequence.
__device__ __forceinline__ bool tree_seq(const TreeParams& p, int b, TreeSeq* s) {
  if (!tree_lengths(p, b, &s->past, &s->fresh)) s->fresh = 0;
  s->k0 = p.window >= 0 ? max(0, s->past - p.window) & ~15 : 0;   // the root sees furthest back
  const int u = (1 << p.unit_log2) - 1;
  s->np = (s->past - s->k0 + u) >> p.unit_log2;
  s->work = s->np + ((s->fresh + u) >> p.unit_log2);
  s->units = s->work + p.cost;
  s->nrt = (s->fresh * p.G + (1 << p.rt_log2) - 1) >> p.rt_log2;
  return s->fresh > 0;
}

// A share of the units, or the piece of a range within it.
struct TreeWalk {
  int b, g, rt, off;       // range, and unit `off` of it
  long long left;          // units of the share from here on
  TreeSeq s;

  __device__ bool enter(const TreeParams& p) {   // the sequence at b, or the next one with work
    for (; b < p.B; ++b)
      if (tree_seq(p, b, &s)) return true;
    return false;
  }
  // The share [u, u + n) of all units; whole warps, n > 0.
  __device__ void start(const TreeParams& p, long long u, long long n) {
    const int lane = threadIdx.x & 31;
    left = n;
    for (b = 0; b < p.B; b += 32) {
      const bool on = b + lane < p.B && tree_seq(p, b + lane, &s);
      long long y = on ? (long long)p.Nkv * s.nrt * s.units : 0;
      const long long own = y;
      for (int o = 1; o < 32; o <<= 1) {
        const long long c = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += c;
      }
      const unsigned past_u = __ballot_sync(0xffffffffu, on && y > u);
      if (past_u) {
        const int at = __ffs(past_u) - 1;
        u -= __shfl_sync(0xffffffffu, y - own, at);
        b += at;
        break;
      }
      u -= __shfl_sync(0xffffffffu, y, 31);
    }
    if (b >= p.B) {   // (u lies below the sum of all units)
      left = 0;
      return;
    }
    tree_seq(p, b, &s);
    const int gr = (int)(u / s.units);
    off = (int)(u - (long long)gr * s.units);
    g = gr / s.nrt;
    rt = gr - g * s.nrt;
    settle(p);
  }
  // Past the end of a range: the next one.
  __device__ void settle(const TreeParams& p) {
    while (left > 0 && off >= s.work) {
      left -= s.units - off;
      off = 0;
      if (++rt == s.nrt) {
        rt = 0;
        if (++g == p.Nkv) {
          g = 0;
          ++b;
          if (left > 0 && !enter(p)) left = 0;
        }
      }
    }
  }
  // Units of this range in the share.
  __device__ int piece() const { return (int)min(left, (long long)(s.work - off)); }
  __device__ void next(const TreeParams& p, int n) {
    off += n;
    left -= n;
    settle(p);
  }
};

// Sum of all units, by one warp.
__device__ __forceinline__ long long tree_units(const TreeParams& p) {
  long long sum = 0;
  TreeSeq s;
  for (int b = threadIdx.x & 31; b < p.B; b += 32)
    if (tree_seq(p, b, &s)) sum += (long long)p.Nkv * s.nrt * s.units;
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Workers that share the units: the grid's, which the host sized for
// total_sequence_length, or one a unit where the lengths leave fewer.
__device__ __forceinline__ long long tree_live(const TreeParams& p, long long units) {
  return max(1LL, min((long long)p.workers, units));
}

// A piece that is all of its range goes to the output. Of the others a worker
// has two at most: one whose range began before its share, slot 2 worker of the
// workspace, and one that begins here and goes on behind it, slot 2 worker + 1.
__device__ __forceinline__ long long tree_slot(long long worker, bool begins) { return 2 * worker + (begins ? 1 : 0); }

// Workers *w0 .. *w1 hold the pieces of the range of units [base, base + work).
__device__ __forceinline__ void tree_pieces(long long base, int work, long long live, long long units, long long* w0,
                                            long long* w1) {
  *w0 = ((base + 1) * live - 1) / units;
  *w1 = ((base + work) * live - 1) / units;
}

cudaError_t launch_tree_attn(const TreeParams& p, cudaStream_t st);
// ... on the tensor cores: fp16, head sizes up to 128.
cudaError_t launch_tree_tc(const TreeParams& p, cudaStream_t st);
cudaError_t launch_tree_merge(const TreeParams& p, cudaStream_t st);
// Rows of a row tile, keys of a unit and shares of the split for a call.
void tree_attn_plan(TreeParams* p);

struct VerifyParams {
  int B, S;
  long long V;
  int half;                  // probabilities in fp16, else fp32
  const int *tokens, *parents;
  int parents_ld;            // S, or 0
  const void *target, *draft;   // draft null: certain drafts
  const float *accept_u, *sample_u;
  const int* new_lens;
  int *path, *path_lens, *next;
  uint32_t* status;
};
cudaError_t launch_tree_verify(const VerifyParams& p, cudaStream_t st);

struct AcceptParams {
  int B, S, Nkv, C, layers;
  int row_bytes;             // of a cache row, a multiple of 16
  const int *path, *path_lens, *seqlens, *new_lens;
  int* into_seqlens;
  uint32_t* status;
  void* cache[2 * kTreeLayers];   // keys and values of every layer
};
cudaError_t launch_tree_accept(const AcceptParams& p, cudaStream_t st);

}  // namespace gqa
