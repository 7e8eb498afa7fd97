// Internal interface of the multi-axis rotary, the block-scaled int8 cache and
// its eviction: parameter blocks and launchers (block_api.cu fills them in).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gqa_internal.h"

namespace gqa {

constexpr int kRotaryChunks = 16;  // 8-pair chunks of a head (head size up to 256)

struct RotaryAxesParams {
  const void *q, *k;        // k null: queries only
  void *qo, *ko;
  const int* pos;           // [axes][tokens]
  const void *cos_c, *sin_c;
  const void *qw, *kw;      // norm weights or null
  uint32_t* status;
  long long tokens;         // B * S
  int N, Nkv, H, pairs, table_rows;
  int table_f32;            // table dtype: 1 fp32, 0 T
  float eps;
  unsigned axis_nibbles[kRotaryChunks];  // axes of pairs 8 l .. 8 l + 7, 4 bits each
  unsigned char chunk_uniform[kRotaryChunks];  // the eight pairs share one axis
};
cudaError_t launch_rotary_axes(const RotaryAxesParams& p, int t_type, cudaStream_t st);

struct BlockParams {
  int B, S, N, Nkv, G, H;
  int C, T;              // cache capacity, total_sequence_length
  int bs_log2, nblk;     // log2 of the block size, blocks of a (b, g)
  int t_type;
  int window;            // -1: none
  float scale, softcap;
  int smooth;
  const void *q, *k, *v;  // k / v null: nothing to append
  void* out;
  int8_t *kc, *vc;
  float *ks, *vs;
  const int *seqlens, *new_lens;
  const void* sink;
  const float* past_w;
  float* present_w;      // null: no weights
  uint32_t* status;
  // split-KV kernel
  int rt_rows, nrt;      // rows of a row tile, row tiles of a (b, g)
  int workers;           // warps of the grid
  int flush;             // fp32 with several row tiles: O summed to nearest every few units
  float *part_o, *part_ml;
  float* stash;          // log2-domain scores [B*Nkv][stash_ld keys][stash_rows] (one row tile), or null
  int stash_ld, stash_rows;
  float* lse;            // log2-domain log-sum-exp [B*Nkv][S*G], or null
  // tensor-core prefill
  int tile_rows;         // rows of a 128-row query tile in use: whole positions of G rows
  int qb_major;          // grid with the query block on the slow axis
  float* o_acc;          // fp32: sums of O, 512 bytes a row of every 128-row query tile, or null
  long long wait_budget;
  int withhold_tile;
};

// Lengths of one sequence; false when they break the contract.
__host__ __device__ inline bool block_lengths(const BlockParams& p, int b, int* total, int* fresh) {
  *total = p.seqlens[b] + 1;
  *fresh = p.new_lens ? p.new_lens[b] : p.S;
  return *total >= 0 && *total <= p.T && *fresh >= 0 && *fresh <= p.S && *fresh <= *total;
}

// Programmatic dependent launch: wait until the kernel ahead on the stream has
// completed (and its writes are visible); allow the next one to start.
__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Packed fp32x2 sum: d = a + b per lane pair.
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  unsigned long long av = *reinterpret_cast<unsigned long long*>(&a);
  unsigned long long bv = *reinterpret_cast<unsigned long long*>(&b);
  unsigned long long dv;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(dv) : "l"(av), "l"(bv));
  return *reinterpret_cast<float2*>(&dv);
}

// Launch that may start before the kernel ahead of it on the stream has
// finished (`early`): it calls dep_wait() before it touches what that one
// writes. What the kernels before those two wrote is complete by then, as the
// one ahead began after them or waited for them before it let this one start.
template <typename K, typename... A>
cudaError_t launch_dependent(bool early, K kern, dim3 grid, unsigned threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_block_append(const BlockParams& p, cudaStream_t st);
// Split-KV attention on warp MMAs, every shape.
constexpr int kBlockUnit = 32;      // keys per work unit
constexpr int kBlockRangeCost = 2;  // work units a range's start and end are counted as
int block_row_tile(int t_type, int H, long long rows);   // query rows per row tile, of `rows` of a (b, g)
int block_workers(const BlockParams& p);
cudaError_t launch_block_attn(const BlockParams& p, cudaStream_t st);
cudaError_t launch_block_merge(const BlockParams& p, cudaStream_t st);
// Tensor-core prefill: head and group sizes up to 128.
constexpr int kPrefillFlush = 512;   // keys after which the fp32 form moves O into sums
cudaError_t launch_block_prefill(const BlockParams& p, cudaStream_t st);
// Attention weights of the cache rows from the log-sum-exp of every query row.
cudaError_t launch_block_weights(const BlockParams& p, cudaStream_t st);
// ... on the tensor cores: where the tensor-core prefill runs with fp16 queries.
cudaError_t launch_block_weights_tc(const BlockParams& p, cudaStream_t st);

struct EvictParams {
  int B, Nkv, H, C, Cto, T;
  int bs_log2, nblk, nblk_to;
  int keep, recent, first;
  int fill;              // GQA_FILL_* bits: what a skipped sequence's entries become -1 of
  const int8_t *kc, *vc;
  const float *ks, *vs;
  int8_t *kc_to, *vc_to;
  float *ks_to, *vs_to;
  const float* w;
  float* w_to;           // or null
  const int* seqlens;
  int *kept, *seqlens_to;
  uint32_t* status;
};
cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t st);
cudaError_t launch_evict_gather(const EvictParams& p, cudaStream_t st);

}  // namespace gqa
