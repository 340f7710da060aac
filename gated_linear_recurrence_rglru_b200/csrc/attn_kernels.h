// Internal interface between the C ABI layer of the local attention operators
// (attn_abi.cu, include/rglru_attn.h) and their kernel launchers.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "rglru_attn.h"

namespace rglru {

constexpr int kMaxSmem = 232448;  // bytes of shared memory a block can opt in to

// Lets `kernel` use `smem` bytes of dynamic shared memory on the current device;
// `done` keeps one bit a device, so that later calls skip the driver.
template <typename K>
cudaError_t opt_in_smem(K kernel, int smem, std::atomic<unsigned long long> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// A strided (B, T, H, dh) tensor, strides in elements.
struct Strided {
  const void *p;
  long long sb, st, sh;
};

// ---------------------------------------------- queries and keys (qk_norm_rope.cu)

constexpr int kMaxPairs = 128;  // rot / 2 at most

struct QkArgs {
  Strided q, k, v;                 // v: append only
  const void *w_q, *w_k;
  const int *positions;            // or null: 0..T-1
  void *q_out, *k_out;             // dq, dk in the backward
  const void *dq_out, *dk_out;     // backward only
  float *dw_q, *dw_k;              // backward only, or null
  void *k_cache, *v_cache;         // append only
  const int *page_table;
  int num_pages, page_size, max_pages;
  int B, T, Hq, Hkv, dh, rot;
  float eps;
  int *dev_status;
  // turn of pair i per unit of position, as a fraction of one turn times 2^64
  unsigned long long phase[kMaxPairs];
};

cudaError_t launch_qk_fwd(const QkArgs &p, int io, cudaStream_t st);
cudaError_t launch_qk_append(const QkArgs &p, int io, cudaStream_t st);
size_t qk_bwd_workspace_bytes(int B, int T, int Hq, int Hkv, int dh);
cudaError_t launch_qk_bwd(const QkArgs &p, int io, void *ws, cudaStream_t st);

// ------------------------------------------------------------- windowed attention

struct AttnArgs {
  Strided q, k, v;
  const int *lens;                 // or null
  void *out;                       // forward: written; backward: read
  float *lse;
  const void *dout;                // backward only (dense)
  void *dq, *dk, *dv;
  int B, T, S, Hq, Hkv, dh, window, sinks;
  float scale;
  int *dev_status;
};

// Key rows of one (batch row, key head) in the backward are cut into tiles of
// `tile` keys. The queries that see a tile, over the query heads that share
// it, are `iters` steps (one head's `step` queries each), cut into pieces of
// at most `len` steps so that short batches fill the GPU: one thread block a
// piece. Tiles that hold sinks are seen by every later query and get more
// pieces. A tile with one piece stores its gradients itself; others leave
// float partial sums that attn_join_kernel adds in the order of the pieces.
struct PiecePlan {
  int tile, step, len;
  int n_tiles, n_sink_tiles;
  int pieces, sink_pieces;         // per tile: grid places (some may be empty)
  int slots;                       // n_sink_tiles * sink_pieces + (n_tiles - n_sink_tiles) * pieces
};

PiecePlan attn_plan(int B, int T, int S, int Hq, int Hkv, int window, int sinks, int tile,
                    int step, int target_blocks, int least);

// Shared by every backward: delta[b, h, t] = sum_d dout * out (float, B * Hq * T,
// its room rounded up), and the join of the pieces' partial sums.
size_t attn_delta_bytes(const AttnArgs &p);
size_t attn_parts_bytes(const AttnArgs &p, const PiecePlan &pl);
cudaError_t launch_attn_delta(const AttnArgs &p, int io, float *delta, cudaStream_t st);
cudaError_t launch_attn_join(const AttnArgs &p, int io, const PiecePlan &pl, const float *parts,
                             cudaStream_t st);

cudaError_t launch_attn_fwd_generic(const AttnArgs &p, int io, cudaStream_t st);
size_t attn_bwd_generic_workspace_bytes(const AttnArgs &p);
cudaError_t launch_attn_bwd_generic(const AttnArgs &p, int io, void *ws, cudaStream_t st);

// Tensor-core kernels: bf16, heads 64, 128 or 256 wide.
bool attn_tc_supported(const AttnArgs &p, int io);
cudaError_t launch_attn_fwd_tc(const AttnArgs &p, cudaStream_t st);
size_t attn_bwd_tc_workspace_bytes(const AttnArgs &p);
cudaError_t launch_attn_bwd_tc(const AttnArgs &p, void *ws, cudaStream_t st);

// ------------------------------------------------ one token over a paged cache

struct DecodeArgs {
  const void *q, *k_cache, *v_cache;
  const int *page_table, *lens;
  void *out;
  int num_pages, page_size, max_pages;
  int B, Hq, Hkv, dh, window, sinks;
  float scale;
  int *dev_status;
};

size_t paged_decode_workspace_bytes(const DecodeArgs &p, int io);
cudaError_t launch_paged_decode(const DecodeArgs &p, int io, void *ws, cudaStream_t st);

}  // namespace rglru
