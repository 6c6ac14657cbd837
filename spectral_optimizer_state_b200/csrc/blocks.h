// Launch interface of the block-wise Muon step (blocks.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/muon.h"

namespace muon {

// The short side of a block is at most this.
constexpr int kBlockMaxShort = 128;
constexpr int kBlockMaxCluster = 8;
constexpr int kBlockMost = 1 << 27;  // blocks of a call

struct BlockParams {
  void* w[MUON_MAX_BATCH];        // W (updated), or Out
  const void* g[MUON_MAX_BATCH];  // G, or X
  float* m[MUON_MAX_BATCH];       // momentum (step only)
  long long ldw, ldg, ldm;        // row strides, elements
  int rows, cols;                 // of every matrix
  int block_rows, block_cols;     // nominal block (the last ones of a matrix may be smaller)
  int grid_cols, per_matrix;      // blocks per block row / per matrix
  int blocks;                     // in the launch
  int ahead;                      // a CTA brings the block this far behind its own to L2 (0: none)
  int slice;                      // long-side elements a CTA of the cluster owns (multiple of 64)
  int cluster;                    // CTAs per block
  int threads;                    // 256 (two CTAs an SM) or 512
  int tmem_cols;
  int alias;                      // the Gram partials of a cluster lie where A will be
  int step;                       // 1: Muon step; 0: orthogonalise only
  int vec;                        // accesses of eight elements allowed (rows and blocks start on multiples)
  float beta, gscale, eps, decay, lr;
  int nesterov, scale_mode;
  float store_scale;              // power of two the iterates are held at
  int k;
  float abc[3 * MUON_MAX_ITERS];
  float* nu;                      // [blocks] ||U||_F
  int* flags;                     // [blocks]
  int* status;
};

// Shared memory of one CTA for blocks of `shorter` (short side) with `slice` long-side elements each.
size_t block_smem_bytes(int shorter, int slice, bool tall, bool f32, int cluster, bool alias);
// `tall`: nominal block_rows > block_cols.
cudaError_t launch_blocks(const BlockParams& p, int blocks, bool tall, bool f32, size_t smem, cudaStream_t stream);

}  // namespace muon
