// Launch interface of the expert products (experts.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace muon {

enum ExpertMode { EXPERT_FORWARD = 0, EXPERT_BACKWARD = 1, EXPERT_WGRAD = 2 };

// Heights of the token box of a K-major B operand: 16 << i rows.
constexpr int kExpertBoxes = 5;

struct alignas(64) ExpertParams {
  CUtensorMap tmA;                // features: W {K, N, E, planes}, or X {K, T, 1, planes} (weight gradient)
  CUtensorMap tmB[kExpertBoxes];  // rows: X / dY {cols, T, 1, planes}; the weight gradient uses tmB[0] alone
  CUtensorMap tmOut;              // fp32 output {columns, rows, experts}, box {32, 16, 1} (with vec)
  const int* offsets;             // [experts + 1], device
  int experts, tokens;
  int features;                   // columns of the output
  int rows;                       // weight gradient: rows of one expert's output (N)
  int k_tiles;                    // products: ceil(contraction / 64)
  int in_f32;                     // fp32 operands: three bf16 planes
  int split;                      // fp32 operands are read at a and b and split by the kernel
  const void* a;                  // split: as tmA and tmB, element strides between rows and experts
  const void* b;
  long long ld_a, s_a, ld_b;
  int pairs_a, pairs_b;           // rows start on 8-byte boundaries and are even
  int contraction;                // products: elements contracted
  void* out;
  long long ld_out, s_out;        // elements between rows / experts of the output
  int out_f32;
  int vec;                        // rows of the output start on 16-byte boundaries
  int clear_rest;                 // zero the rows no segment covers; gradient: all of it if the offsets are bad
  float beta, scale;              // weight gradient: out = beta out + scale acc
  int* status;
};

// `ctas`: persistent CTAs to launch (one per SM at most; an even number of them for pairs).
cudaError_t launch_experts(const ExpertParams& p, ExpertMode mode, bool pair, int ctas, cudaStream_t stream);

// Copies `mats` matrices of rows x cols (row stride ld, matrix stride s) into bf16 planes
// [planes][mats][rows][pitch]: one plane copies bf16 rows that a TMA cannot start on, three split
// fp32 values.  With `offsets`, matrices (experts) whose segment is empty are skipped.
struct PackItem {
  const void* src;
  uint16_t* dst;
  long long ld, s, dst_mat, dst_plane;
  int mats, rows, cols, pitch;
  const int* offsets;
  int block0;  // set by launch_pack
};
struct PackParams {
  PackItem item[2];
  int count;
};
// Both operands of a product in one launch: fp32 sources into three planes, bf16 ones into one.
cudaError_t launch_pack(PackParams& p, bool src_f32, int sm_count, cudaStream_t stream);

}  // namespace muon
