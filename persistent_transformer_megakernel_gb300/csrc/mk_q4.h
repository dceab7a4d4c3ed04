// The 4-bit matrix-vector products' call and the entry of each translation unit of their kernel.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "mk_mma.cuh"

namespace mkq {

struct Q4Params {
  const void *x, *residual;
  void *y;
  const unsigned char *codes;
  const uint16_t *scales;
  const uint8_t *zeros;
  int64_t x_row, residual_row, y_row;
  int m, n, k, groups;
  mkw::Divisor blocks_a_group;   // groups of 128 and more
  mkw::Divisor eighths;          // 8-element parts of a CTA's blocks of k, room for them
  int blocks;           // of k, the last one maybe short
  int cluster;          // CTAs that have a slice of k each
  int inbox;            // byte where the others' sums are put
  int pass_rows;        // x rows of one pass (blockIdx.y)
  int wk;               // warps that share a tile's k: 1, 2, 4, 8 or 16
  int tiles;            // tiles of 16 RT rows
  int pitch;            // bytes from staged column to column
  int vec;              // a block's scales (and zeros) of a row can be loaded at once
};

// launch for x of one type (group: codes a scale)
int run_f32(Q4Params &p, int group, int sms, int dev, cudaStream_t s);
int run_bf16(Q4Params &p, int group, int sms, int dev, cudaStream_t s);

}  // namespace mkq
