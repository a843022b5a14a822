// Newton-Schulz orthogonalisation of any batch of matrices: parameters of the launchers in orth.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ttt {

struct OrthPlan {
  int rows, cols, batch;
  bool bf16, tall;                  // tall: rows > cols, X is the transpose of G
  bool narrow;                      // a launch a step
  int r, c;                         // X is r x c, r <= c
  int tile, tile_sym;               // tile of B X, and of the symmetric products
  int rp, cp;                       // padded sizes
  int norm_blocks;                  // partial sums of squares a matrix
  size_t off_norm, off_rest, off_x[2], off_xt[2], off_a, off_b, total;
};
OrthPlan plan_orth(int rows, int cols, int batch, bool bf16);

struct OrthParams {
  OrthPlan plan;
  const void *g;                    // [batch][rows][cols], row stride ld, matrix stride bs
  int64_t ldg, bsg;
  void *out;
  int64_t ldo, bso;
  float a, b, c, eps;
  int steps;
  char *ws;
};
hipError_t launch_orth(const OrthParams &p, hipStream_t s);

}  // namespace ttt
