// q4.h -- what the 4-bit matrices' translation units share.
#pragma once

#include <atomic>

#include "internal.h"

namespace spmv {
namespace q4 {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 4;  // steps of a warp in flight, the one in use among them

// One launch of the product.
struct RunArgs {
  spmv_q4 a;
  const uint8_t* codesEnd;  // past the last row's last byte
  int n;                    // vectors
  const void* x;
  long long ldx;
  bool xVec;                // x's rows start on 16-byte boundaries
  const void* c;            // or null
  long long ldc;
  int yType;
  void* y;
  long long ldy;
  // the launch's split (make_plan)
  long long tiles;          // of the matrix
  int steps;                // 128 columns each
  int P;                    // blocks of a cluster, along the columns
  int phaseSteps;           // steps whose x is in shared memory at a time
  int maxTiles;             // most tiles of a cluster
};

struct Plan {
  long long tiles, clusters;
  int steps, P, phaseSteps, maxTiles;
  size_t smem;
};
// tileRows: rows of a tile; columns: operand columns; ringBytes: shared memory
// of the warps' rings.
Plan make_plan(const RunArgs& p, int tileRows, int columns, int ringBytes);

// The most dynamic shared memory a block may ask for, allowed once per kernel
// and device (not during a stream capture: one call outside it comes first).
constexpr int kMaxSmem = 227 * 1024;
struct SmemOnce {
  std::atomic<unsigned long long> done{0};
  cudaError_t allow(const void* kernel);
};

template <class X>
cudaError_t launch_run(const RunArgs& p, cudaStream_t s);
template <class X>
constexpr int vectors_per_pass() {
  return sizeof(X) == 4 ? 5 : 16;  // 16 columns, an fp32 vector takes three
}

}  // namespace q4
}  // namespace spmv
