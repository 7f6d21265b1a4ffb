// q4.h -- what the 4-bit matrices' translation units share.
#pragma once

#include <atomic>
#include <mutex>

#include "internal.h"

namespace spmv {
namespace q4 {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTileRows = 32;
// columns of a step with NT * 8 operand columns: 4 KB of codes, or 2 KB to leave
// room for x and the partial sums of more than 8
template <int NT>
constexpr int kStepColsOf = NT == 1 ? 256 : 128;
// steps of a warp held: the one in use and the next ones
template <int NT>
constexpr int kStagesOf = 2;

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
  int P, logP;              // blocks of a cluster, along the columns
  int tileShare, tileRest;  // tiles of a cluster, clusters with one more
  int stepShare, stepRest;  // steps (of kStepColsOf columns) of a block, blocks with one more
  int phaseSteps;           // steps whose x is in shared memory at a time
  int maxTiles;             // most tiles of a cluster
};

struct Plan {
  long long tiles, clusters;
  int steps, P, logP, phaseSteps, maxTiles;
  size_t smem;
};
// What a kernel may hold on the device: asked once per kernel (the GPUs of a
// machine are taken to be alike), outside stream captures, as the attribute is
// set then too.
constexpr int kMaxSmem = 227 * 1024;
struct Residency {
  std::atomic<unsigned long long> devices{0};  // where the attribute is set
  std::mutex mu;
  // clusters of 1, 2, 4, 8 blocks that run at a time, with 1 or 2 blocks on an SM
  int clusters[4][2] = {};
  cudaError_t ask(const void* kernel);
};
// columns: operand columns; ringBytes: shared memory of the warps' rings.
Plan make_plan(const RunArgs& p, int columns, int stepCols, int ringBytes, const Residency& r);

template <class X>
cudaError_t launch_run(const RunArgs& p, cudaStream_t s);
template <class X>
constexpr int vectors_per_pass() {
  return sizeof(X) == 4 ? 5 : 16;  // 16 columns, an fp32 vector takes three
}

}  // namespace q4
}  // namespace spmv
