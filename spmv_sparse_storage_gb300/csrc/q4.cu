// q4.cu -- matrices of 4-bit codes with a scale per group of a row's columns:
// conversion from a dense matrix, products with vectors, rows back in dense
// form.
#include "dtypes.cuh"
#include "device_util.cuh"
#include "internal.h"
#include "q4.h"

namespace spmv {
namespace {

__device__ __forceinline__ float scale_at(const void* scales, int type, long long i) {
  switch (type) {
    case SPMV_F16: return to_f32(static_cast<const __half*>(scales)[i]);
    case SPMV_BF16: return to_f32(static_cast<const __nv_bfloat16*>(scales)[i]);
    default: return static_cast<const float*>(scales)[i];
  }
}

// ---------------------------------------------------------------------------
// Conversion. Of a group: the least and the largest weight, the scale, and per
// weight the code round(w / scale) + zero. Bound by the bytes of W, of the codes
// and of the values where they are asked for, as long as the arithmetic per
// weight stays short: with both the time of its bytes leaves 24 instructions.
// 28672 x 8192 bf16 with zero points and values: 179 us, 5.9 TB/s, 0.87 of a copy
// (0.71 of the issue slots are taken; with 8 weights to a lane, an IEEE division
// each and a branch for ties it took 258).
// ---------------------------------------------------------------------------
constexpr float kMaxFinite = 3.402823466e38f;
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer

struct GroupCodes {
  float step, inv, low, high;  // code - zero is in [low, high]
  unsigned zero;
  bool usable, plain;          // plain: quotients by inv, and never below low
};
// The least normal number of a scale's type: below it a scale is so coarse that
// quotients leave the codes' range, and 1 / scale may overflow.
template <class S>
constexpr float kLeastNormal = 1.2e-37f;
template <>
constexpr float kLeastNormal<__half> = 6.2e-5f;
__device__ __forceinline__ float reciprocal(float v) {  // to 1 unit in the last place
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// w / step from inv = 1 / step (1 + 2^-23): the product's error is taken out by
// the residual w - t step, which fma gives exactly (a Newton correction). What is
// left is 2^-45 of the quotient before the last rounding, so that a half integer,
// which 16-bit weights and scales hit now and then, comes out as one.
__device__ __forceinline__ float quotient(float w, float step, float inv) {
  const float t = w * inv;
  return fmaf(fmaf(-t, step, w), inv, t);
}
// lo <= 0 <= hi: the range of a group's weights (a NaN if one of them is).
template <class S>
__device__ __forceinline__ GroupCodes group_codes(float lo, float hi, bool zeros, S* scale) {
  float raw = zeros ? (hi - lo) * (1.0f / 15.0f) : fmaxf(hi, -lo) * (1.0f / 7.0f);
  if (!(hi <= kMaxFinite && lo >= -kMaxFinite)) raw = __int_as_float(0x7fc00000);
  *scale = from_f32<S>(raw);
  GroupCodes c;
  c.step = to_f32(*scale);
  c.usable = c.step > 0.0f && c.step <= kMaxFinite;
  c.plain = c.usable && c.step >= kLeastNormal<S>;
  c.inv = reciprocal(c.step);
  float zero = 8.0f;
  if (zeros) {
    const float z = c.plain ? quotient(-lo, c.step, c.inv) : -lo / c.step;
    zero = c.usable ? fminf(fmaxf(rintf(z), 0.0f), 15.0f) : 0.0f;
  }
  c.zero = (unsigned)zero;
  c.low = -zero;
  c.high = 15.0f - zero;
  return c;
}
// code - zero + kRound for N weights.
template <int N>
__device__ __forceinline__ void rounded_codes(const float (&w)[N], const GroupCodes& c,
                                              float (&u)[N]) {
  if (c.plain) {
#pragma unroll
    for (int e = 0; e < N; ++e) u[e] = fminf(quotient(w[e], c.step, c.inv), c.high) + kRound;
  } else {
    for (int e = 0; e < N; ++e)
      u[e] = c.usable ? fminf(fmaxf(w[e] / c.step, c.low), c.high) + kRound : kRound;
  }
}

// The range of the 8 H weights of each of the LANES lanes that share a group, in
// pairs for the 16-bit types; NaN wins. hi = max(0, w), lo = min(0, w).
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
template <int LANES, int H>
__device__ __forceinline__ void group_range(const Pack<float, 8> (&v)[H], float& lo, float& hi) {
  float up = 0.0f, down = 0.0f;
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      up = max_nan(up, v[h].v[e]);
      down = max_nan(down, -v[h].v[e]);
    }
#pragma unroll
  for (int off = 1; off < LANES; off *= 2) {
    up = max_nan(up, __shfl_xor_sync(kFullMask, up, off));
    down = max_nan(down, __shfl_xor_sync(kFullMask, down, off));
  }
  hi = up;
  lo = -down;
}
template <int LANES, class P, class W, int H>
__device__ __forceinline__ void pair_range(const Pack<W, 8> (&v)[H], float& lo, float& hi) {
  const P* p = reinterpret_cast<const P*>(&v);
  P up = p[0], down = p[0];
#pragma unroll
  for (int e = 1; e < 4 * H; ++e) {
    up = __hmax2_nan(up, p[e]);
    down = __hmin2_nan(down, p[e]);
  }
  down = __hneg2(down);
  P both;  // (largest, - least)
  both.x = __hmax_nan(up.x, up.y);
  both.y = __hmax_nan(down.x, down.y);
#pragma unroll
  for (int off = 1; off < LANES; off *= 2)
    both = __hmax2_nan(both, __shfl_xor_sync(kFullMask, both, off));
  hi = max_nan(to_f32(both.x), 0.0f);
  lo = -max_nan(to_f32(both.y), 0.0f);
}
template <int LANES, int H>
__device__ __forceinline__ void group_range(const Pack<__half, 8> (&v)[H], float& lo, float& hi) {
  pair_range<LANES, __half2>(v, lo, hi);
}
template <int LANES, int H>
__device__ __forceinline__ void group_range(const Pack<__nv_bfloat16, 8> (&v)[H], float& lo,
                                            float& hi) {
  pair_range<LANES, __nv_bfloat162>(v, lo, hi);
}

// Rows of whole 8-weight pieces on 16-byte boundaries: a lane holds 16
// consecutive weights, a warp 512 of a row, kPieces such stretches in flight; a
// group is G / 16 neighbouring lanes, and 8 codes of a lane are one word.
constexpr int kPieces = 2;
template <class W, class S, int G>
__global__ void __launch_bounds__(256) k_q4_quantize_wide(spmv_q4 a, const W* w, long long ldw,
                                                          W* back, long long ldb,
                                                          unsigned sets) {
  constexpr int LANES = G / 16;
  grid_dependency_wait();
  grid_dependency_trigger();
  const int lane = threadIdx.x & 31;
  const unsigned rows8 = blockIdx.x / sets, set = blockIdx.x - rows8 * sets;
  const long long row = (long long)rows8 * 8 + threadIdx.x / 32;
  if (row >= a.rows) return;
  const int col0 = (int)set * (512 * kPieces) + lane * 16;
  Pack<W, 8> v[kPieces][2];
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = col0 + 512 * i + 8 * h;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][h].v[e] = from_f32<W>(0.0f);
      if (col < a.cols) v[i][h] = *reinterpret_cast<const Pack<W, 8>*>(w + row * ldw + col);
    }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    float lo, hi;
    group_range<LANES>(v[i], lo, hi);
    S scale;
    const GroupCodes c = group_codes<S>(lo, hi, a.zeros != nullptr, &scale);
    const int col = col0 + 512 * i;
    if (col >= a.cols) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (col + 8 * h >= a.cols) break;
      float in[8], u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) in[e] = to_f32(v[i][h].v[e]);
      rounded_codes<8>(in, c, u);
      // code - zero sits in the low bits of u, so the word of codes is the sum
      // of those bits, shifted, and a constant
      unsigned word = (c.zero - 0x4b400000u) * 0x11111111u;
      Pack<W, 8> o;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        word += __float_as_uint(u[e]) << (4 * e);
        o.v[e] = from_f32<W>((u[e] - kRound) * c.step);
      }
      *reinterpret_cast<unsigned*>(a.codes + row * a.ld_codes + (col + 8 * h) / 2) = word;
      if (back) *reinterpret_cast<Pack<W, 8>*>(back + row * ldb + col + 8 * h) = o;
    }
    if (lane % LANES == 0) {
      const int gi = col / G;
      static_cast<S*>(a.scales)[row * a.ld_scales + gi] = scale;
      if (a.zeros) a.zeros[row * a.ld_zeros + gi] = (uint8_t)c.zero;
    }
  }
}

// Any rows: a warp takes 256 columns of a row, read and written element by
// element in the order of the columns, and turned in shared memory into 8
// consecutive ones to a lane. (16384 x 4099 bf16 with zero points and values: 102
// us; two weights to a lane and one group to a warp took 252.)
constexpr int kAnyWarps = 8;
template <class W, class S, int G>
__global__ void __launch_bounds__(32 * kAnyWarps) k_q4_quantize(spmv_q4 a, const W* w,
                                                                long long ldw, W* back,
                                                                long long ldb, unsigned sets) {
  constexpr int LANES = G / 8;
  __shared__ Pack<W, 8> turned[kAnyWarps][32];
  __shared__ unsigned words[kAnyWarps][32];
  grid_dependency_wait();
  grid_dependency_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned rows8 = blockIdx.x / sets, set = blockIdx.x - rows8 * sets;
  const long long row = (long long)rows8 * kAnyWarps + warp;
  if (row >= a.rows) return;
  const int col0 = (int)set * 256;
  const int n = min(a.cols - col0, 256);  // columns here
  W* const elements = reinterpret_cast<W*>(turned[warp]);
  W in[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    in[i] = lane + 32 * i < n ? w[row * ldw + col0 + lane + 32 * i] : from_f32<W>(0.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) elements[lane + 32 * i] = in[i];
  __syncwarp();
  const Pack<W, 8> v[1] = {turned[warp][lane]};
  float lo, hi;
  group_range<LANES>(v, lo, hi);
  S scale;
  const GroupCodes c = group_codes<S>(lo, hi, a.zeros != nullptr, &scale);
  const int mine = min(max(n - 8 * lane, 0), 8);  // of the lane's columns
  float f[8], u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = to_f32(v[0].v[e]);
  rounded_codes<8>(f, c, u);
  unsigned word = (c.zero - 0x4b400000u) * 0x11111111u;
  Pack<W, 8> o;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    word += __float_as_uint(u[e]) << (4 * e);
    o.v[e] = from_f32<W>((u[e] - kRound) * c.step);
  }
  words[warp][lane] = mine == 8 ? word : word & ((1u << (4 * mine)) - 1u);
  if (back) turned[warp][lane] = o;
  if (lane % LANES == 0 && mine > 0) {
    const int gi = (col0 + 8 * lane) / G;
    static_cast<S*>(a.scales)[row * a.ld_scales + gi] = scale;
    if (a.zeros) a.zeros[row * a.ld_zeros + gi] = (uint8_t)c.zero;
  }
  __syncwarp();
  const uint8_t* const bytes = reinterpret_cast<const uint8_t*>(words[warp]);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < (n + 1) / 2)
      a.codes[row * a.ld_codes + col0 / 2 + lane + 32 * i] = bytes[lane + 32 * i];
  if (back)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < n) back[row * ldb + col0 + lane + 32 * i] = elements[lane + 32 * i];
}

// ---------------------------------------------------------------------------
// Rows back in dense form: 8 columns to a lane and load, kRowLoads of them in
// flight, G lanes to a token and stretch. Bound by the bytes written and, 0.55 of
// the issue slots, by the conversions: 4096 rows of 5120 bf16 results 12.0 us, 4.0
// TB/s.
// ---------------------------------------------------------------------------
constexpr int kRowLoads = 4;
template <class O>
__global__ void __launch_bounds__(256) k_embed_q4(spmv_q4 a, int n, int logG, int logGroup,
                                                  const void* tokens, int wide,
                                                  float scale, O* out,
                                                  long long ldo) {
  grid_dependency_wait();
  grid_dependency_trigger();
  const int G = 1 << logG;
  const long long t = (long long)blockIdx.x * (256 >> logG) + (threadIdx.x >> logG);
  if (t >= n) return;
  const long long r = !tokens ? t
                      : wide  ? static_cast<const long long*>(tokens)[t]
                              : (long long)static_cast<const int*>(tokens)[t];
  const bool valid = r >= 0 && r < a.rows;
  constexpr int E = 8;
  const int k0 = ((int)blockIdx.y * kRowLoads * G + (threadIdx.x & (G - 1))) * E;
  unsigned w[kRowLoads];
  float s[kRowLoads], z[kRowLoads];
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) {
    const int k = k0 + i * G * E;
    w[i] = 0;
    s[i] = 0.0f;
    z[i] = 8.0f;
    if (valid && k < a.cols) {
      const uint8_t* q = a.codes + r * a.ld_codes + k / 2;
      w[i] = *reinterpret_cast<const unsigned*>(q);
      s[i] = scale_at(a.scales, a.scale_type, r * a.ld_scales + (k >> logGroup));
      if (a.zeros) z[i] = (float)a.zeros[r * a.ld_zeros + (k >> logGroup)];
    }
  }
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) {
    const int k = k0 + i * G * E;
    if (k >= a.cols) break;
    Pack<O, E> o;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o.v[e] = from_f32<O>(valid ? ((float)((w[i] >> (4 * e)) & 15u) - z[i]) * s[i] * scale : 0.0f);
    *reinterpret_cast<Pack<O, E>*>(out + t * ldo + k) = o;
  }
}

// Any rows: a warp takes 256 columns of a token's row, the codes read byte by byte
// and the results written element by element, turned in shared memory.
template <class O>
__global__ void __launch_bounds__(32 * kAnyWarps) k_embed_q4_any(
    spmv_q4 a, int n, int logGroup, const void* tokens, int wide, float scale,
    O* out, long long ldo) {
  __shared__ Pack<O, 8> turned[kAnyWarps][32];
  __shared__ unsigned words[kAnyWarps][32];
  grid_dependency_wait();
  grid_dependency_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long t = (long long)blockIdx.x * kAnyWarps + warp;
  if (t >= n) return;
  const long long r = !tokens ? t
                      : wide  ? static_cast<const long long*>(tokens)[t]
                              : (long long)static_cast<const int*>(tokens)[t];
  const bool valid = r >= 0 && r < a.rows;
  const int col0 = (int)blockIdx.y * 256;
  const int m = min(a.cols - col0, 256);  // columns here
  uint8_t* const bytes = reinterpret_cast<uint8_t*>(words[warp]);
  float s = 0.0f, z = 8.0f;
  if (valid) {
    uint8_t in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      in[i] = lane + 32 * i < (m + 1) / 2
                  ? a.codes[r * a.ld_codes + col0 / 2 + lane + 32 * i]
                  : (uint8_t)0;
    const int k = min(col0 + 8 * lane, a.cols - 1);
    s = scale_at(a.scales, a.scale_type, r * a.ld_scales + (k >> logGroup));
    if (a.zeros) z = (float)a.zeros[r * a.ld_zeros + (k >> logGroup)];
#pragma unroll
    for (int i = 0; i < 4; ++i) bytes[lane + 32 * i] = in[i];
  }
  __syncwarp();
  const unsigned w = words[warp][lane];
  Pack<O, 8> o;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    o.v[e] = from_f32<O>(valid ? ((float)((w >> (4 * e)) & 15u) - z) * s * scale : 0.0f);
  turned[warp][lane] = o;
  __syncwarp();
  const O* const elements = reinterpret_cast<const O*>(turned[warp]);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (lane + 32 * i < m) out[t * ldo + col0 + lane + 32 * i] = elements[lane + 32 * i];
}

// The host-side checks of a 4-bit matrix: sizes, types and leading dimensions
// always, the arrays when the matrix is not empty.
int check_q4(const spmv_q4* a) {
  if (!a || a->rows < 0 || a->cols < 0 || !dtype_ok(a->scale_type)) return SPMV_ERR_INVALID_ARG;
  if (a->group != 32 && a->group != 64 && a->group != 128) return SPMV_ERR_INVALID_ARG;
  const long long groups = ((long long)a->cols + a->group - 1) / a->group;
  if (a->ld_codes < ((long long)a->cols + 1) / 2 || a->ld_scales < groups)
    return SPMV_ERR_INVALID_ARG;
  if (a->zeros && a->ld_zeros < groups) return SPMV_ERR_INVALID_ARG;
  if (a->rows == 0 || a->cols == 0) return SPMV_OK;
  if (!a->codes || !a->scales || misaligned(a->scales, dtype_bytes(a->scale_type)))
    return SPMV_ERR_INVALID_ARG;
  return SPMV_OK;
}

}  // namespace
}  // namespace spmv

namespace spmv {
namespace q4 {

// The split of a launch: P, the blocks that share a tile's columns, and the
// blocks on an SM, whose cost by this model is the least. In tenths of a
// microsecond, fitted to 8 shapes from 1024 x 1024 to 131072 x 4096: a warp's
// step takes 20 with two blocks on an SM and 14 with one, bringing 4 KB of x
// into shared memory 4, a phase's start 30, a join across the cluster 4 + 2 P
// (8192 x 28672 with one bf16 vector: P = 4 with two blocks 29.5 us, P = 1
// 37.0, one block 43.8; 1024 x 1024: P = 1 4.0, P = 2 4.6; 600 x 16384 with
// two vectors: P = 8 6.2, P = 1 18.0).
Plan make_plan(const RunArgs& p, int columns, int stepCols, int ringBytes, const Residency& res) {
  Plan best{};
  long long bestCost = -1;
  const long long tiles = ((long long)p.a.rows + kTileRows - 1) / kTileRows;
  const int steps = (int)(((long long)p.a.cols + stepCols - 1) / stepCols);
  const int perStep = columns * stepCols * 2;  // x bytes of a step
  const int slot = kTileRows * columns * 4;    // partial sums of a tile and warp
  const int tileSum = kTileRows * p.n * 4;
  for (int i = 0; i < 4 && (1 << i) <= (steps > 0 ? steps : 1); ++i) {
    for (int onSm = 1; onSm <= 2; ++onSm) {
      Plan c{};
      c.P = 1 << i;
      c.logP = i;
      c.tiles = tiles;
      c.steps = steps;
      const int own = steps > 0 ? (steps + c.P - 1) / c.P : 1;
      const long long atOnce = res.clusters[i][onSm - 1];
      if (atOnce < 1) continue;
      // a block's shared memory: its share of an SM's, less the 1 KB that each
      // takes for itself; x in as few phases of equal length as there is room for
      const long long room = (kMaxSmem + 1024) / onSm - 1024 - ringBytes -
                             (long long)(kWarps - 1) * slot;
      long long tilesEach = (tiles + atOnce - 1) / atOnce;
      int phases = 1;
      for (;; ++phases) {
        c.phaseSteps = (own + phases - 1) / phases;
        const long long perTile = slot + (phases > 1 ? tileSum : 0);
        const long long left = room - (long long)c.phaseSteps * perStep;
        if (left >= perTile && (left >= tilesEach * perTile || phases >= 4 || c.phaseSteps == 1)) {
          if (left < tilesEach * perTile) tilesEach = left / perTile;
          break;
        }
        if (c.phaseSteps == 1) {
          tilesEach = 0;
          break;
        }
      }
      if (tilesEach < 1) continue;
      const long long waves = (tiles + atOnce * tilesEach - 1) / (atOnce * tilesEach);
      c.clusters = atOnce * waves < tiles ? atOnce * waves : tiles;
      if (c.clusters < 1) c.clusters = 1;
      c.maxTiles = (int)((tiles + c.clusters - 1) / c.clusters);
      c.smem = (size_t)ringBytes + (size_t)c.phaseSteps * perStep +
               (size_t)(c.maxTiles + kWarps - 1) * slot +
               (phases > 1 ? (size_t)c.maxTiles * tileSum : 0);
      const long long units = ((long long)c.maxTiles * own + kWarps - 1) / kWarps;
      const long long fetches = ((long long)own * perStep + 4095) / 4096;
      const long long cost =
          waves * (units * (onSm == 1 ? 14 : 20) + fetches * 4 + phases * 30) +
          (c.P > 1 ? 4 + 2 * c.P : 0);
      if (bestCost < 0 || cost < bestCost) {
        bestCost = cost;
        best = c;
      }
    }
  }
  return best;
}

cudaError_t Residency::ask(const void* kernel) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (devices.load(std::memory_order_acquire) & bit) return cudaSuccess;
  std::lock_guard<std::mutex> lock(mu);
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < 4 && devices.load(std::memory_order_relaxed) == 0; ++i)
    for (int m = 0; m < 2; ++m) {
      int n = num_sms() * (m + 1);
      if (i > 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(n >> i << i));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = (kMaxSmem + 1024) / (m + 1) - 1024;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1u << i;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess) return e;
      }
      clusters[i][m] = n;
    }
  devices.fetch_or(bit, std::memory_order_release);
  return cudaSuccess;
}

}  // namespace q4
}  // namespace spmv

extern "C" {

int spmv_q4_quantize(const spmv_q4* a, spmv_dtype wType, const void* d_w, int64_t ldw,
                     void* d_back, int64_t ld_back, void* stream) {
  using namespace spmv;
  int st = check_q4(a);
  if (st != SPMV_OK) return st;
  if (!dtype_ok(wType) || ldw < a->cols || (d_back && ld_back < a->cols))
    return SPMV_ERR_INVALID_ARG;
  if (a->rows == 0 || a->cols == 0) return SPMV_OK;
  const int wb = dtype_bytes(wType);
  if (!d_w || misaligned(d_w, wb) || misaligned(d_back, wb)) return SPMV_ERR_INVALID_ARG;
  const long long groups = ((long long)a->cols + a->group - 1) / a->group;
  const void* arr[] = {d_w, a->codes, a->scales, d_back, a->zeros};
  const long long len[] = {extent(a->rows, a->cols, ldw, wb),
                           extent(a->rows, ((long long)a->cols + 1) / 2, a->ld_codes, 1),
                           extent(a->rows, groups, a->ld_scales, dtype_bytes(a->scale_type)),
                           d_back ? extent(a->rows, a->cols, ld_back, wb) : 0,
                           a->zeros ? extent(a->rows, groups, a->ld_zeros, 1) : 0};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j)
      if (overlap(arr[i], len[i], arr[j], len[j]) &&
          !(i == 0 && j == 3 && d_back == d_w && ld_back == ldw))
        return SPMV_ERR_INVALID_ARG;
  st = check_current_device_ptrs(arr, 5);
  if (st != SPMV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = a->cols % 8 == 0 && aligned16(d_w) && ldw * wb % 16 == 0 &&
                    aligned16(d_back) && (!d_back || ld_back * wb % 16 == 0) &&
                    !misaligned(a->codes, 4) && a->ld_codes % 4 == 0;
  const int columns = wide ? 512 * kPieces : 256;  // of a warp
  const long long sets = ((long long)a->cols + columns - 1) / columns;
  const long long blocks = ((long long)a->rows + 7) / 8 * sets;
  if (blocks > 0x7fffffffLL) return SPMV_ERR_TOO_LARGE;
  return record_cuda(with_dtype(wType, [&](auto wv) {
    return with_dtype(a->scale_type, [&](auto sv) {
      using W = decltype(wv);
      using S = decltype(sv);
      const auto kernel =
          wide ? (a->group == 32   ? k_q4_quantize_wide<W, S, 32>
                  : a->group == 64 ? k_q4_quantize_wide<W, S, 64>
                                   : k_q4_quantize_wide<W, S, 128>)
               : (a->group == 32   ? k_q4_quantize<W, S, 32>
                  : a->group == 64 ? k_q4_quantize<W, S, 64>
                                   : k_q4_quantize<W, S, 128>);
      return launch_dependent(kernel, dim3((unsigned)blocks), 256, s, *a,
                              static_cast<const W*>(d_w), (long long)ldw,
                              static_cast<W*>(d_back), (long long)ld_back, (unsigned)sets);
    });
  }));
}

int spmv_q4_run(const spmv_q4* a, int32_t n, spmv_dtype xType, const void* d_x, int64_t ldx,
                const void* d_c, int64_t ldc, spmv_dtype yType, void* d_y, int64_t ldy,
                void* stream) {
  using namespace spmv;
  int st = check_q4(a);
  if (st != SPMV_OK) return st;
  if (n < 0 || !dtype_ok(xType) || !dtype_ok(yType)) return SPMV_ERR_INVALID_ARG;
  if (ldx < a->cols || ldy < a->rows || (d_c && ldc < a->rows)) return SPMV_ERR_INVALID_ARG;
  if (n == 0 || a->rows == 0) return SPMV_OK;
  const int xb = dtype_bytes(xType), yb = dtype_bytes(yType);
  if (!d_y || (a->cols > 0 && !d_x)) return SPMV_ERR_INVALID_ARG;
  if (misaligned(d_x, xb) || misaligned(d_y, yb) || misaligned(d_c, yb))
    return SPMV_ERR_INVALID_ARG;
  const long long yLen = extent(n, a->rows, ldy, yb);
  const long long groups = ((long long)a->cols + a->group - 1) / a->group;
  if (overlap(d_y, yLen, d_x, extent(n, a->cols, ldx, xb)) ||
      overlap(d_y, yLen, a->codes,
              extent(a->rows, ((long long)a->cols + 1) / 2, a->ld_codes, 1)) ||
      overlap(d_y, yLen, a->scales,
              extent(a->rows, groups, a->ld_scales, dtype_bytes(a->scale_type))) ||
      (a->zeros && overlap(d_y, yLen, a->zeros, extent(a->rows, groups, a->ld_zeros, 1))))
    return SPMV_ERR_INVALID_ARG;
  if (d_c && !(d_c == d_y && ldc == ldy) && overlap(d_y, yLen, d_c, extent(n, a->rows, ldc, yb)))
    return SPMV_ERR_INVALID_ARG;
  const void* ptrs[] = {a->cols > 0 ? a->codes : nullptr, a->cols > 0 ? a->scales : nullptr,
                        a->cols > 0 ? a->zeros : nullptr, a->cols > 0 ? d_x : nullptr, d_c, d_y};
  st = check_current_device_ptrs(ptrs, 6);
  if (st != SPMV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  q4::RunArgs r{};
  r.a = *a;
  r.codesEnd = a->codes + extent(a->rows, ((long long)a->cols + 1) / 2, a->ld_codes, 1);
  r.ldx = ldx;
  r.xVec = aligned16(d_x) && (n == 1 || ldx * xb % 16 == 0);
  r.ldc = ldc;
  r.yType = yType;
  r.ldy = ldy;
  return record_cuda(with_dtype(xType, [&](auto xv) {
    using X = decltype(xv);
    constexpr int most = q4::vectors_per_pass<X>();
    for (int j = 0; j < n; j += most) {
      r.n = n - j < most ? n - j : most;
      r.x = static_cast<const X*>(d_x) + j * ldx;
      r.y = static_cast<char*>(d_y) + j * ldy * yb;
      r.c = d_c ? static_cast<const char*>(d_c) + j * ldc * yb : nullptr;
      const cudaError_t e = q4::launch_run<X>(r, s);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }));
}

int spmv_embed_q4(const spmv_q4* a, int32_t nTokens, int32_t indexBytes, const void* d_tokens,
                  float scale, spmv_dtype outType, void* d_out, int64_t ld_out, void* stream) {
  using namespace spmv;
  int st = check_q4(a);
  if (st != SPMV_OK) return st;
  if (nTokens < 0 || !dtype_ok(outType) || ld_out < a->cols) return SPMV_ERR_INVALID_ARG;
  if (indexBytes != 4 && indexBytes != 8) return SPMV_ERR_INVALID_ARG;
  if (nTokens == 0 || a->cols == 0) return SPMV_OK;
  const int ob = dtype_bytes(outType);
  if (!d_out || misaligned(d_out, ob) || misaligned(d_tokens, indexBytes))
    return SPMV_ERR_INVALID_ARG;
  if (!d_tokens && nTokens > a->rows) return SPMV_ERR_INVALID_ARG;
  const long long oLen = extent(nTokens, a->cols, ld_out, ob);
  const long long groups = ((long long)a->cols + a->group - 1) / a->group;
  if (overlap(d_out, oLen, a->codes,
              extent(a->rows, ((long long)a->cols + 1) / 2, a->ld_codes, 1)) ||
      overlap(d_out, oLen, a->scales,
              extent(a->rows, groups, a->ld_scales, dtype_bytes(a->scale_type))) ||
      (a->zeros && overlap(d_out, oLen, a->zeros, extent(a->rows, groups, a->ld_zeros, 1))) ||
      (d_tokens && overlap(d_out, oLen, d_tokens, (long long)nTokens * indexBytes)))
    return SPMV_ERR_INVALID_ARG;
  const void* ptrs[] = {a->rows > 0 ? a->codes : nullptr, a->rows > 0 ? a->scales : nullptr,
                        a->rows > 0 ? a->zeros : nullptr, d_tokens, d_out};
  st = check_current_device_ptrs(ptrs, 5);
  if (st != SPMV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = a->cols % 8 == 0 && aligned16(d_out) && ld_out * ob % 16 == 0 &&
                    !misaligned(a->codes, 4) && a->ld_codes % 4 == 0;
  const int logGroup = a->group == 32 ? 5 : a->group == 64 ? 6 : 7;
  const long long pieces = ((long long)a->cols + 7) / 8;
  int logG = 0;
  while (logG < 5 && (kRowLoads << logG) < pieces) ++logG;
  const int each = wide ? 256 >> logG : kAnyWarps;  // tokens of a block
  const long long y = wide ? (pieces + (kRowLoads << logG) - 1) / (kRowLoads << logG)
                           : ((long long)a->cols + 255) / 256;
  if (y > 65535) return SPMV_ERR_TOO_LARGE;
  const dim3 grid((unsigned)(((long long)nTokens + each - 1) / each), (unsigned)y);
  return record_cuda(with_dtype(outType, [&](auto ov) {
    using O = decltype(ov);
    O* out = static_cast<O*>(d_out);
    return wide ? launch_dependent(k_embed_q4<O>, grid, 256, s, *a, (int)nTokens, logG, logGroup,
                                   d_tokens, (int)(indexBytes == 8), scale, out,
                                   (long long)ld_out)
                : launch_dependent(k_embed_q4_any<O>, grid, 32 * kAnyWarps, s, *a, (int)nTokens,
                                   logGroup, d_tokens, (int)(indexBytes == 8), scale, out,
                                   (long long)ld_out);
  }));
}

}  // extern "C"
