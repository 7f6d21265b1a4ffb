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
// Conversion: one warp per row and group.
// ---------------------------------------------------------------------------
template <class W, class S>
__global__ void __launch_bounds__(256) k_q4_quantize(spmv_q4 a, const W* w, long long ldw,
                                                     W* back, long long ldb) {
  const int groups = (a.cols + a.group - 1) / a.group;
  const long long id = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (id >= (long long)a.rows * groups) return;
  const long long r = id / groups;
  const int gi = (int)(id % groups);
  const int k0 = gi * a.group, k1 = min(k0 + a.group, a.cols);
  float v[4];
  float lo = 0.0f, hi = 0.0f, bad = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = k0 + 2 * lane + (j & 1) + 64 * (j >> 1);
    v[j] = k < k1 ? to_f32(w[r * ldw + k]) : 0.0f;
    lo = fminf(lo, v[j]);
    hi = fmaxf(hi, v[j]);
    if (!(fabsf(v[j]) <= 3.402823466e38f)) bad = 1.0f;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(kFullMask, lo, off));
    hi = fmaxf(hi, __shfl_xor_sync(kFullMask, hi, off));
    bad = fmaxf(bad, __shfl_xor_sync(kFullMask, bad, off));
  }
  float raw = a.zeros ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f;
  if (bad != 0.0f) raw = __int_as_float(0x7fc00000);
  const S held = from_f32<S>(raw);
  const float step = to_f32(held);
  const bool usable = step > 0.0f && step <= 3.402823466e38f;
  float zero = 8.0f;
  if (a.zeros) zero = usable ? fminf(fmaxf(rintf(-lo / step), 0.0f), 15.0f) : 0.0f;
  if (lane == 0) {
    static_cast<S*>(a.scales)[r * a.ld_scales + gi] = held;
    if (a.zeros) a.zeros[r * a.ld_zeros + gi] = (uint8_t)zero;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int k = k0 + 2 * lane + 64 * j;
    if (k >= k1) continue;
    float q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      q[i] = usable ? fminf(fmaxf(rintf(v[2 * j + i] / step) + zero, 0.0f), 15.0f) : zero;
      if (k + i >= k1)
        q[i] = 0.0f;
      else if (back)
        back[r * ldb + k + i] = from_f32<W>((q[i] - zero) * step);
    }
    a.codes[r * a.ld_codes + k / 2] = (uint8_t)((int)q[0] | (int)q[1] << 4);
  }
}

// ---------------------------------------------------------------------------
// Rows back in dense form: one block per token.
// ---------------------------------------------------------------------------
template <class O>
__global__ void __launch_bounds__(256) k_embed_q4(spmv_q4 a, const void* __restrict__ tokens,
                                                  int wide, float scale, O* __restrict__ out,
                                                  long long ldo) {
  const long long t = blockIdx.x;
  const long long r = !tokens ? t
                      : wide  ? static_cast<const long long*>(tokens)[t]
                              : (long long)static_cast<const int*>(tokens)[t];
  const bool valid = r >= 0 && r < a.rows;
  for (int k = threadIdx.x; k < a.cols; k += blockDim.x) {
    float v = 0.0f;
    if (valid) {
      const int gi = k / a.group;
      const int b = a.codes[r * a.ld_codes + k / 2];
      const float zero = a.zeros ? (float)a.zeros[r * a.ld_zeros + gi] : 8.0f;
      v = ((float)((k & 1) ? b >> 4 : b & 15) - zero) *
          scale_at(a.scales, a.scale_type, r * a.ld_scales + gi) * scale;
    }
    out[t * ldo + k] = from_f32<O>(v);
  }
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
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < 4; ++i)
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
  const long long warps = a->rows * groups;
  if ((warps + 7) / 8 > 0x7fffffffLL) return SPMV_ERR_TOO_LARGE;
  return record_cuda(with_dtype(wType, [&](auto wv) {
    return with_dtype(a->scale_type, [&](auto sv) {
      using W = decltype(wv);
      using S = decltype(sv);
      k_q4_quantize<W, S><<<(unsigned)((warps + 7) / 8), 256, 0, s>>>(
          *a, static_cast<const W*>(d_w), ldw, static_cast<W*>(d_back), ld_back);
      note_launches(1);
      return cudaGetLastError();
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
  return record_cuda(with_dtype(outType, [&](auto ov) {
    using O = decltype(ov);
    k_embed_q4<O><<<(unsigned)nTokens, 256, 0, s>>>(*a, d_tokens, indexBytes == 8, scale,
                                                    static_cast<O*>(d_out), ld_out);
    note_launches(1);
    return cudaGetLastError();
  }));
}

}  // extern "C"
