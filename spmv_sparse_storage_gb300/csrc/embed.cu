// embed.cu -- token lookups in a dense table and the gradient of the lookup.
//
// A lookup of T tokens is the product of a T x vocab matrix with one entry
// (scale) per row, at the token's column, and the table; its gradient with
// respect to the table is the transposed product: row v of the gradient is
// scale times the sum of the rows of g whose token is v.
#include "dtypes.cuh"
#include "device_util.cuh"
#include "internal.h"

namespace spmv {
namespace {

__device__ __forceinline__ long long token_at(const void* tokens, int wide, long long i) {
  return wide ? static_cast<const long long*>(tokens)[i]
              : (long long)static_cast<const int*>(tokens)[i];
}

// ---------------------------------------------------------------------------
// Lookup: E elements to a lane and load, kRowLoads of them in flight, G lanes to
// a token and stretch of its row. Bound by the bytes read and written.
// ---------------------------------------------------------------------------
constexpr int kRowLoads = 4;
template <class T, class O, int E>
__global__ void __launch_bounds__(256) k_embed(int n, int vocab, int dim, int logG,
                                               const T* __restrict__ table, long long ldt,
                                               const void* __restrict__ tokens, int wide,
                                               float scale, O* __restrict__ out, long long ldo) {
  grid_dependency_wait();
  grid_dependency_trigger();
  const int G = 1 << logG;
  const long long t = (long long)blockIdx.x * (256 >> logG) + (threadIdx.x >> logG);
  if (t >= n) return;
  const long long token = token_at(tokens, wide, t);
  const bool valid = token >= 0 && token < vocab;
  const int k0 = ((int)blockIdx.y * kRowLoads * G + (threadIdx.x & (G - 1))) * E;
  Pack<T, E> v[kRowLoads];
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) {
    const int k = k0 + i * G * E;
    if (valid && k < dim) v[i] = *reinterpret_cast<const Pack<T, E>*>(table + token * ldt + k);
  }
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) {
    const int k = k0 + i * G * E;
    if (k >= dim) break;
    Pack<O, E> o;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o.v[e] = from_f32<O>(valid ? scale * to_f32(v[i].v[e]) : 0.0f);
    *reinterpret_cast<Pack<O, E>*>(out + t * ldo + k) = o;
  }
}

// ---------------------------------------------------------------------------
// Gradient. The tokens are sorted (equal ones in order); the sorted positions
// are cut into chunks of kSumChunk, each summed by one group of threads that
// hold a slab of columns. A row whose tokens lie inside a chunk is finished
// there; one that crosses chunk borders leaves a partial sum per chunk, and
// the group of the chunk in which it starts adds them up afterwards.
// ---------------------------------------------------------------------------
constexpr int kSumChunk = 32;
constexpr int kSumThreads = 256;

// partial sums of chunk c: [2c] of the row that began before it, [2c + 1] of
// the row that begins in it and goes on after it
__host__ __device__ inline long long sum_chunks(long long n) {
  return (n + kSumChunk - 1) / kSumChunk;
}

template <class O, int E>
__device__ __forceinline__ void finish_row(O* p, const float (&acc)[E], float scale,
                                           int accumulate) {
  Pack<O, E> o;
  if (accumulate) o = *reinterpret_cast<const Pack<O, E>*>(p);
#pragma unroll
  for (int e = 0; e < E; ++e)
    o.v[e] = from_f32<O>(accumulate ? to_f32(o.v[e]) + scale * acc[e] : scale * acc[e]);
  *reinterpret_cast<Pack<O, E>*>(p) = o;
}

// G lanes (a power of two) hold one slab of a row's columns, E each.
template <class T, class O, int E>
__global__ void __launch_bounds__(kSumThreads) k_embed_sum(
    int n, int vocab, int dim, int G, const int* __restrict__ pos, const int* __restrict__ key,
    const T* __restrict__ g, long long ldg, float scale, int accumulate, O* __restrict__ dtable,
    long long ldd, float* __restrict__ part) {
  constexpr int U = 4;  // rows of g in flight
  const int perBlock = kSumThreads / G;
  const long long chunk = (long long)blockIdx.x * perBlock + threadIdx.x / G;
  const long long col = ((long long)blockIdx.y * G + threadIdx.x % G) * E;
  if (chunk >= sum_chunks(n) || col >= dim) return;
  const long long c0 = chunk * kSumChunk;
  const long long c1 = min(c0 + kSumChunk, (long long)n);
  int cur = key[c0];
  if (cur >= vocab) return;
  bool openLeft = c0 > 0 && key[c0 - 1] == cur;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
  auto flush = [&](bool openRight) {
    if (openLeft || openRight) {
      float* p = part + (2 * chunk + (openLeft ? 0 : 1)) * dim + col;
#pragma unroll
      for (int e = 0; e < E; ++e) p[e] = acc[e];
    } else {
      finish_row<O, E>(dtable + cur * ldd + col, acc, scale, accumulate);
    }
  };
  bool done = false;
  for (long long b = c0; b < c1 && !done; b += U) {
    Pack<T, E> v[U];
    int k[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      k[u] = b + u < c1 ? key[b + u] : vocab;
      if (k[u] < vocab) v[u] = *reinterpret_cast<const Pack<T, E>*>(g + pos[b + u] * ldg + col);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k[u] >= vocab) {
        done = true;
        break;
      }
      if (k[u] != cur) {
        flush(false);
        cur = k[u];
        openLeft = false;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += to_f32(v[u].v[e]);
    }
  }
  flush(c1 < n && key[c1] == cur);
}

template <class O, int E>
__global__ void __launch_bounds__(kSumThreads) k_embed_join(
    int n, int vocab, int dim, int G, const int* __restrict__ key,
    const float* __restrict__ part, float scale, int accumulate, O* __restrict__ dtable,
    long long ldd) {
  const int perBlock = kSumThreads / G;
  const long long chunk = (long long)blockIdx.x * perBlock + threadIdx.x / G;
  const long long col = ((long long)blockIdx.y * G + threadIdx.x % G) * E;
  if (chunk >= sum_chunks(n) || col >= dim) return;
  const long long c0 = chunk * kSumChunk;
  long long end = c0 + kSumChunk;
  if (end >= n) return;
  const int row = key[end - 1];
  if (row >= vocab || key[end] != row) return;
  if (key[c0] == row && c0 > 0 && key[c0 - 1] == row) return;  // starts in an earlier chunk
  float acc[E];
  const float* p = part + (2 * chunk + 1) * dim + col;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = p[e];
  for (long long c = chunk + 1;; ++c) {
    p = part + 2 * c * dim + col;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += p[e];
    end += kSumChunk;
    if (end >= n || key[end - 1] != row || key[end] != row) break;
  }
  finish_row<O, E>(dtable + row * ldd + col, acc, scale, accumulate);
}

// Zeros in the rows that no token names, one warp per row.
template <class O>
__global__ void __launch_bounds__(256) k_embed_zero(int n, int vocab, int dim,
                                                    const int* __restrict__ key,
                                                    O* __restrict__ dtable, long long ldd) {
  const long long v = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  if (v >= vocab) return;
  long long lo = 0, hi = n;
  while (lo < hi) {
    const long long mid = (lo + hi) / 2;
    if (key[mid] < v)
      lo = mid + 1;
    else
      hi = mid;
  }
  if (lo < n && key[lo] == v) return;
  for (int k = threadIdx.x % 32; k < dim; k += 32) dtable[v * ldd + k] = from_f32<O>(0.0f);
}

struct GradWork {
  long long sortBytes, partBytes;
};
GradWork grad_work(int vocab, int dim, int n) {
  GradWork w{0, 0};
  if (vocab <= 0 || dim <= 0 || n <= 0) return w;
  w.sortBytes = ((long long)token_sort_scratch_bytes(n, vocab) + 255) & ~255LL;
  w.partBytes = 2 * sum_chunks(n) * (long long)dim * 4;
  return w;
}

}  // namespace
}  // namespace spmv

extern "C" {

int spmv_embed(int32_t vocab, int32_t dim, spmv_dtype tableType, const void* d_table,
               int64_t ld_table, int32_t nTokens, int32_t indexBytes, const void* d_tokens,
               float scale, spmv_dtype outType, void* d_out, int64_t ld_out, void* stream) {
  using namespace spmv;
  if (vocab < 0 || dim < 0 || nTokens < 0 || !dtype_ok(tableType) || !dtype_ok(outType))
    return SPMV_ERR_INVALID_ARG;
  if (indexBytes != 4 && indexBytes != 8) return SPMV_ERR_INVALID_ARG;
  if (ld_table < dim || ld_out < dim) return SPMV_ERR_INVALID_ARG;
  if (nTokens == 0 || dim == 0) return SPMV_OK;
  if (!d_tokens || !d_out || (vocab > 0 && !d_table)) return SPMV_ERR_INVALID_ARG;
  if (misaligned(d_table, dtype_bytes(tableType)) || misaligned(d_out, dtype_bytes(outType)) ||
      misaligned(d_tokens, indexBytes))
    return SPMV_ERR_INVALID_ARG;
  const long long oLen = extent(nTokens, dim, ld_out, dtype_bytes(outType));
  if (overlap(d_out, oLen, d_table, extent(vocab, dim, ld_table, dtype_bytes(tableType))) ||
      overlap(d_out, oLen, d_tokens, (long long)nTokens * indexBytes))
    return SPMV_ERR_INVALID_ARG;
  const void* ptrs[] = {d_table, d_tokens, d_out};
  int st = check_current_device_ptrs(ptrs, 3);
  if (st != SPMV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int tb = dtype_bytes(tableType), ob = dtype_bytes(outType);
  const bool wide = dim % 8 == 0 && aligned16(d_table) && ld_table * tb % 16 == 0 &&
                    aligned16(d_out) && ld_out * ob % 16 == 0;
  const int E = wide ? 8 : 1;
  const long long pieces = ((long long)dim + E - 1) / E;
  int logG = 0;
  while (logG < 5 && (kRowLoads << logG) < pieces) ++logG;
  const long long y = (pieces + (kRowLoads << logG) - 1) / (kRowLoads << logG);
  if (y > 65535) return SPMV_ERR_TOO_LARGE;
  const dim3 grid((unsigned)(((long long)nTokens + (256 >> logG) - 1) / (256 >> logG)), (unsigned)y);
  return record_cuda(with_dtype(tableType, [&](auto tv) {
    return with_dtype(outType, [&](auto ov) {
      using T = decltype(tv);
      using O = decltype(ov);
      return launch_dependent(wide ? k_embed<T, O, 8> : k_embed<T, O, 1>, grid, 256, s,
                              (int)nTokens, (int)vocab, (int)dim, logG,
                              static_cast<const T*>(d_table), (long long)ld_table, d_tokens,
                              (int)(indexBytes == 8), scale, static_cast<O*>(d_out),
                              (long long)ld_out);
    });
  }));
}

int spmv_embed_grad_workspace(int32_t vocab, int32_t dim, int32_t nTokens, int64_t* bytes) {
  if (vocab < 0 || dim < 0 || nTokens < 0 || !bytes) return SPMV_ERR_INVALID_ARG;
  const spmv::GradWork w = spmv::grad_work(vocab, dim, nTokens);
  *bytes = w.sortBytes + w.partBytes;
  return SPMV_OK;
}

int spmv_embed_grad(int32_t vocab, int32_t dim, spmv_dtype gType, const void* d_g, int64_t ld_g,
                    int32_t nTokens, int32_t indexBytes, const void* d_tokens, float scale,
                    int32_t accumulate, spmv_dtype tableType, void* d_dtable, int64_t ld_dtable,
                    void* d_work, int64_t workBytes, void* stream) {
  using namespace spmv;
  if (vocab < 0 || dim < 0 || nTokens < 0 || !dtype_ok(gType) || !dtype_ok(tableType))
    return SPMV_ERR_INVALID_ARG;
  if ((indexBytes != 4 && indexBytes != 8) || (accumulate != 0 && accumulate != 1))
    return SPMV_ERR_INVALID_ARG;
  if (ld_g < dim || ld_dtable < dim || workBytes < 0) return SPMV_ERR_INVALID_ARG;
  if (vocab == 0 || dim == 0 || (nTokens == 0 && accumulate)) return SPMV_OK;
  const GradWork w = grad_work(vocab, dim, nTokens);
  if (!d_dtable || (nTokens > 0 && (!d_g || !d_tokens || !d_work))) return SPMV_ERR_INVALID_ARG;
  if (nTokens > 0 && workBytes < w.sortBytes + w.partBytes) return SPMV_ERR_INVALID_ARG;
  if (misaligned(d_g, dtype_bytes(gType)) || misaligned(d_dtable, dtype_bytes(tableType)) ||
      misaligned(d_tokens, indexBytes) || (nTokens > 0 && misaligned(d_work, 16)))
    return SPMV_ERR_INVALID_ARG;
  const long long gBytes = extent(nTokens, dim, ld_g, dtype_bytes(gType));
  const long long tBytes = extent(vocab, dim, ld_dtable, dtype_bytes(tableType));
  const long long wBytes = nTokens > 0 ? workBytes : 0;
  if (overlap(d_g, gBytes, d_dtable, tBytes) || overlap(d_work, wBytes, d_dtable, tBytes) ||
      overlap(d_work, wBytes, d_g, gBytes) ||
      overlap(d_tokens, (long long)nTokens * indexBytes, d_dtable, tBytes) ||
      overlap(d_tokens, (long long)nTokens * indexBytes, d_work, wBytes))
    return SPMV_ERR_INVALID_ARG;
  const void* ptrs[] = {d_g, d_tokens, d_dtable, d_work};
  int st = check_current_device_ptrs(ptrs, nTokens > 0 ? 4 : 3);
  if (st != SPMV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int *pos = nullptr, *key = nullptr;
  if (nTokens > 0) {
    st = record_cuda(launch_token_sort(nTokens, vocab, d_tokens, indexBytes, d_work, &pos, &key,
                                       s));
    if (st != SPMV_OK) return st;
  }
  float* part = reinterpret_cast<float*>(static_cast<char*>(d_work) + w.sortBytes);
  return record_cuda(with_dtype(gType, [&](auto gv) {
    return with_dtype(tableType, [&](auto ov) {
      using T = decltype(gv);
      using O = decltype(ov);
      O* dt = static_cast<O*>(d_dtable);
      if (!accumulate) {
        k_embed_zero<O><<<(unsigned)(((long long)vocab + 7) / 8), 256, 0, s>>>(
            nTokens, vocab, dim, key, dt, ld_dtable);
        note_launches(1);
      }
      if (nTokens == 0) return cudaGetLastError();
      auto sum = [&](auto width) {
        constexpr int E = decltype(width)::value;
        const long long lanes = (dim + E - 1) / E;
        int G = 1;
        while (G < kSumThreads && G < lanes) G *= 2;
        const dim3 grid((unsigned)((sum_chunks(nTokens) + kSumThreads / G - 1) /
                                   (kSumThreads / G)),
                        (unsigned)((lanes + G - 1) / G));
        k_embed_sum<T, O, E><<<grid, kSumThreads, 0, s>>>(
            nTokens, vocab, dim, G, pos, key, static_cast<const T*>(d_g), ld_g, scale,
            accumulate, dt, ld_dtable, part);
        k_embed_join<O, E><<<grid, kSumThreads, 0, s>>>(nTokens, vocab, dim, G, key, part, scale,
                                                        accumulate, dt, ld_dtable);
        note_launches(2);
        return cudaGetLastError();
      };
      const bool wide = dim % 8 == 0 && ld_g % 8 == 0 && ld_dtable % 8 == 0 &&
                        aligned16(d_g) && aligned16(dt);
      return wide ? sum(std::integral_constant<int, 8>{})
                  : sum(std::integral_constant<int, 1>{});
    });
  }));
}

}  // extern "C"
