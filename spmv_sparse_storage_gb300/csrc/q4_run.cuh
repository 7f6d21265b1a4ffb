// q4_run.cuh -- y_j = A x_j + c_j for a matrix of 4-bit codes (spmv_q4_run).
//
// A[r][k] = s[r][k/G] (q[r][k] - z[r][k/G]), so y[r] is the sum over groups of
// s times the group's sum of (q - z) x. The integers q - z (-15 .. 15) are
// exact in 16 bits and so are the vectors there: the group sums are products of
// small matrices with exact operands and fp32 accumulators, which
// mma.sync.m16n8k16 forms 16 rows and 8 columns at a time. An fp32 x is cut
// into three bf16 parts that add up to it bit for bit (8 + 8 + 8 significant
// bits, by truncation), each a column of its own; their sums are added at the
// end.
//
// What bounds it: the bytes of A, half a byte per entry and one scale per
// group, read once for up to 16 columns; and, close behind, the instructions
// that turn a nibble into a 16-bit operand (11 per 8 entries). mma.sync, not
// tcgen05.mma: with 1 to 16 columns the tensor pipe is idle for most of the
// time either way, and operands go from the code words to the instruction in
// registers, without a second trip through shared memory.
//
// Layout. A tile is 16 * MT rows; a step is 128 columns of it. Each warp brings
// its steps into a ring of kStages buffers of its own by asynchronous 16-byte
// copies (64 bytes per row), so no barrier is taken between steps. Lane (g, c),
// g = lane / 4 and c = lane % 4, holds columns c * G/4 .. of each group of rows g
// and g + 8 (of each 16): any assignment of columns to the k index of an mma is
// as good as another when A and x agree, and this one keeps a group in one mma
// and a lane's codes consecutive. x is staged in the order in which the lanes
// read it, 16 bytes (8 columns: 0 4 1 5 2 6 3 7, as the code words unpack) at a
// time.
//
// Split. The rows' tiles are divided among the clusters of the grid and the
// columns among the P thread blocks of a cluster; inside a block the (tile,
// step) pairs are divided evenly among the warps. A tile's partial sums are
// left in shared memory, one slot per (warp, tile), and joined in a fixed order
// once per block, then (P > 1) across the cluster through distributed shared
// memory: the same result from run to run, and no memory outside the kernel.
#pragma once

#include <cooperative_groups.h>

#include "device_util.cuh"
#include "dtypes.cuh"
#include "internal.h"
#include "q4.h"

namespace spmv {
namespace q4 {

// --- pieces --------------------------------------------------------------------
__device__ __forceinline__ void mma16816(float (&d)[4], const unsigned (&a)[4], unsigned b0,
                                         unsigned b1, __half) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const unsigned (&a)[4], unsigned b0,
                                         unsigned b1, __nv_bfloat16) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A 16-bit operand type: the magic word m such that m | q (q < 128) is base + q
// exactly, and the packed difference.
struct OpHalf {
  using T = __half;
  static constexpr unsigned kMagic = 0x64006400u;  // 1024, unit 1
  static __device__ __forceinline__ unsigned sub(unsigned a, unsigned b) {
    unsigned d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
};
struct OpBf16 {
  using T = __nv_bfloat16;
  static constexpr unsigned kMagic = 0x43004300u;  // 128, unit 1
  static __device__ __forceinline__ unsigned sub(unsigned a, unsigned b) {
    unsigned d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
};
template <class X>
struct OpOf {
  using Op = OpBf16;
  static constexpr int kParts = 3;  // fp32: three bf16 columns
};
template <>
struct OpOf<__half> {
  using Op = OpHalf;
  static constexpr int kParts = 1;
};
template <>
struct OpOf<__nv_bfloat16> {
  using Op = OpBf16;
  static constexpr int kParts = 1;
};

// entries j and j + 4 of a code word, less their zero point (bias = magic | z)
template <class Op>
__device__ __forceinline__ unsigned unpack(unsigned w, int j, unsigned bias) {
  return Op::sub(((w >> (4 * j)) & 0x000f000fu) | Op::kMagic, bias);
}

// 16-byte asynchronous copy of the first `bytes` (1 .. 16) of a 16-byte chunk,
// zeros in the rest.
__device__ __forceinline__ void cp_async16_part(void* smem, const void* gmem, int bytes) {
  const unsigned sa = (unsigned)__cvta_generic_to_shared(smem);
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(sa), "l"(gmem),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Chunk position inside a row's 64 bytes: rows 2 apart are moved so that the
// lanes' 4-, 8- and 16-byte reads of 8 rows fall into different banks.
__device__ __forceinline__ int chunk_at(int row, int j) {
  const int p = (row >> 1) & 3;
  return j ^ (((p & 1) << 1) | (p >> 1));
}

// The 16-bit operands of 8 consecutive columns k .. k + 7 of one vector, in the
// order 0 4 1 5 2 6 3 7, one word per pair; part 0, 1 or 2 of an fp32 vector.
template <class X>
__device__ __forceinline__ void stage_x(const X* x, long long k, long long cols, bool vec,
                                        uint4* out, int stride) {
  Pack<X, 8> v;
  if (vec && k + 8 <= cols) {
    v = *reinterpret_cast<const Pack<X, 8>*>(x + k);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.v[i] = k + i < cols ? x[k + i] : from_f32<X>(0.0f);
  }
  unsigned h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = *reinterpret_cast<const unsigned short*>(&v.v[i]);
  *out = make_uint4(h[0] | h[4] << 16, h[1] | h[5] << 16, h[2] | h[6] << 16, h[3] | h[7] << 16);
}
template <>
__device__ __forceinline__ void stage_x<float>(const float* x, long long k, long long cols,
                                               bool vec, uint4* out, int stride) {
  float v[8];
  if (vec && k + 8 <= cols) {
    const float4 a = *reinterpret_cast<const float4*>(x + k);
    const float4 b = *reinterpret_cast<const float4*>(x + k + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + i < cols ? x[k + i] : 0.0f;
  }
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    unsigned h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      unsigned bits = __float_as_uint(v[i]);
      if ((bits & 0x7f800000u) == 0x7f800000u) {
        // an infinity or a NaN is its first part alone (a NaN kept one by a bit)
        h[i] = (bits >> 16) | ((bits & 0x007fffffu) ? 0x40u : 0u);
        v[i] = 0.0f;
      } else {
        h[i] = bits >> 16;
        v[i] -= __uint_as_float(bits & 0xffff0000u);
      }
    }
    out[p * stride] =
        make_uint4(h[0] | h[4] << 16, h[1] | h[5] << 16, h[2] | h[6] << 16, h[3] | h[7] << 16);
  }
}

__device__ __forceinline__ float scale_value(unsigned raw, int type) {
  if (type == SPMV_F32) return __uint_as_float(raw);
  if (type == SPMV_BF16) return __uint_as_float(raw << 16);
  return __half2float(__ushort_as_half((unsigned short)raw));
}
__device__ __forceinline__ unsigned scale_raw(const void* scales, int type, long long i) {
  return type == SPMV_F32 ? __ldg(static_cast<const unsigned*>(scales) + i)
                          : (unsigned)__ldg(static_cast<const unsigned short*>(scales) + i);
}
__device__ __forceinline__ float load_y(const void* p, int type, long long i) {
  return type == SPMV_F32   ? static_cast<const float*>(p)[i]
         : type == SPMV_F16 ? to_f32(static_cast<const __half*>(p)[i])
                            : to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_y(void* p, int type, long long i, float v) {
  if (type == SPMV_F32)
    static_cast<float*>(p)[i] = v;
  else if (type == SPMV_F16)
    static_cast<__half*>(p)[i] = from_f32<__half>(v);
  else
    static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(v);
}

// --- the kernel ------------------------------------------------------------------
// ALIGNED: every row of codes starts on a 16-byte boundary. Otherwise a row's
// 64 bytes are fetched as the (at most) 5 aligned chunks that hold them and
// shifted into place when read.
template <class X, int G, int NT, int MT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 2) k_q4_run(const RunArgs p) {
  using Op = typename OpOf<X>::Op;
  constexpr int kParts = OpOf<X>::kParts;
  constexpr int kRowBytes = ALIGNED ? 64 : 80;
  constexpr int kStep = 16 * MT * kRowBytes;  // bytes of a stage
  constexpr int kGroups = 128 / G;            // groups of a step
  constexpr int kWords = G / 32;              // code words of a lane, row and group
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const spmv_q4& a = p.a;
  const int NB = p.n * kParts;  // columns
  unsigned char* ring = smem + warp * kStages * kStep;
  uint4* xs = reinterpret_cast<uint4*>(smem + kWarps * kStages * kStep);
  float* slots = reinterpret_cast<float*>(xs + (size_t)p.phaseSteps * 16 * NB);
  const int slotFloats = 16 * MT * NB;
  float* sums = slots + (size_t)(p.maxTiles + kWarps) * slotFloats;

  const int rank = blockIdx.x % p.P;
  const long long cluster = blockIdx.x / p.P, clusters = gridDim.x / p.P;
  const int t0 = (int)(p.tiles * cluster / clusters);
  const int T = (int)(p.tiles * (cluster + 1) / clusters) - t0;
  const int s0 = (int)((long long)p.steps * rank / p.P);
  const int s1 = (int)((long long)p.steps * (rank + 1) / p.P);
  const long long rowBytes = ((long long)a.cols + 1) / 2;
  const int groups = (a.cols + G - 1) / G;
  const X* x = static_cast<const X*>(p.x);
  const int outs = T * 16 * MT * p.n;

  for (int f0 = s0; f0 == s0 || f0 < s1; f0 += p.phaseSteps) {
    const int fs = min(p.phaseSteps, s1 - f0);  // steps of this phase (0: no columns)
    const int units = T * fs;
    const int u0 = (int)((long long)units * warp / kWarps);
    const int u1 = (int)((long long)units * (warp + 1) / kWarps);
    unsigned sc[kStages][2 * MT], zr[kStages][2 * MT];

    // the copies and scale loads of unit u into stage st
    auto issue = [&](int u, int st) {
      if (u < u1) {
        const int t = u / fs, step = f0 + (u - t * fs);
        const long long r0 = (long long)(t0 + t) * (16 * MT);
        unsigned char* dst = ring + st * kStep;
        if (ALIGNED) {
          const long long off = (long long)step * 64 + (lane & 3) * 16;
          const int left = (int)min(rowBytes - off, 16LL);
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) {
            const int row = (lane >> 2) + 8 * i;
            if (left > 0 && r0 + row < a.rows)
              cp_async16_part(dst + row * 64 + chunk_at(row, lane & 3) * 16,
                              a.codes + (r0 + row) * a.ld_codes + off, left);
          }
        } else {
          // 5 chunks of each row, from the aligned address at or below its start
#pragma unroll
          for (int i = 0; i < (5 * 16 * MT + 31) / 32; ++i) {
            const int id = lane + 32 * i;
            const int row = id / 5, j = id - row * 5;
            if (row < 16 * MT && r0 + row < a.rows) {
              const unsigned char* first = a.codes + (r0 + row) * a.ld_codes;
              const unsigned char* src = reinterpret_cast<const unsigned char*>(
                  (reinterpret_cast<uintptr_t>(first + (long long)step * 64) & ~(uintptr_t)15) +
                  16 * j);
              const unsigned char* end = first + rowBytes;
              if (src < end) {
                if (src >= a.codes && src + 16 <= p.codesEnd) {
                  cp_async16_part(dst + row * 80 + j * 16, src, 16);
                } else {  // the ends of the array: byte by byte
                  for (int b = 0; b < 16; ++b)
                    if (src + b >= a.codes && src + b < p.codesEnd)
                      dst[row * 80 + j * 16 + b] = src[b];
                }
              }
            }
          }
        }
        const int gi = step * kGroups + (kGroups == 4 ? c : kGroups == 2 ? c >> 1 : 0);
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
          const long long row = min(r0 + g + 8 * i, (long long)a.rows - 1);
          sc[st][i] = gi < groups ? scale_raw(a.scales, a.scale_type, row * a.ld_scales + gi) : 0u;
          zr[st][i] = a.zeros && gi < groups ? (unsigned)__ldg(a.zeros + row * a.ld_zeros + gi)
                                             : 8u;
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int st = 0; st < kStages - 1; ++st) issue(u0 + st, st);

    // x of this phase, in fragment order: [step][word][column][c]
    if (f0 != s0) __syncthreads();  // the last phase's readers are done
    for (int i = threadIdx.x; i < fs * 16 * p.n; i += kThreads) {
      const int cc = i & 3, v = (i >> 2) % p.n, t = (i >> 2) / p.n;  // t: step * 4 + word
      const int step = t >> 2, word = t & 3;
      const long long k = (long long)(f0 + step) * 128 + (word / kWords) * G + cc * (G / 4) +
                          (word % kWords) * 8;
      stage_x<X>(x + v * p.ldx, k, a.cols, p.xVec, xs + ((size_t)t * NB + v * kParts) * 4 + cc, 4);
    }
    __syncthreads();

    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][nt][i] = 0.0f;

    int tile = fs > 0 ? u0 / fs : 0, at = u0 - tile * fs;  // unit being consumed
    for (int u = u0; u < u1; u += kStages) {
#pragma unroll
      for (int st = 0; st < kStages; ++st) {
        if (u + st < u1) {
          cp_async_wait<kStages - 2>();
          __syncwarp();
          issue(u + st + kStages - 1, (st + kStages - 1) % kStages);
          const unsigned char* buf = ring + st * kStep;
          const uint4* xb = xs + (size_t)at * 16 * NB + c;
#pragma unroll
          for (int gr = 0; gr < kGroups; ++gr) {
            float part[MT][NT][4];
            unsigned bias[2 * MT];
            float s[2 * MT];
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
              unsigned raw = sc[st][i], z = zr[st][i];
              if (kGroups > 1) {
                const int from = (lane & ~3) + gr * (4 / kGroups);
                raw = __shfl_sync(kFullMask, raw, from);
                z = __shfl_sync(kFullMask, z, from);
              }
              s[i] = scale_value(raw, a.scale_type);
              bias[i] = Op::kMagic | z | z << 16;
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[m][nt][i] = 0.0f;
            unsigned w[2 * MT][kWords];
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
              const int row = g + 8 * i;
              if (ALIGNED) {
                const int byte = gr * (G / 2) + c * (G / 8);
                const unsigned char* q =
                    buf + row * 64 + chunk_at(row, byte >> 4) * 16 + (byte & 15);
                if (kWords == 4) {
                  const uint4 v = *reinterpret_cast<const uint4*>(q);
                  w[i][0] = v.x;
                  w[i][1 % kWords] = v.y;
                  w[i][2 % kWords] = v.z;
                  w[i][3 % kWords] = v.w;
                } else if (kWords == 2) {
                  const uint2 v = *reinterpret_cast<const uint2*>(q);
                  w[i][0] = v.x;
                  w[i][1 % kWords] = v.y;
                } else {
                  w[i][0] = *reinterpret_cast<const unsigned*>(q);
                }
              } else {
                const long long r = (long long)(t0 + tile) * (16 * MT) + row;
                const unsigned shift =
                    (unsigned)(reinterpret_cast<uintptr_t>(a.codes + r * a.ld_codes) & 15);
                const unsigned byte = shift + gr * (G / 2) + c * (G / 8);
                const unsigned* q = reinterpret_cast<const unsigned*>(buf + row * 80) + (byte >> 2);
                unsigned lo = q[0];
#pragma unroll
                for (int i2 = 0; i2 < kWords; ++i2) {
                  // the last word's upper neighbour is only needed off a word boundary
                  const unsigned hi = (byte & 3) || i2 + 1 < kWords ? q[i2 + 1] : 0u;
                  w[i][i2] = __funnelshift_r(lo, hi, 8 * (byte & 3));
                  lo = hi;
                }
              }
            }
#pragma unroll
            for (int i2 = 0; i2 < kWords; ++i2) {
              uint4 b[NT];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                b[nt] = make_uint4(0, 0, 0, 0);
                const int col = nt * 8 + g;
                if (col < NB) b[nt] = xb[((gr * kWords + i2) * NB + col) * 4];
              }
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                unsigned lo[4], hi[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  lo[j] = unpack<Op>(w[2 * m][i2], j, bias[2 * m]);
                  hi[j] = unpack<Op>(w[2 * m + 1][i2], j, bias[2 * m + 1]);
                }
                const unsigned f0a[4] = {lo[0], hi[0], lo[1], hi[1]};
                const unsigned f1a[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma16816(part[m][nt], f0a, b[nt].x, b[nt].y, typename Op::T{});
                  mma16816(part[m][nt], f1a, b[nt].z, b[nt].w, typename Op::T{});
                }
              }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  acc[m][nt][i] = fmaf(s[2 * m + (i >> 1)], part[m][nt][i], acc[m][nt][i]);
          }
          ++at;
          if (at == fs || u + st + 1 == u1) {  // the tile's end, or this warp's
            float* slot = slots + (size_t)(tile + warp) * slotFloats;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int col = nt * 8 + 2 * c + (i & 1);
                  if (col < NB) slot[col * (16 * MT) + m * 16 + g + 8 * (i >> 1)] = acc[m][nt][i];
                  acc[m][nt][i] = 0.0f;
                }
            at = 0;
            ++tile;
          }
        }
      }
    }
    cp_async_wait<0>();
    __syncthreads();
    // join the warps' partial sums of each output, in the order of the columns
    const bool last = f0 + p.phaseSteps >= s1;
    for (int o = threadIdx.x; o < outs; o += kThreads) {
      const int row = o % (16 * MT), v = (o / (16 * MT)) % p.n, t = o / (16 * MT * p.n);
      float sum = f0 == s0 ? 0.0f : sums[o];
      if (fs > 0) {
        // the warp that holds unit u: the last w with units * w / kWarps <= u
        const int w0 = (int)((((long long)t * fs + 1) * kWarps - 1) / units);
        const int w1 = (int)((((long long)(t + 1) * fs) * kWarps - 1) / units);
        for (int w = w0; w <= w1; ++w) {
          if ((long long)units * w / kWarps == (long long)units * (w + 1) / kWarps) continue;
#pragma unroll
          for (int q = 0; q < kParts; ++q)
            sum += slots[(size_t)(t + w) * slotFloats + (v * kParts + q) * (16 * MT) + row];
        }
      }
      if (last && p.P == 1) {
        const long long r = (long long)(t0 + t) * (16 * MT) + row;
        if (r < a.rows) {
          if (p.c) sum += load_y(p.c, p.yType, v * p.ldc + r);
          store_y(p.y, p.yType, v * p.ldy + r, sum);
        }
      } else {
        sums[o] = sum;
      }
    }
    if (!last) __syncthreads();
  }
  if (p.P > 1) {
    namespace cgr = cooperative_groups;
    cgr::cluster_group cl = cgr::this_cluster();
    cl.sync();
    for (int o = threadIdx.x + kThreads * rank; o < outs; o += kThreads * p.P) {
      const int row = o % (16 * MT), v = (o / (16 * MT)) % p.n, t = o / (16 * MT * p.n);
      const long long r = (long long)(t0 + t) * (16 * MT) + row;
      if (r >= a.rows) continue;
      float sum = 0.0f;
      for (int q = 0; q < p.P; ++q) sum += *cl.map_shared_rank(sums + o, q);
      if (p.c) sum += load_y(p.c, p.yType, v * p.ldc + r);
      store_y(p.y, p.yType, v * p.ldy + r, sum);
    }
    cl.sync();  // the others may still be reading this block's sums
  }
}

// --- launch --------------------------------------------------------------------------
template <class X, int G, int NT, int MT, bool ALIGNED>
cudaError_t launch_one(const RunArgs& args, cudaStream_t s) {
  constexpr int kRowBytes = ALIGNED ? 64 : 80;
  const Plan plan = make_plan(args, 16 * MT, OpOf<X>::kParts * args.n,
                              kWarps * kStages * 16 * MT * kRowBytes);
  RunArgs p = args;
  p.P = plan.P;
  p.phaseSteps = plan.phaseSteps;
  p.maxTiles = plan.maxTiles;
  p.tiles = plan.tiles;
  p.steps = plan.steps;
  auto kernel = k_q4_run<X, G, NT, MT, ALIGNED>;
  static SmemOnce once;  // one per kernel
  cudaError_t e = once.allow(reinterpret_cast<const void*>(kernel));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(plan.clusters * plan.P));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = plan.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = plan.P;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = plan.P > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kernel, (const RunArgs)p);
  note_launches(1);
  return e;
}

template <class X, int G, bool ALIGNED>
cudaError_t launch_tiles(const RunArgs& p, cudaStream_t s) {
  return OpOf<X>::kParts * p.n <= 8 ? launch_one<X, G, 1, 1, ALIGNED>(p, s)
                                    : launch_one<X, G, 2, 2, ALIGNED>(p, s);
}

// Up to vectors_per_pass<X>() vectors in one launch.
template <class X>
cudaError_t launch_run(const RunArgs& p, cudaStream_t s) {
  const bool aligned = aligned16(p.a.codes) && (p.a.ld_codes % 16 == 0 || p.a.rows <= 1);
  switch (p.a.group) {
    case 32: return aligned ? launch_tiles<X, 32, true>(p, s) : launch_tiles<X, 32, false>(p, s);
    case 64: return aligned ? launch_tiles<X, 64, true>(p, s) : launch_tiles<X, 64, false>(p, s);
    default:
      return aligned ? launch_tiles<X, 128, true>(p, s) : launch_tiles<X, 128, false>(p, s);
  }
}

}  // namespace q4
}  // namespace spmv
