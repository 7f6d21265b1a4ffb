// q4_run.cuh -- y_j = A x_j + c_j for a matrix of 4-bit codes (spmv_q4_run).
//
// A[r][k] = s[r][k/G] (q[r][k] - z[r][k/G]), so y[r] is the sum over groups of
// s times the group's sum of (q - z) x. The integers q - z (-15 .. 15) are
// exact in 16 bits and so are the vectors there: the group sums are products of
// small matrices with exact operands and fp32 accumulators, which
// mma.sync.m16n8k16 forms 16 rows and 8 columns at a time. An fp32 x is cut
// into three bf16 parts, each a column of its own: x = p1 + 2^-7 p2 + 2^-16 p3
// bit for bit, with p1 by truncation, p2 to nearest and p3 what is left (8
// bits). Held so much larger than what they stand for, p2 and p3 lose nothing to
// bf16's least number (2^-133) even of a subnormal x, and no part is larger than
// |x| or 2^-125; their sums are added with these weights at the end.
//
// What bounds it: with 1 to 8 columns latency. The bytes of A, half a byte per entry
// and one scale per group, are read once for up to 16 columns; the instructions that
// turn a nibble into a 16-bit operand (11 per 8 entries) come close behind; but with
// 128 registers, which hold the scales of two steps, only 16 warps run on an SM, DRAM
// is busy for 0.48 to 0.59 of the time and the SM for 0.43 to 0.52 (43 of the 72 forms
// spill, 164 bytes at most, in those with groups of 32 and zero points).
// 131072 x 4096 with an fp32 vector and fp32 scales takes 57.7 us, 4.95 TB/s or
// 0.73 of a copy (46.9 us without the scales' loads, the staging of x and the
// joins); 8192 x 28672 with a bf16 vector 29.4 us, 4.1 TB/s (24.6 without the
// staging and the joins). With 16 columns the fixed parts do: of 36 us for 16384 x
// 5120, about 20 are the steps. mma.sync, not tcgen05.mma: with these columns the
// tensor pipe is idle for three quarters of the time, and operands go from the code
// words to the instruction in registers, without a second trip through shared
// memory.
//
// Layout. A tile is 32 rows; a step is 256 columns of it (128 with more than 8
// operand columns), 4 KB. Each warp
// brings its steps into a ring of kStages buffers of its own by asynchronous
// 16-byte copies, so no barrier is taken between steps. Lane (g, c),
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
// d = A B + c (16 x 16 by 16 x 8)
#define SPMV_MMA16816(TYPE, NAME)                                                              \
  __device__ __forceinline__ void mma16816(float (&d)[4], const unsigned (&a)[4], unsigned b0, \
                                           unsigned b1, float c0, float c1, float c2, float c3,\
                                           TYPE) {                                             \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." NAME "." NAME                                 \
        ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"                       \
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])                                       \
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1),      \
          "f"(c2), "f"(c3));                                                                   \
  }
SPMV_MMA16816(__half, "f16")
SPMV_MMA16816(__nv_bfloat16, "bf16")
#undef SPMV_MMA16816

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

// entries j and j + 4 of a code word, less their zero point (bias = magic | z).
// magic and mask come in registers: as constants they made two instructions of
// the one that masks and sets (8192 x 28672: 113 -> 83 ALU instructions for 16
// rows of 128 columns, 45.7 -> 41.6 us).
template <class Op>
__device__ __forceinline__ unsigned unpack(unsigned w, int j, unsigned mask, unsigned magic,
                                           unsigned bias) {
  unsigned v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w >> (4 * j)), "r"(mask), "r"(magic));
  return Op::sub(v, bias);
}
__device__ __forceinline__ unsigned in_register(unsigned v) {
  asm volatile("" : "+r"(v));
  return v;
}

// 16-byte asynchronous copy of the first `bytes` (1 .. 16) of a 16-byte chunk,
// zeros in the rest.
__device__ __forceinline__ void cp_async16_part(unsigned smem, const void* gmem, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async16(unsigned smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(smem), "l"(gmem)
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
// Shared memory by its own 32-bit addresses (the ring and the staged x).
__device__ __forceinline__ unsigned lds32(unsigned a) {
  unsigned v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(unsigned a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(unsigned a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts8(unsigned a, unsigned v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where 16-byte chunk j of a row's ROW bytes (64 or 128) is kept: moved so that
// the lanes' 4-, 8- and 16-byte reads of 8 rows fall into different banks.
template <int ROW>
__device__ __forceinline__ int chunk_at(int row, int j) {
  if (ROW == 128) return j ^ (((row & 1) << 2) | (row & 2) | ((row >> 2) & 1));
  return j ^ ((row & 2) | ((row >> 2) & 1));
}

// 8 consecutive entries of a vector, zeros past its end.
template <class X>
__device__ __forceinline__ Pack<X, 8> fetch_x(const X* x, long long k, long long cols, bool vec) {
  Pack<X, 8> v;
  if (vec && k + 8 <= cols) {
    v = *reinterpret_cast<const Pack<X, 8>*>(x + k);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.v[i] = k + i < cols ? x[k + i] : from_f32<X>(0.0f);
  }
  return v;
}
__device__ __forceinline__ uint4 in_operand_order(const unsigned (&h)[8]) {
  return make_uint4(h[0] | h[4] << 16, h[1] | h[5] << 16, h[2] | h[6] << 16, h[3] | h[7] << 16);
}
// Their 16-bit operands in the order 0 4 1 5 2 6 3 7; an fp32 vector's three
// parts (p1, p2, p3 above) go to three columns (4 pieces apart).
template <class X>
__device__ __forceinline__ void stage_x(const Pack<X, 8>& v, uint4* out) {
  unsigned h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = *reinterpret_cast<const unsigned short*>(&v.v[i]);
  *out = in_operand_order(h);
}
template <>
__device__ __forceinline__ void stage_x<float>(const Pack<float, 8>& in, uint4* out) {
  float v[8];
  unsigned h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned bits = __float_as_uint(in.v[i]);
    h[i] = bits >> 16;
    if ((bits & 0x7f800000u) == 0x7f800000u) {
      // an infinity or a NaN is its first part alone (a NaN kept one by a bit)
      h[i] |= (bits & 0x007fffffu) ? 0x40u : 0u;
      v[i] = 0.0f;
    } else {
      v[i] = (in.v[i] - __uint_as_float(bits & 0xffff0000u)) * 128.0f;
    }
  }
  out[0] = in_operand_order(h);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
    v[i] = (v[i] - __uint_as_float(h[i] << 16)) * 512.0f;
  }
  out[4] = in_operand_order(h);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = __float_as_uint(v[i]) >> 16;  // (the lower half is 0)
  out[8] = in_operand_order(h);
}
// What a part's sums count for.
__device__ __forceinline__ constexpr float part_weight(int q) {
  return q == 0 ? 1.0f : q == 1 ? 1.0f / 128.0f : 1.0f / 65536.0f;
}

// A scale from its bits: fp32 (shift 0), bf16 (shift 16) or fp16.
__device__ __forceinline__ float scale_value(unsigned raw, int shift, bool half) {
  float f = __uint_as_float(raw << shift);
  if (half) f = __half2float(__ushort_as_half((unsigned short)raw));
  return f;
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

// The warp that holds unit u of `units` divided among the warps (units: tiles and
// steps of which shared memory holds the sums and the x, so well below 2^24).
__device__ __forceinline__ int owner(int u, int units) {
  return ((u + 1) * kWarps - 1) / units;
}

// --- the kernel ------------------------------------------------------------------
// ALIGNED: every row of codes starts on a 16-byte boundary. Otherwise a row's
// bytes are fetched as the aligned chunks that hold them, one more than they
// would fill, and shifted into place when read.
// ZEROS: the matrix has zero points.
template <class X, int G, int NT, bool ALIGNED, bool ZEROS>
__global__ void __launch_bounds__(kThreads, 2) k_q4_run(const RunArgs p) {
  using Op = typename OpOf<X>::Op;
  using OpT = typename Op::T;
  constexpr int kParts = OpOf<X>::kParts;
  constexpr int kStepCols = kStepColsOf<NT>;
  constexpr int kStages = kStagesOf<NT>;
  constexpr int kRow = kStepCols / 2;             // code bytes of a row and step
  constexpr int kPitch = ALIGNED ? kRow : kRow + 16;
  constexpr int kStep = kTileRows * kPitch;       // bytes of a stage
  constexpr int kGroups = kStepCols / G;          // groups of a step
  constexpr int kWords = G / 32;                  // code words of a lane, row and group
  constexpr int kStepWords = kStepCols / 32;      // of a lane, row and step
  constexpr int kRows = kTileRows / 8;            // rows of a lane: g, g + 8, g + 16, g + 24
  // the scales that a lane fetches for the four lanes of its rows: of sRows
  // rows from row sRow0 on and sGroups groups from group sGroup0 on
  constexpr int sRows = kGroups < 4 ? kGroups : 4, sGroups = kGroups < 8 ? 1 : 2;
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const spmv_q4& a = p.a;
  const int NB = p.n * kParts;  // columns
  const unsigned smem0 = (unsigned)__cvta_generic_to_shared(smem);
  const unsigned ring = smem0 + warp * kStages * kStep;
  const unsigned xs0 = smem0 + kWarps * kStages * kStep;
  uint4* xs = reinterpret_cast<uint4*>(smem + kWarps * kStages * kStep);
  float* slots = reinterpret_cast<float*>(xs + (size_t)p.phaseSteps * (kStepCols / 8) * NB);
  const int slotFloats = kTileRows * NB;
  const unsigned mask = in_register(0x000f000fu), magic = in_register(Op::kMagic);

  // this cluster's tiles and this block's steps: equal shares, the first ones
  // one more where they do not divide
  const int rank = p.P > 1 ? blockIdx.x & (p.P - 1) : 0;
  const int cluster = blockIdx.x >> p.logP;
  const int t0 = cluster * p.tileShare + min(cluster, p.tileRest);
  const int T = p.tileShare + (cluster < p.tileRest ? 1 : 0);
  const int s0 = rank * p.stepShare + min(rank, p.stepRest);
  const int s1 = s0 + p.stepShare + (rank < p.stepRest ? 1 : 0);
  // sums of the phases so far, where there are several
  float* sums = slots + (size_t)(p.maxTiles + kWarps - 1) * slotFloats;
  const int xWord4 = NB * 4;  // 16-byte pieces of x from one code word to the next
  const bool phases = p.phaseSteps < p.stepShare + (p.stepRest > 0 ? 1 : 0);
  // vectors joined together (measured: 32 against 36 us for 16 of 16384 x 5120; the
  // other forms lose by it)
  constexpr int kSet = NT == 1 || kParts > 1 || !ALIGNED ? 1 : 4;
  const int sets = kSet == 1 ? p.n : (p.n + kSet - 1) / kSet;
  // (rounded up without passing 32 bits at the largest column counts)
  const int rowBytes = a.cols / 2 + a.cols % 2;
  const int groups = a.cols / G + (a.cols % G != 0);
  const X* x = static_cast<const X*>(p.x);
  const int scaleBytes = a.scale_type == SPMV_F32 ? 4 : 2;
  const int scaleShift = a.scale_type == SPMV_BF16 ? 16 : 0;
  const bool scaleHalf = a.scale_type == SPMV_F16;
  const long long rows8 = 8 * a.ld_codes, scales8 = 8 * a.ld_scales * scaleBytes,
                  zeros8 = 8 * a.ld_zeros;
  const int sRow0 = kGroups == 1 ? c : kGroups == 2 ? 2 * (c & 1) : 0;
  const int sGroup0 = kGroups == 1 ? 0 : kGroups == 2 ? c >> 1 : kGroups == 4 ? c : 2 * c;
  // where the lane's chunks of row g go in a stage, and where its codes of a
  // group and row g are (row g + 8 i: 8 i * kPitch further on)
  unsigned put[kRow / 64];
#pragma unroll
  for (int j = 0; j < kRow / 64; ++j)
    put[j] = ring + g * kPitch + chunk_at<kRow>(g, c + 4 * j) * 16;
  unsigned get[kGroups];
#pragma unroll
  for (int gr = 0; gr < kGroups; ++gr) {
    const int byte = gr * (G / 2) + c * (G / 8);
    get[gr] = ring + g * kPitch + chunk_at<kRow>(g, byte >> 4) * 16 + (byte & 15);
  }

  for (int f0 = s0; f0 == s0 || f0 < s1; f0 += p.phaseSteps) {
    const int fs = min(p.phaseSteps, s1 - f0);  // steps of this phase (0: no columns)
    const int units = T * fs;
    const int u0 = units * warp / kWarps;
    const int u1 = units * (warp + 1) / kWarps;
    unsigned sc[kStages][sRows][sGroups], zr[ZEROS ? kStages : 1][sRows][sGroups];

    // Where this warp's copies are: units left, tile and step, the lane's
    // addresses in row g of the tile.
    int cleft = u1 - u0, ct = fs > 0 ? u0 / fs : 0, cs = u0 - ct * fs;
    const unsigned char *src = nullptr, *scp = nullptr, *zp = nullptr;
    int rowsLeft = 0, bytesLeft = 0, groupsLeft = 0;
    auto enter = [&]() {
      const long long r0 = (long long)(t0 + ct) * kTileRows;
      rowsLeft = (int)min((long long)a.rows - r0, (long long)kTileRows);
      src = a.codes + (r0 + g) * a.ld_codes + ((long long)(f0 + cs) * kRow + c * 16);
      bytesLeft = rowBytes - (f0 + cs) * kRow;
      const int gi = (f0 + cs) * kGroups + sGroup0;
      groupsLeft = groups - gi;
      const long long r = r0 + g + 8 * sRow0;
      scp = static_cast<const unsigned char*>(a.scales) + (r * a.ld_scales + gi) * scaleBytes;
      if (ZEROS) zp = a.zeros + r * a.ld_zeros + gi;
    };
    enter();
    if (f0 == s0) {
      // Launched before the kernel ahead in the stream has ended: only the L2
      // hears of the first codes until it has.
      if (cleft > 0 && lane < rowsLeft)
        prefetch_l2(a.codes + ((long long)(t0 + ct) * kTileRows + lane) * a.ld_codes +
                    (long long)(f0 + cs) * kRow);
      grid_dependency_wait();
      grid_dependency_trigger();
    }
    auto issue = [&](int st) {
      if (cleft > 0) {
        if (ALIGNED) {
          if (rowsLeft == kTileRows && bytesLeft >= kRow) {
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
              const unsigned char* q = src + i * rows8;
#pragma unroll
              for (int j = 0; j < kRow / 64; ++j)
                cp_async16(put[j] + st * kStep + 8 * i * kPitch, q + 64 * j);
            }
          } else {
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
              const unsigned char* q = src + i * rows8;
              const int left = g + 8 * i < rowsLeft ? bytesLeft - c * 16 : 0;
#pragma unroll
              for (int j = 0; j < kRow / 64; ++j)
                if (left > 64 * j)
                  cp_async16_part(put[j] + st * kStep + 8 * i * kPitch, q + 64 * j,
                                  min(left - 64 * j, 16));
            }
          }
        } else {
          // the aligned chunks of each row from its start rounded down
          constexpr int kChunks = kPitch / 16;
          const long long r0 = (long long)(t0 + ct) * kTileRows;
          for (int id = lane; id < kChunks * rowsLeft; id += 32) {
            const int row = id / kChunks, j = id - row * kChunks;
            const unsigned char* first = a.codes + (r0 + row) * a.ld_codes;
            const unsigned char* from =
                reinterpret_cast<const unsigned char*>(
                    reinterpret_cast<uintptr_t>(first + (long long)(f0 + cs) * kRow) &
                    ~(uintptr_t)15) + 16 * j;
            const unsigned to = ring + st * kStep + row * kPitch + j * 16;
            if (from < first + rowBytes) {
              if (from >= a.codes && from + 16 <= p.codesEnd) {
                cp_async16(to, from);
              } else {  // the ends of the array: byte by byte
                for (int b = 0; b < 16; ++b)
                  if (from + b >= a.codes && from + b < p.codesEnd) sts8(to + b, from[b]);
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < sRows; ++i)
#pragma unroll
          for (int l = 0; l < sGroups; ++l) {
            sc[st][i][l] = 0u;
            if (ZEROS) zr[st][i][l] = 8u;
            if (g + 8 * (sRow0 + i) < rowsLeft && l < groupsLeft) {
              const unsigned char* q = scp + i * scales8;
              sc[st][i][l] = scaleBytes == 4
                                 ? reinterpret_cast<const unsigned*>(q)[l]
                                 : (unsigned)reinterpret_cast<const unsigned short*>(q)[l];
              if (ZEROS) zr[st][i][l] = zp[i * zeros8 + l];
            }
          }
        --cleft;
        if (++cs == fs) {
          cs = 0;
          ++ct;
          enter();
        } else {
          src += kRow;
          bytesLeft -= kRow;
          scp += kGroups * scaleBytes;
          groupsLeft -= kGroups;
          if (ZEROS) zp += kGroups;
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int st = 0; st < kStages - 1; ++st) issue(st);

    // x of this phase, in fragment order: [step][word][column][c]
    if (f0 != s0) __syncthreads();  // the last phase's readers are done
    // (a piece: 8 entries of one vector; a thread fetches several at a time, of
    // one vector or of the same columns of several)
    {
      constexpr int kBatch = kParts == 1 ? 4 : 2;
      const int places = fs * kStepWords * 4;
      auto entry = [&](int i) {  // the columns of place i: step, word and c
        const int word = (i >> 2) % kStepWords;
        return (long long)(f0 + (i >> 2) / kStepWords) * kStepCols + (word / kWords) * G +
               (i & 3) * (G / 4) + (word % kWords) * 8;
      };
      Pack<X, 8> held[kBatch];
      if (p.n == 1) {
        for (int i0 = threadIdx.x; i0 < places; i0 += kBatch * kThreads) {
#pragma unroll
          for (int q = 0; q < kBatch; ++q)
            if (i0 + q * kThreads < places)
              held[q] = fetch_x<X>(x, entry(i0 + q * kThreads), a.cols, p.xVec);
#pragma unroll
          for (int q = 0; q < kBatch; ++q) {
            const int i = i0 + q * kThreads;
            if (i < places) stage_x<X>(held[q], xs + (i >> 2) * (kParts * 4) + (i & 3));
          }
        }
      } else {
        const int sets = (p.n + kBatch - 1) / kBatch;
        for (int j = threadIdx.x; j < places * sets; j += kThreads) {
          const int set = j / places, i = j - set * places, v0 = set * kBatch;
          const long long k = entry(i);
          const X* from = x + v0 * p.ldx;
          uint4* to = xs + (i >> 2) * xWord4 + v0 * (kParts * 4) + (i & 3);
#pragma unroll
          for (int q = 0; q < kBatch; ++q)
            if (v0 + q < p.n) held[q] = fetch_x<X>(from + q * p.ldx, k, a.cols, p.xVec);
#pragma unroll
          for (int q = 0; q < kBatch; ++q)
            if (v0 + q < p.n) stage_x<X>(held[q], to + q * (kParts * 4));
        }
      }
    }
    __syncthreads();

    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][nt][i] = 0.0f;

    // The unit being consumed. A column that is not there is read as the last
    // one: what an mma leaves in its place is never looked at.
    int tile = fs > 0 ? u0 / fs : 0, at = u0 - tile * fs;
    unsigned xl[NT];
    const int xWord = xWord4 * 16;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      xl[nt] = xs0 + min(nt * 8 + g, NB - 1) * 64 + c * 16 + at * kStepWords * xWord;
    for (int left = u1 - u0; left > 0;) {
#pragma unroll
      for (int st = 0; st < kStages; ++st) {
        if (left > 0) {
          cp_async_wait<kStages - 2>();
          __syncwarp();
          issue((st + kStages - 1) % kStages);
          // this lane's scales and biases, to be passed among the four
          float sv[sRows][sGroups];
          unsigned zv[sRows][sGroups];
#pragma unroll
          for (int i = 0; i < sRows; ++i)
#pragma unroll
            for (int l = 0; l < sGroups; ++l) {
              sv[i][l] = scale_value(sc[st][i][l], scaleShift, scaleHalf);
              if (ZEROS) zv[i][l] = Op::kMagic + zr[ZEROS ? st : 0][i][l] * 0x00010001u;
            }
          unsigned shift[kRows];
          if (!ALIGNED) {
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
              const long long r = (long long)(t0 + tile) * kTileRows + g + 8 * i;
              shift[i] = (unsigned)(reinterpret_cast<uintptr_t>(a.codes + r * a.ld_codes) & 15);
            }
          }
#pragma unroll
          for (int gr = 0; gr < kGroups; ++gr) {
            float s[kRows];
            unsigned bias[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
              const int from = (lane & ~3) + (kGroups == 1   ? i
                                              : kGroups == 2 ? 2 * gr + (i >> 1)
                                              : kGroups == 4 ? gr
                                                             : gr >> 1);
              const int row = kGroups == 1 ? 0 : kGroups == 2 ? i & 1 : i;
              const int l = kGroups == 8 ? gr & 1 : 0;
              s[i] = __shfl_sync(kFullMask, sv[row][l], from);
              bias[i] = ZEROS ? __shfl_sync(kFullMask, zv[row][l], from) : Op::kMagic + 0x00080008u;
            }
            unsigned w[kRows][kWords];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
              if (ALIGNED) {
                const unsigned q = get[gr] + st * kStep + 8 * i * kPitch;
                if (kWords == 4) {
                  const uint4 v = lds128(q);
                  w[i][0] = v.x;
                  w[i][1 % kWords] = v.y;
                  w[i][2 % kWords] = v.z;
                  w[i][3 % kWords] = v.w;
                } else if (kWords == 2) {
                  const uint2 v = lds64(q);
                  w[i][0] = v.x;
                  w[i][1 % kWords] = v.y;
                } else {
                  w[i][0] = lds32(q);
                }
              } else {
                const unsigned byte = shift[i] + gr * (G / 2) + c * (G / 8);
                const unsigned q = ring + st * kStep + (g + 8 * i) * kPitch + (byte & ~3u);
                unsigned lo = lds32(q);
#pragma unroll
                for (int k = 0; k < kWords; ++k) {
                  // the last word's upper neighbour is only needed off a word boundary
                  const unsigned hi = (byte & 3) || k + 1 < kWords ? lds32(q + 4 * k + 4) : 0u;
                  w[i][k] = __funnelshift_r(lo, hi, 8 * (byte & 3));
                  lo = hi;
                }
              }
            }
            float part[2][NT][4];
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
              uint4 b[NT];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                b[nt] = lds128(xl[nt]);
                xl[nt] += xWord;
              }
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                unsigned lo[4], hi[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  lo[j] = unpack<Op>(w[2 * m][k], j, mask, magic, bias[2 * m]);
                  hi[j] = unpack<Op>(w[2 * m + 1][k], j, mask, magic, bias[2 * m + 1]);
                }
                const unsigned a0[4] = {lo[0], hi[0], lo[1], hi[1]};
                const unsigned a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float(&d)[4] = part[m][nt];
                  if (k == 0)
                    mma16816(d, a0, b[nt].x, b[nt].y, 0.0f, 0.0f, 0.0f, 0.0f, OpT{});
                  else
                    mma16816(d, a0, b[nt].x, b[nt].y, d[0], d[1], d[2], d[3], OpT{});
                  mma16816(d, a1, b[nt].z, b[nt].w, d[0], d[1], d[2], d[3], OpT{});
                }
              }
            }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  acc[m][nt][i] = fmaf(s[2 * m + (i >> 1)], part[m][nt][i], acc[m][nt][i]);
          }
          --left;
          if (++at == fs || left == 0) {  // the tile's end, or this warp's
            float* slot = slots + (size_t)(tile + warp) * slotFloats;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int col = nt * 8 + 2 * c + (i & 1);
                  if (col < NB) slot[col * kTileRows + m * 16 + g + 8 * (i >> 1)] = acc[m][nt][i];
                  acc[m][nt][i] = 0.0f;
                }
            at = 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              xl[nt] = xs0 + min(nt * 8 + g, NB - 1) * 64 + c * 16;
            ++tile;
          }
        }
      }
    }
    cp_async_wait<0>();
    __syncthreads();
    // Join the warps' partial sums of each output, in the order of the columns.
    // What is not finished yet is kept where the first of them was, or with
    // several phases in `sums`.
    const bool last = f0 + p.phaseSteps >= s1;
    for (int item = warp; item < T * sets; item += kWarps) {  // a tile and kSet vectors
      const int t = sets == 1 ? item : item / sets, v0 = (item - t * sets) * kSet;
      const int w0 = fs > 0 ? owner(t * fs, units) : 0;
      const int w1 = fs > 0 ? owner((t + 1) * fs - 1, units) : -1;
      float* const in = slots + (size_t)t * slotFloats + v0 * kParts * kTileRows + lane;
      float* const kept = sums + (t * p.n + v0) * kTileRows + lane;
      const long long r = (long long)(t0 + t) * kTileRows + lane;
      const bool write = last && p.P == 1 && r < a.rows;
      float sum[kSet], c[kSet];
#pragma unroll
      for (int b = 0; b < kSet; ++b) {
        c[b] = write && p.c && v0 + b < p.n ? load_y(p.c, p.yType, (v0 + b) * p.ldc + r) : 0.0f;
        sum[b] = phases && f0 > s0 && v0 + b < p.n ? kept[b * kTileRows] : 0.0f;
      }
      auto add = [&](int w) {
#pragma unroll
        for (int b = 0; b < kSet; ++b)
          if (v0 + b < p.n)
#pragma unroll
            for (int q = kParts - 1; q >= 0; --q)  // (p1 + p2 may overflow where x does not)
              sum[b] = fmaf(in[(size_t)w * slotFloats + (b * kParts + q) * kTileRows],
                            part_weight(q), sum[b]);
      };
      if (units >= kWarps) {
#pragma unroll 4
        for (int w = w0; w <= w1; ++w) add(w);
      } else {
        for (int w = w0; w <= w1; ++w)
          if (owner(units * w / kWarps, units) == w) add(w);  // not an idle one
      }
#pragma unroll
      for (int b = 0; b < kSet; ++b) {
        if (v0 + b >= p.n) break;
        if (write)
          store_y(p.y, p.yType, (v0 + b) * p.ldy + r, sum[b] + c[b]);
        else if (!last || phases)
          kept[b * kTileRows] = sum[b];
        else if (p.P > 1)
          in[(size_t)w0 * slotFloats + b * kParts * kTileRows] = sum[b];
      }
    }
    if (!last) __syncthreads();
  }
  if (p.P > 1) {
    namespace cgr = cooperative_groups;
    cgr::cluster_group cl = cgr::this_cluster();
    cl.sync();
    // blocks with one more step than the others put a tile's first warp elsewhere
    const int more = p.stepShare + 1, less = p.stepShare;
    for (int item = rank * kWarps + warp; item < T * sets; item += kWarps << p.logP) {
      const int t = sets == 1 ? item : item / sets, v0 = (item - t * sets) * kSet;
      const long long r = (long long)(t0 + t) * kTileRows + lane;
      float* const here = sums + (t * p.n + v0) * kTileRows + lane;
      float* const slot0 = slots + (size_t)t * slotFloats + v0 * kParts * kTileRows + lane;
      float* const atMore = slot0 + (size_t)owner(t * more, T * more) * slotFloats;
      float* const atLess = slot0 + (size_t)owner(t * less, T * less) * slotFloats;
      const int apart = phases ? kTileRows : kParts * kTileRows;
      float part[kSet][8], c[kSet];  // all on their way before the first is added
#pragma unroll
      for (int b = 0; b < kSet; ++b)
        c[b] = r < a.rows && p.c && v0 + b < p.n ? load_y(p.c, p.yType, (v0 + b) * p.ldc + r)
                                                 : 0.0f;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float* const from = phases ? here : q < p.stepRest ? atMore : atLess;
#pragma unroll
        for (int b = 0; b < kSet; ++b)
          part[b][q] =
              q < p.P && v0 + b < p.n ? *cl.map_shared_rank(from + b * apart, q) : 0.0f;
      }
#pragma unroll
      for (int b = 0; b < kSet; ++b) {
        float sum = part[b][0];
#pragma unroll
        for (int q = 1; q < 8; ++q) sum += part[b][q];
        if (r < a.rows && v0 + b < p.n)
          store_y(p.y, p.yType, (v0 + b) * p.ldy + r, sum + c[b]);
      }
    }
    cl.sync();  // the others may still be reading this block's sums
  }
}

// --- launch --------------------------------------------------------------------------
template <class X, int G, int NT, bool ALIGNED, bool ZEROS>
cudaError_t launch_one(const RunArgs& args, cudaStream_t s) {
  constexpr int kPitch = kStepColsOf<NT> / 2 + (ALIGNED ? 0 : 16);
  auto kernel = k_q4_run<X, G, NT, ALIGNED, ZEROS>;
  static Residency room;  // one per kernel
  cudaError_t e = room.ask(reinterpret_cast<const void*>(kernel));
  if (e != cudaSuccess) return e;
  const Plan plan = make_plan(args, OpOf<X>::kParts * args.n, kStepColsOf<NT>,
                              kWarps * kStagesOf<NT> * kTileRows * kPitch, room);
  RunArgs p = args;
  p.P = plan.P;
  p.logP = plan.logP;
  p.phaseSteps = plan.phaseSteps;
  p.maxTiles = plan.maxTiles;
  p.tileShare = (int)(plan.tiles / plan.clusters);
  p.tileRest = (int)(plan.tiles % plan.clusters);
  p.stepShare = plan.steps / plan.P;
  p.stepRest = plan.steps % plan.P;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(plan.clusters * plan.P));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = plan.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = plan.P;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = plan.P > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kernel, (const RunArgs)p);
  note_launches(1);
  return e;
}

template <class X, int G, bool ZEROS>
cudaError_t launch_group(const RunArgs& p, cudaStream_t s) {
  const bool aligned = aligned16(p.a.codes) && (p.a.ld_codes % 16 == 0 || p.a.rows <= 1);
  if (OpOf<X>::kParts * p.n <= 8)
    return aligned ? launch_one<X, G, 1, true, ZEROS>(p, s)
                   : launch_one<X, G, 1, false, ZEROS>(p, s);
  return aligned ? launch_one<X, G, 2, true, ZEROS>(p, s)
                 : launch_one<X, G, 2, false, ZEROS>(p, s);
}

// Up to vectors_per_pass<X>() vectors in one launch.
template <class X>
cudaError_t launch_run(const RunArgs& p, cudaStream_t s) {
  const bool z = p.a.zeros != nullptr;
  switch (p.a.group) {
    case 32: return z ? launch_group<X, 32, true>(p, s) : launch_group<X, 32, false>(p, s);
    case 64: return z ? launch_group<X, 64, true>(p, s) : launch_group<X, 64, false>(p, s);
    default: return z ? launch_group<X, 128, true>(p, s) : launch_group<X, 128, false>(p, s);
  }
}

}  // namespace q4
}  // namespace spmv
