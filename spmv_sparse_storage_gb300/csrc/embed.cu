// embed.cu -- token lookups in a dense table and the gradient of the lookup.
//
// A lookup of T tokens is the product of a T x vocab matrix with one entry
// (scale) per row, at the token's column, and the table; its gradient with
// respect to the table is the transposed product: row v of the gradient is
// scale times the sum of the rows of g whose token is v.
#include <cooperative_groups.h>
#include <algorithm>

#include "dtypes.cuh"
#include "device_util.cuh"
#include "internal.h"

namespace spmv {
namespace {

__device__ __forceinline__ long long token_at(const void* tokens, int wide, long long i) {
  return wide ? static_cast<const long long*>(tokens)[i]
              : (long long)static_cast<const int*>(tokens)[i];
}

// How many elements of every row can be taken at once, `most` (8 or 4), 4 or 1, by
// accesses of up to 16 bytes.
inline int elements_at_once(const void* p, long long ld, int dim, int bytes, int most) {
  for (int E = most; E > 2; E /= 2) {
    const int access = E * bytes < 16 ? E * bytes : 16;
    if (dim % E == 0 && !misaligned(p, access) && ld * bytes % access == 0) return E;
  }
  return 1;
}

// ---------------------------------------------------------------------------
// Lookup: E elements to a lane and load, kRowLoads of them in flight, G lanes to
// a token and stretch of its row. Bound by the bytes read and written (32768 rows
// of 4096 fp32 to bf16: 69.8 us, 6.35 TB/s, 0.94 of a copy); with single elements
// (rows off a 16-byte boundary) by the loads and stores themselves. 16384 rows of bf16
// by 8 (4096 columns) 41.5 us, by 4 (4100) 43.6, one by one (4099) 75.
// ---------------------------------------------------------------------------
template <int E>
constexpr int kRowLoads = E == 1 ? 16 : 4;
template <class T, class O, int E>
__global__ void __launch_bounds__(256) k_embed(int n, int vocab, int dim, int logG,
                                               const T* table, long long ldt,
                                               const void* tokens, int wide,
                                               float scale, O* out, long long ldo) {
  grid_dependency_wait();
  grid_dependency_trigger();
  const int G = 1 << logG;
  const long long t = (long long)blockIdx.x * (256 >> logG) + (threadIdx.x >> logG);
  if (t >= n) return;
  const long long token = token_at(tokens, wide, t);
  const bool valid = token >= 0 && token < vocab;
  const int k0 = ((int)blockIdx.y * kRowLoads<E> * G + (threadIdx.x & (G - 1))) * E;
  Pack<T, E> v[kRowLoads<E>];
#pragma unroll
  for (int i = 0; i < kRowLoads<E>; ++i) {
    const int k = k0 + i * G * E;
    if (valid && k < dim) v[i] = *reinterpret_cast<const Pack<T, E>*>(table + token * ldt + k);
  }
#pragma unroll
  for (int i = 0; i < kRowLoads<E>; ++i) {
    const int k = k0 + i * G * E;
    if (k >= dim) break;
    Pack<O, E> o;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o.v[e] = from_f32<O>(valid ? scale * to_f32(v[i].v[e]) : 0.0f);
    *reinterpret_cast<Pack<O, E>*>(out + t * ldo + k) = o;
  }
}

__device__ __forceinline__ int key_of(const void* tokens, int wide, int i, int n, int vocab) {
  if (i >= n) return vocab;
  const long long t = token_at(tokens, wide, i);
  return t >= 0 && t < vocab ? (int)t : vocab;
}

// ---------------------------------------------------------------------------
// Sorting up to kRankMost tokens: an item's place is the number of items with a
// smaller key, or with its own and an earlier place. A block keeps all the keys in
// shared memory and counts for kRankBlock places, a warp for kRankEach of them with
// 128 keys at a time. No block waits for another, which is what a short call gains:
// 64 tokens of 256 fp32 columns 11.1 -> 7.3 us for the whole gradient, 1000 12.6 ->
// 7.9, 2048 15.6 -> 12.2, against the cluster below. The work is the square of the
// number, so that 4096 of 1000 columns would lose by it (30 against 27).
// ---------------------------------------------------------------------------
constexpr int kRankMost = 2048;
constexpr int kRankThreads = 512;
constexpr int kRankEach = 2;
constexpr int kRankLoads = kRankMost / kRankThreads;
constexpr int kRankBlock = kRankThreads / 32 * kRankEach;
static_assert(128 % kRankBlock == 0 && kRankMost % 128 == 0, "");

__global__ void __launch_bounds__(kRankThreads) k_embed_rank(int n, int vocab, const void* tokens,
                                                             int wide, int2* out) {
  __shared__ uint4 keys[kRankMost / 4];
  grid_dependency_wait();
  grid_dependency_trigger();
  unsigned* const key = reinterpret_cast<unsigned*>(keys);
  const int sets = (n + 127) / 128;
  unsigned in[kRankLoads];
#pragma unroll
  for (int l = 0; l < kRankLoads; ++l)
    in[l] = (unsigned)key_of(tokens, wide, threadIdx.x + l * kRankThreads, n, vocab);
#pragma unroll
  for (int l = 0; l < kRankLoads; ++l) key[threadIdx.x + l * kRankThreads] = in[l];
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int at = blockIdx.x * kRankBlock + (threadIdx.x >> 5) * kRankEach;
  unsigned own[kRankEach], count[kRankEach];
#pragma unroll
  for (int r = 0; r < kRankEach; ++r) {
    own[r] = key[at + r];
    count[r] = 0;
  }
  const int here = at / 128;  // the set that holds the warp's places
#pragma unroll 4
  for (int q = 0; q < here; ++q) {
    const uint4 k = keys[q * 32 + lane];
#pragma unroll
    for (int r = 0; r < kRankEach; ++r)
      count[r] += (k.x <= own[r]) + (k.y <= own[r]) + (k.z <= own[r]) + (k.w <= own[r]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = here * 128 + e * 32 + lane;
#pragma unroll
    for (int r = 0; r < kRankEach; ++r)
      count[r] += key[i] < own[r] || (key[i] == own[r] && i < at + r);
  }
#pragma unroll 4
  for (int q = here + 1; q < sets; ++q) {
    const uint4 k = keys[q * 32 + lane];
#pragma unroll
    for (int r = 0; r < kRankEach; ++r)
      count[r] += (k.x < own[r]) + (k.y < own[r]) + (k.z < own[r]) + (k.w < own[r]);
  }
#pragma unroll
  for (int r = 0; r < kRankEach; ++r) {
    const unsigned place = __reduce_add_sync(kFullMask, count[r]);
    if (lane == r && at + r < n) out[place] = make_int2((int)own[r], at + r);
  }
}

// ---------------------------------------------------------------------------
// Sorting up to kSortMost tokens in one launch: one cluster of 4 or 8 blocks holds
// them all in its shared memory, kSortThreads * IPT to a block, and sorts them
// by least-significant-digit radix passes (stable; 9 bits at most a pass, so two
// for vocabularies below 2^18). Per pass a warp ranks its own items against each
// other (by the lanes with an equal digit, found by a ballot per bit, round after
// round), the block adds the warps before it, the cluster the blocks before it,
// and every item is stored at its place, in whichever block that is. Bound by the
// shared-memory round trips and the cluster's barriers: 19 us for 32768 tokens
// (matching whole digits took 23). The general path launches three
// kernels for every 8 bits (65537 tokens: 57 us in all against 50 for 65536;
// a cluster of 16 gained nothing: 67 against 68 us for 131072 tokens).
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxBits = 9;
constexpr int kSortMaxBlocks = 8;
constexpr int kSortMaxItems = 8;  // a thread's
constexpr int kSortMost = kSortMaxBlocks * kSortThreads * kSortMaxItems;

// Shared memory of a block: items[2][kSortThreads * IPT] (key, place), counts
// [kSortWarps][1 << bits] (16 bits each), totals, starts.
struct SortItem {
  int key, pos;
};
inline size_t sort_smem(int ipt, int bits) {
  return 2 * sizeof(SortItem) * (size_t)kSortThreads * ipt +
         sizeof(unsigned short) * ((size_t)kSortWarps << bits) + sizeof(int) * (2u << bits) +
         sizeof(int) * 64;
}

template <int IPT>
__global__ void __launch_bounds__(kSortThreads, 1) k_embed_sort(
    int n, int vocab, const void* tokens, int wide, int passes, int bits,
    int2* out) {
  extern __shared__ __align__(16) unsigned char smem[];
  grid_dependency_wait();
  grid_dependency_trigger();
  namespace cgr = cooperative_groups;
  cgr::cluster_group cl = cgr::this_cluster();
  const int blocks = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  constexpr int kTile = kSortThreads * IPT;
  const int D = 1 << bits, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  SortItem* items = reinterpret_cast<SortItem*>(smem);
  unsigned short* counts = reinterpret_cast<unsigned short*>(items + 2 * kTile);
  int* totals = reinterpret_cast<int*>(counts + ((size_t)kSortWarps << bits));
  int* starts = totals + D;
  int* sums = starts + D;  // one per warp
  SortItem it[IPT];
  const int first = warp * 32 * IPT + lane;  // in the tile: the thread's items are 32 apart
#pragma unroll
  for (int r = 0; r < IPT; ++r) {
    const int i = rank * kTile + first + 32 * r;
    it[r] = {key_of(tokens, wide, i, n, vocab), i};
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * bits;
    SortItem* next = items + (pass & 1 ? kTile : 0);
    if (pass > 0) {
      const SortItem* prev = items + (pass & 1 ? 0 : kTile);
#pragma unroll
      for (int r = 0; r < IPT; ++r) it[r] = prev[first + 32 * r];
    }
    for (int i = tid; i < kSortWarps * D / 2; i += kSortThreads)
      reinterpret_cast<unsigned*>(counts)[i] = 0u;
    __syncthreads();
    // rank among the warp's items of the same digit
    unsigned short* mine = counts + warp * D;
    int rk[IPT];
#pragma unroll
    for (int r = 0; r < IPT; ++r) {
      const int d = (it[r].key >> shift) & (D - 1);
      unsigned peers = kFullMask;  // the lanes with the same digit, bit by bit
      for (int b = 0; b < bits; ++b) {
        const unsigned set = __ballot_sync(kFullMask, d >> b & 1);
        peers &= d >> b & 1 ? set : ~set;
      }
      const int before = mine[d];
      __syncwarp();
      rk[r] = before + __popc(peers & lanemask_lt());
      if (lane == __ffs(peers) - 1) mine[d] = (unsigned short)(before + __popc(peers));
      __syncwarp();
    }
    __syncthreads();
    // counts of the warps before, and the block's totals
    for (int d = tid; d < D; d += kSortThreads) {
      int run = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = counts[w * D + d];
        counts[w * D + d] = (unsigned short)run;
        run += c;
      }
      totals[d] = run;
    }
    cl.sync();
    // where the block's items of each digit start: all smaller digits, and the
    // same digit in the blocks before
    int all = 0, before = 0;
    if (tid < D) {
#pragma unroll
      for (int q = 0; q < kSortMaxBlocks; ++q) {
        const int c = q < blocks ? *cl.map_shared_rank(totals + tid, q) : 0;
        all += c;
        before += q < rank ? c : 0;
      }
    }
    int inc = all;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(kFullMask, inc, off);
      if (lane >= off) inc += o;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
      int x = sums[lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(kFullMask, x, off);
        if (lane >= off) x += o;
      }
      sums[lane] = x;
    }
    __syncthreads();
    if (tid < D) starts[tid] = inc - all + (warp > 0 ? sums[warp - 1] : 0) + before;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < IPT; ++r) {
      const int d = (it[r].key >> shift) & (D - 1);
      const int to = starts[d] + mine[d] + rk[r];
      if (pass == passes - 1) {
        if (to < n) out[to] = make_int2(it[r].key, it[r].pos);
      } else {
        *cl.map_shared_rank(next + to % kTile, to / kTile) = it[r];
      }
    }
    cl.sync();  // every item is in place (and no block leaves while it is written to)
  }
}

// ---------------------------------------------------------------------------
// Gradient. The sorted positions are cut into chunks, each summed by one group of
// G threads that hold a slab of columns, E each. The group in whose chunk a row's
// tokens begin finishes the row, as far as the end of the next chunk; a row that
// goes on beyond that leaves a partial sum in every chunk it touches, and a
// second kernel adds those up. Either way the terms are added in order, a chunk's
// at a time: nothing depends on the order in which blocks run. When the gradient
// is overwritten, further blocks of the same launch write zeros into the rows
// that no token names. Bound by the bytes of g and of the gradient: 32768 tokens of
// 4096 bf16 columns into 131072 rows take 197 us here, 6.7 TB/s or 0.98 of a copy,
// between the sort (19 us) and the second kernel (9 us).
// ---------------------------------------------------------------------------
constexpr int kSumThreads = 256;
constexpr int kSumChunk = 32;       // positions of a chunk, at most
constexpr int kSumChunkLeast = 4;
constexpr int kSumWanted = 608;     // blocks: four for each of 152 SMs (a fixed number, so that
                                    // the workspace is the same size wherever it is asked for)
constexpr int kSumStaged = 1024;    // positions of a block, at most
constexpr int kZeroRows = 64;       // rows of a zeroing block
constexpr int kJoinChunks = 1024;   // chunks that a block of the second kernel looks at
constexpr int kJoinBlocks = 32;     // blocks that share the rows found there
constexpr int kJoinRows = 4;        // partial sums in flight there

// The sorted tokens' numbers and places, `stride` ints apart.
struct SortedTokens {
  const int* key;
  const int* pos;
  int stride;
  __device__ __forceinline__ int key_at(long long i) const { return key[i * stride]; }
  __device__ __forceinline__ int pos_at(long long i) const { return pos[i * stride]; }
};

struct SumShape {
  int G, chunk;
  long long chunks, blocksX, slabs;
};
// Chunks of 32 positions, shorter ones where those would not fill the GPU
// (2048 tokens of 1000 columns: 4 positions, 8.4 us against 24 with 32).
SumShape sum_shape(int n, int dim, int E) {
  SumShape s;
  const long long lanes = ((long long)dim + E - 1) / E;
  s.G = 1;
  while (s.G < kSumThreads && s.G < lanes) s.G *= 2;
  s.slabs = (lanes + s.G - 1) / s.G;
  s.chunk = kSumChunk;
  while (kSumThreads / s.G * s.chunk > kSumStaged) s.chunk /= 2;
  for (;; s.chunk /= 2) {
    s.chunks = ((long long)n + s.chunk - 1) / s.chunk;
    s.blocksX = (s.chunks + kSumThreads / s.G - 1) / (kSumThreads / s.G);
    if (s.chunk == kSumChunkLeast || s.blocksX * s.slabs >= kSumWanted) return s;
  }
}

// A row of zeros by a warp: 16 bytes at a time between the boundaries it spans.
template <class O>
__device__ __forceinline__ void zero_row(O* row, int dim, int lane) {
  constexpr int E = 16 / (int)sizeof(O);
  const int head =
      min(dim, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(O));
  const int whole = (dim - head) / E;
  if (lane < head) row[lane] = from_f32<O>(0.0f);
  uint4* const body = reinterpret_cast<uint4*>(row + head);
  for (int k = lane; k < whole; k += 32) body[k] = make_uint4(0u, 0u, 0u, 0u);
  if (lane < dim - head - whole * E) row[head + whole * E + lane] = from_f32<O>(0.0f);
}

// The first position of the sorted keys that is not below v, by a warp: 32 places
// at a time, so that 32768 keys take three rounds.
__device__ __forceinline__ int lower_bound_warp(const SortedTokens& in, int n, long long v) {
  const int lane = threadIdx.x & 31;
  long long lo = 0, hi = n;  // the answer is in [lo, hi]
  while (lo < hi) {
    const long long at = lo + (hi - lo) * lane / 32;
    const unsigned below = __ballot_sync(kFullMask, in.key_at(at) < v);
    // places 0 .. popc - 1 are below v
    const int c = __popc(below);
    if (c == 0) return (int)lo;
    const long long next = c < 32 ? lo + (hi - lo) * c / 32 : hi;
    lo = lo + (hi - lo) * (c - 1) / 32 + 1;
    hi = next;
  }
  return (int)lo;
}

// Zeros in those of kZeroRows rows that no token names.
template <class O>
__device__ void zero_rows(long long v0, int n, int vocab, int dim, const SortedTokens& in,
                          O* dtable, long long ldd) {
  __shared__ int bound[2];
  __shared__ unsigned named[kZeroRows / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < kZeroRows / 32) named[threadIdx.x] = 0u;
  if (warp < 2) {
    const int at = lower_bound_warp(in, n, v0 + warp * kZeroRows);
    if (lane == 0) bound[warp] = at;
  }
  __syncthreads();
  for (int i = bound[0] + threadIdx.x; i < bound[1]; i += kSumThreads) {
    const int r = (int)(in.key_at(i) - v0);
    atomicOr(&named[r >> 5], 1u << (r & 31));
  }
  __syncthreads();
  for (int i = warp; i < kZeroRows && v0 + i < vocab; i += kSumThreads / 32)
    if (!(named[i >> 5] >> (i & 31) & 1u)) zero_row(dtable + (v0 + i) * ldd, dim, lane);
}

// E elements of a row: next to each other, or (APART) `step` apart and of those the
// ones before `left` (any others are read as the last: loads without a condition are
// all on their way before the first is waited for).
template <bool APART, class V, int E>
__device__ __forceinline__ Pack<V, E> take(const V* p, int step, int left) {
  Pack<V, E> v;
  if (!APART) return *reinterpret_cast<const Pack<V, E>*>(p);
#pragma unroll
  for (int e = 0; e < E; ++e) v.v[e] = p[min(e * step, left - 1)];
  return v;
}
template <bool APART, class V, int E>
__device__ __forceinline__ void put(V* p, const Pack<V, E>& v, int step, int left) {
  if (!APART) {
    *reinterpret_cast<Pack<V, E>*>(p) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (e * step < left) p[e * step] = v.v[e];
}
template <bool ADD, class O, int E>
__device__ __forceinline__ Pack<O, E> finished(const float (&acc)[E], float scale,
                                               const Pack<O, E>& old) {
  Pack<O, E> o;
#pragma unroll
  for (int e = 0; e < E; ++e)
    o.v[e] = from_f32<O>(ADD ? to_f32(old.v[e]) + scale * acc[e] : scale * acc[e]);
  return o;
}

// Partial sums of chunk c: part[2c] of the row that began before it, part[2c + 1]
// of the row that begins in it. Blocks from sumBlocks on (in the first slab) zero
// rows. The keys and places of a block's chunks, and the keys around them, wait in
// shared memory, so that only the rows of g (and those added to) are waited for.
// A thread's share of a row (8 or 16 bytes, E = 8 or 4) is fetched 7 rows ahead, by
// asynchronous copies into its own places in shared memory (kSlots of them), which
// takes no registers and no barrier. Rows of any alignment (APART) come by single elements, 4
// to a thread as far apart as the threads of its group, R rows at a time into
// registers (16384 tokens of 4099 bf16 columns 152 us; one element to a thread, four
// times the groups, 200; loads under conditions 231). (4 rows
// into registers with E = 8 left the kernel waiting: 283 us for 32768 tokens of
// 4096 bf16 columns into 131072 rows, 196 with the copies.)
// E is 8 where g and the gradient are both of 16 bits, else 4 at most: 32 bytes to a
// lane as two pieces would take every sector of a row twice (16384 tokens of fp32 g
// and gradient, 4096 columns with 8, 4100 with 4: 221 against 169 us; bf16 g 169
// against 155). Rows that allow 4 alone: 4100 bf16 columns 104 us, element by element
// 197; 100000 tokens of 300 columns 88 against 144.
constexpr int sum_most(int gBytes, int tableBytes) {
  return gBytes == 2 && tableBytes == 2 ? 8 : 4;
}
constexpr int kSlots = 8;
template <class T, class O, int E, bool ADD>
constexpr int kSlotBytes = E * (int)(sizeof(T) + (ADD ? sizeof(O) : 0));
template <class T, class O, int E, bool ADD>
constexpr int kSumSmem = kSlots * kSumThreads * kSlotBytes<T, O, E, ADD>;
// A thread's share, to shared memory and from there.
template <int BYTES>
__device__ __forceinline__ void fetch_share(unsigned char* all, const void* gmem) {
  static_assert(BYTES == 8 || BYTES == 16, "one access");
  unsigned char* const to = all + threadIdx.x * BYTES;
  if constexpr (BYTES == 16)
    cp_async16(to, gmem);
  else
    cp_async_small<BYTES>(to, gmem);
}
template <class V>
__device__ __forceinline__ V own_share(const unsigned char* all) {
  static_assert(sizeof(V) == 8 || sizeof(V) == 16, "one access");
  return reinterpret_cast<const V*>(all)[threadIdx.x];
}

template <class T, class O, int E, bool APART, bool ADD>
__global__ void __launch_bounds__(kSumThreads, 3) k_embed_sum(
    int n, int vocab, int dim, int G, int chunkRows, long long chunks, unsigned sumBlocks,
    const SortedTokens in, const T* g,
    long long ldg, float scale, O* dtable, long long ldd, float* part,
    unsigned char* goesOn) {
  extern __shared__ __align__(16) unsigned char ring[];
  constexpr int kKeys = kSumStaged + 2 * kSumChunk + 2;
  __shared__ int sKey[kKeys], sPos[kSumStaged + kSumChunk];
  grid_dependency_wait();
  grid_dependency_trigger();
  if (blockIdx.x >= sumBlocks) {
    if (blockIdx.y == 0)
      zero_rows((long long)(blockIdx.x - sumBlocks) * kZeroRows, n, vocab, dim, in, dtable, ldd);
    return;
  }
  // keys from one chunk and one position before the block's first chunk to one
  // chunk and one position past its last: sKey[i - base]
  const int perBlock = kSumThreads / G;
  const long long b0 = (long long)blockIdx.x * perBlock * chunkRows;
  const long long base = b0 - chunkRows - 1;
  const int held = perBlock * chunkRows;
  for (int i = threadIdx.x; i < held + 2 * chunkRows + 2; i += kSumThreads) {
    const long long at = base + i;
    sKey[i] = at < 0 ? -1 : at < n ? in.key_at(at) : vocab;
    if (i < held + chunkRows) sPos[i] = b0 + i < n ? in.pos_at(b0 + i) : 0;
  }
  __syncthreads();
  const long long chunk = (long long)blockIdx.x * perBlock + threadIdx.x / G;
  const long long col = APART ? (long long)blockIdx.y * G * E + threadIdx.x % G
                              : ((long long)blockIdx.y * G + threadIdx.x % G) * E;
  if (chunk >= chunks || col >= dim) return;
  const int columns = dim - (int)col;  // from the thread's first one on
  const int here = (threadIdx.x / G) * chunkRows;  // of the block's positions
  const int* const k = sKey + here + chunkRows + 1;  // k[i]: key of the chunk's position i
  const int* const at = sPos + here;
  const int len = (int)min((long long)chunkRows, n - chunk * chunkRows);
  const int head = k[0], tail = k[len - 1], after = k[len];
  // whether the tail's row begins here and goes on beyond the next chunk, for the
  // second kernel
  if (col == 0)
    goesOn[chunk] = tail < vocab && after == tail && k[len + chunkRows] == tail &&
                    !(k[-1] == head && head == tail);
  if (head >= vocab) return;
  // the head's row began earlier: the chunk before finishes it if it began there
  // and ends here
  const bool openLeft = k[-1] == head;
  const bool skipHead =
      openLeft && k[-chunkRows - 1] != head && (tail != head || after != head);
  // the tail's row goes on: finished here if it began here and ends in the next chunk
  const bool finish =
      after == tail && !(openLeft && head == tail) && k[len + chunkRows] != tail;
  const int most = finish ? len + chunkRows : len;
  int begin = 0;
  if (skipHead)
    while (begin < len && k[begin] == head) ++begin;
  // whether position i is one of this group's
  auto mine = [&](int i) { return i < most && k[i] < vocab && (i < len || k[i] == tail); };
  int cur = head;
  bool open = openLeft;
  float acc[E], first[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = first[e] = 0.0f;
  auto add = [&](int i, const Pack<T, E>& v, const Pack<O, E>& old) {
    if (k[i] != cur) {
      cur = k[i];
      open = false;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    }
    if (i == len) {  // the next chunk's terms are a sum of their own
#pragma unroll
      for (int e = 0; e < E; ++e) {
        first[e] = acc[e];
        acc[e] = 0.0f;
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += to_f32(v.v[e]);
    const bool ends = k[i + 1] != cur;
    if (ends && !open) {
      if (i >= len)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += first[e];
      put<APART>(dtable + cur * ldd + col, finished<ADD>(acc, scale, old), G, columns);
    } else if (ends || (i + 1 == len && !finish)) {
      Pack<float, E> p;
#pragma unroll
      for (int e = 0; e < E; ++e) p.v[e] = acc[e];
      put<APART>(part + (2 * chunk + (open ? 0 : 1)) * dim + col, p, G, columns);
    }
  };
  if constexpr (!APART) {
    constexpr int kD = kSlots, kT = E * (int)sizeof(T), kO = E * (int)sizeof(O);
    // slot j: every thread's share of a row of g, then of the row added to
    auto slot = [&](int j) { return ring + (size_t)j * kSumThreads * kSlotBytes<T, O, E, ADD>; };
    int next = begin;  // the next position to fetch
    auto fetch = [&](int j) {
      if (mine(next)) {
        fetch_share<kT>(slot(j), g + at[next] * ldg + col);
        if (ADD && k[next + 1] != k[next])  // what a row that ends here is added to
          fetch_share<kO>(slot(j) + kSumThreads * kT, dtable + k[next] * ldd + col);
      }
      ++next;
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int j = 0; j < kD - 1; ++j) fetch(j);
    int j = 0;
    for (int i = begin; mine(i); ++i) {
      fetch(j == 0 ? kD - 1 : j - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kD - 1) : "memory");
      const Pack<T, E> v = own_share<Pack<T, E>>(slot(j));
      Pack<O, E> old;
      if (ADD) old = own_share<Pack<O, E>>(slot(j) + kSumThreads * kT);
      add(i, v, old);
      j = j + 1 == kD ? 0 : j + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    constexpr int R = ADD ? 4 : 8;
    for (int b = begin; mine(b); b += R) {
      Pack<T, E> v[R];
      Pack<O, E> old[R];
#pragma unroll
      for (int u = 0; u < R; ++u)
        v[u] = take<true, T, E>(g + at[mine(b + u) ? b + u : b] * ldg + col, G, columns);
      if (ADD)
#pragma unroll
        for (int u = 0; u < R; ++u)
          if (mine(b + u) && k[b + u + 1] != k[b + u])
            old[u] = take<true, O, E>(dtable + k[b + u] * ldd + col, G, columns);
#pragma unroll
      for (int u = 0; u < R; ++u) {
        if (!mine(b + u)) return;
        add(b + u, v[u], old[u]);
      }
    }
  }
}

// The rows that go on beyond the chunk after the one they begin in, as the sums have
// marked them: kJoinBlocks blocks look at the marks of the same kJoinChunks chunks
// and take the marked ones in turn; a block's kSumThreads / L groups of L lanes add a
// run of the row's partial sums each. (A block for every 4 chunks, most of which
// found nothing, 17 us instead of 9 for 32768 tokens of 4096 bf16 columns; 2048 tokens
// 23.4 -> 17.4 in all. 16 blocks to the same marks 231 us in all, 32 227, 64 226; with
// 128 lanes to a group the long rows of a vocabulary of 3 take 48 us, with 64 38.)
template <class O, int E, bool ADD>
__global__ void __launch_bounds__(kSumThreads, 4) k_embed_join(
    int dim, int logL, int chunkRows, long long chunks, const SortedTokens in,
    const unsigned char* goesOn, const float* part, float scale, O* dtable, long long ldd) {
  __shared__ __align__(16) float sums[kSumThreads * E];
  __shared__ unsigned begins[kJoinChunks / 32];
  static_assert(kJoinChunks == 32 * 32, "a word of begins to a lane");
  grid_dependency_wait();
  grid_dependency_trigger();
  const int L = 1 << logL, groups = kSumThreads >> logL;
  const int group = threadIdx.x >> logL, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long col = ((long long)blockIdx.y * L + (threadIdx.x & (L - 1))) * E;
  const long long chunk0 = (long long)(blockIdx.x / kJoinBlocks) * kJoinChunks;
#pragma unroll
  for (int w = warp; w < kJoinChunks / 32; w += kSumThreads / 32) {
    const long long c = chunk0 + w * 32 + lane;
    const unsigned found = __ballot_sync(kFullMask, c < chunks && goesOn[c] != 0);
    if (lane == 0) begins[w] = found;
  }
  __syncthreads();
  // every warp: how many begins there are, and before each word of them
  const unsigned word = begins[lane];
  int upTo = __popc(word);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(kFullMask, upTo, off);
    if (lane >= off) upTo += o;
  }
  const int total = __shfl_sync(kFullMask, upTo, 31);
  for (int item = blockIdx.x % kJoinBlocks; item < total; item += kJoinBlocks) {
    const int w = __ffs(__ballot_sync(kFullMask, upTo > item)) - 1;  // it is in this word
    unsigned bits = __shfl_sync(kFullMask, word, w);
    for (int skip = item - (__shfl_sync(kFullMask, upTo, w) - __popc(bits)); skip > 0; --skip)
      bits &= bits - 1;
    const long long chunk = chunk0 + w * 32 + __ffs(bits) - 1;
    const int row = in.key_at((chunk + 1) * chunkRows - 1);
    // the chunks after it that begin with the row: m of them
    long long m = 0;
    for (int found = kSumThreads; found == kSumThreads; m += found) {
      const long long c = chunk + 1 + m + threadIdx.x;
      found = __syncthreads_count(c < chunks && in.key_at(c < chunks ? c * chunkRows : 0) == row);
    }
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    const long long a = chunk + 1 + m * group / groups, b = chunk + 1 + m * (group + 1) / groups;
    if (col < dim)
      for (long long c = a; c < b; c += kJoinRows) {
        Pack<float, E> v[kJoinRows];
#pragma unroll
        for (int u = 0; u < kJoinRows; ++u)
          if (c + u < b)
            v[u] = *reinterpret_cast<const Pack<float, E>*>(part + 2 * (c + u) * dim + col);
#pragma unroll
        for (int u = 0; u < kJoinRows; ++u)
          if (c + u < b)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += v[u].v[e];
      }
#pragma unroll
    for (int e = 0; e < E; ++e) sums[threadIdx.x * E + e] = acc[e];
    for (int half = groups / 2; half > 0; half /= 2) {  // groups 0 .. half - 1 take the others'
      __syncthreads();
      if (group < half)
#pragma unroll
        for (int e = 0; e < E; ++e)
          sums[threadIdx.x * E + e] += sums[(threadIdx.x + half * L) * E + e];
    }
    if (group == 0 && col < dim) {
      O* const to = dtable + row * ldd + col;
      Pack<O, E> old;
      if (ADD) old = *reinterpret_cast<const Pack<O, E>*>(to);
      const Pack<float, E> q =
          *reinterpret_cast<const Pack<float, E>*>(part + (2 * chunk + 1) * dim + col);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = q.v[e] + sums[threadIdx.x * E + e];
      *reinterpret_cast<Pack<O, E>*>(to) = finished<ADD>(acc, scale, old);
    }
    __syncthreads();  // sums is free again
  }
}

struct GradWork {
  long long sortBytes, partBytes, markBytes;  // (a mark for each chunk)
  long long all() const { return sortBytes + partBytes + markBytes; }
};
GradWork grad_work(int vocab, int dim, int n) {
  GradWork w{0, 0, 0};
  if (vocab <= 0 || dim <= 0 || n <= 0) return w;
  w.sortBytes = n <= kSortMost ? 2LL * n * (long long)sizeof(int)
                               : (long long)token_sort_scratch_bytes(n, vocab);
  w.sortBytes = (w.sortBytes + 255) & ~255LL;
  for (const int E : {8, 4}) {  // whichever the pointers will allow
    const long long chunks = sum_shape(n, dim, E).chunks;
    w.partBytes = std::max(w.partBytes, 2 * chunks * dim * 4);
    w.markBytes = std::max(w.markBytes, chunks);
  }
  return w;
}

// Sorts up to kSortMost tokens.
template <int IPT>
cudaError_t launch_sort(int n, int vocab, const void* tokens, int wide, int blocks, int2* out,
                        cudaStream_t s) {
  int keyBits = 1;
  while (keyBits < 31 && (1LL << keyBits) <= vocab) ++keyBits;
  const int passes = (keyBits + kSortMaxBits - 1) / kSortMaxBits;
  const int bits = (keyBits + passes - 1) / passes;
  static KernelOnce once;
  cudaError_t e = once.allow(reinterpret_cast<const void*>(k_embed_sort<IPT>),
                            (int)sort_smem(IPT, kSortMaxBits));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = sort_smem(IPT, bits);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)blocks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, k_embed_sort<IPT>, n, vocab, tokens, wide, passes, bits, out);
  note_launches(1);
  return e;
}

// The sums, zeros and, where a row can go on beyond the next chunk, the join. With
// E = 1 (rows of any alignment) a thread of the sums has 4 columns apart.
template <class T, class O, int E, bool ADD>
cudaError_t launch_sums(const SumShape& shape, dim3 grid, int n, int vocab, int dim,
                        const SortedTokens& sorted, const T* g, long long ldg, float scale,
                        O* dtable, long long ldd, float* part, unsigned char* goesOn,
                        cudaStream_t s) {
  const auto sum = k_embed_sum<T, O, E == 1 ? 4 : E, E == 1, ADD>;
  constexpr int smem = E == 1 ? 0 : kSumSmem<T, O, E, ADD>;
  static KernelOnce once;
  cudaError_t e = once.allow(reinterpret_cast<const void*>(sum), smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent_smem(sum, grid, kSumThreads, smem, s, n, vocab, dim, shape.G, shape.chunk,
                            shape.chunks, (unsigned)shape.blocksX, sorted, g, ldg, scale, dtable,
                            ldd, part, goesOn);
  if (e != cudaSuccess || shape.chunks <= 2) return e;
  constexpr int kJoinE = E < 4 ? E : 4;
  const long long lanes = ((long long)dim + kJoinE - 1) / kJoinE;
  int logL = 0;
  while (logL < 6 && (1 << logL) < lanes) ++logL;
  const long long looks = (shape.chunks + kJoinChunks - 1) / kJoinChunks;
  return launch_dependent(k_embed_join<O, kJoinE, ADD>,
                          dim3((unsigned)(looks * kJoinBlocks),
                               (unsigned)((lanes + (1 << logL) - 1) >> logL)),
                          kSumThreads, s, dim, logL, shape.chunk, shape.chunks, sorted,
                          (const unsigned char*)goesOn, (const float*)part, scale, dtable, ldd);
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
  const int E = std::min(elements_at_once(d_table, ld_table, dim, tb, 8),
                         elements_at_once(d_out, ld_out, dim, ob, 8));
  const long long pieces = ((long long)dim + E - 1) / E;
  const int loads = E == 1 ? kRowLoads<1> : kRowLoads<8>;
  int logG = 0;
  while (logG < 5 && (loads << logG) < pieces) ++logG;
  const long long y = (pieces + (loads << logG) - 1) / (loads << logG);
  if (y > 65535) return SPMV_ERR_TOO_LARGE;
  const dim3 grid((unsigned)(((long long)nTokens + (256 >> logG) - 1) / (256 >> logG)), (unsigned)y);
  return record_cuda(with_dtype(tableType, [&](auto tv) {
    return with_dtype(outType, [&](auto ov) {
      using T = decltype(tv);
      using O = decltype(ov);
      const auto kernel = E == 8   ? k_embed<T, O, 8>
                          : E == 4 ? k_embed<T, O, 4>
                                   : k_embed<T, O, 1>;
      return launch_dependent(kernel, grid, 256, s, (int)nTokens, (int)vocab, (int)dim, logG,
                              static_cast<const T*>(d_table), (long long)ld_table, d_tokens,
                              (int)(indexBytes == 8), scale, static_cast<O*>(d_out),
                              (long long)ld_out);
    });
  }));
}

int spmv_embed_grad_workspace(int32_t vocab, int32_t dim, int32_t nTokens, int64_t* bytes) {
  if (vocab < 0 || dim < 0 || nTokens < 0 || !bytes) return SPMV_ERR_INVALID_ARG;
  const spmv::GradWork w = spmv::grad_work(vocab, dim, nTokens);
  *bytes = w.all();
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
  if (nTokens > 0 && workBytes < w.all()) return SPMV_ERR_INVALID_ARG;
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
  const int gb = dtype_bytes(gType), tb = dtype_bytes(tableType);
  const int most = sum_most(gb, tb);
  const int E = std::min(elements_at_once(d_g, ld_g, dim, gb, most),
                         elements_at_once(d_dtable, ld_dtable, dim, tb, most));
  const SumShape shape = sum_shape(nTokens, dim, std::max(E, 4));
  const long long zeroBlocks = accumulate ? 0 : ((long long)vocab + kZeroRows - 1) / kZeroRows;
  // (the second kernel's slabs are of 64 lanes with 4 columns at most)
  if (((long long)dim + 63) / 64 > 65535 || shape.blocksX + zeroBlocks > 0x7fffffffLL)
    return SPMV_ERR_TOO_LARGE;
  const void* ptrs[] = {d_g, d_tokens, d_dtable, d_work};
  int st = check_current_device_ptrs(ptrs, nTokens > 0 ? 4 : 3);
  if (st != SPMV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* part = reinterpret_cast<float*>(static_cast<char*>(d_work) + w.sortBytes);
  unsigned char* goesOn = static_cast<unsigned char*>(d_work) + w.sortBytes + w.partBytes;
  SortedTokens sorted{nullptr, nullptr, 1};
  if (nTokens > kSortMost) {
    st = record_cuda(launch_token_sort(nTokens, vocab, d_tokens, indexBytes, d_work, &sorted.pos,
                                       &sorted.key, s));
  } else if (nTokens > 0 && nTokens <= kRankMost) {
    int2* const out = static_cast<int2*>(d_work);
    st = record_cuda(launch_dependent(
        k_embed_rank, dim3((unsigned)((nTokens + kRankBlock - 1) / kRankBlock)), kRankThreads, s,
        (int)nTokens, (int)vocab, d_tokens, (int)(indexBytes == 8), out));
    sorted = {&out->x, &out->y, 2};
  } else if (nTokens > 0) {
    int2* const out = static_cast<int2*>(d_work);
    // as few items to a thread as the cluster's blocks allow
    const int blocks = nTokens <= 4 * kSortThreads ? 4 : kSortMaxBlocks;
    int ipt = 1;
    while (blocks * kSortThreads * ipt < nTokens) ipt *= 2;
    const auto sort = ipt == 1   ? launch_sort<1>
                      : ipt == 2 ? launch_sort<2>
                      : ipt == 4 ? launch_sort<4>
                                 : launch_sort<8>;
    st = record_cuda(sort(nTokens, vocab, d_tokens, indexBytes == 8, blocks, out, s));
    sorted = {&out->x, &out->y, 2};
  }
  if (st != SPMV_OK) return st;
  const dim3 grid((unsigned)(shape.blocksX + zeroBlocks), (unsigned)shape.slabs);
  return record_cuda(with_dtype(gType, [&](auto gv) {
    return with_dtype(tableType, [&](auto ov) {
      using T = decltype(gv);
      using O = decltype(ov);
      constexpr int kMost = sum_most(sizeof(T), sizeof(O));
      const auto launch = E == kMost ? (accumulate ? launch_sums<T, O, kMost, true>
                                                   : launch_sums<T, O, kMost, false>)
                          : E == 4   ? (accumulate ? launch_sums<T, O, 4, true>
                                                   : launch_sums<T, O, 4, false>)
                                     : (accumulate ? launch_sums<T, O, 1, true>
                                                   : launch_sums<T, O, 1, false>);
      return launch(shape, grid, (int)nTokens, (int)vocab, (int)dim, sorted,
                    static_cast<const T*>(d_g), (long long)ld_g, scale,
                    static_cast<O*>(d_dtable), (long long)ld_dtable, part, goesOn, s);
    });
  }));
}

}  // extern "C"
