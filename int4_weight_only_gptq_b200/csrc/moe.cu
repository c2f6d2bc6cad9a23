// Token movement of a mixture-of-experts layer: tokens sorted by expert, the
// experts' rows combined back into tokens, and the gradients of both.
//
// With expert ids e(m, j) (token m's j-th choice, pair p = m * topk + j) and
// the stable order of the pairs by expert,
//   dest[p]   = #{q : e(q) < e(p)} + #{q < p : e(q) = e(p)}   (-1 if dropped)
//   x_sorted[dest[p]] = x[m]
//   out[m]    = sum_j w[p] * y_sorted[dest[p]]
//   dy_sorted[dest[p]] = w[p] * dout[m],  dw[p] = <dout[m], y_sorted[dest[p]]>
// and the gradient of x is the weightless sum of its rows' gradients, which is
// the combine with w = 1.  All of it is bound by memory traffic (or, for a few
// tokens, by launch latency): rows move in 16-byte chunks, each input row is
// read once, sums are FP32 in a fixed order (bitwise reproducible), and every
// result is rounded once.
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "gptq_w4a16.h"
#include "kernels.h"

namespace gptq {

namespace {

__device__ __forceinline__ void wait_previous_grid() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void let_next_grid_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Streaming 16-byte load on the coherent path: these grids may start while the
// previous one still runs, so nothing it writes is read as read-only data
// (for the same reason the kernels' pointers carry no __restrict__).
__device__ __forceinline__ uint4 ld_row_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

__device__ __forceinline__ float2 half2_to_float2(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

__device__ __forceinline__ uint32_t floats_to_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The expert of a pair, or E if the id names no expert (the pair is dropped).
template <typename Id>
__device__ __forceinline__ int key_of(const Id* ids, int64_t p, int E) {
  const Id v = ids[p];
  return v >= 0 && v < (Id)E ? (int)v : E;
}

// The lanes whose key equals this lane's: one ballot per bit.  (A warp match
// instruction takes a time that grows with the number of different keys: with
// it the places of 65,536 pairs of 128 experts took 23.8 us instead of 12.8.)
__device__ __forceinline__ unsigned lanes_with_equal(int key, int key_bits) {
  unsigned same = 0xffffffffu;
  for (int b = 0; b < key_bits; ++b) {
    const unsigned set = __ballot_sync(0xffffffffu, (key >> b) & 1);
    same &= (key >> b) & 1 ? set : ~set;
  }
  return same;
}

// ---- sort, few pairs: one launch ------------------------------------------
//
// Every CTA holds all keys in shared memory and counts the places of its own
// tokens' pairs directly from the definition of dest: O(pairs) work per pair,
// which for up to kSortSmallPairs pairs takes less time than a second launch.
// A key is expert * 4096 + p, so that dest is the number of smaller keys.
// The last CTA writes the experts' offsets (a histogram and a scan).
constexpr int kSortSmallShift = 12;
constexpr int kSortSmallPairs = 1 << kSortSmallShift;
constexpr int kSmallThreads = 256;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kSmallAhead = 3;  // 16-byte chunks of a row per thread loaded ahead

template <typename Id>
__global__ void __launch_bounds__(kSmallThreads, 8)
    sort_small_kernel(const uint16_t* x, const Id* ids, int M, int H,
                      int topk, int E, uint16_t* x_sorted,
                      int32_t* offsets, int32_t* dest) {
  extern __shared__ __align__(16) int keys[];
  __shared__ int places[GPTQ_MOE_MAX_TOPK];
  __shared__ int counts[GPTQ_MOE_MAX_EXPERTS];
  wait_previous_grid();
  let_next_grid_start();
  const int P = M * topk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 4
  for (int p = threadIdx.x; p < P; p += kSmallThreads)
    keys[p] = key_of(ids, p, E) << kSortSmallShift | p;
  // to a multiple of four keys: the largest key there is
  if ((int)threadIdx.x < 3) keys[P + threadIdx.x] = 0x7FFFFFFF;
  if ((int)blockIdx.x == gridDim.x - 1) {
    for (int e = threadIdx.x; e < E; e += kSmallThreads) counts[e] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < P; p += kSmallThreads) {
      const int e = keys[p] >> kSortSmallShift;
      if (e < E) atomicAdd(&counts[e], 1);
    }
    __syncthreads();
    if (warp == 0) {
      int before = 0;
      for (int e0 = 0; e0 < E; e0 += 32) {
        const int c = e0 + lane < E ? counts[e0 + lane] : 0;
        int s = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += v;
        }
        if (e0 + lane < E) offsets[e0 + lane] = before + s - c;
        before += __shfl_sync(0xffffffffu, s, 31);
      }
      if (lane == 0) offsets[E] = before;
    }
    return;
  }
  __syncthreads();
  for (int m = blockIdx.x; m < M; m += gridDim.x - 1) {
    // the row's first chunks are under way while the places are counted
    const uint4* src = reinterpret_cast<const uint4*>(x + (int64_t)m * H);
    const int chunks = H / 8;
    uint4 v[kSmallAhead];
#pragma unroll
    for (int i = 0; i < kSmallAhead; ++i)
      if ((int)threadIdx.x + i * kSmallThreads < chunks)
        v[i] = ld_row_v4(src + threadIdx.x + i * kSmallThreads);
    for (int j = warp; j < topk; j += kSmallWarps) {
      const int p = m * topk + j, key = keys[p];
      int n = -1;
      if (key >> kSortSmallShift < E) {
        n = 0;
        for (int q = lane; 4 * q < P; q += 32) {
          const int4 k = reinterpret_cast<const int4*>(keys)[q];
          n += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
        }
        n = __reduce_add_sync(0xffffffffu, n);
      }
      if (lane == 0) {
        places[j] = n;
        dest[p] = n;
      }
    }
    __syncthreads();
    for (int j = 0; j < topk; ++j) {
      if (places[j] < 0) continue;
      uint4* out = reinterpret_cast<uint4*>(x_sorted + (int64_t)places[j] * H);
#pragma unroll
      for (int i = 0; i < kSmallAhead; ++i)
        if ((int)threadIdx.x + i * kSmallThreads < chunks)
          out[threadIdx.x + i * kSmallThreads] = v[i];
    }
    for (int c = threadIdx.x + kSmallAhead * kSmallThreads; c < chunks; c += kSmallThreads) {
      const uint4 more = ld_row_v4(src + c);
      for (int j = 0; j < topk; ++j)
        if (places[j] >= 0)
          reinterpret_cast<uint4*>(x_sorted + (int64_t)places[j] * H)[c] = more;
    }
    __syncthreads();
  }
}

// ---- sort, more pairs: one launch, every CTA counts all ids --------------------
//
// One CTA per SM takes a run of tokens.  It asks for their rows (into L2),
// reads every id while they arrive, counts the pairs of each expert before its
// own run and in all, ranks its own pairs, and moves its rows.  Reading all ids
// on every SM costs less than a launch of its own for the places, while there
// are few of them and few rows: against the two launches below, in us,
//   tokens x choices x H   520 x 8 x 2048   4000 x 4 x 512   16000 x 1 x 64
//     two launches              8.3              8.7              7.8
//     this one                  5.7              7.3              6.4
// With more bytes the copy decides, and 32 warps an SM keep less of it in flight
// than the grid of sort_rows: at 16,384 pairs 42 MB took 12.4 for 13.0, 98 MB
// 22.4 for 21.6, and 8192 x 2 x 5120 (252 MB) 50 for 44.  Moving the rows by
// bulk copies through shared memory instead (four warps, up to eight rows each)
// narrowed that to 48 and cost the small ones half a microsecond.
constexpr int kSortMidPairs = 16384;
constexpr int64_t kSortMidBytes = 48 << 20;
constexpr int kMidThreads = 1024;
constexpr int kMidWarps = kMidThreads / 32;
constexpr int kMidIds = 8;    // of a thread at once, all loads in flight
constexpr int kMidChunks = 4;  // 16-byte chunks of a row per lane
constexpr int kMidOwn = 256;  // pairs of one CTA: its tokens' choices

template <typename Id>
__global__ void __launch_bounds__(kMidThreads, 1)
    sort_mid_kernel(const uint16_t* x, const Id* ids, int M, int H, int topk, int E,
                    uint16_t* x_sorted, int32_t* offsets, int32_t* dest) {
  __shared__ int before[GPTQ_MOE_MAX_EXPERTS];  // pairs of the expert before this run
  __shared__ int total[GPTQ_MOE_MAX_EXPERTS];   // ... in all; then its next place
  __shared__ int warp_sums[kMidWarps];
  __shared__ int places[kMidOwn];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m0 = (int)((int64_t)blockIdx.x * M / gridDim.x);
  const int m1 = (int)((int64_t)(blockIdx.x + 1) * M / gridDim.x);
  const int P = M * topk, p0 = m0 * topk, p1 = m1 * topk;
  before[threadIdx.x] = 0;
  total[threadIdx.x] = 0;
  wait_previous_grid();
  let_next_grid_start();
  {
    const char* rows = reinterpret_cast<const char*>(x + (int64_t)m0 * H);
    const int64_t bytes = (int64_t)(m1 - m0) * H * 2;
    for (int64_t b = 128 * (int64_t)threadIdx.x; b < bytes; b += 128 * kMidThreads)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(rows + b));
  }
  __syncthreads();
  const int key_bits = 32 - __clz(E);  // keys are 0 .. E
  for (int q = threadIdx.x; q < P; q += kMidIds * kMidThreads) {
    int key[kMidIds];
#pragma unroll
    for (int i = 0; i < kMidIds; ++i)
      key[i] = q + i * kMidThreads < P ? key_of(ids, q + i * kMidThreads, E) : E;
#pragma unroll
    for (int i = 0; i < kMidIds; ++i) {
      if (key[i] == E) continue;
      atomicAdd(&total[key[i]], 1);
      if (q + i * kMidThreads < p0) atomicAdd(&before[key[i]], 1);
    }
  }
  __syncthreads();
  // thread e: the expert's first row, and this run's first place in it
  const int all = (int)threadIdx.x < E ? total[threadIdx.x] : 0;
  int scan = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) warp_sums[warp] = scan;
  __syncthreads();
  int prior = lane < warp ? warp_sums[lane] : 0;  // 32 warps: one lane each
  prior = __reduce_add_sync(0xffffffffu, prior);
  const int start = prior + scan - all;
  if ((int)threadIdx.x < E) {
    total[threadIdx.x] = start + before[threadIdx.x];
    if (blockIdx.x == 0) {
      offsets[threadIdx.x] = start;
      if ((int)threadIdx.x == E - 1) offsets[E] = start + all;
    }
  }
  __syncthreads();
  if (warp == 0) {
    for (int p = p0; p < p1; p += 32) {
      const int k = p + lane < p1 ? key_of(ids, p + lane, E) : E;
      const unsigned same = lanes_with_equal(k, key_bits);
      const int lower = __popc(same & ((1u << lane) - 1u));
      const int at = k < E ? total[k] : 0;
      __syncwarp();
      if (k < E && lower == 0) total[k] = at + __popc(same);
      __syncwarp();
      if (p + lane < p1) {
        const int d = k < E ? at + lower : -1;
        places[p + lane - p0] = d;
        dest[p + lane] = d;
      }
    }
  }
  __syncthreads();
  const int chunks = H / 8, segments = (chunks + 32 * kMidChunks - 1) / (32 * kMidChunks);
  for (int u = warp; u < (m1 - m0) * segments; u += kMidWarps) {
    const int mm = u / segments, c0 = (u - mm * segments) * (32 * kMidChunks) + lane;
    const uint4* src = reinterpret_cast<const uint4*>(x + (int64_t)(m0 + mm) * H);
    uint4 v[kMidChunks];
#pragma unroll
    for (int i = 0; i < kMidChunks; ++i)
      if (c0 + 32 * i < chunks) v[i] = ld_row_v4(src + c0 + 32 * i);
    for (int j = 0; j < topk; ++j) {
      const int d = places[mm * topk + j];
      if (d < 0) continue;
      uint4* out = reinterpret_cast<uint4*>(x_sorted + (int64_t)d * H);
#pragma unroll
      for (int i = 0; i < kMidChunks; ++i)
        if (c0 + 32 * i < chunks) out[c0 + 32 * i] = v[i];
    }
  }
}

// ---- sort, many pairs: places by one cluster, then the rows ------------------
//
// One cluster of eight CTAs; every warp owns a contiguous run of pairs and
// walks it twice: once counting its pairs per expert, once handing out places
// in order from its running base per expert.  Between the walks the counts
// are turned into bases: over the warps of a CTA, over the CTAs (distributed
// shared memory), over the experts.  The order of pairs is kept throughout, so
// the sort is stable, and it needs no scratch memory.
constexpr int kPlaceCtas = 8;
constexpr int kPlaceThreads = 1024;
constexpr int kPlaceWarps = kPlaceThreads / 32;
constexpr int kPlaceKeys = 8;  // pairs per lane whose ids are loaded together

constexpr size_t place_smem_bytes(int E) { return ((size_t)kPlaceWarps + 2) * E * sizeof(int); }

__device__ __forceinline__ int ld_dsmem_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Keys of pairs p, p + 32, ..., all loads in flight at once.
template <typename Id>
__device__ __forceinline__ void load_keys(const Id* ids, int64_t p, int64_t end, int E,
                                          int (&key)[kPlaceKeys]) {
#pragma unroll
  for (int i = 0; i < kPlaceKeys; ++i) key[i] = p + 32 * i < end ? key_of(ids, p + 32 * i, E) : E;
}

template <typename Id>
__global__ void __cluster_dims__(kPlaceCtas, 1, 1) __launch_bounds__(kPlaceThreads)
    sort_place_kernel(const Id* ids, int64_t P, int E,
                      int32_t* offsets, int32_t* dest) {
  // warp w's count, then base, of expert e: base[w * E + e]; this CTA's total
  // of expert e: total[e]; the first place of expert e: first[e]
  extern __shared__ int sm[];
  int* base = sm;
  int* total = sm + kPlaceWarps * E;
  int* first = total + E;
  __shared__ int warp_sums[kPlaceWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = (int)cluster_ctarank();
  wait_previous_grid();
  // After the wait, never before: sort_rows_kernel reads x as soon as every CTA
  // has said this, so it must mean that the work before this launch is done.
  let_next_grid_start();
  const int64_t w = (int64_t)cta * kPlaceWarps + warp;
  constexpr int64_t W = kPlaceCtas * kPlaceWarps;
  const int64_t begin = P * w / W, end = P * (w + 1) / W;
  int* mine = base + warp * E;
  for (int e = lane; e < E; e += 32) mine[e] = 0;
  __syncwarp();
  int key[kPlaceKeys];
  for (int64_t p0 = begin; p0 < end; p0 += 32 * kPlaceKeys) {
    load_keys(ids, p0 + lane, end, E, key);
#pragma unroll
    for (int i = 0; i < kPlaceKeys; ++i) {
      if (p0 + 32 * i >= end) break;
      if (key[i] < E) atomicAdd(&mine[key[i]], 1);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kPlaceThreads) {
    int c[kPlaceWarps];
#pragma unroll
    for (int v = 0; v < kPlaceWarps; ++v) c[v] = base[v * E + e];
    int sum = 0;
#pragma unroll
    for (int v = 0; v < kPlaceWarps; ++v) {
      base[v * E + e] = sum;
      sum += c[v];
    }
    total[e] = sum;
  }
  cluster_sync_all();
  // thread e (E <= 1024 threads): this expert's pairs in all CTAs and in the
  // CTAs before this one, then the scan over the experts
  int before = 0, all = 0;
  if ((int)threadIdx.x < E) {
#pragma unroll
    for (int c = 0; c < kPlaceCtas; ++c) {
      const int n = ld_dsmem_s32(map_to_rank(smem_u32(&total[threadIdx.x]), (uint32_t)c));
      if (c < cta) before += n;
      all += n;
    }
  }
  int scan = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) warp_sums[warp] = scan;
  __syncthreads();
  int prior = lane < warp ? warp_sums[lane] : 0;  // 32 warps: one lane each
  prior = __reduce_add_sync(0xffffffffu, prior);
  const int start = prior + scan - all;  // the expert's first row
  if ((int)threadIdx.x < E) {
    first[threadIdx.x] = start + before;
    if (cta == 0) {
      offsets[threadIdx.x] = start;
      if ((int)threadIdx.x == E - 1) offsets[E] = start + all;
    }
  }
  // no CTA leaves while another may still read its totals: this one has read
  // them, and waits for the others at its end
  cluster_arrive();
  __syncthreads();  // first[] is complete
  for (int e = lane; e < E; e += 32) mine[e] += first[e];
  __syncwarp();
  const int key_bits = 32 - __clz(E);  // keys are 0 .. E
  const bool kept = end - begin <= 32 * kPlaceKeys;  // the first walk's keys are all still here
  for (int64_t p0 = begin; p0 < end; p0 += 32 * kPlaceKeys) {
    if (!kept) load_keys(ids, p0 + lane, end, E, key);
#pragma unroll
    for (int i = 0; i < kPlaceKeys; ++i) {
      const int64_t p = p0 + 32 * i + lane;
      if (p - lane >= end) break;
      const unsigned same = lanes_with_equal(key[i], key_bits);
      const int lower = __popc(same & ((1u << lane) - 1u));
      const int at = key[i] < E ? mine[key[i]] : 0;
      __syncwarp();
      if (key[i] < E && lower == 0) mine[key[i]] = at + __popc(same);
      __syncwarp();
      if (p < end) dest[p] = key[i] < E ? at + lower : -1;
    }
  }
  cluster_wait();
}

// Rows: a warp takes 1024 values (four 16-byte chunks per lane) of one token,
// reads them once and writes them to each of the token's places.  The grid
// starts once every CTA of the places' launch has passed its own wait for
// earlier work, so x is complete by then and its first loads run beside that
// launch; only the places wait for it.
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kGatherChunks = 4;

__global__ void __launch_bounds__(kRowThreads)
    sort_rows_kernel(const uint16_t* x, const int32_t* dest, int64_t M, int H,
                     int topk, int segments, uint16_t* x_sorted) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int64_t m = unit / segments;
  if (m >= M) {
    wait_previous_grid();
    return;
  }
  const int c0 = (int)(unit - m * segments) * (32 * kGatherChunks) + lane, chunks = H / 8;
  const uint4* src = reinterpret_cast<const uint4*>(x + m * H);
  uint4 v[kGatherChunks];
#pragma unroll
  for (int i = 0; i < kGatherChunks; ++i)
    if (c0 + 32 * i < chunks) v[i] = ld_row_v4(src + c0 + 32 * i);
  wait_previous_grid();
  let_next_grid_start();
  for (int j0 = 0; j0 < topk; j0 += 32) {
    const int mine = j0 + lane < topk ? dest[m * topk + j0 + lane] : -1;
    const int n = min(32, topk - j0);
    for (int j = 0; j < n; ++j) {
      const int d = __shfl_sync(0xffffffffu, mine, j);
      if (d < 0) continue;
      uint4* out = reinterpret_cast<uint4*>(x_sorted + (int64_t)d * H);
#pragma unroll
      for (int i = 0; i < kGatherChunks; ++i)
        if (c0 + 32 * i < chunks) out[c0 + 32 * i] = v[i];
    }
  }
}

// ---- combine -----------------------------------------------------------------

// A place read from dest: -1 if the pair was dropped; one outside the rows is
// reported and treated as dropped.
__device__ __forceinline__ int checked_place(int d, int64_t R, int* err) {
  if (d >= R) {
    atomicCAS(err, 0, kDeviceErrIndex);
    return -1;
  }
  return d < 0 ? -1 : d;
}

// A warp takes 512 values (two chunks per lane) of one token and adds its
// rows in the order of the choices, FP32, four rows' loads in flight.
constexpr int kCombineChunks = 2;
constexpr int kCombineAhead = 4;

template <bool WEIGHTED>
__global__ void __launch_bounds__(kRowThreads)
    combine_kernel(const uint16_t* y, const int32_t* dest,
                   const float* weights, int64_t M, int H, int topk, int64_t R,
                   int segments, uint16_t* out, int* err) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  wait_previous_grid();
  let_next_grid_start();
  const int64_t m = unit / segments;
  if (m >= M) return;
  const int c0 = (int)(unit - m * segments) * (32 * kCombineChunks) + lane, chunks = H / 8;
  float acc[kCombineChunks][8];
#pragma unroll
  for (int i = 0; i < kCombineChunks; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[i][q] = 0.f;
  for (int j0 = 0; j0 < topk; j0 += 32) {
    const int n = min(32, topk - j0);
    const int64_t p = m * topk + j0 + lane;
    const int place = lane < n ? checked_place(dest[p], R, err) : -1;
    const float weight = WEIGHTED && lane < n ? weights[p] : 1.f;
    for (int j = 0; j < n; j += kCombineAhead) {
      uint4 v[kCombineAhead][kCombineChunks];
      int d[kCombineAhead];
#pragma unroll
      for (int a = 0; a < kCombineAhead; ++a) {
        d[a] = j + a < n ? __shfl_sync(0xffffffffu, place, j + a) : -1;
        const uint4* src = reinterpret_cast<const uint4*>(y + (int64_t)d[a] * H);
#pragma unroll
        for (int i = 0; i < kCombineChunks; ++i)
          if (d[a] >= 0 && c0 + 32 * i < chunks) v[a][i] = ld_row_v4(src + c0 + 32 * i);
      }
#pragma unroll
      for (int a = 0; a < kCombineAhead; ++a) {
        if (d[a] < 0) continue;  // the same for the whole warp
        const float w = __shfl_sync(0xffffffffu, weight, j + a);
#pragma unroll
        for (int i = 0; i < kCombineChunks; ++i) {
          const uint32_t h[4] = {v[a][i].x, v[a][i].y, v[a][i].z, v[a][i].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 f = half2_to_float2(h[q]);
            acc[i][2 * q] = fmaf(w, f.x, acc[i][2 * q]);
            acc[i][2 * q + 1] = fmaf(w, f.y, acc[i][2 * q + 1]);
          }
        }
      }
    }
  }
  uint4* dst = reinterpret_cast<uint4*>(out + m * H);
#pragma unroll
  for (int i = 0; i < kCombineChunks; ++i)
    if (c0 + 32 * i < chunks)
      dst[c0 + 32 * i] = make_uint4(floats_to_half2(acc[i][0], acc[i][1]),
                                    floats_to_half2(acc[i][2], acc[i][3]),
                                    floats_to_half2(acc[i][4], acc[i][5]),
                                    floats_to_half2(acc[i][6], acc[i][7]));
}

// ---- combine, backward ---------------------------------------------------------

// One CTA per token, CHOICES choices at a time: each thread takes AHEAD chunks
// of dout and the rows' chunks beside them (all loads in flight together),
// stores w * dout (one rounding) and adds up its part of the dot products;
// lanes by shuffles, warps in order.  CHOICES * AHEAD = 8 keeps the loads in
// flight, and with them the bandwidth, the same for few choices as for many:
// two choices of 8192 x 5120 took 101 us with AHEAD = 1 (4.2 TB/s).
constexpr int kBackThreads = 128;
constexpr int kBackWarps = kBackThreads / 32;

template <int CHOICES, int AHEAD>
__global__ void __launch_bounds__(kBackThreads)
    combine_backward_kernel(const uint16_t* dout, const uint16_t* y, const int32_t* dest,
                            const float* weights, int H, int topk, int64_t R, uint16_t* dy,
                            float* dw, int* err) {
  __shared__ float part[kBackWarps][CHOICES];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_previous_grid();
  let_next_grid_start();
  const int64_t m = blockIdx.x;
  const int chunks = H / 8;
  const uint4* g = reinterpret_cast<const uint4*>(dout + m * H);
  for (int j0 = 0; j0 < topk; j0 += CHOICES) {
    int d[CHOICES];
    float w[CHOICES], dot[CHOICES];
#pragma unroll
    for (int j = 0; j < CHOICES; ++j) {
      const int64_t p = m * topk + j0 + j;
      d[j] = j0 + j < topk ? checked_place(dest[p], R, err) : -1;
      w[j] = j0 + j < topk ? weights[p] : 0.f;
      dot[j] = 0.f;
    }
    for (int c0 = threadIdx.x; c0 < chunks; c0 += kBackThreads * AHEAD) {
      uint4 gv[AHEAD], v[AHEAD][CHOICES];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int c = c0 + a * kBackThreads;
        if (c >= chunks) break;
        gv[a] = ld_row_v4(g + c);
#pragma unroll
        for (int j = 0; j < CHOICES; ++j)
          if (d[j] >= 0)
            v[a][j] = ld_row_v4(reinterpret_cast<const uint4*>(y + (int64_t)d[j] * H) + c);
      }
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int c = c0 + a * kBackThreads;
        if (c >= chunks) break;
        const float2 g0 = half2_to_float2(gv[a].x), g1 = half2_to_float2(gv[a].y);
        const float2 g2 = half2_to_float2(gv[a].z), g3 = half2_to_float2(gv[a].w);
#pragma unroll
        for (int j = 0; j < CHOICES; ++j) {
          if (d[j] < 0) continue;
          fma8(dot[j], v[a][j], g0, g1, g2, g3);
          reinterpret_cast<uint4*>(dy + (int64_t)d[j] * H)[c] =
              make_uint4(floats_to_half2(w[j] * g0.x, w[j] * g0.y),
                         floats_to_half2(w[j] * g1.x, w[j] * g1.y),
                         floats_to_half2(w[j] * g2.x, w[j] * g2.y),
                         floats_to_half2(w[j] * g3.x, w[j] * g3.y));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < CHOICES; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_down_sync(0xffffffffu, dot[j], o);
      if (lane == 0) part[warp][j] = dot[j];
    }
    __syncthreads();
    if ((int)threadIdx.x < CHOICES && j0 + (int)threadIdx.x < topk) {
      float s = 0.f;
      for (int v = 0; v < kBackWarps; ++v) s += part[v][threadIdx.x];
      dw[m * topk + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

// A launch that may begin while the previous kernel of the stream ends.  Every
// kernel above waits for that one before it reads or writes anything, but for
// sort_rows_kernel, which reads x before it waits for the places' launch (see
// there for why x is complete).
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  Launch(int64_t grid, int block, size_t smem, cudaStream_t stream) {
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

template <typename Id>
cudaError_t launch_sort(const uint16_t* x, const Id* ids, int64_t M, int64_t H, int topk, int E,
                        uint16_t* x_sorted, int32_t* offsets, int32_t* dest, cudaStream_t stream,
                        const DeviceInfo& dev) {
  const int64_t P = M * topk;
  if (P <= kSortSmallPairs) {
    // one CTA per token up to eight per SM, and the one that writes offsets
    const int64_t ctas = std::min<int64_t>(M, 8 * (int64_t)dev.num_sms) + 1;
    const Launch l(ctas, kSmallThreads, (size_t)(P + 3) * sizeof(int), stream);
    return cudaLaunchKernelEx(&l.cfg, sort_small_kernel<Id>, x, ids, (int)M, (int)H, topk, E,
                              x_sorted, offsets, dest);
  }
  const int64_t ctas = std::min<int64_t>(M, dev.num_sms);
  if (P <= kSortMidPairs && M * H * 2 * (topk + 1) <= kSortMidBytes &&
      (M + ctas - 1) / ctas * topk <= kMidOwn) {
    const Launch l(ctas, kMidThreads, 0, stream);
    return cudaLaunchKernelEx(&l.cfg, sort_mid_kernel<Id>, x, ids, (int)M, (int)H, topk, E,
                              x_sorted, offsets, dest);
  }
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  const int di = dev.device & 63;
  std::call_once(once[di], [&] {
    attr_err[di] = cudaFuncSetAttribute(sort_place_kernel<Id>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)place_smem_bytes(GPTQ_MOE_MAX_EXPERTS));
  });
  if (attr_err[di] != cudaSuccess) return attr_err[di];
  const size_t smem = place_smem_bytes(E);
  cudaError_t e;
  const Launch place(kPlaceCtas, kPlaceThreads, smem, stream);
  e = cudaLaunchKernelEx(&place.cfg, sort_place_kernel<Id>, ids, P, E, offsets, dest);
  if (e != cudaSuccess) return e;
  const int segments = (int)((H / 8 + 32 * kGatherChunks - 1) / (32 * kGatherChunks));
  const int64_t units = M * segments;
  const Launch rows((units + kRowWarps - 1) / kRowWarps, kRowThreads, 0, stream);
  return cudaLaunchKernelEx(&rows.cfg, sort_rows_kernel, x, (const int32_t*)dest, M, (int)H, topk,
                            segments, x_sorted);
}

}  // namespace

cudaError_t launch_moe_sort(const uint16_t* x, const void* ids, int id_bytes, int64_t M,
                            int64_t H, int topk, int E, uint16_t* x_sorted, int32_t* offsets,
                            int32_t* dest, cudaStream_t stream, const DeviceInfo& dev) {
  if (id_bytes == 8)
    return launch_sort(x, static_cast<const int64_t*>(ids), M, H, topk, E, x_sorted, offsets,
                       dest, stream, dev);
  return launch_sort(x, static_cast<const int32_t*>(ids), M, H, topk, E, x_sorted, offsets, dest,
                     stream, dev);
}

cudaError_t launch_moe_combine(const uint16_t* y, const int32_t* dest, const float* weights,
                               int64_t M, int64_t H, int topk, int64_t R, uint16_t* out,
                               cudaStream_t stream, const DeviceInfo& dev) {
  const int segments = (int)((H / 8 + 32 * kCombineChunks - 1) / (32 * kCombineChunks));
  const int64_t units = M * segments;
  // few tokens: one warp per CTA, so that their loads spread over the SMs
  const int warps = units < 8 * (int64_t)dev.num_sms ? 1 : kRowWarps;
  const Launch l((units + warps - 1) / warps, 32 * warps, 0, stream);
  return weights ? cudaLaunchKernelEx(&l.cfg, combine_kernel<true>, y, dest, weights, M, (int)H,
                                      topk, R, segments, out, dev.error_word)
                 : cudaLaunchKernelEx(&l.cfg, combine_kernel<false>, y, dest, weights, M, (int)H,
                                      topk, R, segments, out, dev.error_word);
}

cudaError_t launch_moe_combine_backward(const uint16_t* dout, const uint16_t* y,
                                        const int32_t* dest, const float* weights, int64_t M,
                                        int64_t H, int topk, int64_t R, uint16_t* dy, float* dw,
                                        cudaStream_t stream, const DeviceInfo& dev) {
  const Launch l(M, kBackThreads, 0, stream);
  const auto kernel = topk == 1   ? combine_backward_kernel<1, 8>
                      : topk == 2 ? combine_backward_kernel<2, 4>
                      : topk <= 4 ? combine_backward_kernel<4, 2>
                                  : combine_backward_kernel<8, 1>;
  return cudaLaunchKernelEx(&l.cfg, kernel, dout, y, dest, weights, (int)H, topk, R, dy, dw,
                            dev.error_word);
}

}  // namespace gptq
