// The experts' products for few rows per expert (decoding):
//   Y[rows of e] = X[rows of e] . dequant(qweight[e], scales[e])
// streaming each chosen expert's weights once.
//
// The transposed product of the decode kernel (a CTA owns 128 weight columns,
// one TMEM lane each; the tokens are the MMA's N), with the token tiles cut
// from the experts' rows (experts.cuh) and one persistent CTA per SM walking
// the (token tile, column block) items, column block fastest:
//
// * Two rings of 256-k stages, each with a producer warp: the qweight box [32
//   packed rows x 128 columns] (16 KB) with its scale rows, freed as soon as
//   its words are read, and X [ROWS x 256 k], freed by its MMAs.  (In one ring
//   the weights stayed until the MMAs were done, and the loads in flight were
//   too few.)  Rows of X past the tile belong to other experts, each a column of
//   the accumulator that is never stored.
// * Four groups of four warps take the stages in turn; stage f goes to TMEM A
//   slot f mod 3: a thread turns the 32 words of its column into 128 cells.
//   One wait for the stage, one for the slot and one arrival per 32 words: with
//   sixteen words per warp between the barriers the waits were a third of all
//   instructions.
// * Weights are written in natural k order (12 operations a word for scales
//   below 2^-5).  The decode kernel's paired order needs 11, and X permuted in
//   place with a fence for the tensor cores: no faster here.
// * One elected lane issues the MMAs into one of two accumulators; four warps
//   of their own read a finished item out and store it while the next one is
//   multiplied.  An MMA of 16 tokens takes 15 cycles, into one accumulator or
//   into four in turn; a stage's sixteen with their commits 320 alone, 460
//   beside warps that keep the issue slots busy.
// * Few items (splits > 1): the CTAs of a cluster share one item, each taking
//   a range of K, and add their partial sums in rank order through
//   distributed shared memory.
//
// Weights are dequantised exactly as defined, fp16((q - 8) * s), FP32
// accumulation, one rounding; the order of the sums is fixed, so results are
// bitwise reproducible.  Every wait is bounded in time; on expiry the kernel
// records GPTQ_ERR_TIMEOUT in the device error word, drains its own copies
// and MMAs, frees TMEM and exits.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "experts.cuh"
#include "gptq_w4a16.h"
#include "kernels.h"
#include "tc05.cuh"
#include "tmap.h"

namespace gptq {

namespace {

constexpr int BW = 128;        // weight columns per item (MMA M)
constexpr int BK = 256;        // k per stage and A slot fill (16 MMAs of k16)
constexpr int PR = BK / 8;     // packed rows per stage
constexpr int WPT = 8;         // words per TMEM store (32 columns)
constexpr int GROUPS = 4;      // dequantisation groups: stage f goes to group f mod 4
constexpr int SLOTS = 3;       // A slots: stage f goes to slot f mod 3
constexpr int DQ_WARP0 = 2;    // warps 0, 1: weight producer, MMA issuer
constexpr int EPI_WARP0 = DQ_WARP0 + 4 * GROUPS;  // four read-out warps
constexpr int X_WARP = EPI_WARP0 + 4;             // X's producer
constexpr int THREADS = (X_WARP + 1) * 32;
constexpr int QW_BYTES = PR * BW * 4;
constexpr int QW_ROW_BYTES = BW * 4;
constexpr int S_ROW_BYTES = BW * 2;
constexpr int W_MAX = 10, X_MAX = 6;  // ring stages, at most
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t D_COL = 0;     // two accumulators of up to 32 columns
constexpr uint32_t D_NEXT = 64;
constexpr uint32_t A_COL = 128;   // A slots: [128, 512), 128 columns each
constexpr uint32_t A_SLOT_COLS = BK / 2;
constexpr uint64_t kWaitLimitNs = 4000000000ull;
constexpr uint64_t kDrainLimitNs = 200000000ull;
static_assert(A_COL + SLOTS * A_SLOT_COLS <= TMEM_COLS, "TMEM budget");
static_assert(GROUPS < 2 * SLOTS, "see Bars::aempty");
static_assert(EPI_WARP0 % 4 == 2 && DQ_WARP0 % 4 == 2, "quarters by warp % 4");

struct Bars {
  // Use v of weight stage s landed: barrier s + stages * (v & 1).  A group can
  // come to wait for a load that is not issued yet, with the stage's load
  // before it (another group's, when the ring is no multiple of the groups)
  // still under way: the two parities of one barrier could not tell them apart.
  uint64_t wfull[2 * W_MAX];
  uint64_t wempty[W_MAX];      // stage read by its group's warps
  uint64_t xfull[X_MAX];       // X stage landed
  uint64_t xempty[X_MAX];      // MMAs reading it done
  uint64_t afull[SLOTS];       // A slot written by a group's warps
  // MMAs reading use u of slot a done: barrier a + SLOTS * (u & 1).  A group
  // can come to wait for use u - 1 = stage f - 3 while the MMAs of stage f - 6
  // (use u - 2) still run, which one barrier per slot and its parity could not
  // tell from use u - 1 having finished; those of stage f - 9 are done, since
  // the group's own stage f - 4 waited for stage f - 7.
  uint64_t aempty[2 * SLOTS];
  uint64_t dfull[2];           // MMAs of item j done (accumulator j % 2)
  uint64_t dempty[2];          // accumulator read out
  uint32_t tmem_base;
  int abort_flag;
};

// Shared memory: the rings of X and of the weights, the barriers, the table of
// token tiles.
constexpr int kSmemLimit = 227 * 1024 - 1024;

struct Shape {
  int scale_rows, w_bytes, w_stages, smem_bytes;
};

// X stages: enough that a stage's X, asked for when the MMAs of the stage that
// many before are done, lands before its weights are dequantised.
template <int ROWS>
constexpr int x_stages() {
  return ROWS >= 32 ? 5 : 6;
}

template <int ROWS>
Shape shape_of(int group_shift, int E) {
  Shape d;
  const int gs = group_shift < 30 ? group_shift : 30;
  d.scale_rows = (BK >> gs) > 1 ? (BK >> gs) : 1;
  d.w_bytes = QW_BYTES + d.scale_rows * S_ROW_BYTES;
  const int rest =
      x_stages<ROWS>() * ROWS * BK * 2 + (int)sizeof(Bars) + ExpertTable<ROWS, ROWS>::bytes(E);
  d.w_stages = std::min(W_MAX, (kSmemLimit - rest) / d.w_bytes);
  d.smem_bytes = 1024 + d.w_stages * d.w_bytes + rest;
  return d;
}

// One stage's 32 words of a thread's column into its 128 TMEM cells of an A
// slot: eight words at a time, the next eight under way meanwhile.  SMALL: the
// scales allow the form with fewer operations (same values; every lane of the
// warp).  `ready` waits for the slot, after the first eight words are done.
template <int WPS, bool SMALL, class Ready>
__device__ __forceinline__ bool dequant_stage(const uint8_t* qw, const uint8_t* sc, int gs,
                                              uint32_t a_cells, Ready ready) {
  uint32_t w[2][WPT];
#pragma unroll
  for (int i = 0; i < WPT; ++i) w[0][i] = *reinterpret_cast<const uint32_t*>(qw + i * QW_ROW_BYTES);
#pragma unroll
  for (int c = 0; c < PR / WPT; ++c) {
    if (c + 1 < PR / WPT) {
#pragma unroll
      for (int i = 0; i < WPT; ++i)
        w[(c + 1) & 1][i] =
            *reinterpret_cast<const uint32_t*>(qw + (WPT * (c + 1) + i) * QW_ROW_BYTES);
    }
    uint32_t cells[4 * WPT];
#pragma unroll
    for (int g = 0; g < WPT / WPS; ++g) {
      const int srow = (8 * (WPT * c + WPS * g)) >> gs;
      const uint32_t s2 =
          half2_broadcast(*reinterpret_cast<const uint16_t*>(sc + srow * S_ROW_BYTES));
      uint32_t b2, c2;
      if (SMALL) natural_form_constants(s2, b2, c2);
#pragma unroll
      for (int i = 0; i < WPS; ++i) {
        const uint32_t word = w[c & 1][WPS * g + i];
        uint32_t* out = cells + 4 * (WPS * g + i);
        if (SMALL)
          dequant_word_natural_small_scale(word, b2, c2, out);
        else
          dequant_word_natural(word, s2, out);
      }
    }
    if (c == 0 && !ready()) return false;
    tmem_st_32x32b_x32(a_cells + 4 * WPT * c, cells);
  }
  return true;
}

// WPS: consecutive words of a thread that share one scale (2: group 16, 4:
// group 32, 8: larger ones).  x3d: X as one 3-D box per stage (K a multiple of
// 64), else one 2-D box per 64 k.  gridDim.y: CTAs (a cluster) that share an
// item along K.  ROWS: rows of a token tile, at most.
template <int WPS, int ROWS>
__global__ void __launch_bounds__(THREADS, 1)
    experts_decode_kernel(const __grid_constant__ CUtensorMap x_map,
                          const __grid_constant__ CUtensorMap qw_map,
                          const __grid_constant__ CUtensorMap s_map, const int32_t* offsets,
                          uint16_t* y, int R, int K, int N, int E, int group_shift, int stages,
                          int w_bytes, int x3d, int* err) {
  constexpr int ATOM_BYTES = ROWS * 128;     // X: 64-k atoms of ROWS 128-byte rows
  constexpr int X_BYTES = 4 * ATOM_BYTES;
  constexpr int XS = x_stages<ROWS>();
  using Table = ExpertTable<ROWS, ROWS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* w_ring = ring + XS * X_BYTES;
  Bars* bar = reinterpret_cast<Bars*>(w_ring + stages * w_bytes);
  volatile int* abort_flag = &bar->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gs = min(group_shift, 30);
  const int splits = gridDim.y;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * stages; ++s) mbar_init(&bar->wfull[s], 1);
    for (int s = 0; s < stages; ++s) mbar_init(&bar->wempty[s], 4);
    for (int s = 0; s < XS; ++s) {
      mbar_init(&bar->xfull[s], 1);
      mbar_init(&bar->xempty[s], 1);
    }
    for (int a = 0; a < SLOTS; ++a) mbar_init(&bar->afull[a], 4);
    for (int a = 0; a < 2 * SLOTS; ++a) mbar_init(&bar->aempty[a], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->dfull[i], 1);
      mbar_init(&bar->dempty[i], 4);
    }
    bar->abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&x_map);
    prefetch_tensormap(&qw_map);
    prefetch_tensormap(&s_map);
  }
  if (warp == 1) {
    tmem_alloc(&bar->tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  // the offsets and X may come from the previous kernel of the stream
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Table table;
  table.place(bar + 1, E);
  tc_fence_before();
  table.build(offsets, R, THREADS, err);  // ends with a barrier of the CTA
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;

  const int nblk = (N + BW - 1) / BW;
  const int items = table.tiles() * nblk;
  const int first = blockIdx.x, step = gridDim.x;
  const int n_items = first < items ? (items - first + step - 1) / step : 0;
  const int NS = (K + BK - 1) / BK;
  const int st0 = (int)((int64_t)blockIdx.y * NS / splits);  // this CTA's stages of an item
  const int n_st = (int)((int64_t)(blockIdx.y + 1) * NS / splits) - st0;

  if (warp == 0) {
    // ---------------- weight producer (converged; one elected lane issues) ----------------
    int issued = 0, s = 0, v = 0;  // ring stage, and which use of it
    bool ok = true;
    for (int j = 0; j < n_items && ok; ++j) {
      const int item = first + j * step;
      const int n0 = (item % nblk) * BW, e = table.find(item / nblk).e;
      for (int t = 0; t < n_st; ++t) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bar->wempty[s], (uint32_t)(v & 1) ^ 1u,
                                                       abort_flag, kWaitLimitNs));
        if (!ok) {
          if (lane == 0) record_timeout(err, bar);
          break;
        }
        if (elect_one()) {
          uint8_t* st = w_ring + s * w_bytes;
          uint64_t* full = &bar->wfull[s + stages * (v & 1)];
          const int k0 = (st0 + t) * BK;
          mbar_arrive_expect_tx(full, w_bytes);
          tma_load_3d(st, &qw_map, n0, k0 >> 3, e, full);
          tma_load_3d(st + QW_BYTES, &s_map, n0, k0 >> gs, e, full);
        }
        __syncwarp();
        ++issued;
        if (++s == stages) {
          s = 0;
          ++v;
        }
      }
    }
    if (*abort_flag) {
      // drain: wait (bounded) for the last load issued into each slot
      int never = 0;
      for (int i = issued - 1; i >= 0 && i >= issued - stages; --i)
        mbar_wait_bounded(&bar->wfull[i % (2 * stages)], (uint32_t)(i / (2 * stages)) & 1u,
                          &never, kDrainLimitNs);
    }
    // all copies are issued: the next kernel in the stream may start its
    // prologue (it waits for this grid before touching its inputs)
    if (lane == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncwarp();
  } else if (warp == X_WARP) {
    // ---------------- X producer (converged; one elected lane issues) ----------------
    int issued = 0, s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int j = 0; j < n_items && ok; ++j) {
      const int row0 = table.find((first + j * step) / nblk).row0;
      for (int t = 0; t < n_st; ++t) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bar->xempty[s], ph ^ 1u, abort_flag,
                                                       kWaitLimitNs));
        if (!ok) {
          if (lane == 0) record_timeout(err, bar);
          break;
        }
        if (elect_one()) {
          uint8_t* st = ring + s * X_BYTES;
          const int k0 = (st0 + t) * BK;
          // 64-k atoms of X that hold k below K (a 3-D box always fills four)
          const int atoms = x3d ? 4 : min(4, (K - k0 + 63) / 64);
          mbar_arrive_expect_tx(&bar->xfull[s], atoms * ATOM_BYTES);
          if (x3d) {
            tma_load_3d(st, &x_map, 0, row0, k0 >> 6, &bar->xfull[s]);
          } else {
            for (int a = 0; a < atoms; ++a)
              tma_load_2d(st + a * ATOM_BYTES, &x_map, k0 + 64 * a, row0, &bar->xfull[s]);
          }
        }
        __syncwarp();
        ++issued;
        if (++s == XS) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (*abort_flag) {
      int never = 0;
      for (int i = issued - 1; i >= 0 && i >= issued - XS; --i)
        mbar_wait_bounded(&bar->xfull[i % XS], (uint32_t)(i / XS) & 1u, &never, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer (one lane does it all) ----------------
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_f16_f32(BW, ROWS);
      bool ok = true;
      int s = 0, a = 0, use = 0;
      uint32_t xph = 0;
      for (int j = 0; j < n_items && ok; ++j) {
        const uint32_t d = tmem + D_COL + (uint32_t)(j & 1) * D_NEXT;
        if (j >= 2) {
          ok = mbar_wait_bounded(&bar->dempty[j & 1], (uint32_t)((j - 2) >> 1) & 1u, abort_flag,
                                 kWaitLimitNs);
          if (!ok) break;
        }
        for (int t = 0; t < n_st; ++t) {
          // both asked at once first: a wait costs 200 cycles even when there is
          // nothing to wait for
          const bool there = mbar_test_wait(smem_u32(&bar->xfull[s]), xph) &
                             mbar_test_wait(smem_u32(&bar->afull[a]), (uint32_t)use & 1u);
          if (!there)
            ok = mbar_wait_bounded(&bar->xfull[s], xph, abort_flag, kWaitLimitNs) &&
                 mbar_wait_bounded(&bar->afull[a], (uint32_t)use & 1u, abort_flag, kWaitLimitNs);
          if (!ok) break;
          tc_fence_after();
          const uint64_t x_desc = smem_desc_sw128(smem_u32(ring + s * X_BYTES));
          const uint32_t a_base = tmem + A_COL + a * A_SLOT_COLS;
          const int nk = min(BK, K - (st0 + t) * BK) / 16;  // k16 steps below K
          const uint32_t keep = t > 0 ? 1u : 0u;
          if (nk == BK / 16) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma_f16_ts(d, a_base + 8 * kk,
                         x_desc + (uint64_t)(((kk >> 2) * ATOM_BYTES + (kk & 3) * 32) >> 4),
                         idesc, kk > 0 ? 1u : keep);
          } else {
#pragma unroll 1
            for (int kk = 0; kk < nk; ++kk)
              mma_f16_ts(d, a_base + 8 * kk,
                         x_desc + (uint64_t)(((kk >> 2) * ATOM_BYTES + (kk & 3) * 32) >> 4),
                         idesc, kk > 0 ? 1u : keep);
          }
          mma_commit(&bar->aempty[a + SLOTS * (use & 1)]);
          mma_commit(&bar->xempty[s]);
          if (t == n_st - 1) mma_commit(&bar->dfull[j & 1]);
          if (++a == SLOTS) {
            a = 0;
            ++use;
          }
          if (++s == XS) {
            s = 0;
            xph ^= 1u;
          }
        }
      }
      if (!ok) {
        record_timeout(err, bar);
        // wait (bounded) for the MMAs already issued before TMEM is freed
        uint64_t* last = &bar->aempty[a + SLOTS * (use & 1)];
        mma_commit(last);
        int never = 0;
        mbar_wait_bounded(last, (uint32_t)(use >> 1) & 1u, &never, kDrainLimitNs);
      }
    }
    __syncwarp();
  } else if (warp < EPI_WARP0) {
    // ---------------- dequantisation ----------------
    const int grp = (warp - DQ_WARP0) >> 2;
    const int quarter = warp & 3;            // TMEM lanes 32*quarter .. +31
    const int col = 32 * quarter + lane;
    const uint32_t a_lane = tmem + ((uint32_t)(32 * quarter) << 16) + A_COL;
    const int total = n_items * n_st;
    int s = grp % stages, v = grp / stages;        // ring stage, and which use of it
    int a = grp % SLOTS, use = grp / SLOTS;  // A slot, and which use of it
    bool ok = true;
    for (int f = grp; f < total; f += GROUPS) {
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bar->wfull[s + stages * (v & 1)],
                                                     (uint32_t)(v >> 1) & 1u, abort_flag,
                                                     kWaitLimitNs));
      if (!ok) break;
      const uint8_t* qw = w_ring + s * w_bytes + col * 4;
      const uint8_t* sc = w_ring + s * w_bytes + QW_BYTES + col * 2;
      // the A slot is free once the MMAs of its previous use have completed
      const auto ready = [&]() -> bool {
        const bool free =
            __all_sync(0xffffffffu, mbar_wait_bounded(&bar->aempty[a + SLOTS * ((use - 1) & 1)],
                                                      (uint32_t)((use - 1) >> 1) & 1u, abort_flag,
                                                      kWaitLimitNs));
        tc_fence_after();
        return free;
      };
      // one form for the whole stage, so that its branch is the warp's
      bool small = WPS >= 4;
      if (WPS >= 4) {
#pragma unroll
        for (int g = 0; g < PR / WPS; ++g)
          small &= scale_fits_natural_form(*reinterpret_cast<const uint16_t*>(
              sc + ((8 * WPS * g) >> gs) * S_ROW_BYTES));  // every load in flight at once
        small = __all_sync(0xffffffffu, small);
      }
      const uint32_t a_cells = a_lane + a * A_SLOT_COLS;
      ok = small ? dequant_stage<WPS, true>(qw, sc, gs, a_cells, ready)
                 : dequant_stage<WPS, false>(qw, sc, gs, a_cells, ready);
      // qweight and scales of the stage are read (a lane's words were used
      // before it got here)
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->wempty[s]);
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->afull[a]);
      a += GROUPS % SLOTS;
      use += GROUPS / SLOTS;
      if (a >= SLOTS) {
        a -= SLOTS;
        ++use;
      }
      s += GROUPS;
      if (s >= stages) {
        s -= stages;
        ++v;
      }
    }
    if (!ok && lane == 0) record_timeout(err, bar);
    __syncwarp();
  } else {
    // ---------------- read-out ----------------
    const int quarter = warp & 3;
    const int col = 32 * quarter + lane;
    const uint32_t lane_addr = (uint32_t)(32 * quarter) << 16;
    float* part = reinterpret_cast<float*>(ring);  // [token][column], splits > 1
    for (int j = 0; j < n_items; ++j) {
      const int item = first + j * step;
      const ExpertTile tt = table.find(item / nblk);
      const int n = (item % nblk) * BW + col;
      if (!__all_sync(0xffffffffu,
                      mbar_wait_bounded<true>(&bar->dfull[j & 1], (uint32_t)(j >> 1) & 1u,
                                              abort_flag, kWaitLimitNs))) {
        if (lane == 0) record_timeout(err, bar);
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + lane_addr + D_COL + (uint32_t)(j & 1) * D_NEXT;
      uint16_t* out = y + (int64_t)tt.row0 * N + n;
      const int blocks = (tt.rows + 15) / 16;
#pragma unroll 1
      for (int tb = 0; tb < blocks; ++tb) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(d + 16 * tb, v);
        tmem_wait_ld();
        if (tb == blocks - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->dempty[j & 1]);  // it may be overwritten
        }
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const float acc = __uint_as_float(v[q]);
          const int tok = 16 * tb + q;
          if (splits > 1 && tok < tt.rows)
            part[tok * BW + col] = acc;
          else if (tok < tt.rows && n < N)
            out[(int64_t)tok * N] = __half_as_ushort(__float2half_rn(acc));
        }
      }
    }
    __syncwarp();
  }

  // Each CTA-wide barrier has a single call site reached by every thread.
  tc_fence_before();
  __syncthreads();
  if (splits > 1) {
    // one item per cluster: its CTAs add their ranges of K in rank order
    cluster_sync_all();
    if (first < items) {
      const ExpertTile tt = table.find(first / nblk);
      const int n0 = (first % nblk) * BW, rank = (int)cluster_ctarank();
      const int count = tt.rows * BW;
      const uint32_t base = smem_u32(ring);
      for (int i = rank * count / splits + (int)threadIdx.x; i < (rank + 1) * count / splits;
           i += THREADS) {
        const int tok = i / BW, c = i - tok * BW;
        if (n0 + c >= N) continue;
        float sum = 0.f;
        for (int r = 0; r < splits; ++r) sum += ld_dsmem_f32(map_to_rank(base + 4u * i, r));
        y[(int64_t)(tt.row0 + tok) * N + n0 + c] = __half_as_ushort(__float2half_rn(sum));
      }
    }
    cluster_sync_all();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int WPS, int ROWS>
cudaError_t launch_t(const CUtensorMap& x_map, const CUtensorMap& qw_map, const CUtensorMap& s_map,
                     const int32_t* offsets, uint16_t* y, int64_t R, int64_t K, int64_t N,
                     int64_t E, int group_shift, const Shape& d, int x3d, int64_t items,
                     int splits, cudaStream_t stream, const DeviceInfo& dev) {
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  const int di = dev.device & 63;
  std::call_once(once[di], [&] {
    attr_err[di] = cudaFuncSetAttribute(experts_decode_kernel<WPS, ROWS>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        1024 + kSmemLimit);
  });
  if (attr_err[di] != cudaSuccess) return attr_err[di];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(items, std::max(1, dev.num_sms / splits)),
                     (unsigned)splits, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = (size_t)d.smem_bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = (unsigned)splits;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, experts_decode_kernel<WPS, ROWS>, x_map, qw_map, s_map, offsets,
                            y, (int)R, (int)K, (int)N, (int)E, group_shift, d.w_stages,
                            d.w_bytes, x3d, dev.error_word);
}

// CTAs that share an item along K: as many as the SMs hold when every item is
// there, each with two stages at least (a shorter range does not pay for the
// reduction).
int pick_splits(int64_t items, int64_t K, const DeviceInfo& dev) {
  const int64_t stages = (K + BK - 1) / BK;
  int64_t s = std::min<int64_t>(8, dev.num_sms / items);
  s = std::min(s, stages / 2);
  return s < 1 ? 1 : (int)s;
}

template <int ROWS>
cudaError_t launch_rows(const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                      const int32_t* offsets, uint16_t* y, int64_t R, int64_t K, int64_t N,
                      int64_t E, int group_shift, cudaStream_t stream, const DeviceInfo& dev) {
  const Shape d = shape_of<ROWS>(group_shift, (int)E);
  if (d.w_stages < GROUPS) return cudaErrorInvalidValue;
  const int64_t n_groups = (group_shift == 62 || (int64_t(1) << group_shift) >= K)
                               ? 1 : (K + (int64_t(1) << group_shift) - 1) >> group_shift;
  CUtensorMap x_map, qw_map, s_map;
  const int x3d = K % 64 == 0;
  const uint64_t dims[3] = {64, (uint64_t)R, (uint64_t)(K / 64)};
  const uint64_t strides[2] = {(uint64_t)K * 2, 128};
  const uint32_t box[3] = {64, ROWS, BK / 64};
  if (!(x3d ? encode_map_3d(&x_map, x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dims, strides, box,
                            CU_TENSOR_MAP_SWIZZLE_128B)
            : encode_map_2d(&x_map, x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (uint64_t)K, (uint64_t)R,
                            (uint64_t)K * 2, 64, ROWS, CU_TENSOR_MAP_SWIZZLE_128B)))
    return cudaErrorInvalidValue;
  const uint64_t qdims[3] = {(uint64_t)N, (uint64_t)(K / 8), (uint64_t)E};
  const uint64_t qstrides[2] = {(uint64_t)N * 4, (uint64_t)(K / 8) * N * 4};
  const uint32_t qbox[3] = {BW, PR, 1};
  const uint64_t sdims[3] = {(uint64_t)N, (uint64_t)n_groups, (uint64_t)E};
  const uint64_t sstrides[2] = {(uint64_t)N * 2, (uint64_t)n_groups * N * 2};
  const uint32_t sbox[3] = {BW, (uint32_t)d.scale_rows, 1};
  if (!encode_map_3d(&qw_map, qweight, CU_TENSOR_MAP_DATA_TYPE_INT32, qdims, qstrides, qbox,
                     CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !encode_map_3d(&s_map, scales, CU_TENSOR_MAP_DATA_TYPE_UINT16, sdims, sstrides, sbox,
                     CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  // the most items there can be: a tile per row, or one per expert and one
  // more for every ROWS rows beyond that
  const int64_t tiles = std::min<int64_t>(R, E + R / ROWS);
  const int64_t items = tiles * ((N + BW - 1) / BW);
  const int splits = pick_splits(items, K, dev);
  const auto launch = group_shift == 4   ? launch_t<2, ROWS>
                      : group_shift == 5 ? launch_t<4, ROWS>
                                         : launch_t<WPT, ROWS>;
  return launch(x_map, qw_map, s_map, offsets, y, R, K, N, E, group_shift, d, x3d, items, splits,
                stream, dev);
}

}  // namespace

cudaError_t launch_experts_decode(const uint16_t* x, const int32_t* qweight,
                                  const uint16_t* scales, const int32_t* offsets, uint16_t* y,
                                  int64_t R, int64_t K, int64_t N, int64_t E, int group_shift,
                                  int tile, cudaStream_t stream, const DeviceInfo& dev) {
  const auto launch = tile <= 16 ? launch_rows<16> : launch_rows<32>;
  return launch(x, qweight, scales, offsets, y, R, K, N, E, group_shift, stream, dev);
}

}  // namespace gptq
