// The experts' products on CTA pairs: for every expert e and its rows
//   Y[rows of e] = X[rows of e] . dequant(qweight[e], scales[e])
// and the gradient with respect to the rows,
//   dX[rows of e] = dY[rows of e] . dequant(qweight[e], scales[e])^T,
// with tcgen05.mma.cta_group::2.
//
// The transposed product of the pair prefill kernel (256 output columns per
// CTA pair as the MMA's M, dequantised into TMEM; tokens as its N, half of the
// token tile loaded by each CTA; persistent clusters walking the tiles), with
// the token tiles cut from the experts' rows:
//
// * The experts' row counts are known on the device only.  Every CTA builds
//   the same table of token tiles from the offsets (experts.cuh) and cluster c
//   takes tiles c, c + clusters, ..., column pair fastest.
// * A tile holds up to BT = 128 or 256 rows of one expert; the MMA's width is
//   the rows rounded up to 32, so an expert with few rows pays for those only.
//   The copy box of X has half as many rows per CTA (a tensor map for each
//   width), so that a tile reads no more of X from L2 than it multiplies: with
//   128 rows per expert all column pairs together read 9.7 TB/s.  Rows that a
//   box reads past the tile belong to other experts (or read as zero past the
//   tensor): each is a column of the accumulator of its own, which is never
//   stored.
// * Four warps of their own read a finished accumulator out.  Tiles of up to
//   128 rows alternate between the two halves of the accumulator columns, so
//   the next tile's MMAs run meanwhile: with few rows per expert a tile takes
//   a few microseconds, and waiting for its read-out took a fifth of them.
// * Stores: 32-row blocks wholly inside the tile go through TMA, the others
//   as 16-byte rows, so that no other expert's row is written.
//
// In the gradient the roles of K and N are exchanged: the pair's 256 columns
// are k, the contraction runs over n.  The weight tile of a stage is the same
// box of 16 packed rows x 128 columns, but a TMEM lane is now one k.  A thread
// takes half a packed word (four k) of four neighbouring columns at a time:
// one byte permute collects a byte of two columns' words, whose two nibbles
// are two k of that column pair.  Stored in the 16-lane, 256-bit form of
// tcgen05.st, a thread's four k lie in TMEM lanes r, r + 8, r + 16 and r + 24
// of its quarter.  (With a lane per thread, every word was read by eight
// threads and shared memory bound the kernel.)
//
// So TMEM lane l of a quarter holds output column 4 (l mod 8) + l / 8 (the
// forward dequantisation reads its words accordingly), and the 16-lane form of
// tcgen05.ld hands a thread four neighbouring columns of a token: the read-out
// packs and stores them eight bytes at a time.
//
// Every wait is bounded in time; on expiry the CTA records GPTQ_ERR_TIMEOUT
// in the device error word and winds down.  Both CTAs always reach the final
// cluster barrier, so neither leaves while the other may still signal it.

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

constexpr int BW = 128;   // output columns per CTA (TMEM lanes); 256 per pair (MMA M)
constexpr int BK = 128;   // contraction per A slot (eight k16 MMAs)
constexpr int XS = 3;     // X ring stages
constexpr int WS_MAX = 8;  // weight-tile ring stages (qweight + scales), at most
constexpr int AS = 4;     // A slots in TMEM (BK each)
constexpr int FS = 4;     // barriers of ready stages
constexpr int DQ_GROUPS = 4;             // dequantisation groups: group g takes slots' worth g mod 4
constexpr int DQ_WARPS = 4 * DQ_GROUPS;  // one warp per TMEM lane quarter in each group
// Warps: dequantisation from 0, four for the read-out, the producers, the MMA
// issuer.  In that order: beside warps of arithmetic alone, a warp behind them
// got to issue twice as often as one before them (a loop of 16 MMAs and their
// commits took 1860 cycles there, 4230 as warp 0).  Here that gives 1 % with 32
// rows per expert (42.3 -> 41.8 us, 64 experts of 2048 x 2048).
constexpr int EPI_WARP0 = DQ_WARPS;
constexpr int X_WARP = EPI_WARP0 + 4, W_WARP = X_WARP + 1, MMA_WARP = W_WARP + 1;
constexpr int THREADS = (MMA_WARP + 1) * 32;
constexpr int S_ROW_BYTES = BW * 2;                // a scale row of 128 columns: 256 B
constexpr int X_STAGE_BYTES = 32 * 1024;           // 128 rows x 128 or 64 rows x 256 columns
constexpr int W_RING_BYTES = 80 * 1024;
constexpr int Y_ROWS = 32;                         // tokens per store block
constexpr int Y_BLOCK_BYTES = Y_ROWS * 32 * 2;     // ... of a read-out warp's 32 columns
constexpr int Y_BLOCKS = 2;                        // per read-out warp, in turn
constexpr int W_OFF = XS * X_STAGE_BYTES;
constexpr int Y_OFF = W_OFF + W_RING_BYTES;
constexpr int BAR_OFF = Y_OFF + 4 * Y_BLOCKS * Y_BLOCK_BYTES;
constexpr int LIST_OFF = BAR_OFF + 512;
constexpr int TABLE_OFF = LIST_OFF + 256 * 16;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t D_COL = 0;              // accumulators: columns [0, 256)
constexpr uint32_t D_HALF = 128;           // ... tiles of up to 128 rows alternate
constexpr uint32_t A_COL = 256;            // A slots: [256, 256 + 4 * 64)
constexpr uint32_t A_STAGE_COLS = BK / 2;  // two FP16 per 32-bit column
constexpr uint16_t kPairMask = 0x3;        // both CTAs of the cluster
constexpr uint64_t kWaitLimitNs = 4000000000ull;
constexpr uint64_t kDrainLimitNs = 200000000ull;
static_assert(A_COL + AS * A_STAGE_COLS <= TMEM_COLS, "TMEM budget");
static_assert(AS == DQ_GROUPS, "A slot j is written by group j");

// A ring stage holds KST of the contraction: 128 with tiles of 256 tokens, 256
// (two A slots' worth) with smaller ones, whose MMAs are so short that the
// producers' and the MMA warp's work per stage sets the pace.
template <int BT>
struct Geo {
  using Table = ExpertTable<BT, 32>;
  static constexpr int KST = BT <= 128 ? 256 : 128;
  static constexpr int H = KST / BK;                 // A slots per stage
  static constexpr int ATOMS = KST / 64;             // 64-column atoms of X per stage
  static constexpr int QW_BYTES = BW * (KST / 8) * 4;
  // scale rows of 16 k each at most (group 16)
  static constexpr int W_STAGE_BYTES = QW_BYTES + KST / 16 * S_ROW_BYTES;
  static constexpr int WS = W_RING_BYTES / W_STAGE_BYTES;
  static_assert(BT / 2 * KST * 2 == X_STAGE_BYTES, "an X stage");
  static_assert(WS == 8 / H && WS <= WS_MAX, "weight stage f / H mod WS comes round to group j");
};
static_assert(1024 + TABLE_OFF + ExpertTable<256, 32>::bytes(GPTQ_MOE_MAX_EXPERTS) <= 227 * 1024,
              "shared memory per CTA");

// Both CTAs hold the full set; full and dempty are only used in the even CTA.
// dfull and dempty of tile i: entry i mod 2.
struct PairBarriers {
  // Stage f is ready, entry f mod 4: both halves of X landed, and the group
  // warps of both CTAs wrote its A slots: one barrier for the MMA lane to ask.
  // (Nobody signals stage f before stage f - 4 is done: X waits for
  // f - 3, an A slot for its last use, two or four stages before.)
  uint64_t full[FS];
  uint64_t xempty[XS];  // pair MMAs reading the X stage done
  uint64_t wfull[WS_MAX];   // this CTA's qweight and scale tiles landed
  uint64_t wempty[WS_MAX];  // weight tiles read by this CTA's group warps
  uint64_t aempty[AS];  // pair MMAs reading the A slot done
  uint64_t dfull[2];    // all MMAs of the tile done
  uint64_t dempty[2];   // accumulator read out by both CTAs' read-out warps (even CTA)
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(PairBarriers) <= 512, "barrier area");

// X in boxes of 16, 32, ... rows per CTA: half of each MMA width.
template <int BT>
struct XMaps {
  CUtensorMap width[BT / 32];
};

// The tiles of one cluster: tile = cluster + i * clusters for i = 0, 1, ...;
// column pair fastest.  The first LISTED are looked up once, all threads at a
// time, and kept in shared memory: a search of the table takes over 500 cycles,
// in the MMA warp as long as two of a small tile's stages.
constexpr int LISTED = (TABLE_OFF - LIST_OFF) / 16;
struct ListedTile {
  int e, row0, rows_n, o0;  // rows | n << 16; first column of the pair
};
static_assert(sizeof(ListedTile) == 16, "one 16-byte load");

template <class Table>
struct Walk {
  int cluster, clusters, n_pairs, tiles;
  Table table;
  ListedTile* list;
  __device__ int count() const {
    return cluster < tiles ? (tiles - cluster + clusters - 1) / clusters : 0;
  }
  __device__ ExpertTile find(int i, int& o0) const {
    const int tile = cluster + i * clusters;
    o0 = 2 * (tile % n_pairs) * BW;
    return table.find(tile / n_pairs);
  }
  // Called by every thread of the CTA (`threads` of them); a barrier must
  // follow.
  __device__ void fill(int threads) {
    const int n = min(count(), LISTED);
    for (int i = threadIdx.x; i < n; i += threads) {
      int o0;
      const ExpertTile t = find(i, o0);
      list[i] = ListedTile{t.e, t.row0, t.rows | t.n << 16, o0};
    }
  }
  // This CTA's first output column in tile i, and the token tile.
  __device__ ExpertTile at(int i, uint32_t rank, int& o0) const {
    ExpertTile t;
    if (i < LISTED) {
      const int4 v = *reinterpret_cast<const int4*>(list + i);
      t = ExpertTile{v.x, v.y, v.z & 0xFFFF, v.z >> 16};
      o0 = v.w;
    } else {
      t = find(i, o0);
    }
    o0 += (int)rank * BW;
    return t;
  }
};

// C: the contraction length (K, or N in the gradient); O: the output width
// (N, or K in the gradient).  scale_bytes: scales of a stage.
// x3d: X is read through a [C/64][R][64] view, one copy per stage (C a
// multiple of 64); otherwise through [R][C], one copy per 64-column atom.
// WPS: consecutive packed words of a column that share one scale (2, 4, 8 or,
// for groups of 128 and more, 16; not used in the gradient).
template <bool DX, int BT, int WPS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    experts_pair_kernel(const __grid_constant__ XMaps<BT> x_maps,
                        const __grid_constant__ CUtensorMap qw_map,
                        const __grid_constant__ CUtensorMap s_map,
                        const __grid_constant__ CUtensorMap y_map, const int32_t* offsets, int R,
                        int C, int O, int E, int group_shift, int scale_bytes, int x3d,
                        int n_pairs, uint16_t* y, int* err) {
  using G_ = Geo<BT>;
  constexpr int KST = G_::KST, H = G_::H, WS = G_::WS;
  constexpr int QW_BYTES = G_::QW_BYTES, W_STAGE_BYTES = G_::W_STAGE_BYTES;
  constexpr int QW_ROW_BYTES = (DX ? KST : BW) * 4;  // a packed row of the weight tile
  constexpr int SC_ROW_BYTES = (DX ? KST : BW) * 2;
  extern __shared__ uint8_t smem_raw[];
  // 1024-byte aligned base; the same offset in both CTAs, so that one MMA
  // descriptor and one barrier offset name the matching buffers of the pair
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* xs = smem;
  PairBarriers* bar = reinterpret_cast<PairBarriers*>(smem + BAR_OFF);
  volatile int* abort_flag = &bar->abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: even CTA (issues the MMAs), 1: odd CTA
  const bool even = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < XS; ++s) {
      mbar_init(&bar->xempty[s], 1);  // one pair commit
    }
    for (int j = 0; j < WS; ++j) {
      mbar_init(&bar->wfull[j], 1);
      mbar_init(&bar->wempty[j], 4 * H);  // the four warps of each of its groups
    }
    for (int j = 0; j < AS; ++j) {
      mbar_init(&bar->aempty[j], 1);      // one pair commit
    }
    // the even CTA's expect_tx (bytes from both CTAs), and the group warps of
    // the stage's slots in both
    for (int f = 0; f < FS; ++f) mbar_init(&bar->full[f], 1 + 2 * 4 * H);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->dfull[i], 1);       // one pair commit per tile
      mbar_init(&bar->dempty[i], 2 * 4);  // the read-out warps of both CTAs
    }
    bar->abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == X_WARP && lane == 0) {
    for (int i = 0; i < BT / 32; ++i) prefetch_tensormap(&x_maps.width[i]);
    prefetch_tensormap(&qw_map);
    prefetch_tensormap(&s_map);
    prefetch_tensormap(&y_map);
  }
  __syncwarp();
  if (warp == MMA_WARP) {
    tmem_alloc_pair(&bar->tmem_base, TMEM_COLS);
    tmem_relinquish_pair();
  }
  // both CTAs' barriers are initialised and TMEM is allocated before any thread
  // signals the other CTA: this one says so now, and asks for the other's word
  // once its table is built
  tc_fence_before();
  cluster_arrive();
  // the offsets and X may come from the previous kernel of the stream
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Walk<typename G_::Table> walk;
  walk.cluster = (int)(blockIdx.x >> 1);
  walk.clusters = (int)(gridDim.x >> 1);
  walk.n_pairs = n_pairs;
  walk.table.place(smem + TABLE_OFF, E);
  walk.table.build(offsets, R, THREADS, err);
  walk.tiles = walk.table.tiles() * n_pairs;
  walk.list = reinterpret_cast<ListedTile*>(smem + LIST_OFF);
  walk.fill(THREADS);
  const int NT = walk.count();          // tiles of this cluster
  const int KB = (C + KST - 1) / KST;   // stages per tile
  const int G = NT * KB;                // stages of this cluster, over all its tiles
  __syncthreads();  // the list is complete
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  // the even CTA's barriers that both CTAs signal
  const uint32_t full_even = map_to_rank(smem_u32(&bar->full[0]), 0);
  const uint32_t dempty_even = map_to_rank(smem_u32(&bar->dempty[0]), 0);

  if (warp == X_WARP || warp == W_WARP) {
    // ---------------- TMA producers: X half, weights ----------------
    // Converged warps; one elected lane issues.
    int kb = 0, it = 0, o0 = 0, s = 0, issued = 0;
    uint32_t ph = 0;
    ExpertTile tt{0, 0, 0, 32};
    if (NT > 0) tt = walk.at(0, rank, o0);
    bool ok = true;
    uint64_t* const empty = warp == X_WARP ? bar->xempty : bar->wempty;
    const int ring = warp == X_WARP ? XS : WS;
    for (int g = 0; g < G; ++g) {
      ok = __all_sync(0xffffffffu,
                      mbar_wait_bounded(&empty[s], ph ^ 1u, abort_flag, kWaitLimitNs));
      if (!ok) {
        if (lane == 0) record_timeout(err, bar);
        break;
      }
      const int c0 = kb * KST;
      if (warp == X_WARP) {
        // The odd CTA's half of the token tile may lie wholly past the last
        // row of X: then it loads nothing and the even CTA expects only its
        // own bytes; the MMA reads stale shared memory for token columns that
        // are never stored.
        const int row = tt.row0 + (int)rank * (tt.n / 2);
        const CUtensorMap* x_map = &x_maps.width[tt.n / 32 - 1];
        const bool odd_rows = tt.row0 + tt.n / 2 < R;
        if (elect_one()) {
          uint8_t* dst = xs + s * X_STAGE_BYTES;
          const uint32_t bar_c = full_even + 8u * (uint32_t)(g % FS);
          const uint32_t atom_bytes = tt.n / 2 * 128;
          // atoms that hold columns below C (a 3-D box always fills all)
          const int atoms = x3d ? G_::ATOMS : min(G_::ATOMS, (C - c0 + 63) / 64);
          if (even)
            mbar_arrive_expect_tx(&bar->full[g % FS], (odd_rows ? 2u : 1u) * atoms * atom_bytes);
          if (even || odd_rows) {
            if (x3d) {
              tma_load_3d_pair(dst, x_map, 0, row, c0 / 64, bar_c);
            } else {
              for (int a = 0; a < atoms; ++a)
                tma_load_2d_pair(dst + a * atom_bytes, x_map, c0 + 64 * a, row, bar_c);
            }
          }
        }
      } else if (elect_one()) {
        uint8_t* wst = smem + W_OFF + s * W_STAGE_BYTES;
        if (o0 < O) {
          // first column and first k of the stage's weight tile
          const int n0 = DX ? c0 : o0, k0 = DX ? o0 : c0;
          mbar_arrive_expect_tx(&bar->wfull[s], QW_BYTES + scale_bytes);
          tma_load_3d(wst, &qw_map, n0, k0 / 8, tt.e, &bar->wfull[s]);
          tma_load_3d(wst + QW_BYTES, &s_map, n0, (int)((int64_t)k0 >> group_shift), tt.e,
                      &bar->wfull[s]);
        } else {
          mbar_arrive(&bar->wfull[s]);  // padding CTA: no columns, nothing to load
        }
      }
      __syncwarp();
      ++issued;
      if (++s == ring) {
        s = 0;
        ph ^= 1u;
      }
      if (++kb == KB) {
        kb = 0;
        if (++it < NT) tt = walk.at(it, rank, o0);
      }
    }
    if (*abort_flag && (even || warp == W_WARP)) {
      // drain: wait for the last loads issued into each slot (the odd CTA's X
      // loads complete on the even CTA's barriers, which the even CTA drains;
      // where a stage's A slots are never written, the limit is that wait)
      int never = 0;
      uint64_t* const full = warp == X_WARP ? bar->full : bar->wfull;
      const int entries = warp == X_WARP ? FS : ring;
      for (int i = issued - 1; i >= 0 && i >= issued - ring; --i)
        mbar_wait_bounded(&full[i % entries], (uint32_t)(i / entries) & 1u, &never,
                          kDrainLimitNs);
    }
    // all copies are issued: the next kernel in the stream may start its
    // prologue (it waits for this grid before touching its inputs)
    if (warp == W_WARP && lane == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncwarp();  // the whole warp reaches the cluster barrier below together
  } else if (warp == MMA_WARP) {
    // ---------------- pair MMA issuer (even CTA; one lane does it all) ----------------
    if (even && elect_one()) {
      bool ok = true;
      int it = 0, f = 0, s = 0, a = 0, last_n = 0;  // tile; stage, its X stage and A slot
      for (; it < NT && ok; ++it) {
        int o0;
        const int n = walk.at(it, rank, o0).n;
        const uint32_t idesc = idesc_f16_f32(2 * BW, n);
        const uint32_t atom_bytes = n / 2 * 128;
        const uint32_t d = tmem + D_COL + (n <= (int)D_HALF ? (it & 1) * D_HALF : 0u);
        // the tile before the last has been read out; the last one too, where
        // the two share accumulator columns
        if (it > 1)
          ok = mbar_wait_bounded(&bar->dempty[it & 1], (uint32_t)((it - 2) >> 1) & 1u, abort_flag,
                                 kWaitLimitNs);
        if (ok && it > 0 && max(n, last_n) > (int)D_HALF)
          ok = mbar_wait_bounded(&bar->dempty[(it - 1) & 1], (uint32_t)((it - 1) >> 1) & 1u,
                                 abort_flag, kWaitLimitNs);
        if (!ok) break;
        tc_fence_after();
        last_n = n;
        for (int kb = 0; kb < KB; ++kb) {
          // the stage's A slots: a, and with two per stage a + 1 (a is even then)
          ok = mbar_wait_bounded(&bar->full[f % FS], (uint32_t)(f / FS) & 1u, abort_flag,
                                 kWaitLimitNs);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const uint64_t b_lo = smem_desc_sw128(smem_u32(xs + s * X_STAGE_BYTES)) +
                                  (uint64_t)((2 * h * atom_bytes) >> 4);
            const uint64_t b_hi = b_lo + (uint64_t)(atom_bytes >> 4);
            const uint32_t a_base = tmem + A_COL + (a + h) * A_STAGE_COLS;
            // k16 steps that hold columns below C
            const int nk = min(BK, C - kb * KST - h * BK + 15) / 16;
            const uint32_t keep = kb > 0 || h > 0 ? 1u : 0u;
            if (nk == BK / 16) {
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)
                mma_f16_ts_pair(d, a_base + kk * 8,
                                (kk < 4 ? b_lo : b_hi) + (uint64_t)(((kk & 3) * 32) >> 4), idesc,
                                kk > 0 ? 1u : keep);
            } else {
#pragma unroll 1
              for (int kk = 0; kk < nk; ++kk)
                mma_f16_ts_pair(d, a_base + kk * 8,
                                (kk < 4 ? b_lo : b_hi) + (uint64_t)(((kk & 3) * 32) >> 4), idesc,
                                kk > 0 ? 1u : keep);
            }
            mma_commit_pair(&bar->aempty[a + h], kPairMask);
          }
          mma_commit_pair(&bar->xempty[s], kPairMask);
          if (kb == KB - 1) mma_commit_pair(&bar->dfull[it & 1], kPairMask);  // tile done
          ++f;
          if (++s == XS) s = 0;
          a = (a + H) % AS;
        }
      }
      if (!ok) {
        record_timeout(err, bar);
        // wait for the MMAs already issued before anyone frees TMEM
        mma_commit_pair(&bar->aempty[a + H - 1], kPairMask);
        int never = 0;
        mbar_wait_bounded(&bar->aempty[a + H - 1], (uint32_t)(f * H / AS) & 1u, &never,
                          kDrainLimitNs);
      }
    }
    __syncwarp();  // the whole warp reaches the cluster barrier below together
  } else if (warp < EPI_WARP0) {
    // ---------------- dequantisation ----------------
    const int quarter = warp & 3;            // TMEM lanes 32*quarter .. +31
    const int j = warp >> 2;    // group: slots' worth f = j mod 4, A slot j
    const uint32_t a_slot =
        tmem + ((uint32_t)(32 * quarter) << 16) + A_COL + j * A_STAGE_COLS;
    // forward: this thread's column in weight slot 0; gradient: its packed
    // row, its four columns of every sixteen, and its half of their words
    const int col = 32 * quarter + 4 * (lane & 7) + (lane >> 3);
    const int prow = 4 * quarter + (lane >> 3);
    // ... in its half of a stage
    const int hf = j % H;
    const uint8_t* qw0 = smem + W_OFF +
                         (DX ? prow * QW_ROW_BYTES + (BK * hf + 4 * (lane & 3)) * 4
                             : BK / 8 * hf * QW_ROW_BYTES + col * 4);
    const int gs = min(group_shift, 30);
    const uint8_t* sc0 =
        smem + W_OFF + QW_BYTES +
        (DX ? (gs >= 7 ? 0 : (prow * 8) >> gs) * SC_ROW_BYTES + (BK * hf + 4 * (lane & 3)) * 2
            : ((BK * hf) >> gs) * SC_ROW_BYTES + col * 2);
    const uint32_t half = (uint32_t)(lane >> 2) & 1u;  // k 0..3 or 4..7 of the words
    const uint32_t pick_lo = half ? 0x6622u : 0x4400u;  // first byte of two words' halves
    const uint32_t pick_hi = half ? 0x7733u : 0x5511u;  // second byte

    bool ok = true;
    int jw = j / H, f = j / H;   // weight stage's slot, the stage
    uint32_t pw = 0, ph = 0;     // phases of the weight slot and the A slot
    for (int g = j; g < G * H; g += DQ_GROUPS) {
      const uint8_t* qw = qw0 + jw * W_STAGE_BYTES;
      const uint8_t* sc = sc0 + jw * W_STAGE_BYTES;
      // qweight and scale tiles of the stage have landed
      ok = __all_sync(0xffffffffu,
                      mbar_wait_bounded<true>(&bar->wfull[jw], pw, abort_flag, kWaitLimitNs));
      if (!ok) break;
      bool small = false;  // one form for the whole stage, so that its branch is the warp's
      if constexpr (!DX) {
        small = true;
#pragma unroll
        for (int r = 0; r < BK / 8; r += WPS)
          small &= scale_fits_natural_form(*reinterpret_cast<const uint16_t*>(
              sc + r / WPS * SC_ROW_BYTES));  // every load in flight at once
        small = __all_sync(0xffffffffu, small);
      }
      // the stage's 128 k (or n), one half (32 TMEM columns) at a time
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t cells[32];
        if constexpr (DX) {
          // cells 0..15: k 0 and 1 of the thread's half words, 16..31: k 2 and 3
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // sixteen columns n, four of them this thread's
            const uint4 w = *reinterpret_cast<const uint4*>(qw + (64 * h + 16 * i) * 4);
            const uint2 s4 = *reinterpret_cast<const uint2*>(sc + (64 * h + 16 * i) * 2);
            const uint32_t lo[2] = {prmt(w.x, w.y, pick_lo), prmt(w.z, w.w, pick_lo)};
            const uint32_t hi[2] = {prmt(w.x, w.y, pick_hi), prmt(w.z, w.w, pick_hi)};
            const uint32_t s2[2] = {s4.x, s4.y};
#pragma unroll
            for (int q = 0; q < 2; ++q) {  // column pairs: q - 8 exactly, then one rounding
              cells[4 * i + q] = hmul2_rn(
                  hsub2_rn(lop3_and_or(lo[q], 0x000F000Fu, kMagic1024), kMinus1032), s2[q]);
              cells[4 * i + 2 + q] =
                  hmul2_rn(hfma2_rn(lop3_and_or(lo[q], 0x00F000F0u, kMagic1024), kOneSixteenth,
                                    kMinus72), s2[q]);
              cells[16 + 4 * i + q] = hmul2_rn(
                  hsub2_rn(lop3_and_or(hi[q], 0x000F000Fu, kMagic1024), kMinus1032), s2[q]);
              cells[16 + 4 * i + 2 + q] =
                  hmul2_rn(hfma2_rn(lop3_and_or(hi[q], 0x00F000F0u, kMagic1024), kOneSixteenth,
                                    kMinus72), s2[q]);
            }
          }
        } else {
          uint32_t w[8];
#pragma unroll
          for (int r = 0; r < 8; ++r)
            w[r] = *reinterpret_cast<const uint32_t*>(qw + (8 * h + r) * QW_ROW_BYTES);
          constexpr int PER = WPS < 8 ? WPS : 8;  // words of this half that share a scale
#pragma unroll
          for (int r0 = 0; r0 < 8; r0 += PER) {
            const uint32_t s2 = half2_broadcast(*reinterpret_cast<const uint16_t*>(
                sc + (8 * h + r0) / WPS * SC_ROW_BYTES));
            if (small) {
              uint32_t b2, c2;
              natural_form_constants(s2, b2, c2);
#pragma unroll
              for (int r = r0; r < r0 + PER; ++r)
                dequant_word_natural_small_scale(w[r], b2, c2, cells + 4 * r);
            } else {
#pragma unroll
              for (int r = r0; r < r0 + PER; ++r) dequant_word_natural(w[r], s2, cells + 4 * r);
            }
          }
        }
        if (h == 0) {
          // the A slot is free once the pair MMAs of its previous use completed
          ok = __all_sync(0xffffffffu, mbar_wait_bounded<true>(&bar->aempty[j], ph ^ 1u,
                                                               abort_flag, kWaitLimitNs));
          if (!ok) break;
          tc_fence_after();
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->wempty[jw]);  // weight tiles of the stage read
        }
        if constexpr (DX) {
          tmem_st_16x256b_x4(a_slot + 32 * h, cells);
          tmem_st_16x256b_x4(a_slot + (16u << 16) + 32 * h, cells + 16);
        } else {
          tmem_st_32x32b_x32(a_slot + 32 * h, cells);
        }
      }
      if (!ok) break;
      tmem_wait_st();  // the whole warp's cells are in TMEM
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(full_even + 8u * (uint32_t)(f % FS));
      f += DQ_GROUPS / H;
      ph ^= 1u;
      jw += DQ_GROUPS / H;
      if (jw >= WS) {
        jw -= WS;
        pw ^= 1u;
      }
    }
    if (!ok && lane == 0) record_timeout(err, bar);
    __syncwarp();
  } else {
    // ---------------- accumulator read-out ----------------
    const int quarter = warp & 3;
    const uint32_t lane_addr = (uint32_t)(32 * quarter) << 16;
    uint8_t* ystage = smem + Y_OFF + (warp - EPI_WARP0) * Y_BLOCKS * Y_BLOCK_BYTES;
    // of every eight tokens this thread reads 2 (lane mod 4) and the next, four
    // columns each; the block's 64-byte rows have the 64-byte swizzle
    const int tok0 = 2 * (lane & 3);
    const uint32_t ybyte = (uint32_t)(lane & 4) << 1;  // which half of a 16-byte chunk
    const uint32_t ychunk = (uint32_t)lane >> 3;
    int blk = 0;
    for (int it = 0; it < NT; ++it) {
      int o0;
      const ExpertTile tt = walk.at(it, rank, o0);
      const int c0 = o0 + 32 * quarter;
      if (!__all_sync(0xffffffffu,
                      mbar_wait_bounded<true>(&bar->dfull[it & 1], (uint32_t)(it >> 1) & 1u,
                                              abort_flag, kWaitLimitNs))) {
        if (lane == 0) record_timeout(err, bar);
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + lane_addr + D_COL + (tt.n <= (int)D_HALF ? (it & 1) * D_HALF : 0u);
      const int blocks = c0 < O ? (tt.rows + Y_ROWS - 1) / Y_ROWS : 0;
#pragma unroll 1
      for (int b = 0; b < blocks; ++b) {
        uint32_t va[16], vb[16];  // the thread's columns 0 and 1, 2 and 3
        tmem_ld_16x256b_x4(d + Y_ROWS * b, va);
        tmem_ld_16x256b_x4(d + (16u << 16) + Y_ROWS * b, vb);
        // the store that used this block last has read it: all but the latest
        if (lane == 0) bulk_wait_read_but_one();
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && b == blocks - 1)  // all read: the MMAs may overwrite it
          mbar_arrive_cluster(dempty_even + 8u * (uint32_t)(it & 1));
        uint8_t* yb = ystage + blk * Y_BLOCK_BYTES;
        blk ^= 1;
#pragma unroll
        for (int g = 0; g < Y_ROWS / 8; ++g) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int tok = 8 * g + tok0 + t;
            const __half2 lo = __floats2half2_rn(__uint_as_float(va[4 * g + t]),
                                                 __uint_as_float(va[4 * g + 2 + t]));
            const __half2 hi = __floats2half2_rn(__uint_as_float(vb[4 * g + t]),
                                                 __uint_as_float(vb[4 * g + 2 + t]));
            *reinterpret_cast<uint2*>(yb + tok * 64 + ((ychunk ^ ((tok >> 1) & 3)) << 4) + ybyte) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                           *reinterpret_cast<const uint32_t*>(&hi));
          }
        }
        const int row = tt.row0 + Y_ROWS * b, live = min(Y_ROWS, tt.rows - Y_ROWS * b);
        if (live == Y_ROWS) {
          fence_proxy_async_smem();  // the staging writes are visible to the store
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&y_map, yb, c0, row);
            bulk_commit_group();
          }
        } else {
          // the tile ends inside the block: its rows only, 16 bytes at a time
          __syncwarp();
          for (int i = lane; i < 4 * live; i += 32) {
            const int c = c0 + 8 * (i & 3);
            if (c < O)
              *reinterpret_cast<uint4*>(y + (int64_t)(row + (i >> 2)) * O + c) =
                  *reinterpret_cast<const uint4*>(yb + (i >> 2) * 64 +
                                                  (((i & 3) ^ ((i >> 3) & 3)) << 4));
          }
          // (an empty group keeps the count of groups and blocks in step)
          if (lane == 0) bulk_commit_group();
          __syncwarp();
        }
      }
      if (blocks == 0) {  // none of the warp's columns exist
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(dempty_even + 8u * (uint32_t)(it & 1));
      }
    }
    if (lane == 0) bulk_wait_all();  // this warp's stores have completed
    __syncwarp();
  }

  // neither CTA leaves (or frees TMEM) while the pair's MMAs, loads or
  // signals may still touch it
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

template <bool DX, int BT, int WPS>
cudaError_t launch_bt(const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                        const int32_t* offsets, uint16_t* y, int64_t R, int64_t K, int64_t N,
                        int64_t E, int group_shift, cudaStream_t stream, const DeviceInfo& dev) {
  const int64_t C = DX ? N : K, O = DX ? K : N;
  const int64_t n_groups = (group_shift == 62 || (int64_t(1) << group_shift) >= K)
                               ? 1 : (K + (int64_t(1) << group_shift) - 1) >> group_shift;
  using G_ = Geo<BT>;
  // scale rows that a stage's k touch (KST of them, or the CTA's 128 in the
  // gradient), and its columns
  const int span = DX ? BW : G_::KST;
  const int scale_rows = group_shift >= 30 || (span >> group_shift) < 1 ? 1 : span >> group_shift;
  const int scale_cols = DX ? G_::KST : BW;
  XMaps<BT> x_maps;
  CUtensorMap qw_map, s_map, y_map;
  // X as [C/64][R][64] (one copy of all the 64-column atoms per stage) when C
  // is a multiple of 64, else as [R][C] (one copy per atom); rows at or beyond R
  // and columns at or beyond C read as zero either way
  const int x3d = C % 64 == 0;
  for (int i = 0; i < BT / 32; ++i) {
    const uint32_t rows = 16u * (i + 1);
    const uint64_t dims[3] = {64, (uint64_t)R, (uint64_t)(C / 64)};
    const uint64_t strides[2] = {(uint64_t)C * 2, 128};
    const uint32_t box[3] = {64, rows, G_::ATOMS};
    if (!(x3d ? encode_map_3d(&x_maps.width[i], x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dims, strides,
                              box, CU_TENSOR_MAP_SWIZZLE_128B)
              : encode_map_2d(&x_maps.width[i], x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (uint64_t)C,
                              (uint64_t)R, (uint64_t)C * 2, 64, rows, CU_TENSOR_MAP_SWIZZLE_128B)))
      return cudaErrorInvalidValue;
  }
  const uint64_t qdims[3] = {(uint64_t)N, (uint64_t)(K / 8), (uint64_t)E};
  const uint64_t qstrides[2] = {(uint64_t)N * 4, (uint64_t)(K / 8) * N * 4};
  const uint32_t qbox[3] = {(uint32_t)scale_cols, (uint32_t)span / 8, 1};
  const uint64_t sdims[3] = {(uint64_t)N, (uint64_t)n_groups, (uint64_t)E};
  const uint64_t sstrides[2] = {(uint64_t)N * 2, (uint64_t)n_groups * N * 2};
  const uint32_t sbox[3] = {(uint32_t)scale_cols, (uint32_t)scale_rows, 1};
  if (!encode_map_3d(&qw_map, qweight, CU_TENSOR_MAP_DATA_TYPE_INT32, qdims, qstrides, qbox,
                     CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !encode_map_3d(&s_map, scales, CU_TENSOR_MAP_DATA_TYPE_UINT16, sdims, sstrides, sbox,
                     CU_TENSOR_MAP_SWIZZLE_NONE) ||
      // Y blocks of 32 columns x 32 tokens
      !encode_map_2d(&y_map, y, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (uint64_t)O, (uint64_t)R,
                     (uint64_t)O * 2, 32, Y_ROWS, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  static std::once_flag attr_once[64];
  static cudaError_t attr_err[64];
  const int d = dev.device & 63;
  std::call_once(attr_once[d], [&] {
    attr_err[d] = cudaFuncSetAttribute(experts_pair_kernel<DX, BT, WPS>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       1024 + TABLE_OFF + Geo<BT>::Table::bytes(GPTQ_MOE_MAX_EXPERTS));
  });
  if (attr_err[d] != cudaSuccess) return attr_err[d];
  // column pairs of 2 x 128 (with an odd count of 128-column tiles the last
  // pair's odd CTA has no columns: it loads no weights and stores nothing);
  // at most one token tile per row, and fewer than one per 64 rows beyond one
  // per expert
  const int64_t n_pairs = ((O + BW - 1) / BW + 1) / 2;
  const int64_t tiles = n_pairs * std::min<int64_t>(R, E + R / 64);
  const int64_t clusters = std::min<int64_t>(tiles, std::max(1, dev.num_sms / 2));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * clusters), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = 1024 + TABLE_OFF + Geo<BT>::Table::bytes((int)E);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, experts_pair_kernel<DX, BT, WPS>, x_maps, qw_map, s_map, y_map, offsets,
                            (int)R, (int)C, (int)O, (int)E, group_shift,
                            scale_rows * scale_cols * 2, x3d,
                            (int)n_pairs, y, dev.error_word);
}

// The token tile.  256 tokens move half the weights per product, 128 waste
// less on ragged row counts, give more tiles and overlap their read-out.  In us
// with 128 / 256 tokens, by rows per expert on average:
//   64 experts of 2048 x 2048, 64: 50 / 65, 128: 72 / 83, 256: 120 / 128,
//     512: 223 / 230 (the gradient 128: 75 / 84, 256: 125 / 130)
//   8 experts of 5120 x 17408, 64: 116 / 146, 128: 176 / 180, 256: 292 / 292,
//     512: 541 / 528
//   the gradient of 8 experts of 17408 x 5120, under sustained load, 192:
//     288 / 284, 256: 354 / 350, 384: 498 / 474, 512: 656 / 622
template <bool DX, int WPS>
cudaError_t launch_pair(const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                        const int32_t* offsets, uint16_t* y, int64_t R, int64_t K, int64_t N,
                        int64_t E, int group_shift, cudaStream_t stream, const DeviceInfo& dev) {
  const int64_t n_pairs = ((DX ? K : N) + 2 * BW - 1) / (2 * BW);
  const bool few = (E + R / 256) * n_pairs < dev.num_sms / 2;  // not a tile for each cluster
  const auto launch = R <= 256 * E || few ? launch_bt<DX, 128, WPS> : launch_bt<DX, 256, WPS>;
  return launch(x, qweight, scales, offsets, y, R, K, N, E, group_shift, stream, dev);
}

}  // namespace

cudaError_t launch_experts_pair(const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                                const int32_t* offsets, uint16_t* y, int64_t R, int64_t K,
                                int64_t N, int64_t E, int group_shift, cudaStream_t stream,
                                const DeviceInfo& dev) {
  const auto launch = group_shift == 4   ? launch_pair<false, 2>
                      : group_shift == 5 ? launch_pair<false, 4>
                      : group_shift == 6 ? launch_pair<false, 8>
                                         : launch_pair<false, 16>;
  return launch(x, qweight, scales, offsets, y, R, K, N, E, group_shift, stream, dev);
}

cudaError_t launch_experts_dx(const uint16_t* dy, const int32_t* qweight, const uint16_t* scales,
                              const int32_t* offsets, uint16_t* dx, int64_t R, int64_t K,
                              int64_t N, int64_t E, int group_shift, cudaStream_t stream,
                              const DeviceInfo& dev) {
  return launch_pair<true, 16>(dy, qweight, scales, offsets, dx, R, K, N, E, group_shift, stream,
                               dev);
}

}  // namespace gptq
