// The linear layer's bf16 products on the tensor cores, two SMs to a tile.
//
//   C(m, n) = sum over k of A(m, k) B(n, k), then z = C + bias, y = act(z) + residual
//
// Bound by the tensor pipe and, in a long run, by the power limit: 32768 x 4096 x
// 4096 keeps the pipe 95 % active and takes 550 to 600 us by the clock the GPU then
// holds (1.8 to 2.0 PFLOP/s).  A pair of CTAs owns a 256 x 256 tile: each CTA
// holds 128 rows of A and 128 rows of B, the pair's tcgen05.mma reads both
// halves, and each CTA's tensor memory receives 128 rows x 256 columns.  Against
// one CTA on 128 x 256 this halves the B bytes that each SM loads per product
// (62 instead of 94 bytes a clock for each SM, of what L2 gives 152 of them).
// Both accumulators of the 512 tensor-memory columns are used in turn, so the
// epilogue of a tile runs under the products of the next.  One warp a CTA
// issues the TMA loads (six stages of 64 k), one warp of the leader CTA the
// products, eight warps the epilogue.  Blocks are persistent.
//
// Either operand may lie with its rows contiguous instead of its k (the
// backward's dz^T x and dz W): TMA then brings 64-row blocks with k across, and
// the descriptors say so; nothing is transposed in memory.
#include "linear.cuh"
#include "pair.cuh"

namespace kda {
namespace dense {
namespace {

constexpr int kTile = 256;     // rows of a pair's tile
constexpr int kHalf = 128;     // a CTA's rows of A
constexpr int kStep = 64;      // k of a stage: 128 bytes, one swizzle line
constexpr int kStages = 6;
constexpr int kABytes = kHalf * kStep * 2;  // 16 KB: a CTA's A of a stage
constexpr int kEpilogueWarps = 8;
constexpr int kTcThreads = (kEpilogueWarps + 2) * 32;
constexpr int kGroup = 8;      // row tiles that share a band of column tiles (L2 reuse)
// BN columns of a tile, half of them from each CTA's B: 256, or 128 for few tiles.
constexpr int b_bytes(int bn) { return bn / 2 * kStep * 2; }
constexpr int stage_bytes(int bn) { return kABytes + b_bytes(bn); }

struct Shared {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  uint32_t gave_up;  // a wait of either CTA did
  uint32_t issued;   // stages that this CTA's loading warp issued
};
constexpr int smem_bytes(int bn) {
  return 1024 /* alignment */ + kStages * stage_bytes(bn) + kEpilogueWarps * 4096 + 256;
}
static_assert(sizeof(Shared) <= 256, "");

// Nonzero once a bounded wait of any launch on this device gave up (never cleared).
__device__ int g_gave_up;

// The schedule: `whole` tiles with their full k axis, then the other tiles with
// theirs in `splits` parts of k_per stages, whose sums tc_join_kernel adds.
struct Schedule {
  int tiles, whole, units;  // below 2^30 (launch_tc)
  int splits, k_per, bn;
};

struct TcArgs {
  Product p;
  Schedule s;
  float *part;  // [tiles - whole][splits][256][bn]
  int row_tiles, col_tiles;
  bool grid;   // output rows on 16-byte boundaries
  int polls;   // limit of a wait, and where one that gave up leaves 1 (NULL: g_gave_up)
  int *err;
};

struct Unit {
  int64_t m0, n0;
  int k_first, k_count;  // in stages
  float *part;           // where its sums go, NULL: a whole tile
};
// Tiles go in bands of kGroup row tiles, down the band first.
__device__ __forceinline__ void tile_of(const TcArgs &a, int t, int64_t *m0, int64_t *n0) {
  const int per_band = kGroup * a.col_tiles;
  const int band = t / per_band, in = t - band * per_band;
  const int rows = min(kGroup, a.row_tiles - band * kGroup);
  const int col = in / rows;
  *m0 = (int64_t)(band * kGroup + in - col * rows) * kTile;
  *n0 = (int64_t)col * a.s.bn;
}
__device__ __forceinline__ Unit unit_of(const TcArgs &a, int u) {
  Unit r;
  const int kb = (int)((a.p.K + kStep - 1) / kStep);
  if (u < a.s.whole) {
    tile_of(a, u, &r.m0, &r.n0);
    r.k_first = 0;
    r.k_count = kb;
    r.part = nullptr;
    return r;
  }
  const int v = u - a.s.whole, t = v / a.s.splits, split = v - t * a.s.splits;
  tile_of(a, a.s.whole + t, &r.m0, &r.n0);
  r.k_first = split * a.s.k_per;
  r.k_count = min(a.s.k_per, kb - r.k_first);
  r.part = a.part + (int64_t)v * (kTile * a.s.bn);
  return r;
}

// ---- epilogue ----
// A warp takes 32 rows x 32 columns of the accumulator at a time.  Tensor memory
// gives each lane one row; through 4 KB of shared memory (16-byte chunks swizzled
// by the row, no bank conflicts) the warp turns that into rows across lanes, so
// that its reads and writes of y, preact and residual are whole 64-byte pieces of
// rows, and partial sums whole 128-byte lines.
constexpr int kStageRow = 128;  // bytes of a staged row: 32 fp32

__device__ __forceinline__ uint32_t staged(int row, int chunk) {
  return (uint32_t)(row * kStageRow + ((chunk ^ (row & 7)) << 4));
}
__device__ __forceinline__ float4 lds4(const unsigned char *p) { return *reinterpret_cast<const float4 *>(p); }

__device__ __forceinline__ void stage_rows(unsigned char *sm, int lane, const float (&v)[32]) {
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<float4 *>(sm + staged(lane, j)) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  __syncwarp();
}

// Staged rows m0 .. m0 + 31, columns n0 .. n0 + 31: four rows' 8 columns a lane.
template <int ACT>
__device__ __forceinline__ void finish_vec(const Product &P, const unsigned char *sm, int lane, int64_t m0, int64_t n0,
                                           const Vec<__nv_bfloat16, 8> (&res)[4]) {
  const int q = lane & 3, r0 = lane >> 2;
  const int64_t n = n0 + q * 8;
  if (n >= P.N) return;
  float bias[8];
  if (P.bias != nullptr) bias_8(P, n, bias);
  int64_t at = (m0 + r0) * P.N + n;
  const int left = (int)min(P.M - m0, (int64_t)32);
  float4 x[4], y[4];  // all of them before the first store, which the loads could not pass
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = lds4(sm + staged(i * 8 + r0, 2 * q));
    y[i] = lds4(sm + staged(i * 8 + r0, 2 * q + 1));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i, at += 8 * P.N) {
    if (i * 8 + r0 < left) {
      float c[8] = {x[i].x, x[i].y, x[i].z, x[i].w, y[i].x, y[i].y, y[i].z, y[i].w};
      if (P.bias != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] += bias[e];
      }
      finish_8<ACT>(P, at, c, res[i]);
    }
  }
}
// The same one column a lane, for rows off the 16-byte grid.
template <int ACT>
__device__ __forceinline__ void finish_scalar(const Product &P, const unsigned char *sm, int lane, int64_t m0,
                                              int64_t n0) {
  const int64_t n = n0 + lane;
  if (n >= P.N) return;
  const int rows = (int)min((int64_t)32, P.M - m0);
  if (rows <= 0) return;
  typedef __nv_bfloat16 B;
  const float bias = P.bias != nullptr ? to_f(static_cast<const B *>(P.bias)[n]) : 0.f;
  const int64_t at = m0 * P.N + n;
  const B *res = P.residual != nullptr ? static_cast<const B *>(P.residual) + at : nullptr;
  B *z = P.preact != nullptr ? static_cast<B *>(P.preact) + at : nullptr, *y = static_cast<B *>(P.y) + at;
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 8) {
    float add[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) add[i] = res != nullptr && r0 + i < rows ? to_f(res[(r0 + i) * P.N]) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + i;
      if (r >= rows) break;
      const float c = *reinterpret_cast<const float *>(sm + staged(r, lane >> 2) + (lane & 3) * 4) + bias;
      if (z != nullptr) z[r * P.N] = from_f<B>(c);
      y[r * P.N] = from_f<B>(act_value<ACT, true>(c) + add[i]);
    }
  }
}
// Partial sums to a tile of [256][BN] fp32.
template <int BN>
__device__ __forceinline__ void store_part(float *tile, const unsigned char *sm, int lane, int row0, int col0) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + (lane >> 3), j = lane & 7;
    *reinterpret_cast<float4 *>(tile + (row0 + r) * BN + col0 + j * 4) = lds4(sm + staged(r, j));
  }
}

__device__ __forceinline__ bool wait(const TcArgs &a, uint64_t *bar, uint32_t parity, int polls) {
  if (pair::wait_cluster(bar, parity, polls)) return true;
  atomicExch(a.err != nullptr ? a.err : &g_gave_up, 1);
  return false;
}

// After a wait that gave up, once both CTAs' roles have ended: the products and the
// copies that are still in flight are waited for, since they read and write shared
// and tensor memory that ends with the block.  The leader does it for both: its
// barriers count both CTAs' copies.  A CTA may have issued up to kStages stages
// that the other did not (no stage is issued again before it was consumed, which
// takes both CTAs' halves): their barriers lack the other's bytes, or the leader's
// own arrival, which are made up for first.
__device__ __forceinline__ void settle(const TcArgs &a, Shared &sh, int warp, uint32_t stage_bytes) {
  if (warp == kEpilogueWarps + 1) {
    if (pair::elect()) pair::commit(&sh.drain);  // the lane that issued the products
    __syncwarp();
    wait(a, &sh.drain, 0, (int)umma::kSpinLimit);
  } else if (warp == kEpilogueWarps && pair::elect()) {
    const int n0 = (int)sh.issued, n1 = (int)pair::load_at(&sh.issued, 1);
    for (int s = 0; s < kStages; ++s) {
      // the last stage of this slot that each has issued, or below 0
      const int last0 = n0 - 1 - (n0 - 1 - s + kStages) % kStages, last1 = n1 - 1 - (n1 - 1 - s + kStages) % kStages;
      const int last = last0 > last1 ? last0 : last1;
      if (last < 0) continue;
      if (last1 < last)
        pair::complete_tx(&sh.full[s], stage_bytes);
      else if (last0 < last)
        pair::arrive_expect(&sh.full[s], stage_bytes);
      wait(a, &sh.full[s], (last / kStages) & 1, (int)umma::kSpinLimit);
    }
  }
  __syncwarp();
}

template <bool AK, bool BK, int ACT, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTcThreads, 1)
linear_tc_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap map_a,
                 const __grid_constant__ CUtensorMap map_b) {
  constexpr int kStageBytes = stage_bytes(BN), kTmemCols = 2 * BN;
  extern __shared__ unsigned char raw[];
  // the tiles' addresses agree in both CTAs: the dynamic shared base does
  unsigned char *tiles = reinterpret_cast<unsigned char *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  Shared &sh = *reinterpret_cast<Shared *>(tiles + kStages * kStageBytes + kEpilogueWarps * 32 * kStageRow);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = pair::cluster_rank();
  const int units = a.s.units, first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      umma::bar_init(&sh.full[i], 1);
      umma::bar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      umma::bar_init(&sh.acc_full[i], 1);
      umma::bar_init(&sh.acc_empty[i], 2 * kEpilogueWarps);
    }
    umma::bar_init(&sh.drain, 1);
    sh.gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 0) pair::tmem_alloc(&sh.tmem, kTmemCols);
  if (warp == kEpilogueWarps && lane == 0) {
    pair::prefetch_map(&map_a);
    pair::prefetch_map(&map_b);
  }
  umma::fence_before();
  __syncthreads();
  pair::cluster_sync();
  umma::fence_after();
  wait_for_stream();  // all above is the block's own
  const uint32_t tmem = sh.tmem;
  const uint32_t base = umma::smem_u32(tiles);
  bool ok = true;  // no wait of this warp gave up

  // The two issuing warps stay converged and elect a lane for each instruction: a
  // lane alone in a divergent branch issues them so slowly that the pipe waits
  // (606 clocks a stage against 519, and 575 against 517 where a stage takes four
  // loads).
  if (warp == kEpilogueWarps) {  // TMA, both CTAs
    uint32_t it = 0;
    for (int u = first; u < units && ok; u += stride) {
      const Unit w = unit_of(a, u);
      const int m = (int)w.m0 + (int)rank * kHalf, n = (int)w.n0 + (int)rank * (BN / 2);
      for (int kb = 0; kb < w.k_count; ++kb, ++it) {
        const int s = it % kStages;
        if (it >= kStages &&
            !__all_sync(0xffffffffu, wait(a, &sh.empty[s], (it / kStages - 1) & 1, a.polls))) {
          ok = false;
          break;
        }
        const uint32_t bar = pair::at_rank(&sh.full[s], 0);
        const uint32_t da = base + s * kStageBytes, db = da + kABytes;
        const int k = (w.k_first + kb) * kStep;
        if (pair::elect()) {
          if (rank == 0) pair::arrive_expect(&sh.full[s], 2 * kStageBytes);
          if (AK) {
            pair::tma_load_2d(da, &map_a, k, m, bar);
          } else {
            pair::tma_load_2d(da, &map_a, m, k, bar);
            pair::tma_load_2d(da + kABytes / 2, &map_a, m + 64, k, bar);
          }
          if (BK) {
            pair::tma_load_2d(db, &map_b, k, n, bar);
          } else {
            pair::tma_load_2d(db, &map_b, n, k, bar);
            if (BN == 256) pair::tma_load_2d(db + kABytes / 2, &map_b, n + 64, k, bar);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0) sh.issued = it;
  } else if (warp == kEpilogueWarps + 1) {  // products, leader CTA
    if (rank == 0) {
      const uint32_t idesc = umma::idesc_bf16(kTile, BN) | (AK ? 0u : 1u << 15) | (BK ? 0u : 1u << 16);
      const uint32_t d0 = __shfl_sync(0xffffffffu, tmem, 0);
      uint32_t it = 0, tile = 0;
      bool have = false;  // have: the stage's data was seen to be there
      for (int u = first; u < units && ok; u += stride, ++tile) {
        const int count = unit_of(a, u).k_count;
        const int acc = tile & 1;
        if (tile >= 2 && !__all_sync(0xffffffffu, wait(a, &sh.acc_empty[acc], (tile / 2 - 1) & 1, a.polls))) {
          ok = false;
          break;
        }
        umma::fence_after();
        for (int kb = 0; kb < count; ++kb, ++it) {
          const int s = it % kStages;
          if (!__all_sync(0xffffffffu, have || wait(a, &sh.full[s], (it / kStages) & 1, a.polls))) {
            ok = false;
            break;
          }
          umma::fence_after();
          const uint32_t da = base + s * kStageBytes, db = da + kABytes;
          have = __all_sync(0xffffffffu, pair::peek(&sh.full[(it + 1) % kStages], ((it + 1) / kStages) & 1));
          if (pair::elect()) {
#pragma unroll
            for (int k = 0; k < kStep / 16; ++k) {
              const uint64_t ad = AK ? umma::desc_sw128(da + k * 32) : pair::desc_mn(da + k * 2048);
              const uint64_t bd = BK ? umma::desc_sw128(db + k * 32) : pair::desc_mn(db + k * 2048);
              pair::mma(d0 + acc * BN, ad, bd, idesc, kb > 0 || k > 0);
            }
            pair::commit_both(&sh.empty[s]);
            if (kb == count - 1) pair::commit_both(&sh.acc_full[acc]);
          }
          __syncwarp();
        }
      }
    }
  } else {  // epilogue: warp w reads lanes 32 (w % 4) of its CTA's tensor memory, half of the columns
    const int quarter = warp & 3, side = warp >> 2;
    unsigned char *stage = tiles + kStages * kStageBytes + warp * (32 * kStageRow);
    uint32_t tile = 0;
    for (int u = first; u < units; u += stride, ++tile) {
      const Unit w = unit_of(a, u);
      const int acc = tile & 1;
      if (!__all_sync(0xffffffffu, wait(a, &sh.acc_full[acc], (tile / 2) & 1, a.polls))) {
        ok = false;
        break;
      }
      umma::fence_after();
      const int row0 = rank * kHalf + quarter * 32;
      const int64_t m0 = w.m0 + row0;
#pragma unroll 1
      for (int c = 0; c < BN / 64; ++c) {
        const int col0 = side * (BN / 2) + c * 32;
        const int64_t n0 = w.n0 + col0;
        Vec<__nv_bfloat16, 8> res[4];
        if (a.p.residual != nullptr && w.part == nullptr && a.grid) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + i * 8 + (lane >> 2), n = n0 + (lane & 3) * 8;
            if (m < a.p.M && n < a.p.N)
              res[i] = ldvec<__nv_bfloat16, 8>(static_cast<const __nv_bfloat16 *>(a.p.residual) + m * a.p.N + n);
          }
        }
        float v[32];
        umma::tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + acc * BN + col0, v);
        if (c == BN / 64 - 1) {  // the accumulator is read: the next but one tile may overwrite it
          umma::fence_before();
          __syncwarp();
          if (lane == 0) pair::arrive_remote(pair::at_rank(&sh.acc_empty[acc], 0));
        }
        stage_rows(stage, lane, v);
        if (w.part != nullptr)
          store_part<BN>(w.part, stage, lane, row0, col0);
        else if (a.grid)
          finish_vec<ACT>(a.p, stage, lane, m0, n0, res);
        else
          finish_scalar<ACT>(a.p, stage, lane, m0, n0);
      }
    }
  }
  if (!ok && lane == 0) {
    pair::store_at(&sh.gave_up, 0, 1);
    pair::store_at(&sh.gave_up, 1, 1);
  }
  __syncwarp();
  umma::fence_before();
  __syncthreads();
  pair::cluster_sync();
  umma::fence_after();
  if (sh.gave_up != 0) {  // the same in both CTAs
    if (rank == 0) settle(a, sh, warp, kStageBytes);
    __syncthreads();
    pair::cluster_sync();
  }
  if (warp == 0) pair::tmem_free(tmem, kTmemCols);
}

// [rows][cols] with rows `ld` apart, k or rows contiguous: boxes of 64 elements
// (128 bytes, swizzled) by `box` rows, or 64 k; elements outside arrive as zeros.
cudaError_t operand_map(CUtensorMap *m, const Operand &o, int64_t rows, int64_t k, int box) {
  return o.k_major ? encode_2d(m, o.p, k, rows, o.ld, kStep, box) : encode_2d(m, o.p, rows, k, o.ld, 64, kStep);
}

template <bool AK, bool BK, int ACT, int BN>
cudaError_t launch_bn(const TcArgs &a, const CUtensorMap &ma, const CUtensorMap &mb, unsigned grid, cudaStream_t s) {
  auto kernel = linear_tc_kernel<AK, BK, ACT, BN>;
  static std::atomic<int> granted[64];
  const cudaError_t e = allow_smem(kernel, granted, smem_bytes(BN));
  if (e != cudaSuccess) return e;
  KDA_LAUNCH("linear_tc_kernel", s, start_kernel(kernel, grid, kTcThreads, smem_bytes(BN), s, a, ma, mb));
  return cudaGetLastError();
}
template <bool AK, bool BK, int ACT>
cudaError_t launch(const TcArgs &a, const CUtensorMap &ma, const CUtensorMap &mb, unsigned grid, cudaStream_t s) {
  return a.s.bn == 256 ? launch_bn<AK, BK, ACT, 256>(a, ma, mb, grid, s)
                       : launch_bn<AK, BK, ACT, 128>(a, ma, mb, grid, s);
}

int64_t tiles_of(int64_t n, int per) { return (n + per - 1) / per; }

// Whole tiles fill as many full waves of the SM pairs as they can.  The tiles
// left over (all of them when there are fewer than pairs) have their k axis cut
// into the number of parts with the least estimated time, in clocks: a stage costs
// 520 (measured; 512 at the pair's 8192 products a clock), or 330 with 128 columns,
// whose operands shared memory delivers no faster; filling and draining 6000 or
// 4500; the join a launch (about 5000) and the fp32 sums written and read (about
// 6000 bytes a clock, mostly in L2).  4096 x 4096 x 4096 has 256 tiles for 76 pairs:
// 3 waves and 28 tiles, which in 8 parts take 3/8 of a wave instead of one (83 us
// instead of 99 when this came in).  Tiles of 128 columns are for products that
// leave pairs idle: the forward of 1531 x 1001 x 2047 has 24 tiles of 256 columns
// (25.5 us) or 48 of 128 (18.2 us).
Schedule schedule_of(int64_t M, int64_t N, int64_t K, int sms) {
  const int64_t kb = (K + kStep - 1) / kStep, pairs = sms / 2;
  Schedule S{0, 0, 0, 1, (int)kb, 0};
  double best = 0;
  for (const int bn : {256, 128}) {
    const int64_t tiles = tiles_of(M, kTile) * tiles_of(N, bn), left = tiles % pairs;
    const double stage = bn == 256 ? 520.0 : 330.0, fill = bn == 256 ? 6000.0 : 4500.0;
    const double waves = (double)(tiles / pairs) * (stage * (double)kb);
    const auto consider = [&](double t, const Schedule &c) {
      if (S.bn == 0 || t < best) {
        best = t;
        S = c;
      }
    };
    consider(waves + (left != 0 ? stage * (double)kb : 0.0) + fill, Schedule{(int)tiles, (int)tiles, (int)tiles, 1, (int)kb, bn});
    for (int64_t want = 2; left != 0 && want <= 64 && want * 2 <= kb; ++want) {
      const int64_t per = (kb + want - 1) / want, n = (kb + per - 1) / per;
      const double tail = (double)((left * n + pairs - 1) / pairs) * (stage * (double)per);
      const double join = 5000.0 + 8.0 * (double)(n * left) * kTile * bn / 6000.0;
      consider(waves + tail + fill + join, Schedule{(int)tiles, (int)(tiles - left), (int)(tiles - left + left * n), (int)n, (int)per, bn});
    }
  }
  return S;
}

size_t part_bytes_of(const Schedule &S) {
  return S.whole < S.tiles ? sizeof(float) * (size_t)(S.tiles - S.whole) * S.splits * kTile * S.bn : 0;
}

// Adds the parts of the split tiles, in order, and finishes the outputs: a block
// takes 16 rows of a tile, a thread 8 columns of two rows (adjacent ones where
// they are read and written as vectors, else 32 apart).
template <int ACT, bool GRID>
__global__ void __launch_bounds__(256) tc_join_kernel(const __grid_constant__ TcArgs a) {
  wait_for_stream();
  const int t = blockIdx.x >> 4;
  int64_t m0, n0;
  tile_of(a, a.s.whole + t, &m0, &n0);
  const int bn = a.s.bn, step = kTile * bn;
  const float *part = a.part + (int64_t)t * a.s.splits * step;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = (int)(blockIdx.x & 15) * 16 + i * 8 + (threadIdx.x >> 5);
    const int64_t m = m0 + row;
    if (m >= a.p.M) return;
    float c[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if constexpr (GRID) {
      const int64_t n = n0 + lane * 8;
      if (lane * 8 >= bn || n >= a.p.N) return;
      const float *p = part + row * bn + lane * 8;
#pragma unroll 4
      for (int k = 0; k < a.s.splits; ++k, p += step) {
        const float4 x = *reinterpret_cast<const float4 *>(p), y = *reinterpret_cast<const float4 *>(p + 4);
        c[0] += x.x, c[1] += x.y, c[2] += x.z, c[3] += x.w;
        c[4] += y.x, c[5] += y.y, c[6] += y.z, c[7] += y.w;
      }
      float bias[8];
      bias_8(a.p, n, bias);
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] += bias[e];
      const int64_t at = m * a.p.N + n;
      Vec<__nv_bfloat16, 8> res;
      if (a.p.residual != nullptr) res = ldvec<__nv_bfloat16, 8>(static_cast<const __nv_bfloat16 *>(a.p.residual) + at);
      finish_8<ACT>(a.p, at, c, res);
    } else {
      const float *p = part + row * bn + lane;
#pragma unroll 4
      for (int k = 0; k < a.s.splits; ++k, p += step)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (32 * e < bn) c[e] += p[32 * e];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (32 * e < bn && n0 + lane + 32 * e < a.p.N) finish_one<__nv_bfloat16, ACT>(a.p, m, n0 + lane + 32 * e, c[e]);
    }
  }
}

cudaError_t launch_join(const TcArgs &a, cudaStream_t s) {
  const unsigned grid = (unsigned)((a.s.tiles - a.s.whole) * 16);
  DENSE_ACT_SWITCH(a.p.act, {
    if (a.grid)
      KDA_LAUNCH("tc_join_kernel", s, start_kernel(tc_join_kernel<ACT, true>, grid, 256, 0, s, a));
    else
      KDA_LAUNCH("tc_join_kernel", s, start_kernel(tc_join_kernel<ACT, false>, grid, 256, 0, s, a));
  });
  return cudaGetLastError();
}

}  // namespace

cudaError_t linear_status_word(int **p) {
  void *q = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&q, g_gave_up);
  *p = static_cast<int *>(q);
  return e;
}

size_t tc_part_bytes(int64_t M, int64_t N, int64_t K, int sms) { return part_bytes_of(schedule_of(M, N, K, sms)); }

cudaError_t launch_tc(const Product &P, float *part, int sms, cudaStream_t s, const Waits &waits) {
  const Schedule S = schedule_of(P.M, P.N, P.K, sms);
  const TcArgs a{P, S, part, (int)tiles_of(P.M, kTile), (int)tiles_of(P.N, S.bn), rows_on_grid(P), waits.polls, waits.err};
  CUtensorMap ma, mb;
  cudaError_t e = operand_map(&ma, P.a, P.M, P.K, kHalf);
  if (e == cudaSuccess) e = operand_map(&mb, P.b, P.N, P.K, S.bn / 2);
  if (e != cudaSuccess) return e;
  const int64_t pairs = sms / 2;
  const unsigned grid = (unsigned)(2 * (a.s.units < pairs ? a.s.units : pairs));
  if (!P.a.k_major) {
    e = launch<false, false, KDA_ACT_NONE>(a, ma, mb, grid, s);
  } else if (!P.b.k_major) {
    e = launch<true, false, KDA_ACT_NONE>(a, ma, mb, grid, s);
  } else {
    DENSE_ACT_SWITCH(P.act, e = (launch<true, true, ACT>(a, ma, mb, grid, s)));
  }
  return e == cudaSuccess && a.s.whole < a.s.tiles ? launch_join(a, s) : e;
}

}  // namespace dense
}  // namespace kda
