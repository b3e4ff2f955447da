// Matrix product on the fp32 pipes, with the linear layer's epilogue: the whole
// of the fp32 path (fp32 arithmetic throughout).
//
// C(m, n) = sum over k of A(m, k) B(n, k) for any strides.  A block of 128 threads
// owns 128 x 128 outputs, 16 x 8 a thread, over k slices of 16 held twice in shared
// memory: the next slice is read into registers while this one is multiplied.
// Bound by the fp32 FMA rate; the products are packed pairs of rows
// (fma.rn.f32x2), which leave issue slots for the six 16-byte operand loads of
// each k: 4096 x 4096 x 4096 takes 2.59 ms so, 3.35 with single FMAs.
//
// Two blocks a SM share the work evenly whatever the number of tiles: the slices of
// all tiles, one tile after the other, are dealt out in equal runs.  A run that
// covers a tile finishes it; the pieces of a tile that several runs share go to the
// workspace, two at most a block, and simt_join_kernel adds them in order.  2048 x
// 1024 x 1024, 128 tiles: 100 us, against 112 with its k axis cut in two and 127
// with a tile a block.
//
// A few rows (a serving step) are bound by reading B = W once instead:
// linear_few32_kernel streams it through registers.
#include "linear.cuh"

namespace kda {
namespace dense {
namespace {

constexpr int kBM = 128, kBN = 128, kBK = 16, kSimtThreads = 128;

__device__ __forceinline__ void fma2(uint64_t &d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;\n" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t twice(float x) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %1};\n" : "=l"(d) : "r"(__float_as_uint(x)));
  return d;
}
__device__ __forceinline__ float half_of(uint64_t v, int h) {
  return __uint_as_float(h ? (uint32_t)(v >> 32) : (uint32_t)v);
}

// One operand's slice: rows [row0, row0 + 128) x k [k0, k0 + 16), 16 elements a thread, zero outside.
struct SliceLoad {
  const float *p;
  int64_t ld, rows, k_end;
  bool k_major, vec;
  int r, k;  // this thread's first element within the slice
  __device__ __forceinline__ void init(const Operand &o, int64_t row0, int64_t rows_, int64_t k_end_) {
    p = static_cast<const float *>(o.p);
    ld = o.ld;
    k_major = o.k_major;
    k_end = k_end_;
    rows = rows_ - row0;
    vec = (ld & 3) == 0 && ((uintptr_t)p & 15) == 0;
    if (k_major) {
      r = threadIdx.x;
      k = 0;
      p += (row0 + r) * ld;
    } else {
      r = (threadIdx.x & 7) * 16;
      k = threadIdx.x >> 3;
      p += row0 + r;
    }
  }
  __device__ __forceinline__ void load(int64_t k0, float (&v)[16]) const {
    const int64_t kk = k0 + k;
    const float *q = k_major ? p + kk : p + kk * ld;
    // elements that exist along the contiguous axis
    const int64_t left = k_major ? (r < rows ? k_end - kk : 0) : (kk < k_end ? rows - r : 0);
    if (vec && left >= 16) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(v + i) = *reinterpret_cast<const float4 *>(q + i);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = i < left ? q[i] : 0.f;
    }
  }
  __device__ __forceinline__ void store(float (*sm)[kBM + 4], const float (&v)[16]) const {
    if (k_major) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sm[i][r] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(&sm[k][r + i]) = *reinterpret_cast<const float4 *>(v + i);
    }
  }
};

// A thread's operands of one k: 16 rows of A (4 of every 32), 8 of B (4 of every 64).
struct Fragment {
  uint64_t a[8];  // pairs of rows
  float b[8];
  __device__ __forceinline__ void load(const float (*as)[kBM + 4], const float (*bs)[kBN + 4], int k, int ty, int tx) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(&as[k][i * 32 + ty * 4]);
      a[2 * i] = v.x, a[2 * i + 1] = v.y;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<float4 *>(b + 4 * j) = *reinterpret_cast<const float4 *>(&bs[k][j * 64 + tx * 4]);
  }
};

// The epilogue of four outputs of one row from n on.
template <int ACT>
__device__ __forceinline__ void finish_4(const Product &P, int64_t m, int64_t n, float4 c, bool grid) {
  if (!grid || n + 4 > P.N) {
    const float v[4] = {c.x, c.y, c.z, c.w};
    for (int e = 0; e < 4; ++e)
      if (n + e < P.N) finish_one<float, ACT>(P, m, n + e, v[e]);
    return;
  }
  const int64_t at = m * P.N + n;
  if (P.bias != nullptr) {
    const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(P.bias) + n);
    c.x += b.x, c.y += b.y, c.z += b.z, c.w += b.w;
  }
  if (P.preact != nullptr) *reinterpret_cast<float4 *>(static_cast<float *>(P.preact) + at) = c;
  c = make_float4(act_value<ACT, false>(c.x), act_value<ACT, false>(c.y), act_value<ACT, false>(c.z),
                  act_value<ACT, false>(c.w));
  if (P.residual != nullptr) {
    const float4 r = *reinterpret_cast<const float4 *>(static_cast<const float *>(P.residual) + at);
    c.x += r.x, c.y += r.y, c.z += r.z, c.w += r.w;
  }
  *reinterpret_cast<float4 *>(static_cast<float *>(P.y) + at) = c;
}

struct Runs {
  int64_t slices;  // of all tiles
  int per_tile;    // slices of a tile's k axis
  int col_tiles, blocks;
  __host__ __device__ int64_t begin(int64_t b) const { return b * slices / blocks; }
  // the block whose run holds a slice
  __host__ __device__ int block_of(int64_t slice) const { return (int)(((slice + 1) * blocks - 1) / slices); }
};

// part: [2 blocks][128][128]: a run's piece of the tile it starts in, then of the
// tile that it starts itself and does not finish.
template <int ACT>
__global__ void __launch_bounds__(kSimtThreads) linear_simt_kernel(Product P, Runs R, float *part, bool grid) {
  wait_for_stream();
  __shared__ __align__(16) float as[2][kBK][kBM + 4];
  __shared__ __align__(16) float bs[2][kBK][kBN + 4];
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int64_t first = R.begin(blockIdx.x), last = R.begin(blockIdx.x + 1);
#pragma unroll 1
  for (int64_t at = first; at < last;) {
    const int64_t tile = at / R.per_tile;
    const int from = (int)(at - tile * R.per_tile), count = (int)min(last - at, (int64_t)(R.per_tile - from));
    const int64_t m0 = tile / R.col_tiles * kBM, n0 = tile % R.col_tiles * kBN;
    const int64_t kb = (int64_t)from * kBK, ke = min(P.K, kb + (int64_t)count * kBK);
    SliceLoad la, lb;
    la.init(P.a, m0, P.M, ke);
    lb.init(P.b, n0, P.N, ke);
    uint64_t acc[8][8];  // pairs of rows x columns
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = 0;
    int cur = 0;
    float va[16], vb[16];
    la.load(kb, va);
    lb.load(kb, vb);
    __syncthreads();  // the tile before has been multiplied
    la.store(as[0], va);
    lb.store(bs[0], vb);
    __syncthreads();
#pragma unroll 1
    for (int64_t k0 = kb; k0 < ke; k0 += kBK) {
      const bool more = k0 + kBK < ke;
      if (more) {
        la.load(k0 + kBK, va);
        lb.load(k0 + kBK, vb);
      }
#pragma unroll
      for (int k = 0; k < kBK; ++k) {
        Fragment g;
        g.load(as[cur], bs[cur], k, ty, tx);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint64_t b2 = twice(g.b[j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) fma2(acc[i][j], g.a[i], b2);
        }
      }
      if (more) {
        cur ^= 1;
        la.store(as[cur], va);
        lb.store(bs[cur], vb);
        __syncthreads();
      }
    }
    const bool whole = count == R.per_tile;
    float *piece = part + (2 * (int64_t)blockIdx.x + (from == 0 && at != first ? 1 : 0)) * (kBM * kBN);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = (i >> 2) * 32 + ty * 4 + (i & 3);
      const int64_t m = m0 + row;
      if (whole && m >= P.M) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = j * 64 + tx * 4;
        float c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = half_of(acc[i >> 1][4 * j + e], i & 1);
        const float4 v = make_float4(c[0], c[1], c[2], c[3]);
        if (!whole)
          *reinterpret_cast<float4 *>(piece + row * kBN + col) = v;
        else if (n0 + col < P.N)
          finish_4<ACT>(P, m, n0 + col, v, grid);
      }
    }
    at += count;
  }
}

// Adds the pieces of a shared tile in the order of their runs and finishes the
// outputs: a block takes 8 rows, a thread 4 columns of one; four pieces' loads at once.
constexpr int kJoinRows = 8;
template <int ACT>
__global__ void __launch_bounds__(256) simt_join_kernel(Product P, Runs R, const float *__restrict__ part, bool grid) {
  wait_for_stream();
  constexpr int kBlocks = kBM / kJoinRows;
  const int64_t tile = blockIdx.x / kBlocks, slice = tile * R.per_tile;
  const int b0 = R.block_of(slice), b1 = R.block_of(slice + R.per_tile - 1);
  if (b0 == b1) return;  // one run had all of it
  const int row = (int)(blockIdx.x % kBlocks) * kJoinRows + (threadIdx.x >> 5), col = (threadIdx.x & 31) * 4;
  const int64_t m = tile / R.col_tiles * kBM + row, n = tile % R.col_tiles * kBN + col;
  if (m >= P.M || n >= P.N) return;
  // the first run's piece is its second one unless the run starts with this tile
  const float *p = part + row * kBN + col + (R.begin(b0) != slice ? kBM * kBN : 0);
  float4 c = *reinterpret_cast<const float4 *>(p + 2 * (int64_t)b0 * (kBM * kBN));
  p = part + row * kBN + col;
#pragma unroll 4
  for (int b = b0 + 1; b <= b1; ++b) {
    const float4 v = *reinterpret_cast<const float4 *>(p + 2 * (int64_t)b * (kBM * kBN));
    c.x += v.x, c.y += v.y, c.z += v.z, c.w += v.w;
  }
  finish_4<ACT>(P, m, n, c, grid);
}

// Two blocks a SM (one waits for its slice while the other multiplies), none with
// less than 8 slices.
Runs runs_of(int64_t M, int64_t N, int64_t K, int sms) {
  Runs R;
  R.per_tile = (int)((K + kBK - 1) / kBK);
  R.col_tiles = (int)((N + kBN - 1) / kBN);
  R.slices = (M + kBM - 1) / kBM * R.col_tiles * R.per_tile;
  const int64_t most = 2 * (int64_t)sms, want = R.slices / 8;
  R.blocks = (int)(want < 1 ? 1 : want < most ? want : most);
  return R;
}
// Whether a tile is shared: unless every run is whole tiles.
bool shares(const Runs &R) {
  return R.slices > 0 && (R.slices % R.blocks != 0 || R.slices / R.blocks % R.per_tile != 0);
}

// ---- a few rows ----
// A block takes four rows of W, its eight warps 128 k at a time each; a lane holds
// 4 contiguous k of every row against the same k of up to MT rows of x. The lanes'
// sums are added by shuffles, the warps' in shared memory, in a fixed order. 4096 x
// 4096: 12.7 us for 1 row (9.9 by its bytes), 18.6 for 4, 71 for 16, where x comes
// from L2 once a block (88 on 128 x 128 tiles).
constexpr int kFewWarps = 8, kWRows = 4;

template <bool VEC>
__device__ __forceinline__ float4 load4(const float *row, int64_t k, int64_t K) {
  if (VEC) return k < K ? __ldg(reinterpret_cast<const float4 *>(row + k)) : make_float4(0.f, 0.f, 0.f, 0.f);
  return make_float4(k < K ? row[k] : 0.f, k + 1 < K ? row[k + 1] : 0.f, k + 2 < K ? row[k + 2] : 0.f,
                     k + 3 < K ? row[k + 3] : 0.f);
}

template <int MT, bool VEC, int ACT>
__global__ void __launch_bounds__(kFewWarps * 32) linear_few32_kernel(const Product P) {
  wait_for_stream();
  __shared__ float sums[kFewWarps][kWRows * MT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n0 = (int64_t)blockIdx.x * kWRows;
  const float *w = static_cast<const float *>(P.b.p), *x = static_cast<const float *>(P.a.p);
  float acc[kWRows][MT];
#pragma unroll
  for (int r = 0; r < kWRows; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = 0.f;
#pragma unroll(MT > 4 ? 1 : 2)
  for (int64_t k = warp * 128 + lane * 4; k < P.K; k += kFewWarps * 128) {
    float4 wv[kWRows];
#pragma unroll
    for (int r = 0; r < kWRows; ++r) wv[r] = load4<VEC>(w + min(n0 + r, P.N - 1) * P.K, k, P.K);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m < P.M) {
        const float4 xv = load4<VEC>(x + m * P.K, k, P.K);
#pragma unroll
        for (int r = 0; r < kWRows; ++r) {
          acc[r][m] = fmaf(wv[r].x, xv.x, acc[r][m]);
          acc[r][m] = fmaf(wv[r].y, xv.y, acc[r][m]);
          acc[r][m] = fmaf(wv[r].z, xv.z, acc[r][m]);
          acc[r][m] = fmaf(wv[r].w, xv.w, acc[r][m]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kWRows; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[r][m] += __shfl_xor_sync(0xffffffffu, acc[r][m], o);
      if (lane == 0) sums[warp][r * MT + m] = acc[r][m];
    }
  __syncthreads();
  if (threadIdx.x >= kWRows * MT) return;
  const int r = threadIdx.x / MT, m = threadIdx.x % MT;
  if (m >= P.M || n0 + r >= P.N) return;
  float c = 0.f;
#pragma unroll
  for (int v = 0; v < kFewWarps; ++v) c += sums[v][threadIdx.x];
  finish_one<float, ACT>(P, m, n0 + r, c);
}

template <int MT>
cudaError_t few(const Product &P, cudaStream_t s) {
  const bool vec = P.K % 4 == 0 && (((uintptr_t)P.a.p | (uintptr_t)P.b.p) & 15) == 0;
  const unsigned grid = (unsigned)((P.N + kWRows - 1) / kWRows);
  DENSE_ACT_SWITCH(P.act, {
    if (vec)
      KDA_LAUNCH("linear_few32_kernel", s,
                 start_kernel(linear_few32_kernel<MT, true, ACT>, grid, kFewWarps * 32, 0, s, P));
    else
      KDA_LAUNCH("linear_few32_kernel", s,
                 start_kernel(linear_few32_kernel<MT, false, ACT>, grid, kFewWarps * 32, 0, s, P));
  });
  return cudaGetLastError();
}

}  // namespace

size_t simt_part_bytes(int64_t M, int64_t N, int64_t K, int sms) {
  const Runs R = runs_of(M, N, K, sms);
  return shares(R) ? sizeof(float) * 2 * (size_t)R.blocks * kBM * kBN : 0;
}

cudaError_t launch_simt(const Product &P, float *part, int sms, cudaStream_t s) {
  const Runs R = runs_of(P.M, P.N, P.K, sms);
  const uintptr_t bits = (uintptr_t)P.y | (uintptr_t)P.preact | (uintptr_t)P.residual | (uintptr_t)P.bias;
  const bool grid = P.N % 4 == 0 && (bits & 15) == 0;
  DENSE_ACT_SWITCH(P.act, {
    KDA_LAUNCH("linear_simt_kernel", s,
               start_kernel(linear_simt_kernel<ACT>, (unsigned)R.blocks, kSimtThreads, 0, s, P, R, part, grid));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !shares(R)) return e;
    KDA_LAUNCH("simt_join_kernel", s,
               start_kernel(simt_join_kernel<ACT>, (unsigned)(R.slices / R.per_tile * (kBM / kJoinRows)), 256, 0, s, P, R, part, grid));
  });
  return cudaGetLastError();
}

cudaError_t launch_few32(const Product &P, cudaStream_t s) {
  if (P.M <= 1) return few<1>(P, s);
  if (P.M <= 4) return few<4>(P, s);
  if (P.M <= 8) return few<8>(P, s);
  return few<kFewRows32>(P, s);
}

}  // namespace dense
}  // namespace kda
