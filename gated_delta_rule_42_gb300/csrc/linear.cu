// The linear layer: dispatch of its products and the elementwise passes beside them.
//
//   z = x W^T + b, y = act(z) + r;  dz = dy act'(z), dx = dz W, dW = dz^T x, db = sum of dz's rows
#include "linear.cuh"

namespace kda {
namespace dense {
namespace {

// dz = dy act'(z) and the partial sums of its columns, one pass over dy and z.
// In bf16, dz is rounded for the two products, whose operands the tensor cores take
// in bf16 (a second term for the lost bits would double their time), and z is what
// the forward rounded (in fp32 it would be twice the bytes there and here).  The two
// roundings put dx and dweight 2.4e-3 (relative RMS) from 64 bits, where rounding the
// results alone puts them 1.7e-3.  dbias sums the unrounded dz.
// A block works on 32 column vectors x 8 rows at a time down its slab of rows
// (blockIdx.y), four such loads in flight; dz (rows ld_dz apart) or NULL,
// dbias or NULL; several slabs leave their sums in part [gridDim.y][N].
constexpr int kDzRows = 4;
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(256)
linear_dz_kernel(const T *__restrict__ dy, const T *__restrict__ z, T *__restrict__ dz, int64_t ld_dz,
                 float *__restrict__ part, T *__restrict__ dbias, int64_t M, int N) {
  wait_for_stream();
  __shared__ float sm[8][32 * VEC + 1];
  const int cv = blockIdx.x * 32 + threadIdx.x;  // this thread's column vector
  const bool on = (int64_t)cv * VEC < N;
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  if (on) {
    const int64_t step = (int64_t)gridDim.y * 8;
    for (int64_t r0 = (int64_t)blockIdx.y * 8 + threadIdx.y; r0 < M; r0 += kDzRows * step) {
      Vec<T, VEC> d[kDzRows], zz[kDzRows];
#pragma unroll
      for (int k = 0; k < kDzRows; ++k) {
        const int64_t r = r0 + k * step, at = r * N + (int64_t)cv * VEC;
        if (r < M) {
          d[k] = ldvec<T, VEC>(dy + at);
          if constexpr (ACT != KDA_ACT_NONE) zz[k] = ldvec<T, VEC>(z + at);
        }
      }
#pragma unroll
      for (int k = 0; k < kDzRows; ++k) {
        const int64_t r = r0 + k * step;
        if (r >= M) break;
        float g[VEC], zf[VEC];
        unpack(d[k], g);
        if constexpr (ACT != KDA_ACT_NONE) unpack(zz[k], zf);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          if constexpr (ACT != KDA_ACT_NONE) g[e] *= act_slope<ACT, sizeof(T) == 2>(zf[e]);
          acc[e] += g[e];
        }
        if (dz != nullptr) stvec<T, VEC>(dz + r * ld_dz + (int64_t)cv * VEC, pack<T, VEC>(g));
      }
    }
  }
  if (dbias == nullptr) return;
#pragma unroll
  for (int e = 0; e < VEC; ++e) sm[threadIdx.y][threadIdx.x * VEC + e] = acc[e];
  __syncthreads();
  for (int c = threadIdx.y * 32 + threadIdx.x; c < 32 * VEC; c += 256) {
    const int64_t col = (int64_t)blockIdx.x * 32 * VEC + c;
    if (col >= N) continue;
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) a += sm[k][c];
    if (gridDim.y == 1)
      dbias[col] = from_f<T>(a);
    else
      part[(int64_t)blockIdx.y * N + col] = a;
  }
}

// Slabs of rows: enough blocks for 8 a SM, no slab below 8 rows.
constexpr int kOneSlabRows = 64;
int dz_slabs(int64_t M, int N, int vec, int sms) {
  const int64_t cols = (N + 32 * vec - 1) / (32 * vec), rows8 = (M + 7) / 8;
  int64_t want = (sms * 8 + cols - 1) / cols;
  want = want < rows8 ? want : rows8;
  // one slab leaves no partial sums to add: 3.7 us against 4.2 for 64 x 4096, with its launch
  if (M <= kOneSlabRows) want = 1;
  return (int)(want < 1 ? 1 : want > 1024 ? 1024 : want);
}

template <typename T>
cudaError_t run_dz(const Linear &L, const void *dy, const void *z, void *dz, int64_t ld_dz, float *part, void *dbias,
                   int sms, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const uintptr_t bits = (uintptr_t)dy | (L.act != KDA_ACT_NONE ? (uintptr_t)z : 0) | (uintptr_t)dz;
  const bool vec = L.outs % V == 0 && (bits & 15) == 0;
  const int slabs = dz_slabs(L.rows, L.outs, vec ? V : 1, sms);
  const int w = 32 * (vec ? V : 1);
  const dim3 grid((unsigned)((L.outs + w - 1) / w), (unsigned)slabs), block(32, 8);
  const T *d = static_cast<const T *>(dy), *zt = static_cast<const T *>(z);
  T *o = static_cast<T *>(dz), *db = static_cast<T *>(dbias);
  DENSE_ACT_SWITCH(L.act, {
    if (vec)
      KDA_LAUNCH("linear_dz_kernel", s,
                 start_kernel(linear_dz_kernel<T, V, ACT>, grid, block, 0, s, d, zt, o, ld_dz, part, db, L.rows, L.outs));
    else
      KDA_LAUNCH("linear_dz_kernel", s,
                 start_kernel(linear_dz_kernel<T, 1, ACT>, grid, block, 0, s, d, zt, o, ld_dz, part, db, L.rows, L.outs));
  });
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || dbias == nullptr || slabs == 1) return e;
  return launch_column_reduce(part, slabs, L.outs, L.outs, dbias, nullptr, 0, L.bf16, s);
}

int sms_or_default() {
  int sms = 0;
  return sm_count(&sms) == cudaSuccess ? sms : 152;
}

// ---- operands off the 16-byte grid ----
// TMA reads rows that start on 16-byte boundaries; other matrices are copied
// once to rows of a multiple of 8 elements.  The copy costs its bytes (rows x
// cols x 2, twice); the products read every element many times.  Two matrices at
// most (x and the weight), in one launch.
struct Pad {
  const __nv_bfloat16 *src;
  __nv_bfloat16 *dst;
  int64_t rows;
  int cols, ld;
};
__global__ void __launch_bounds__(256) pad_rows_kernel(Pad a, Pad b) {
  wait_for_stream();
  const Pad &p = blockIdx.y ? b : a;
  const int per_row = p.ld / 8;
  const int64_t total = p.rows * per_row, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
    const int64_t r = i / per_row;
    const int c = (int)(i - r * per_row) * 8;
    Vec<__nv_bfloat16, 8> v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v.e[e] = c + e < p.cols ? p.src[r * p.cols + c + e] : __float2bfloat16_rn(0.f);
    stvec<__nv_bfloat16, 8>(p.dst + r * p.ld + c, v);
  }
}

int64_t round8(int64_t n) { return (n + 7) & ~(int64_t)7; }
bool off_grid(const void *p, int cols) { return cols % 8 != 0 || ((uintptr_t)p & 15) != 0; }
size_t pad_bytes(const void *p, int64_t rows, int cols) {
  return off_grid(p, cols) ? align256(2 * (size_t)rows * round8(cols)) : 0;
}
// The operands as TMA can read them: x and the weight themselves, or copies at
// x_room and w_room.
struct OnGrid {
  Operand x, w;
};
cudaError_t on_grid(const Linear &L, bool need_x, bool need_w, char *x_room, char *w_room, int sms, OnGrid *g,
                    cudaStream_t s) {
  g->x = Operand{L.x, L.ins, true};
  g->w = Operand{L.weight, L.ins, true};
  Pad pads[2];
  int n = 0;
  int64_t blocks = 0;
  const auto add = [&](Operand &o, int64_t rows, char *room) {
    pads[n++] = Pad{static_cast<const __nv_bfloat16 *>(o.p), reinterpret_cast<__nv_bfloat16 *>(room), rows, L.ins,
                    (int)round8(L.ins)};
    const int64_t m = (rows * (round8(L.ins) / 8) + 255) / 256;
    blocks = m > blocks ? m : blocks;
    o.p = room;
    o.ld = round8(L.ins);
  };
  if (need_x && off_grid(L.x, L.ins)) add(g->x, L.rows, x_room);
  if (need_w && off_grid(L.weight, L.ins)) add(g->w, L.outs, w_room);
  if (n == 0) return cudaSuccess;
  const dim3 grid((unsigned)(blocks < sms * 16 ? blocks : sms * 16), (unsigned)n);
  KDA_LAUNCH("pad_rows_kernel", s, start_kernel(pad_rows_kernel, grid, 256, 0, s, pads[0], pads[n - 1]));
  return cudaGetLastError();
}

size_t part_bytes(int64_t M, int64_t N, int64_t K, bool bf16, int sms) {
  return align256(bf16 ? tc_part_bytes(M, N, K, sms) : simt_part_bytes(M, N, K, sms));
}

// One product with its epilogue.
cudaError_t product(const Product &P, bool bf16, float *part, int sms, cudaStream_t s, const Waits &waits = kWaits) {
  return bf16 ? launch_tc(P, part, sms, s, waits) : launch_simt(P, part, sms, s);
}

// Up to 32 bf16 rows on the 16-byte grid, 16 off it, and 16 fp32 rows stream the
// weight through registers instead of taking tiles (4096 x 4096 bf16: 7.3 us for 1
// row, 12.1 for 32, against 17.2 to 22 on tiles; 1001 x 2047, off the grid: 9.6 us
// for 16 rows against 15.2, but 21 to 27 for 17 to 32 rows, since elements are
// loaded one by one).
bool few_rows(const Linear &L) {
  if (!L.bf16) return L.rows <= kFewRows32;
  const bool off = off_grid(L.x, L.ins) || off_grid(L.weight, L.ins);
  return L.rows <= (off ? kFewRows / 2 : kFewRows);
}

// Forward workspace: x and weight on the grid | parts of a split product.
struct FwdLayout {
  size_t w, part, total;
};
FwdLayout fwd_layout(const Linear &L, int sms) {
  FwdLayout f;
  if (few_rows(L)) return FwdLayout{0, 0, 0};
  f.w = L.bf16 ? pad_bytes(L.x, L.rows, L.ins) : 0;
  f.part = f.w + (L.bf16 ? pad_bytes(L.weight, L.outs, L.ins) : 0);
  f.total = f.part + part_bytes(L.rows, L.outs, L.ins, L.bf16, sms);
  return f;
}

// Backward workspace: dz | column partials | x and weight on the grid | parts of
// a split product.  In bf16 dz has its place without an activation too: dy may
// lie off the grid.
struct BwdLayout {
  size_t cols, x, w, part, total;
  int64_t ld_dz;
};
BwdLayout bwd_layout(const Linear &L, int sms) {
  BwdLayout w;
  w.ld_dz = L.bf16 ? round8(L.outs) : L.outs;
  w.cols = L.bf16 || L.act != KDA_ACT_NONE ? align256((L.bf16 ? 2 : 4) * (size_t)L.rows * w.ld_dz) : 0;
  int slabs = 1;
  for (const int vec : {1, L.bf16 ? 8 : 4}) {
    const int n = dz_slabs(L.rows, L.outs, vec, sms);
    slabs = n > slabs ? n : slabs;
  }
  w.x = w.cols + align256(sizeof(float) * (size_t)slabs * L.outs);
  w.w = w.x + (L.bf16 ? pad_bytes(L.x, L.rows, L.ins) : 0);
  w.part = w.w + (L.bf16 ? pad_bytes(L.weight, L.outs, L.ins) : 0);
  const size_t a = part_bytes(L.rows, L.ins, L.outs, L.bf16, sms),
               b = part_bytes(L.outs, L.ins, L.rows, L.bf16, sms);
  w.total = w.part + (a > b ? a : b);
  return w;
}

}  // namespace

size_t linear_fwd_workspace(const Linear &L) { return fwd_layout(L, sms_or_default()).total; }
size_t linear_bwd_workspace(const Linear &L) { return bwd_layout(L, sms_or_default()).total; }

bool linear_uses_tensor_cores(const Linear &L) { return L.bf16 && L.rows > 0 && !few_rows(L); }

cudaError_t launch_linear_fwd(const Linear &L, void *y, void *preact, char *ws, cudaStream_t s, const Waits &waits) {
  if (L.rows == 0) return cudaSuccess;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const FwdLayout f = fwd_layout(L, sms);
  Product P{L.rows, L.outs, L.ins, {L.x, L.ins, true}, {L.weight, L.ins, true}, L.bias, L.residual, L.act, y,
            preact};
  if (few_rows(L)) return L.bf16 ? launch_few(P, s) : launch_few32(P, s);
  if (L.bf16) {
    OnGrid g;
    if ((e = on_grid(L, true, true, ws, ws + f.w, sms, &g, s)) != cudaSuccess) return e;
    P.a = g.x;
    P.b = g.w;
  }
  return product(P, L.bf16, reinterpret_cast<float *>(ws + f.part), sms, s, waits);
}

cudaError_t launch_linear_bwd(const Linear &L, const void *dy, const void *preact, void *dx, void *dweight,
                              void *dbias, char *ws, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const BwdLayout w = bwd_layout(L, sms);
  float *cols = reinterpret_cast<float *>(ws + w.cols), *part = reinterpret_cast<float *>(ws + w.part);
  const bool products = dx != nullptr || dweight != nullptr;
  // dz is dy itself without an activation, where the products can read it
  const bool make = products && (L.act != KDA_ACT_NONE || (L.bf16 && off_grid(dy, L.outs)));
  void *made = make ? ws : nullptr;
  if (L.rows > 0 && (make || dbias != nullptr)) {
    e = L.bf16 ? run_dz<__nv_bfloat16>(L, dy, preact, made, w.ld_dz, cols, dbias, sms, s)
               : run_dz<float>(L, dy, preact, made, w.ld_dz, cols, dbias, sms, s);
    if (e != cudaSuccess) return e;
  }
  const void *dz = make ? made : dy;
  const int64_t ld = make ? w.ld_dz : L.outs;
  if (L.rows == 0) {  // dx is empty, dweight and dbias are empty sums
    const size_t es = L.bf16 ? 2 : 4;
    if (dbias != nullptr && (e = cudaMemsetAsync(dbias, 0, es * L.outs, s)) != cudaSuccess) return e;
    return dweight == nullptr ? cudaSuccess : cudaMemsetAsync(dweight, 0, es * (size_t)L.outs * L.ins, s);
  }
  OnGrid g{{L.x, L.ins, true}, {L.weight, L.ins, true}};
  if (L.bf16) {
    e = on_grid(L, dweight != nullptr, dx != nullptr, ws + w.x, ws + w.w, sms, &g, s);
    if (e != cudaSuccess) return e;
  }
  if (dx != nullptr) {
    const Product P{L.rows, L.ins, L.outs, {dz, ld, true}, {g.w.p, g.w.ld, false}, nullptr, nullptr, KDA_ACT_NONE, dx,
                    nullptr};
    if ((e = product(P, L.bf16, part, sms, s)) != cudaSuccess) return e;
  }
  if (dweight != nullptr) {
    const Product P{L.outs, L.ins, L.rows, {dz, ld, false}, {g.x.p, g.x.ld, false}, nullptr, nullptr, KDA_ACT_NONE,
                    dweight, nullptr};
    e = product(P, L.bf16, part, sms, s);
  }
  return e;
}

}  // namespace dense
}  // namespace kda
