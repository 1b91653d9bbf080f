// Layer norm over rows, forward and backward, with the gradients of its
// weight and bias reduced per worker.
//
//   forward    mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps)
//              y = (x - mu) r w + b
//   backward   xh = (x - mu) r, g = dy w
//              dx = r (g - mean(g) - xh mean(g xh))
//              dw[m] = sum over worker m's rows of dy xh,  db[m] = sum of dy
//
// All of it is bound by memory: forward reads x and writes y, backward reads
// x and dy and writes dx, each once.  A row is held in the registers of the
// group of threads that works on it (kE elements a thread), so both of the
// variance's passes and the backward's two sums cost no second read; groups
// walk over rows with the next row's loads in flight.  The backward adds dy xh
// and dy of its rows to per-thread column sums, adds those of a block's groups
// in shared memory, and leaves one row of partial sums a block; a second
// launch adds a worker's blocks.  All sums have a fixed order.
#include "layers.cuh"

using namespace signmuon;

namespace {

constexpr int kMaxThreads = 1024;     // forward: threads a block at most
constexpr int kBwdThreads = 512;      // backward: its column sums need up to 128 registers a thread
constexpr int kGroupThreads = 256;    // threads a block where a row needs fewer
constexpr int kWideThreads = 512;     // rows too long for registers

// Rows and columns of one call.
struct NormArgs {
  int64_t rows;
  int32_t cols, tpr;                  // threads a row (a multiple of 32)
  const void* x;
  const void* dy;
  void* out;                          // y or dx
  int64_t ld_x, ld_dy, ld_out;
  const void* w;
  const void* b;
  int32_t w_bf16;
  float eps;
  float* mean;
  float* rstd;
  float* part;                        // backward: [blocks][sums][cols]
  int32_t n_workers, has_bias;
};
// Barrier of one group of a block (1 .. 8; 0 is __syncthreads').
__device__ __forceinline__ void group_sync(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

template <typename T, int VEC, int E>
struct Row {
  static constexpr int kChunks = E / VEC;
  typename RawVec<T, VEC>::type raw[kChunks];
  __device__ __forceinline__ void load(const T* p, int t, int tpr, int cols) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int col = (c * tpr + t) * VEC;
      if (col < cols) raw[c] = load_stream<T, VEC>(p + col);
    }
  }
  // Elements past the last column are 0.
  __device__ __forceinline__ void get(float (&v)[E], int t, int tpr, int cols) const {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float u[VEC];
      unpack(raw[c], u);
      const bool in = (c * tpr + t) * VEC < cols;
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[c * VEC + j] = in ? u[j] : 0.f;
    }
  }
};

template <int VEC, int E>
__device__ __forceinline__ void load_weights(const void* w, int bf16, int t, int tpr, int cols, float (&v)[E]) {
#pragma unroll
  for (int c = 0; c < E / VEC; ++c)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int col = (c * tpr + t) * VEC + j;
      v[c * VEC + j] = col < cols ? load_elem(w, col, bf16) : 0.f;
    }
}

// --------------------------------------------------------------- forward
// The variance is centred: each warp takes its part's own mean and sum of
// squares about it, and the parts are joined as
//   M2 = sum M2_i + sum n_i (mu_i - mu)^2
// so that one exchange through shared memory serves both passes.
template <typename T, int VEC, int E>
__global__ void __launch_bounds__(kMaxThreads) norm_forward_kernel(const NormArgs a) {
  __shared__ float2 sh[2][32];
  __shared__ float sh_n[32];  // elements of a row that each warp of a group holds
  const int tpr = a.tpr, t = threadIdx.x % tpr, group = threadIdx.x / tpr, groups = blockDim.x / tpr;
  const int lane = threadIdx.x & 31, warps = tpr / 32, w0 = group * warps, cols = a.cols;
  float w[E], b[E];
  load_weights<VEC, E>(a.w, a.w_bf16, t, tpr, cols, w);
  if (a.b) load_weights<VEC, E>(a.b, a.w_bf16, t, tpr, cols, b);
  else
#pragma unroll
    for (int i = 0; i < E; ++i) b[i] = 0.f;
  float mine = 0.f;  // this thread's elements
#pragma unroll
  for (int c = 0; c < E / VEC; ++c) mine += (c * tpr + t) * VEC < cols ? (float)VEC : 0.f;
  const float n_warp = warp_sum(mine), inv_cols = 1.f / (float)cols;
  if (threadIdx.x < tpr && lane == 0) sh_n[threadIdx.x / 32] = n_warp;
  __syncthreads();
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.out);

  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t row = (int64_t)blockIdx.x * groups + group;
  Row<T, VEC, E> cur, next;
  if (row < a.rows) cur.load(x + row * a.ld_x, t, tpr, cols);
  for (int it = 0; row < a.rows; row += step, it ^= 1) {
    if (row + step < a.rows) next.load(x + (row + step) * a.ld_x, t, tpr, cols);
    float v[E];
    cur.get(v, t, tpr, cols);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += v[i];
    s = warp_sum(s);
    float mean = warps == 1 ? s * inv_cols : n_warp > 0.f ? s / n_warp : 0.f;
    float m2 = 0.f;
#pragma unroll
    for (int c = 0; c < E / VEC; ++c)
      if ((c * tpr + t) * VEC < cols)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d = v[c * VEC + j] - mean;
          m2 = fmaf(d, d, m2);
        }
    m2 = warp_sum(m2);
    if (warps > 1) {
      if (lane == 0) sh[it][threadIdx.x / 32] = make_float2(s, m2);
      group_sync(group, tpr);
      float total = 0.f;
      for (int i = 0; i < warps; ++i) total += sh[it][w0 + i].x;
      mean = total * inv_cols;
      m2 = 0.f;
      for (int i = 0; i < warps; ++i) {
        const float n = sh_n[i];
        if (n > 0.f) {
          const float2 p = sh[it][w0 + i];
          const float d = __fdividef(p.x, n) - mean;
          m2 += p.y + n * d * d;
        }
      }
    }
    const float r = rsqrtf(m2 * inv_cols + a.eps);
    if (t == 0) a.mean[row] = mean, a.rstd[row] = r;
#pragma unroll
    for (int c = 0; c < E / VEC; ++c) {
      const int col = (c * tpr + t) * VEC;
      if (col < cols) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = fmaf((v[c * VEC + j] - mean) * r, w[c * VEC + j], b[c * VEC + j]);
        store_stream<T, VEC>(y + row * a.ld_out + col, o);
      }
    }
    cur = next;
  }
}

// Sum over the block in a fixed order (every thread gets it).
__device__ __forceinline__ float block_sum(float v, float* sh) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < (int)blockDim.x / 32; ++i) s += sh[i];
  return s;
}

// Rows longer than a block's registers hold: one block a row, which reads it
// three times (the second and third time mostly from L2).
template <typename T, int VEC>
__global__ void __launch_bounds__(kWideThreads) norm_forward_wide_kernel(const NormArgs a) {
  __shared__ float sh[32];
  const int cols = a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    T* y = static_cast<T*>(a.out) + row * a.ld_out;
    float u[VEC], s = 0.f;
    for (int col = threadIdx.x * VEC; col < cols; col += kWideThreads * VEC) {
      unpack(*reinterpret_cast<const typename RawVec<T, VEC>::type*>(x + col), u);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += u[j];
    }
    const float mean = block_sum(s, sh) / (float)cols;
    s = 0.f;
    for (int col = threadIdx.x * VEC; col < cols; col += kWideThreads * VEC) {
      unpack(*reinterpret_cast<const typename RawVec<T, VEC>::type*>(x + col), u);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s = fmaf(u[j] - mean, u[j] - mean, s);
    }
    const float r = rsqrtf(block_sum(s, sh) / (float)cols + a.eps);
    if (threadIdx.x == 0) a.mean[row] = mean, a.rstd[row] = r;
    for (int col = threadIdx.x * VEC; col < cols; col += kWideThreads * VEC) {
      unpack(*reinterpret_cast<const typename RawVec<T, VEC>::type*>(x + col), u);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        u[j] = fmaf((u[j] - mean) * r, load_elem(a.w, col + j, a.w_bf16), a.b ? load_elem(a.b, col + j, a.w_bf16) : 0.f);
      store_stream<T, VEC>(y + col, u);
    }
  }
}

// -------------------------------------------------------------- backward
template <typename T, int VEC, int E>
__global__ void __launch_bounds__(kBwdThreads)
norm_backward_kernel(const NormArgs a, const __grid_constant__ WorkerRows rows, const __grid_constant__ WorkerBlocks share) {
  extern __shared__ float cols_sh[];  // [sums][cols] (blocks of more than one group)
  __shared__ float2 sh[2][32];
  const int tpr = a.tpr, t = threadIdx.x % tpr, group = threadIdx.x / tpr, groups = blockDim.x / tpr;
  const int lane = threadIdx.x & 31, warps = tpr / 32, w0 = group * warps, cols = a.cols;
  const int m = worker_of_block(share, a.n_workers, blockIdx.x);
  const int blocks = share.begin[m + 1] - share.begin[m];
  float w[E], dw[E], db[E];
  load_weights<VEC, E>(a.w, a.w_bf16, t, tpr, cols, w);
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.f;
  const float inv_cols = 1.f / (float)cols;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  T* dx = static_cast<T*>(a.out);

  const int64_t step = (int64_t)blocks * groups, end = rows.begin[m + 1];
  int64_t row = rows.begin[m] + (int64_t)(blockIdx.x - share.begin[m]) * groups + group;
  Row<T, VEC, E> cx, cg, nx, ng;
  float mean = 0.f, r = 0.f, mean_next = 0.f, r_next = 0.f;
  if (row < end) {
    cx.load(x + row * a.ld_x, t, tpr, cols);
    cg.load(dy + row * a.ld_dy, t, tpr, cols);
    mean = a.mean[row], r = a.rstd[row];
  }
  for (int it = 0; row < end; row += step, it ^= 1) {
    if (row + step < end) {
      nx.load(x + (row + step) * a.ld_x, t, tpr, cols);
      ng.load(dy + (row + step) * a.ld_dy, t, tpr, cols);
      mean_next = a.mean[row + step], r_next = a.rstd[row + step];
    }
    float xh[E], g[E], s1 = 0.f, s2 = 0.f;
    cx.get(xh, t, tpr, cols);
    cg.get(g, t, tpr, cols);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      xh[i] = (xh[i] - mean) * r;  // past the last column g is 0, so this drops out
      db[i] += g[i];
      dw[i] += (i / VEC * tpr + t) * VEC < cols ? g[i] * xh[i] : 0.f;
      g[i] *= w[i];
      s1 += g[i];
      s2 += (i / VEC * tpr + t) * VEC < cols ? g[i] * xh[i] : 0.f;
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (warps > 1) {
      if (lane == 0) sh[it][threadIdx.x / 32] = make_float2(s1, s2);
      group_sync(group, tpr);
      s1 = s2 = 0.f;
      for (int i = 0; i < warps; ++i) {
        const float2 p = sh[it][w0 + i];
        s1 += p.x;
        s2 += p.y;
      }
    }
    s1 *= inv_cols;
    s2 *= inv_cols;
#pragma unroll
    for (int c = 0; c < E / VEC; ++c) {
      const int col = (c * tpr + t) * VEC;
      if (col < cols) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = r * (g[c * VEC + j] - s1 - xh[c * VEC + j] * s2);
        store_stream<T, VEC>(dx + row * a.ld_out + col, o);
      }
    }
    cx = nx, cg = ng, mean = mean_next, r = r_next;
  }

  // The block's partial sums: its groups one after another.
  const int sums = a.has_bias ? 2 : 1;
  float* part = a.part + (int64_t)blockIdx.x * sums * cols;
  float* acc = groups > 1 ? cols_sh : part;
  for (int g = 0; g < groups; ++g) {
    if (g) __syncthreads();
    if (g == group)
#pragma unroll
      for (int c = 0; c < E / VEC; ++c)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int col = (c * tpr + t) * VEC + j;
          if (col < cols) {
            acc[col] = (g ? acc[col] : 0.f) + dw[c * VEC + j];
            if (a.has_bias) acc[cols + col] = (g ? acc[cols + col] : 0.f) + db[c * VEC + j];
          }
        }
  }
  if (groups > 1) {
    __syncthreads();
    for (int i = threadIdx.x; i < sums * cols; i += blockDim.x) part[i] = cols_sh[i];
  }
}

// Rows longer than a block's registers hold: dx by a block a row, which reads
// dy and x twice.
template <typename T, int VEC>
__global__ void __launch_bounds__(kWideThreads) norm_backward_wide_kernel(const NormArgs a) {
  __shared__ float sh[32];
  const int cols = a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy;
    T* dx = static_cast<T*>(a.out) + row * a.ld_out;
    const float mean = a.mean[row], r = a.rstd[row];
    float u[VEC], g[VEC], s1 = 0.f, s2 = 0.f;
    for (int col = threadIdx.x * VEC; col < cols; col += kWideThreads * VEC) {
      unpack(*reinterpret_cast<const typename RawVec<T, VEC>::type*>(x + col), u);
      unpack(*reinterpret_cast<const typename RawVec<T, VEC>::type*>(dy + col), g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float q = g[j] * load_elem(a.w, col + j, a.w_bf16);
        s1 += q;
        s2 = fmaf(q, (u[j] - mean) * r, s2);
      }
    }
    s1 = block_sum(s1, sh) / (float)cols;
    s2 = block_sum(s2, sh) / (float)cols;
    for (int col = threadIdx.x * VEC; col < cols; col += kWideThreads * VEC) {
      unpack(*reinterpret_cast<const typename RawVec<T, VEC>::type*>(x + col), u);
      unpack(*reinterpret_cast<const typename RawVec<T, VEC>::type*>(dy + col), g);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        u[j] = r * (g[j] * load_elem(a.w, col + j, a.w_bf16) - s1 - (u[j] - mean) * r * s2);
      store_stream<T, VEC>(dx + col, u);
    }
  }
}

// ... and the column sums by blocks of 32 columns x 8 warps over the rows that
// a block of the other kernel would have had.
template <typename T>
__global__ void __launch_bounds__(256)
norm_columns_kernel(const NormArgs a, const __grid_constant__ WorkerRows rows, const __grid_constant__ WorkerBlocks share) {
  __shared__ float sh[2][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, cols = a.cols, col = blockIdx.y * 32 + lane;
  const int m = worker_of_block(share, a.n_workers, blockIdx.x);
  const int blocks = share.begin[m + 1] - share.begin[m];
  float dw = 0.f, db = 0.f;
  if (col < cols)
    for (int64_t row = rows.begin[m] + (int64_t)(blockIdx.x - share.begin[m]) * 8 + warp; row < rows.begin[m + 1];
         row += (int64_t)blocks * 8) {
      float u[1], g[1];
      unpack(*reinterpret_cast<const typename RawVec<T, 1>::type*>(static_cast<const T*>(a.x) + row * a.ld_x + col), u);
      unpack(*reinterpret_cast<const typename RawVec<T, 1>::type*>(static_cast<const T*>(a.dy) + row * a.ld_dy + col), g);
      db += g[0];
      dw = fmaf(g[0], (u[0] - a.mean[row]) * a.rstd[row], dw);
    }
  sh[0][warp][lane] = dw;
  sh[1][warp][lane] = db;
  __syncthreads();
  const int sums = a.has_bias ? 2 : 1;
  if (warp < sums && col < cols) {
    float s = 0.f;
    for (int i = 0; i < 8; ++i) s += sh[warp][i][lane];
    a.part[((int64_t)blockIdx.x * sums + warp) * cols + col] = s;
  }
}

// Adds a worker's blocks: 32 columns a block, 8 warps each taking every
// eighth block's row.
__global__ void __launch_bounds__(256)
norm_finalize_kernel(const float* part, int cols, int sums, int w_bf16, const __grid_constant__ WorkerBlocks share,
                     const __grid_constant__ WorkerPtrs dw, const __grid_constant__ WorkerPtrs db) {
  __shared__ float sh[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, col = blockIdx.x * 32 + lane;
  const int m = blockIdx.y, which = blockIdx.z;
  float s = 0.f;
  if (col < cols)
#pragma unroll 4
    for (int b = share.begin[m] + warp; b < share.begin[m + 1]; b += 8) s += part[((int64_t)b * sums + which) * cols + col];
  sh[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < cols) {
    s = 0.f;
    for (int i = 0; i < 8; ++i) s += sh[i][lane];
    store_elem(which ? db.p[m] : dw.p[m], col, w_bf16, s);
  }
}

// ------------------------------------------------------------------ host
// Elements a thread holds and threads a row for rows of `cols` elements:
// 8 elements up to `threads` x 8 columns, else 16; 0 where a block's threads
// cannot hold the row.
struct RowShape {
  int e, tpr;
};
RowShape row_shape(int cols, int threads, int vec) {
  RowShape s;
  s.e = cols <= 8 * kGroupThreads ? 8 : 16;
  if (s.e < vec) s.e = vec;
  s.tpr = (cols + 32 * s.e - 1) / (32 * s.e) * 32;
  if (s.tpr > threads) s.e = 0;
  return s;
}
int groups_of(int tpr) { return tpr >= kGroupThreads ? 1 : kGroupThreads / tpr; }

template <typename T, int VEC>
void forward_launch(const NormArgs& a, RowShape s, int sms, cudaStream_t st) {
  if (!s.e) {
    const int64_t grid = a.rows < (int64_t)sms * 4 ? a.rows : (int64_t)sms * 4;
    norm_forward_wide_kernel<T, VEC><<<(unsigned)grid, kWideThreads, 0, st>>>(a);
    return;
  }
  const int groups = groups_of(s.tpr), threads = groups * s.tpr;
  int64_t grid = ceil_div(a.rows, groups);
  const int64_t most = (int64_t)sms * (1024 / threads > 0 ? 1024 / threads : 1);
  if (grid > most) grid = most;
  if (s.e == 8) norm_forward_kernel<T, VEC, 8><<<(unsigned)grid, threads, 0, st>>>(a);
  else norm_forward_kernel<T, VEC, 16><<<(unsigned)grid, threads, 0, st>>>(a);
}

// Blocks of the backward pass, shared out over the workers by their rows: a
// worker with rows has at least one.
int block_share(int n_workers, const int64_t* row_begin, int groups, int most, WorkerBlocks* share) {
  const int64_t rows = row_begin[n_workers];
  int n = 0;
  for (int m = 0; m < n_workers; ++m) {
    const int64_t mine = row_begin[m + 1] - row_begin[m];
    int64_t b = rows ? (int64_t)((double)mine / (double)rows * most) : 0;
    const int64_t useful = ceil_div(mine, groups);
    if (b > useful) b = useful;
    if (b < 1 && mine > 0) b = 1;
    share->begin[m] = n;
    n += (int)b;
  }
  share->begin[n_workers] = n;
  return n;
}

constexpr int kBwdBlocksPerSm = 2;
// Of blocks at most: those of every SM, and one more for each worker whose
// share rounds to none.
int bwd_max_blocks(int sms, int n_workers) { return sms * kBwdBlocksPerSm + n_workers; }

template <typename T, int VEC>
void backward_launch(const NormArgs& a, RowShape s, const WorkerRows& rows, const int64_t* row_begin, int sms,
                     WorkerBlocks* share, cudaStream_t st) {
  if (!s.e) {
    block_share(a.n_workers, row_begin, 64, sms, share);
    const int blocks = share->begin[a.n_workers];
    const int64_t grid = a.rows < (int64_t)sms * 4 ? a.rows : (int64_t)sms * 4;
    if (a.rows) {
      norm_backward_wide_kernel<T, VEC><<<(unsigned)grid, kWideThreads, 0, st>>>(a);
      norm_columns_kernel<T><<<dim3((unsigned)blocks, (unsigned)ceil_div(a.cols, 32)), 256, 0, st>>>(a, rows, *share);
    }
    return;
  }
  const int groups = groups_of(s.tpr), threads = groups * s.tpr;
  const int blocks = block_share(a.n_workers, row_begin, groups, sms * kBwdBlocksPerSm, share);
  if (!blocks) return;
  const size_t smem = groups > 1 ? (size_t)(a.has_bias ? 2 : 1) * a.cols * 4 : 0;  // at most 16 KB
  if (s.e == 8) norm_backward_kernel<T, VEC, 8><<<blocks, threads, smem, st>>>(a, rows, *share);
  else norm_backward_kernel<T, VEC, 16><<<blocks, threads, smem, st>>>(a, rows, *share);
}

template <typename F>
void by_vec(signmuon_dtype t, int vec, F f) {
  using bf16 = __nv_bfloat16;
  if (t == SIGNMUON_F32) vec == 4 ? f(float(), std::integral_constant<int, 4>()) : f(float(), std::integral_constant<int, 1>());
  else if (vec == 8) f(bf16(), std::integral_constant<int, 8>());
  else if (vec == 2) f(bf16(), std::integral_constant<int, 2>());
  else f(bf16(), std::integral_constant<int, 1>());
}

}  // namespace

extern "C" {

signmuon_status signmuon_layer_norm_forward(int64_t rows, int32_t cols, signmuon_dtype x_dtype, const void* x,
                                            int64_t ld_x, signmuon_dtype w_dtype, const void* weight, const void* bias,
                                            float eps, void* y, int64_t ld_y, float* mean, float* rstd, void* stream) {
  if (cols > kMaxCols) return SIGNMUON_ERR_UNSUPPORTED;
  if (rows < 0 || cols <= 0 || !known_dtype(x_dtype) || !known_dtype(w_dtype) || !weight || ld_x < cols || ld_y < cols ||
      !(eps >= 0.f))
    return SIGNMUON_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !y || !mean || !rstd)) return SIGNMUON_ERR_INVALID_ARG;
  const int xb = dtype_bytes(x_dtype), wb = dtype_bytes(w_dtype);
  if (!aligned_to(x, xb) || !aligned_to(y, xb) || !aligned_to(weight, wb) || !aligned_to(bias, wb) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return SIGNMUON_ERR_ALIGNMENT;
  if (!rows) return SIGNMUON_OK;
  int vec = vec_width(x_dtype, cols);
  vec = vec_narrow(vec, x_dtype, x, ld_x);
  vec = vec_narrow(vec, x_dtype, y, ld_y);
  NormArgs a = {};
  a.rows = rows, a.cols = cols, a.x = x, a.out = y, a.ld_x = ld_x, a.ld_out = ld_y, a.w = weight, a.b = bias;
  a.w_bf16 = w_dtype == SIGNMUON_BF16, a.eps = eps, a.mean = mean, a.rstd = rstd;
  const RowShape s = row_shape(cols, kMaxThreads, vec);
  a.tpr = s.tpr;
  by_vec(x_dtype, vec, [&](auto t, auto v) {
    forward_launch<decltype(t), decltype(v)::value>(a, s, current_sms(), static_cast<cudaStream_t>(stream));
  });
  return cuda_status(cudaGetLastError());
}

size_t signmuon_layer_norm_backward_workspace_bytes(int32_t cols, int n_workers, const int64_t* row_begin) {
  if (cols <= 0 || n_workers <= 0 || n_workers > SIGNMUON_MAX_WORKERS || !row_begin ||
      !valid_splits(row_begin, n_workers, row_begin[n_workers]))
    return 0;
  return kWsHeaderBytes + round_up((size_t)bwd_max_blocks(current_sms(), n_workers) * 2 * cols * 4, 256);
}

signmuon_status signmuon_layer_norm_backward(int32_t cols, int n_workers, const int64_t* row_begin,
                                             signmuon_dtype x_dtype, const void* dy, int64_t ld_dy, const void* x,
                                             int64_t ld_x, signmuon_dtype w_dtype, const void* weight,
                                             const float* mean, const float* rstd, void* dx, int64_t ld_dx,
                                             void* const* dweight, void* const* dbias, void* workspace,
                                             size_t ws_bytes, void* stream) {
  if (cols > kMaxCols) return SIGNMUON_ERR_UNSUPPORTED;
  if (cols <= 0 || n_workers <= 0 || n_workers > SIGNMUON_MAX_WORKERS || !row_begin ||
      !valid_splits(row_begin, n_workers, row_begin[n_workers]) || !known_dtype(x_dtype) || !known_dtype(w_dtype) ||
      !weight || !dweight || ld_dy < cols || ld_x < cols || ld_dx < cols)
    return SIGNMUON_ERR_INVALID_ARG;
  const int64_t n = row_begin[n_workers];
  if (n > 0 && (!dy || !x || !mean || !rstd || !dx)) return SIGNMUON_ERR_INVALID_ARG;
  const int xb = dtype_bytes(x_dtype), wb = dtype_bytes(w_dtype);
  if (!aligned_to(dy, xb) || !aligned_to(x, xb) || !aligned_to(dx, xb) || !aligned_to(weight, wb) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return SIGNMUON_ERR_ALIGNMENT;
  WorkerPtrs dw = {}, db = {};
  for (int m = 0; m < n_workers; ++m) {
    dw.p[m] = dweight[m];
    if (dbias) db.p[m] = dbias[m];
    if (!dw.p[m] || (dbias && !db.p[m])) return SIGNMUON_ERR_INVALID_ARG;
    if (!aligned_to(dw.p[m], wb) || !aligned_to(db.p[m], wb)) return SIGNMUON_ERR_ALIGNMENT;
  }
  const signmuon_status st =
      check_ws(workspace, ws_bytes, signmuon_layer_norm_backward_workspace_bytes(cols, n_workers, row_begin));
  if (st) return st;
  int vec = vec_width(x_dtype, cols);
  vec = vec_narrow(vec, x_dtype, x, ld_x);
  vec = vec_narrow(vec, x_dtype, dy, ld_dy);
  vec = vec_narrow(vec, x_dtype, dx, ld_dx);
  NormArgs a = {};
  a.rows = n, a.cols = cols, a.x = x, a.dy = dy, a.out = dx, a.ld_x = ld_x, a.ld_dy = ld_dy, a.ld_out = ld_dx;
  a.w = weight, a.w_bf16 = w_dtype == SIGNMUON_BF16, a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWsHeaderBytes);
  a.n_workers = n_workers, a.has_bias = dbias != nullptr;
  const RowShape s = row_shape(cols, kBwdThreads, vec);
  a.tpr = s.tpr;
  WorkerRows rows = {};
  for (int m = 0; m <= n_workers; ++m) rows.begin[m] = row_begin[m];
  WorkerBlocks share = {};
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  by_vec(x_dtype, vec, [&](auto t, auto v) {
    backward_launch<decltype(t), decltype(v)::value>(a, s, rows, row_begin, current_sms(), &share, cs);
  });
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_status(e);
  norm_finalize_kernel<<<dim3((unsigned)ceil_div(cols, 32), (unsigned)n_workers, dbias ? 2u : 1u), 256, 0, cs>>>(
      a.part, cols, dbias ? 2 : 1, a.w_bf16, share, dw, db);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
