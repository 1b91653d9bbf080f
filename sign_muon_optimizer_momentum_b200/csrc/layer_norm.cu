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
// walk over rows, and each thread keeps its part of the next rows coming by
// asynchronous copies into a ring of its own in shared memory (no barrier:
// a thread reads back only what it copied).  The backward adds dy xh
// and dy of its rows to per-thread column sums, adds those of a block's groups
// in shared memory, and leaves one row of partial sums a block; a second
// launch adds a worker's blocks.  All sums have a fixed order.
#include "layers.cuh"

using namespace signmuon;

namespace {

constexpr int kWarpCols = 1024;       // longest row that one warp takes (32 elements a lane)
constexpr int kThreads = 256;         // threads a block where a warp or less takes a row
constexpr int kBlockElems = 16;       // elements a thread where a block takes a row
constexpr int kBlockThreads = 512;    // threads of such a block at most (8192 columns)
constexpr int kWideThreads = 512;     // rows longer still

// Rows and columns of one call.
struct NormArgs {
  int64_t rows;
  int32_t cols;
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
// A thread's part of a row: chunk c is the VEC elements from column
// (c * tpr + t) * VEC, tpr threads to a row.  Rows come through kSlots slots
// of shared memory; single bf16 (2 bytes, below what can be copied
// asynchronously) are loaded when they are needed.
template <typename T, int VEC, int E, int kSlots>
struct Rows {
  using Raw = typename RawVec<T, VEC>::type;
  static constexpr int kChunks = E / VEC;
  static constexpr bool kAsync = sizeof(Raw) >= 4;
  static constexpr size_t bytes(int threads) { return kAsync ? (size_t)kSlots * kChunks * sizeof(Raw) * threads : 0; }
  Raw* ring;
  int t, tpr, cols;
  // Slots past the last column are 0 from the start and stay so.
  __device__ __forceinline__ Rows(void* smem, int t, int tpr, int cols)
      : ring(static_cast<Raw*>(smem) + threadIdx.x), t(t), tpr(tpr), cols(cols) {
    if constexpr (kAsync) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        if ((c * tpr + t) * VEC >= cols)
#pragma unroll
          for (int i = 0; i < kSlots; ++i) ring[(i * kChunks + c) * blockDim.x] = Raw{};
    }
  }
  __device__ __forceinline__ void fetch(const T* p, int slot) const {
    if constexpr (kAsync) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int col = (c * tpr + t) * VEC;
        if (col < cols) copy_async<sizeof(Raw)>(ring + (slot * kChunks + c) * blockDim.x, p + col);
      }
    }
  }
  // Elements past the last column are 0.
  __device__ __forceinline__ void get(float (&v)[E], const T* p, int slot) const {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float u[VEC];
      if constexpr (kAsync) {
        unpack(ring[(slot * kChunks + c) * blockDim.x], u);
      } else {
        const int col = (c * tpr + t) * VEC;
        u[0] = 0.f;
        if (col < cols) unpack(load_stream<T, VEC>(p + col), u);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[c * VEC + j] = u[j];
    }
  }
};
// Slots of a ring: about 192 bytes of rows a thread, two rows at least.
template <typename T, int E>
constexpr int kRowSlots = 192 / (E * (int)sizeof(T)) < 2 ? 2 : 192 / (E * (int)sizeof(T)) > 4 ? 4 : 192 / (E * (int)sizeof(T));

// A thread's weights (zero past the last column).  Where a block takes a row:
// in registers, as they are stored (W is the type).  Where a warp or less
// takes a row, a thread has too many for that: fp32 in shared memory, each
// group of four of the kTpr lanes side by side, so that reads meet no bank
// conflict (rows of eight by lane cost twice the reads, which then bound the
// forward kernel).
template <typename W, int VEC, int E>
struct RegWeights {
  static constexpr bool kBf16 = sizeof(W) == 2;
  uint32_t reg[kBf16 ? E / 2 : E];
  __device__ __forceinline__ void load(const void* w, int, float*, int t, int tpr, int cols) {
    uint32_t v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int col = (i / VEC * tpr + t) * VEC + i % VEC;
      v[i] = w && col < cols ? __float_as_uint(load_elem(w, col, kBf16)) : 0u;
    }
#pragma unroll
    for (int i = 0; i < (kBf16 ? E / 2 : E); ++i) reg[i] = kBf16 ? v[2 * i % E] >> 16 | v[(2 * i + 1) % E] : v[i];
  }
  __device__ __forceinline__ void get(int c, float (&v)[VEC]) const {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int i = c * VEC + j;
      if constexpr (kBf16) v[j] = i % 2 ? bf16_hi(reg[i / 2]) : bf16_lo(reg[i / 2]);
      else v[j] = __uint_as_float(reg[i]);
    }
  }
};
template <int VEC, int E, int kTpr>
struct SharedWeights {
  const float* sh;  // this lane's first
  __device__ __forceinline__ void load(const void* w, int bf16, float* smem, int t, int, int cols) {
    // Element q of group g (of min(VEC, 4)) of chunk c of lane l.
    for (int col = threadIdx.x; col < E * kTpr; col += kThreads) {
      const int c = col / (kTpr * VEC), l = col / VEC % kTpr, j = col % VEC;
      smem[at(c, j) + l * kGroup] = w && col < cols ? load_elem(w, col, bf16) : 0.f;
    }
    sh = smem + t * kGroup;
  }
  static constexpr int kGroup = VEC < 4 ? VEC : 4;
  __device__ __forceinline__ static int at(int c, int j) { return (c * (VEC / kGroup) + j / kGroup) * kTpr * kGroup + j % kGroup; }
  __device__ __forceinline__ void get(int c, float (&v)[VEC]) const {
#pragma unroll
    for (int j = 0; j < VEC; j += kGroup) {
      if constexpr (kGroup == 4) {
        const float4 q = *reinterpret_cast<const float4*>(sh + at(c, j));
        v[j] = q.x, v[j + 1] = q.y, v[j + 2] = q.z, v[j + 3] = q.w;
      } else if constexpr (kGroup == 2) {
        const float2 q = *reinterpret_cast<const float2*>(sh + at(c, j));
        v[j] = q.x, v[j + 1] = q.y;
      } else {
        v[j] = sh[at(c, j)];
      }
    }
  }
};
template <typename W, int VEC, int E, int kTpr>
using Weights = std::conditional_t<kTpr == 0, RegWeights<W, VEC, E>, SharedWeights<VEC, E, kTpr>>;

// Sum over the kTpr lanes of a row's group (kTpr <= 32), or over the block
// (kTpr == 0) by way of sh.  Blocks alternate between two arrays, so that one
// barrier a sum does.
template <int kTpr>
__device__ __forceinline__ float row_sum(float v, float* sh) {
#pragma unroll
  for (int o = (kTpr ? kTpr : 32) / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (kTpr == 0) {
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x / 32] = v;
    __syncthreads();
    const float4* q = reinterpret_cast<const float4*>(sh);
    v = 0.f;
    for (int i = 0; i < (int)blockDim.x / 32; i += 4) {
      const float4 p = q[i / 4];  // zero past the block's warps
      v += (p.x + p.y) + (p.z + p.w);
    }
  }
  return v;
}

// --------------------------------------------------------------- forward
// kTpr lanes (8, 16 or 32) a row, or 0: a block a row.  The variance is taken
// about the mean, from the values in registers.
template <typename T, typename W, int VEC, int E, int kTpr>
__global__ void __launch_bounds__(kTpr ? kThreads : kBlockThreads) norm_forward_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float sh[2][kBlockThreads / 32];
  constexpr bool kBlock = kTpr == 0;
  constexpr int kSlots = kRowSlots<T, E>;
  const int tpr = kBlock ? blockDim.x : kTpr, t = threadIdx.x % tpr, cols = a.cols;
  constexpr int groups = kBlock ? 1 : kThreads / (kBlock ? 1 : kTpr);
  const float inv_cols = 1.f / (float)cols;
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.out);

  // All lanes of a warp run the same iterations (`first` is the row of the
  // warp's first lane); rows past the end are masked.
  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t row = (int64_t)blockIdx.x * groups + threadIdx.x / tpr;
  int64_t first = (int64_t)blockIdx.x * groups + threadIdx.x / 32 * 32 / tpr;
  const Rows<T, VEC, E, kSlots> in(smem, t, tpr, cols);
#pragma unroll
  for (int i = 0; i < kSlots - 1; ++i) {
    if (row + i * step < a.rows) in.fetch(x + (row + i * step) * a.ld_x, i);
    copy_commit();
  }
  float* w_sh = reinterpret_cast<float*>(smem + Rows<T, VEC, E, kSlots>::bytes(blockDim.x));
  Weights<W, VEC, E, kTpr> w, b;
  w.load(a.w, a.w_bf16, w_sh, t, tpr, cols);
  b.load(a.b, a.w_bf16, w_sh + E * kTpr, t, tpr, cols);
  if (threadIdx.x < 2 * kBlockThreads / 32) sh[0][threadIdx.x] = 0.f;
  __syncthreads();

  int slot = 0;
  for (; first < a.rows; row += step, first += step) {
    const int64_t ahead = row + (kSlots - 1) * step;
    if (ahead < a.rows) in.fetch(x + ahead * a.ld_x, slot == 0 ? kSlots - 1 : slot - 1);
    copy_commit();
    copy_wait<kSlots - 1>();
    const bool valid = row < a.rows;
    float v[E];
    in.get(v, x + (valid ? row : 0) * a.ld_x, slot);
    slot = slot == kSlots - 1 ? 0 : slot + 1;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += v[i];
    const float mean = row_sum<kTpr>(s, sh[0]) * inv_cols;
    s = 0.f;
#pragma unroll
    for (int c = 0; c < E / VEC; ++c)
      if ((c * tpr + t) * VEC < cols)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[c * VEC + j] -= mean;
          s = fmaf(v[c * VEC + j], v[c * VEC + j], s);
        }
    const float r = rsqrtf(row_sum<kTpr>(s, sh[1]) * inv_cols + a.eps);
    if (t == 0 && valid) a.mean[row] = mean, a.rstd[row] = r;
#pragma unroll
    for (int c = 0; c < E / VEC; ++c) {
      const int col = (c * tpr + t) * VEC;
      if (col < cols && valid) {
        float o[VEC], wv[VEC], bv[VEC];
        w.get(c, wv);
        b.get(c, bv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = fmaf(v[c * VEC + j] * r, wv[j], bv[j]);
        store_stream<T, VEC>(y + row * a.ld_out + col, o);
      }
    }
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
template <typename T, typename W, int VEC, int E, int kTpr>
__global__ void __launch_bounds__(kTpr ? kThreads : kBlockThreads)
norm_backward_kernel(const NormArgs a, const __grid_constant__ WorkerRows rows, const __grid_constant__ WorkerBlocks share) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float sh[2][2][kBlockThreads / 32];
  constexpr bool kBlock = kTpr == 0;
  constexpr int kSlots = kRowSlots<T, 2 * E>;
  const int tpr = kBlock ? blockDim.x : kTpr, t = threadIdx.x % tpr, cols = a.cols;
  constexpr int groups = kBlock ? 1 : kThreads / (kBlock ? 1 : kTpr);
  const int m = worker_of_block(share, a.n_workers, blockIdx.x);
  const int blocks = share.begin[m + 1] - share.begin[m];
  const float inv_cols = 1.f / (float)cols;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  T* dx = static_cast<T*>(a.out);

  const int64_t step = (int64_t)blocks * groups, end = rows.begin[m + 1];
  int64_t first = rows.begin[m] + (int64_t)(blockIdx.x - share.begin[m]) * groups;
  int64_t row = first + threadIdx.x / tpr;
  first += threadIdx.x / 32 * 32 / tpr;
  using Ring = Rows<T, VEC, E, kSlots>;
  const Ring in_x(smem, t, tpr, cols), in_g(smem + Ring::bytes(blockDim.x), t, tpr, cols);
#pragma unroll
  for (int i = 0; i < kSlots - 1; ++i) {
    if (row + i * step < end) in_x.fetch(x + (row + i * step) * a.ld_x, i), in_g.fetch(dy + (row + i * step) * a.ld_dy, i);
    copy_commit();
  }
  float mean_next = 0.f, r_next = 0.f;
  if (row < end) mean_next = a.mean[row], r_next = a.rstd[row];
  Weights<W, VEC, E, kTpr> w;
  w.load(a.w, a.w_bf16, reinterpret_cast<float*>(smem + 2 * Ring::bytes(blockDim.x)), t, tpr, cols);
  if (threadIdx.x < 4 * kBlockThreads / 32) sh[0][0][threadIdx.x] = 0.f;
  __syncthreads();

  float dw[E], db[E];
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.f;
  int slot = 0;
  for (int it = 0; first < end; row += step, first += step, it ^= 1) {
    const int64_t ahead = row + (kSlots - 1) * step;
    if (ahead < end) {
      const int to = slot == 0 ? kSlots - 1 : slot - 1;
      in_x.fetch(x + ahead * a.ld_x, to), in_g.fetch(dy + ahead * a.ld_dy, to);
    }
    copy_commit();
    const float mean = mean_next, r = r_next;
    if (row + step < end) mean_next = a.mean[row + step], r_next = a.rstd[row + step];
    copy_wait<kSlots - 1>();
    const bool valid = row < end;
    float xh[E], g[E], s1 = 0.f, s2 = 0.f;
    in_x.get(xh, x + (valid ? row : 0) * a.ld_x, slot);
    in_g.get(g, dy + (valid ? row : 0) * a.ld_dy, slot);
    slot = slot == kSlots - 1 ? 0 : slot + 1;
#pragma unroll
    for (int c = 0; c < E / VEC; ++c) {
      const int col = (c * tpr + t) * VEC;
      if (col < cols && valid) {
        float wv[VEC];
        w.get(c, wv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int i = c * VEC + j;
          xh[i] = (xh[i] - mean) * r;
          db[i] += g[i];
          dw[i] = fmaf(g[i], xh[i], dw[i]);
          g[i] *= wv[j];
          s1 += g[i];
          s2 = fmaf(g[i], xh[i], s2);
        }
      }
    }
    if constexpr (kBlock) {
      // Both sums with one barrier; the arrays alternate by rows.
      s1 = warp_sum(s1);
      s2 = warp_sum(s2);
      if ((threadIdx.x & 31) == 0) sh[it][0][threadIdx.x / 32] = s1, sh[it][1][threadIdx.x / 32] = s2;
      __syncthreads();
      s1 = s2 = 0.f;
      for (int i = 0; i < (int)blockDim.x / 32; i += 4) {
        const float4 p = *reinterpret_cast<const float4*>(&sh[it][0][i]), q = *reinterpret_cast<const float4*>(&sh[it][1][i]);
        s1 += (p.x + p.y) + (p.z + p.w);
        s2 += (q.x + q.y) + (q.z + q.w);
      }
    } else {
      s1 = row_sum<kTpr>(s1, nullptr);
      s2 = row_sum<kTpr>(s2, nullptr);
    }
    const float c1 = -r * s1 * inv_cols, c2 = -r * s2 * inv_cols;
#pragma unroll
    for (int c = 0; c < E / VEC; ++c) {
      const int col = (c * tpr + t) * VEC;
      if (col < cols && valid) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = fmaf(xh[c * VEC + j], c2, fmaf(g[c * VEC + j], r, c1));
        store_stream<T, VEC>(dx + row * a.ld_out + col, o);
      }
    }
  }

  // The block's partial sums.
  const int sums = a.has_bias ? 2 : 1;
  float* part = a.part + (int64_t)blockIdx.x * sums * cols;
  if constexpr (kBlock) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int col = (i / VEC * tpr + t) * VEC + i % VEC;
      if (col < cols) {
        part[col] = dw[i];
        if (a.has_bias) part[cols + col] = db[i];
      }
    }
  } else {
    // Every group's in shared memory (over the rings and weights), then added
    // by column in the groups' order; one sum after the other, which bounds
    // the room at 4 kThreads E bytes.
    float* all = reinterpret_cast<float*>(smem);
    constexpr int kCols = kTpr * E;
    for (int q = 0; q < sums; ++q) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int col = (i / VEC * kTpr + t) * VEC + i % VEC;
        all[threadIdx.x / kTpr * kCols + col] = q ? db[i] : dw[i];
      }
      __syncthreads();
      for (int col = threadIdx.x; col < cols; col += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int g = 0; g < groups; ++g) s += all[g * kCols + col];
        part[q * cols + col] = s;
      }
    }
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
template <int N>
using Int = std::integral_constant<int, N>;
// f(elements a lane, lanes a row) for the kernels where a warp or less takes
// a row: as few lanes as hold it with 8 elements each, then more elements.
template <typename F>
void by_lanes(int cols, F f) {
  if (cols <= 64) f(Int<8>(), Int<8>());
  else if (cols <= 128) f(Int<8>(), Int<16>());
  else if (cols <= 256) f(Int<8>(), Int<32>());
  else if (cols <= 512) f(Int<16>(), Int<32>());
  else if (cols <= 768) f(Int<24>(), Int<32>());
  else f(Int<32>(), Int<32>());
}
template <typename F>
void by_weight(int bf16, F f) {
  if (bf16) f(__nv_bfloat16());
  else f(float());
}
int block_threads(int cols) { return (int)round_up((size_t)ceil_div(cols, kBlockElems), 32); }

template <typename T, int VEC>
void forward_launch(const NormArgs& a, int sms, cudaStream_t st) {
  auto grid = [&](int64_t rows_a_block, int64_t blocks_an_sm) {
    const int64_t n = ceil_div(a.rows, rows_a_block), most = sms * blocks_an_sm;
    return (unsigned)(n < most ? n : most);
  };
  const int threads = block_threads(a.cols);
  if (a.cols <= kWarpCols)
    by_lanes(a.cols, [&](auto e, auto lanes) {
      constexpr int kE = decltype(e)::value, kTpr = decltype(lanes)::value;
      constexpr auto k = norm_forward_kernel<T, float, VEC, kE, kTpr>;
      const size_t smem = Rows<T, VEC, kE, kRowSlots<T, kE>>::bytes(kThreads) + 2 * 4 * kE * kTpr;
      k<<<grid(kThreads / kTpr, resident_blocks<k>(kThreads, smem)), kThreads, smem, st>>>(a);
    });
  else if (threads <= kBlockThreads) {
    const size_t smem = Rows<T, VEC, kBlockElems, kRowSlots<T, kBlockElems>>::bytes(threads);
    by_weight(a.w_bf16, [&](auto w) {
      constexpr auto k = norm_forward_kernel<T, decltype(w), VEC, kBlockElems, 0>;
      k<<<grid(1, resident_blocks<k>(threads, smem)), threads, smem, st>>>(a);
    });
  } else {
    norm_forward_wide_kernel<T, VEC><<<grid(1, 4), kWideThreads, 0, st>>>(a);
  }
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

constexpr int kBwdBlocksPerSm = 8;
// Of blocks at most: those of every SM, and one more for each worker whose
// share rounds to none.
int bwd_max_blocks(int sms, int n_workers) { return sms * kBwdBlocksPerSm + n_workers; }

template <typename T, int VEC>
void backward_launch(const NormArgs& a, const WorkerRows& rows, const int64_t* row_begin, int sms, WorkerBlocks* share,
                     cudaStream_t st) {
  auto blocks = [&](int rows_a_block, int blocks_an_sm) {
    return block_share(a.n_workers, row_begin, rows_a_block,
                       sms * (blocks_an_sm < kBwdBlocksPerSm ? blocks_an_sm : kBwdBlocksPerSm), share);
  };
  const int threads = block_threads(a.cols);
  if (!a.rows) return;
  if (a.cols <= kWarpCols)
    by_lanes(a.cols, [&](auto e, auto lanes) {
      constexpr int kE = decltype(e)::value, kTpr = decltype(lanes)::value;
      constexpr auto k = norm_backward_kernel<T, float, VEC, kE, kTpr>;
      const size_t rings = 2 * Rows<T, VEC, kE, kRowSlots<T, 2 * kE>>::bytes(kThreads) + 4 * kE * kTpr;
      const size_t sums = 4 * kThreads * kE, smem = rings > sums ? rings : sums;
      const int n = blocks(kThreads / kTpr, resident_blocks<k>(kThreads, smem));
      k<<<n, kThreads, smem, st>>>(a, rows, *share);
    });
  else if (threads <= kBlockThreads) {
    const size_t smem = 2 * Rows<T, VEC, kBlockElems, kRowSlots<T, 2 * kBlockElems>>::bytes(threads);
    by_weight(a.w_bf16, [&](auto w) {
      constexpr auto k = norm_backward_kernel<T, decltype(w), VEC, kBlockElems, 0>;
      const int n = blocks(1, resident_blocks<k>(threads, smem));
      k<<<n, threads, smem, st>>>(a, rows, *share);
    });
  } else {
    const int64_t most = (int64_t)sms * 4;
    norm_backward_wide_kernel<T, VEC><<<(unsigned)(a.rows < most ? a.rows : most), kWideThreads, 0, st>>>(a);
    const int n = blocks(64, 1);
    norm_columns_kernel<T><<<dim3((unsigned)n, (unsigned)ceil_div(a.cols, 32)), 256, 0, st>>>(a, rows, *share);
  }
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
  by_vec(x_dtype, vec, [&](auto t, auto v) {
    forward_launch<decltype(t), decltype(v)::value>(a, current_sms(), static_cast<cudaStream_t>(stream));
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
  WorkerRows rows = {};
  for (int m = 0; m <= n_workers; ++m) rows.begin[m] = row_begin[m];
  WorkerBlocks share = {};
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  by_vec(x_dtype, vec, [&](auto t, auto v) {
    backward_launch<decltype(t), decltype(v)::value>(a, rows, row_begin, current_sms(), &share, cs);
  });
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_status(e);
  norm_finalize_kernel<<<dim3((unsigned)ceil_div(cols, 32), (unsigned)n_workers, dbias ? 2u : 1u), 256, 0, cs>>>(
      a.part, cols, dbias ? 2 : 1, a.w_bf16, share, dw, db);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
