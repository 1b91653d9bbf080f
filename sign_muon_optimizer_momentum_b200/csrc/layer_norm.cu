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
// x and dy and writes dx, each once.  A row is held in the registers of kTpr
// threads (a part of a warp, a warp, or several warps),
// so both of the variance's passes and the backward's two sums cost no second
// read; each group of threads walks over rows, and each thread keeps its part
// of the next rows coming by asynchronous copies into a ring of its own in
// shared memory (no barrier: a thread reads back only what it copied).
//
// Rows of any length are read and written 16 bytes at a time.  Where a row's
// stride is not a multiple of that, rows start at different places within 16
// bytes, the same place again after `period` rows: a block takes only rows
// that start at the same place (`shift` elements into their first 16 bytes),
// so that a thread keeps its columns and masks for the whole call.
//
// The backward adds dy xh and dy of its rows to per-thread column sums, adds
// those of a block's groups in shared memory, and leaves one row of partial
// sums a block; a second launch adds a worker's blocks.  All sums have a fixed
// order.
#include "layers.cuh"

using namespace signmuon;

namespace {

constexpr int kThreads = 256;         // threads a block for rows of up to that many
constexpr int kWideThreads = 512;     // threads a block for rows that registers do not hold
constexpr int kBwdHeldCols = 8192;    // the backward's widest rows that they hold

// Rows and columns of one call.
struct NormArgs {
  int64_t rows;
  int32_t cols;
  int32_t period;                     // rows after which starts within 16 bytes repeat
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

// What a thread has of a row: chunk c is the VEC elements from column
// col(c) = (c * kTpr + t) * VEC - shift.  Bit i of `mask` says whether element
// i is in the row: some of the first chunk of a row may lie before it, some of
// the last after it, unless rows start on 16 bytes and end with a chunk
// (kWhole).
template <int VEC, int E, int kTpr, bool kWhole>
struct Part {
  int t, cols, shift;
  uint32_t mask;
  __device__ __forceinline__ Part(int t, int cols, int shift) : t(t), cols(cols), shift(kWhole ? 0 : shift), mask(0) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int at = col(i / VEC) + i % VEC;
      mask |= at >= 0 && at < cols ? 1u << i : 0u;
    }
  }
  __device__ __forceinline__ int col(int c) const { return (c * kTpr + t) * VEC - (kWhole ? 0 : shift); }
  __device__ __forceinline__ bool in(int c, int j) const { return mask >> (c * VEC + j) & 1; }
  __device__ __forceinline__ bool any(int c) const { return kWhole || VEC == 1 ? in(c, 0) : (mask >> c * VEC & kFull) != 0; }
  __device__ __forceinline__ bool whole(int c) const { return kWhole || VEC == 1 ? in(c, 0) : (mask >> c * VEC & kFull) == kFull; }
  // The same, with tests of the mask to be made where they are used: their
  // results, kept over the loop over rows, would take more registers than the
  // row.
  __device__ __forceinline__ Part again() const {
    Part p = *this;
    asm volatile("" : "+r"(p.mask));
    return p;
  }
  static constexpr uint32_t kFull = (1u << VEC) - 1;
};

// Rows come through kSlots slots of shared memory; single bf16 (2 bytes, below
// what can be copied asynchronously) are loaded when they are needed.
template <typename T, int VEC, int E, int kTpr, bool kWhole, int kSlots, int kBlock>
struct Rows {
  using Raw = typename RawVec<T, VEC>::type;
  using P = Part<VEC, E, kTpr, kWhole>;
  static constexpr int kChunks = E / VEC;
  static constexpr bool kAsync = sizeof(Raw) >= 4;
  static constexpr size_t kBytes = kAsync ? (size_t)kSlots * kChunks * sizeof(Raw) * kBlock : 0;
  Raw* ring;
  // Slots without columns are 0 from the start and stay so.
  __device__ __forceinline__ Rows(void* smem, const P& p) : ring(static_cast<Raw*>(smem) + threadIdx.x) {
    if constexpr (kAsync) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        if (!p.any(c))
#pragma unroll
          for (int i = 0; i < kSlots; ++i) ring[(i * kChunks + c) * kBlock] = Raw{};
    }
  }
  __device__ __forceinline__ void fetch(const P& p, const T* row, int slot) const {
    if constexpr (kAsync) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        // What a chunk has after the row's end is not read, but zero.
        if (p.any(c))
          copy_async<sizeof(Raw), kWhole>(ring + (slot * kChunks + c) * kBlock, row + p.col(c),
                                          min(VEC, p.cols - p.col(c)) * (int)sizeof(T));
    }
  }
  // The elements outside the row are 0.
  __device__ __forceinline__ void get(const P& p, float (&v)[E], const T* row, int slot) const {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float u[VEC];
      if constexpr (kAsync) {
        unpack(ring[(slot * kChunks + c) * kBlock], u);
        if (!kWhole && c == 0 && !p.whole(0)) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) u[j] = p.in(0, j) ? u[j] : 0.f;
        }
      } else {
        u[0] = 0.f;
        if (p.any(c)) unpack(load_stream<T, VEC>(row + p.col(c)), u);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[c * VEC + j] = u[j];
    }
  }
};
// Slots of a ring: about 192 bytes of rows a thread, two rows at least.
template <typename T, int E>
constexpr int kRowSlots = 192 / (E * (int)sizeof(T)) < 2 ? 2 : 192 / (E * (int)sizeof(T)) > 4 ? 4 : 192 / (E * (int)sizeof(T));

// A thread's weights (zero outside the row): fp32 in shared memory, groups of
// four of a row's threads side by side, so that reads meet no bank conflict.
// (In registers they would halve the threads an SM holds; with a thread's
// eight together, reads take twice as long and bound the forward kernel.)
template <int VEC, int E, int kTpr, bool kWhole>
struct Weights {
  using P = Part<VEC, E, kTpr, kWhole>;
  static constexpr int kGroup = VEC < 4 ? VEC : 4;
  static constexpr size_t kBytes = 4 * E * kTpr;
  const float* sh;  // this thread's first
  __device__ __forceinline__ Weights(void* smem, const P& p, const void* w, int bf16)
      : sh(static_cast<float*>(smem) + p.t * kGroup) {
    for (int i = threadIdx.x; i < E * kTpr; i += blockDim.x) {
      const int j = i % VEC, l = i / VEC % kTpr, c = i / VEC / kTpr, col = i - p.shift;
      static_cast<float*>(smem)[at(c, j) + l * kGroup] = w && col >= 0 && col < p.cols ? load_elem(w, col, bf16) : 0.f;
    }
  }
  __device__ __forceinline__ static constexpr int at(int c, int j) {
    return (c * (VEC / kGroup) + j / kGroup) * kTpr * kGroup + j % kGroup;
  }
  __device__ __forceinline__ void get(int c, float (&v)[VEC]) const {
#pragma unroll
    for (int j = 0; j < VEC; j += kGroup) {
      if constexpr (kGroup == 4) {
        const float4 q = *reinterpret_cast<const float4*>(sh + at(c, j));
        v[j] = q.x, v[j + 1] = q.y, v[j + 2] = q.z, v[j + 3] = q.w;
      } else {
        v[j] = sh[at(c, j)];
      }
    }
  }
};

// Sums of N values over the kTpr threads of a row.  Groups of more than a warp
// exchange their warps' sums by `sh`, one of two arrays that a caller uses in
// turn: then one barrier a sum does.
template <int kTpr, int N>
struct RowSum {
  struct Shared {
    float warp[2][kTpr > kThreads ? kTpr / 32 : kThreads / 32][N];
  };
  __device__ __forceinline__ static void run(float (&v)[N], Shared& sh, int turn) {
#pragma unroll
    for (int o = (kTpr < 32 ? kTpr : 32) / 2; o; o >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    if constexpr (kTpr > 32) {
      const int group = threadIdx.x / kTpr, warp = threadIdx.x / 32;
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int n = 0; n < N; ++n) sh.warp[turn][warp][n] = v[n];
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kTpr) : "memory");
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] = 0.f;
#pragma unroll
      for (int i = 0; i < kTpr / 32; ++i)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += sh.warp[turn][group * (kTpr / 32) + i][n];
    }
  }
};

// Writes a chunk: whole chunks at once, the ends of a row by elements.
template <typename T, int VEC, int E, int kTpr, bool kWhole>
__device__ __forceinline__ void store_chunk(const Part<VEC, E, kTpr, kWhole>& p, T* row, int c, const float (&o)[VEC]) {
  if (kWhole || VEC == 1 || p.whole(c)) {
    store_stream<T, VEC>(row + p.col(c), o);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (p.in(c, j)) store_elem(row, p.col(c) + j, sizeof(T) == 2, o[j]);
  }
}

// --------------------------------------------------------------- forward
// The variance is taken about the mean, from the values in registers.  Bound by
// memory: 32768 rows of 4096 bf16 in 91 us (floor 83; 32 elements a thread, 128
// threads a row; without the rings 210).
template <typename T, int VEC, int E, int kTpr, bool kWhole>
struct Forward {
  static constexpr int kBlock = kTpr > kThreads ? kTpr : kThreads, kGroups = kBlock / kTpr;
  using Ring = Rows<T, VEC, E, kTpr, kWhole, kRowSlots<T, E>, kBlock>;
  using W = Weights<VEC, E, kTpr, kWhole>;
  static constexpr size_t kSmem = Ring::kBytes + 2 * W::kBytes;
};
template <typename T, int VEC, int E, int kTpr, bool kWhole>
__global__ void __launch_bounds__(kTpr > kThreads ? kTpr : kThreads, VEC > 1 && kTpr >= 64 && kTpr <= kThreads && E == 32 ? 4 : 1)
norm_forward_kernel(const NormArgs a) {
  using F = Forward<T, VEC, E, kTpr, kWhole>;
  using Sum = RowSum<kTpr, 1>;
  constexpr int kSlots = kRowSlots<T, E>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ typename Sum::Shared sh;
  // Each of a period's blocks takes rows that start at the same place.
  const int64_t step = (int64_t)(gridDim.x / a.period) * F::kGroups * a.period;
  const int64_t row0 = (int64_t)(blockIdx.x / a.period) * F::kGroups * a.period + blockIdx.x % a.period;
  const float inv_cols = 1.f / (float)a.cols;
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.out);
  // All threads of a warp run the same iterations (`first` is the row of the
  // warp's first thread); rows past the end are masked.
  int64_t row = row0 + (int64_t)(threadIdx.x / kTpr) * a.period;
  int64_t first = row0 + (int64_t)(threadIdx.x / 32 * 32 / kTpr) * a.period;
  const Part<VEC, E, kTpr, kWhole> part_of(threadIdx.x % kTpr, a.cols, (int)(row0 * a.ld_x % VEC));

  const typename F::Ring in(smem, part_of);
#pragma unroll
  for (int i = 0; i < kSlots - 1; ++i) {
    if (row + i * step < a.rows) in.fetch(part_of, x + (row + i * step) * a.ld_x, i);
    copy_commit();
  }
  const typename F::W w(smem + F::Ring::kBytes, part_of, a.w, a.w_bf16);
  const typename F::W b(smem + F::Ring::kBytes + F::W::kBytes, part_of, a.b, a.w_bf16);
  __syncthreads();

  int slot = 0;
  for (; first < a.rows; row += step, first += step) {
    const auto p = part_of.again();
    const int64_t ahead = row + (kSlots - 1) * step;
    if (ahead < a.rows) in.fetch(p, x + ahead * a.ld_x, slot == 0 ? kSlots - 1 : slot - 1);
    copy_commit();
    copy_wait<kSlots - 1>();
    const bool valid = row < a.rows;
    float u[E];
    in.get(p, u, x + (valid ? row : 0) * a.ld_x, slot);
    slot = slot == kSlots - 1 ? 0 : slot + 1;
    Pair v[E / 2], sum(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) v[i] = Pair(u[2 * i], u[2 * i + 1]), sum = sum + v[i];
    float s[1] = {sum.lo() + sum.hi()};
    Sum::run(s, sh, 0);
    const float mean = s[0] * inv_cols;
    const Pair minus(-mean, -mean);
    sum = Pair(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < E / VEC; ++c) {
      if constexpr (VEC == 1) {
        if (c % 2 == 0) {
          v[c / 2] = v[c / 2] + minus;
          v[c / 2] = Pair(p.any(c) ? v[c / 2].lo() : 0.f, p.any(c + 1) ? v[c / 2].hi() : 0.f);
          sum = fma(v[c / 2], v[c / 2], sum);
        }
      } else if (p.any(c)) {
        const bool whole = kWhole || p.whole(c);
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          Pair& q = v[(c * VEC + j) / 2];
          q = q + minus;
          if (!whole) q = Pair(p.in(c, j) ? q.lo() : 0.f, p.in(c, j + 1) ? q.hi() : 0.f);
          sum = fma(q, q, sum);
        }
      }
    }
    s[0] = sum.lo() + sum.hi();
    Sum::run(s, sh, 1);
    const float r = rsqrtf(s[0] * inv_cols + a.eps);
    if (p.t == 0 && valid) a.mean[row] = mean, a.rstd[row] = r;
    const Pair rr(r, r);
    T* out = y + row * a.ld_out;
#pragma unroll
    for (int c = 0; c < E / VEC; ++c) {
      if (p.any(c) && valid) {
        float o[VEC], wv[VEC], bv[VEC];
        w.get(c, wv);
        b.get(c, bv);
        if constexpr (VEC == 1) {
          o[0] = fmaf((c % 2 ? v[c / 2].hi() : v[c / 2].lo()) * r, wv[0], bv[0]);
        } else {
#pragma unroll
          for (int j = 0; j < VEC; j += 2) {
            const Pair q = fma(v[(c * VEC + j) / 2] * rr, Pair(wv[j], wv[j + 1]), Pair(bv[j], bv[j + 1]));
            o[j] = q.lo(), o[j + 1] = q.hi();
          }
        }
        store_chunk<T>(p, out, c, o);
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
// three times (the second and third time mostly from L2; 4096 rows of 16384
// bf16: 105 us, floor 42; a cluster of blocks that holds the row took longer, for
// its two barriers a row).
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
// Bound by memory as well: eight workers' 65536 rows of 768 bf16 in 49 us, and the
// second launch 2 us more (floor 47; without the rings 143).  9001 rows of 1000
// fp32, 17 rows a group of threads: 19 us (floor 17).
template <typename T, int VEC, int E, int kTpr, bool kWhole>
struct Backward {
  static constexpr int kBlock = kTpr > kThreads ? kTpr : kThreads, kGroups = kBlock / kTpr;
  using Ring = Rows<T, VEC, E, kTpr, kWhole, kRowSlots<T, 2 * E>, kBlock>;
  using W = Weights<VEC, E, kTpr, kWhole>;
  static constexpr size_t kRun = 2 * Ring::kBytes + W::kBytes, kSums = kGroups > 1 ? 4 * kBlock * E : 0;
  static constexpr size_t kSmem = kRun > kSums ? kRun : kSums;
};
template <typename T, int VEC, int E, int kTpr, bool kWhole>
__global__ void __launch_bounds__(kTpr > kThreads ? kTpr : kThreads)
norm_backward_kernel(const NormArgs a, const __grid_constant__ WorkerRows rows, const __grid_constant__ WorkerBlocks share) {
  allow_next_kernel();
  using B = Backward<T, VEC, E, kTpr, kWhole>;
  using Sum = RowSum<kTpr, 2>;
  using Ring = typename B::Ring;
  constexpr int kSlots = kRowSlots<T, 2 * E>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ typename Sum::Shared sh;
  const int m = worker_of_block(share, a.n_workers, blockIdx.x);
  const int blocks = share.begin[m + 1] - share.begin[m], mine = blockIdx.x - share.begin[m];
  const float inv_cols = 1.f / (float)a.cols;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  T* dx = static_cast<T*>(a.out);
  const int64_t step = (int64_t)(blocks / a.period) * B::kGroups * a.period, end = rows.begin[m + 1];
  const int64_t row0 = rows.begin[m] + (int64_t)(mine / a.period) * B::kGroups * a.period + mine % a.period;
  int64_t row = row0 + (int64_t)(threadIdx.x / kTpr) * a.period;
  int64_t first = row0 + (int64_t)(threadIdx.x / 32 * 32 / kTpr) * a.period;
  const Part<VEC, E, kTpr, kWhole> part_of(threadIdx.x % kTpr, a.cols, (int)(row0 * a.ld_x % VEC));

  const Ring in_x(smem, part_of), in_g(smem + Ring::kBytes, part_of);
#pragma unroll
  for (int i = 0; i < kSlots - 1; ++i) {
    const int64_t at = row + i * step;
    if (at < end) in_x.fetch(part_of, x + at * a.ld_x, i), in_g.fetch(part_of, dy + at * a.ld_dy, i);
    copy_commit();
  }
  float mean_next = 0.f, r_next = 0.f;
  if (row < end) mean_next = a.mean[row], r_next = a.rstd[row];
  const typename B::W w(smem + 2 * Ring::kBytes, part_of, a.w, a.w_bf16);
  __syncthreads();

  Pair dw[E / 2], db[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) dw[i] = db[i] = Pair(0.f, 0.f);
  int slot = 0;
  for (int turn = 0; first < end; row += step, first += step, turn ^= 1) {
    const auto p = part_of.again();
    const int64_t ahead = row + (kSlots - 1) * step;
    if (ahead < end) {
      const int to = slot == 0 ? kSlots - 1 : slot - 1;
      in_x.fetch(p, x + ahead * a.ld_x, to), in_g.fetch(p, dy + ahead * a.ld_dy, to);
    }
    copy_commit();
    const float mean = mean_next, r = r_next;
    if (row + step < end) mean_next = a.mean[row + step], r_next = a.rstd[row + step];
    copy_wait<kSlots - 1>();
    const bool valid = row < end;
    Pair xh[E / 2], g[E / 2], s1(0.f, 0.f), s2(0.f, 0.f);
    {
      float u[E];
      in_x.get(p, u, x + (valid ? row : 0) * a.ld_x, slot);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) xh[i] = Pair(u[2 * i], u[2 * i + 1]);
      in_g.get(p, u, dy + (valid ? row : 0) * a.ld_dy, slot);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) g[i] = Pair(u[2 * i], u[2 * i + 1]);
    }
    slot = slot == kSlots - 1 ? 0 : slot + 1;
    const Pair minus(-mean, -mean), rr(r, r);
#pragma unroll
    for (int c = 0; c < E / VEC; ++c) {
      if constexpr (VEC == 1) {
        if (c % 2 == 0 && p.any(c) && valid) {
          float w0[1], w1[1];
          w.get(c, w0), w.get(c + 1, w1);
          const Pair q = (xh[c / 2] + minus) * rr;
          xh[c / 2] = Pair(q.lo(), p.any(c + 1) ? q.hi() : 0.f);
          db[c / 2] = db[c / 2] + g[c / 2];
          dw[c / 2] = fma(g[c / 2], xh[c / 2], dw[c / 2]);
          g[c / 2] = g[c / 2] * Pair(w0[0], w1[0]);
          s1 = s1 + g[c / 2];
          s2 = fma(g[c / 2], xh[c / 2], s2);
        }
      } else if (p.any(c) && valid) {
        const bool whole = kWhole || p.whole(c);
        float wv[VEC];
        w.get(c, wv);
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          const int i = (c * VEC + j) / 2;
          xh[i] = (xh[i] + minus) * rr;
          // Elements outside the row: xh may be anything there, dy is 0.
          if (!whole) xh[i] = Pair(p.in(c, j) ? xh[i].lo() : 0.f, p.in(c, j + 1) ? xh[i].hi() : 0.f);
          db[i] = db[i] + g[i];
          dw[i] = fma(g[i], xh[i], dw[i]);
          g[i] = g[i] * Pair(wv[j], wv[j + 1]);
          s1 = s1 + g[i];
          s2 = fma(g[i], xh[i], s2);
        }
      }
    }
    float s[2] = {s1.lo() + s1.hi(), s2.lo() + s2.hi()};
    Sum::run(s, sh, turn);
    const float c1 = -r * s[0] * inv_cols, c2 = -r * s[1] * inv_cols;
    const Pair cc1(c1, c1), cc2(c2, c2);
    T* out = dx + row * a.ld_out;
#pragma unroll
    for (int c = 0; c < E / VEC; ++c) {
      if (p.any(c) && valid) {
        float o[VEC];
        if constexpr (VEC == 1) {
          const Pair q = fma(xh[c / 2], cc2, fma(g[c / 2], rr, cc1));
          o[0] = c % 2 ? q.hi() : q.lo();
        } else {
#pragma unroll
          for (int j = 0; j < VEC; j += 2) {
            const int i = (c * VEC + j) / 2;
            const Pair q = fma(xh[i], cc2, fma(g[i], rr, cc1));
            o[j] = q.lo(), o[j + 1] = q.hi();
          }
        }
        store_chunk<T>(p, out, c, o);
      }
    }
  }

  // The block's partial sums.
  const auto& p = part_of;
  const int sums = a.has_bias ? 2 : 1;
  float* part = a.part + (int64_t)blockIdx.x * sums * a.cols;
  if constexpr (B::kGroups == 1) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = i / VEC, j = i % VEC;
      if (p.in(c, j)) {
        part[p.col(c) + j] = i % 2 ? dw[i / 2].hi() : dw[i / 2].lo();
        if (a.has_bias) part[a.cols + p.col(c) + j] = i % 2 ? db[i / 2].hi() : db[i / 2].lo();
      }
    }
  } else {
    // Every group's in shared memory (over the rings and weights), then added
    // by column in the groups' order, one sum after the other.
    float* all = reinterpret_cast<float*>(smem);
    constexpr int kCols = kTpr * E;
    for (int q = 0; q < sums; ++q) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const Pair s = q ? db[i / 2] : dw[i / 2];
        all[threadIdx.x / kTpr * kCols + (i / VEC * kTpr + p.t) * VEC + i % VEC] = i % 2 ? s.hi() : s.lo();
      }
      __syncthreads();
      for (int col = threadIdx.x; col < a.cols; col += B::kBlock) {
        float s = 0.f;
#pragma unroll 8
        for (int g = 0; g < B::kGroups; ++g) s += all[g * kCols + col + p.shift];
        part[q * a.cols + col] = s;
      }
    }
  }
}

// Rows longer than a block's registers hold: dx by a block a row, which reads
// dy and x twice (4096 rows of 16384 bf16 with the column sums: 184 us, floor 62,
// of 232 for what is read twice and a third time).
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

// ... and, before it, the column sums by blocks of 32 x VEC columns x 8 warps over
// the rows that a block of the other kernel would have had.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
norm_columns_kernel(const NormArgs a, const __grid_constant__ WorkerRows rows, const __grid_constant__ WorkerBlocks share) {
  __shared__ float sh[2][8][VEC][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, cols = a.cols, col = (blockIdx.y * 32 + lane) * VEC;
  const int m = worker_of_block(share, a.n_workers, blockIdx.x);
  const int blocks = share.begin[m + 1] - share.begin[m];
  const int64_t step = (int64_t)blocks * 8, end = rows.begin[m + 1];
  const T* x = static_cast<const T*>(a.x) + col;
  const T* dy = static_cast<const T*>(a.dy) + col;
  float dw[VEC] = {}, db[VEC] = {};
  if (col < cols)
#pragma unroll 4
    for (int64_t row = rows.begin[m] + (int64_t)(blockIdx.x - share.begin[m]) * 8 + warp; row < end; row += step) {
      float u[VEC], g[VEC];
      unpack(*reinterpret_cast<const typename RawVec<T, VEC>::type*>(x + row * a.ld_x), u);
      unpack(*reinterpret_cast<const typename RawVec<T, VEC>::type*>(dy + row * a.ld_dy), g);
      const float mean = a.mean[row], r = a.rstd[row];
#pragma unroll
      for (int j = 0; j < VEC; ++j) db[j] += g[j], dw[j] = fmaf(g[j], (u[j] - mean) * r, dw[j]);
    }
#pragma unroll
  for (int j = 0; j < VEC; ++j) sh[0][warp][j][lane] = dw[j], sh[1][warp][j][lane] = db[j];
  __syncthreads();
  const int sums = a.has_bias ? 2 : 1;
  for (int i = threadIdx.x; i < sums * 32 * VEC; i += 256) {
    const int which = i / (32 * VEC), c = i % (32 * VEC), at = blockIdx.y * 32 * VEC + c;
    if (at >= cols) continue;
    float s = 0.f;
    for (int w = 0; w < 8; ++w) s += sh[which][w][c % VEC][c / VEC];
    a.part[((int64_t)blockIdx.x * sums + which) * cols + at] = s;
  }
}

// Adds a worker's blocks: 32 columns a block, 8 warps each taking every
// eighth block's row.  Bound by latency; launched while the blocks still run.
__global__ void __launch_bounds__(256)
norm_finalize_kernel(const float* part, int cols, int sums, int w_bf16, const __grid_constant__ WorkerBlocks share,
                     const __grid_constant__ WorkerPtrs dw, const __grid_constant__ WorkerPtrs db) {
  __shared__ float sh[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, col = blockIdx.x * 32 + lane;
  const int m = blockIdx.y, which = blockIdx.z;
  wait_for_kernel_before();
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
// f(elements a thread, threads a row) for rows that reach over `span`
// elements, false where no kernel holds them.  Few threads with 8 elements
// each, up to a warp, then more elements (fewer threads have less to exchange),
// then more warps.  The backward's column sums leave room for 16 elements a
// thread where several warps have a row.
template <bool kBackward, typename F>
bool by_span(int span, F f) {
  if (span <= 8) return f(Int<8>(), Int<1>());
  if (span <= 16) return f(Int<8>(), Int<2>());
  if (span <= 32) return f(Int<8>(), Int<4>());
  if (span <= 64) return f(Int<8>(), Int<8>());
  if (span <= 128) return f(Int<8>(), Int<16>());
  if (span <= 256) return f(Int<8>(), Int<32>());
  if (span <= 512) return f(Int<16>(), Int<32>());
  if (span <= 768) return f(Int<24>(), Int<32>());
  if (span <= 1024) return f(Int<32>(), Int<32>());
  if constexpr (kBackward) {
    if (span <= 2048) return f(Int<16>(), Int<128>());
    if (span <= 4096) return f(Int<16>(), Int<256>());
    if (span <= kBwdHeldCols) return f(Int<16>(), Int<512>());
  } else {
    if (span <= 1536) return f(Int<24>(), Int<64>());
    if (span <= 2048) return f(Int<32>(), Int<64>());
    if (span <= 4096) return f(Int<32>(), Int<128>());
    if (span <= 8192) return f(Int<32>(), Int<256>());
    if (span <= 12288) return f(Int<32>(), Int<384>());
  }
  return false;
}

template <typename T, int VEC, bool kWhole>
void forward_launch(const NormArgs& a, int sms, cudaStream_t st) {
  const bool held = by_span<false>(a.cols + (a.period > 1 ? VEC - 1 : 0), [&](auto e, auto tpr) {
    constexpr int kE = decltype(e)::value, kTpr = decltype(tpr)::value;
    using F = Forward<T, VEC, kE, kTpr, kWhole>;
    constexpr auto k = norm_forward_kernel<T, VEC, kE, kTpr, kWhole>;
    const int64_t most = (int64_t)sms * resident_blocks<k>(F::kBlock, F::kSmem) / a.period * a.period;
    int64_t blocks = ceil_div(a.rows, (int64_t)F::kGroups * a.period) * a.period;
    if (blocks > most) blocks = most < a.period ? a.period : most;
    k<<<(unsigned)blocks, F::kBlock, F::kSmem, st>>>(a);
    return true;
  });
  if (!held) {
    const int64_t most = (int64_t)sms * 4;
    norm_forward_wide_kernel<T, kWhole ? VEC : 1><<<(unsigned)(a.rows < most ? a.rows : most), kWideThreads, 0, st>>>(a);
  }
}

// Blocks of the backward pass, shared out over the workers by their rows: a
// whole number of periods for each, none for one without rows.
int block_share(int n_workers, const int64_t* row_begin, int rows_a_block, int most, int period, WorkerBlocks* share) {
  const int64_t rows = row_begin[n_workers];
  int n = 0;
  for (int m = 0; m < n_workers; ++m) {
    const int64_t mine = row_begin[m + 1] - row_begin[m];
    int64_t b = rows ? (int64_t)((double)mine / (double)rows * (most / period)) : 0;
    const int64_t useful = ceil_div(mine, (int64_t)rows_a_block * period);
    if (b > useful) b = useful;
    if (b < 1 && mine > 0) b = 1;
    share->begin[m] = n;
    n += (int)b * period;
  }
  share->begin[n_workers] = n;
  return n;
}

constexpr int kBwdBlocksPerSm = 8;
constexpr int kColumnRows = 64;     // rows a block of their column sums at least
constexpr int kMaxPeriod = 8;
// Blocks at most, whatever the type and the addresses: those of every SM (the
// column sums have one) and for each worker whose share rounds to none a period
// more, and no more than a worker has rows for.
int64_t bwd_max_blocks(int sms, int32_t cols, int n_workers, const int64_t* row_begin) {
  const bool wide = cols > kBwdHeldCols;
  const int64_t most = wide ? (int64_t)sms + n_workers : (int64_t)sms * kBwdBlocksPerSm + kMaxPeriod * n_workers;
  int64_t useful = 0;
  for (int m = 0; m < n_workers; ++m) {
    const int64_t rows = row_begin[m + 1] - row_begin[m];
    if (rows) useful += wide ? ceil_div(rows, kColumnRows) : rows + kMaxPeriod - 1;
  }
  return useful < most ? useful : most;
}

template <typename T, int VEC, bool kWhole>
void backward_launch(const NormArgs& a, const WorkerRows& rows, const int64_t* row_begin, int sms, WorkerBlocks* share,
                     cudaStream_t st) {
  if (!a.rows) return;
  const bool held = by_span<true>(a.cols + (a.period > 1 ? VEC - 1 : 0), [&](auto e, auto tpr) {
    constexpr int kE = decltype(e)::value, kTpr = decltype(tpr)::value;
    using B = Backward<T, VEC, kE, kTpr, kWhole>;
    constexpr auto k = norm_backward_kernel<T, VEC, kE, kTpr, kWhole>;
    const int resident = resident_blocks<k>(B::kBlock, B::kSmem);
    const int blocks = block_share(a.n_workers, row_begin, B::kGroups,
                                   sms * (resident < kBwdBlocksPerSm ? resident : kBwdBlocksPerSm), a.period, share);
    k<<<blocks, B::kBlock, B::kSmem, st>>>(a, rows, *share);
    return true;
  });
  if (!held) {
    // The column sums first: dx may take dy's place.
    constexpr int kVec = kWhole ? VEC : 1;
    const int blocks = block_share(a.n_workers, row_begin, kColumnRows, sms, 1, share);
    norm_columns_kernel<T, kVec><<<dim3((unsigned)blocks, (unsigned)ceil_div(a.cols, 32 * kVec)), 256, 0, st>>>(a, rows, *share);
    const int64_t most = (int64_t)sms * 4;
    norm_backward_wide_kernel<T, kVec><<<(unsigned)(a.rows < most ? a.rows : most), kWideThreads, 0, st>>>(a);
  }
}

// How rows are accessed: 16 bytes at a time if every buffer starts on 16 bytes
// and the buffers' rows start at the same place within 16 bytes, else element
// by element.
struct Access {
  bool wide;
  int period;
};
Access access_of(signmuon_dtype t, int n, const void* const* p, const int64_t* ld) {
  const int vec = 16 / dtype_bytes(t);
  for (int i = 0; i < n; ++i)
    if (!aligned_to(p[i], 16) || ld[i] % vec != ld[0] % vec) return {false, 1};
  int period = 1;
  while (ld[0] * period % vec) period *= 2;
  return {true, period};
}

// f(type, elements an access, whether rows are whole accesses)
template <typename F>
void by_access(signmuon_dtype t, const Access& access, int cols, F f) {
  const bool whole = access.period == 1 && cols % (16 / dtype_bytes(t)) == 0;
  if (t == SIGNMUON_F32) {
    if (!access.wide) f(float(), Int<1>(), std::true_type());
    else if (whole) f(float(), Int<4>(), std::true_type());
    else f(float(), Int<4>(), std::false_type());
  } else {
    if (!access.wide) f(__nv_bfloat16(), Int<1>(), std::true_type());
    else if (whole) f(__nv_bfloat16(), Int<8>(), std::true_type());
    else f(__nv_bfloat16(), Int<8>(), std::false_type());
  }
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
  const void* const bufs[2] = {x, y};
  const int64_t lds[2] = {ld_x, ld_y};
  const Access access = access_of(x_dtype, 2, bufs, lds);
  NormArgs a = {};
  a.period = access.period;
  a.rows = rows, a.cols = cols, a.x = x, a.out = y, a.ld_x = ld_x, a.ld_out = ld_y, a.w = weight, a.b = bias;
  a.w_bf16 = w_dtype == SIGNMUON_BF16, a.eps = eps, a.mean = mean, a.rstd = rstd;
  by_access(x_dtype, access, cols, [&](auto t, auto v, auto whole) {
    forward_launch<decltype(t), decltype(v)::value, decltype(whole)::value>(a, current_sms(), static_cast<cudaStream_t>(stream));
  });
  return cuda_status(cudaGetLastError());
}

size_t signmuon_layer_norm_backward_workspace_bytes(int32_t cols, int n_workers, const int64_t* row_begin) {
  if (cols <= 0 || n_workers <= 0 || n_workers > SIGNMUON_MAX_WORKERS || !row_begin ||
      !valid_splits(row_begin, n_workers, row_begin[n_workers]))
    return 0;
  return kWsHeaderBytes + round_up((size_t)bwd_max_blocks(current_sms(), cols, n_workers, row_begin) * 2 * cols * 4, 256);
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
  const void* const bufs[3] = {x, dy, dx};
  const int64_t lds[3] = {ld_x, ld_dy, ld_dx};
  const Access access = access_of(x_dtype, 3, bufs, lds);
  NormArgs a = {};
  a.period = access.period;
  a.rows = n, a.cols = cols, a.x = x, a.dy = dy, a.out = dx, a.ld_x = ld_x, a.ld_dy = ld_dy, a.ld_out = ld_dx;
  a.w = weight, a.w_bf16 = w_dtype == SIGNMUON_BF16, a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWsHeaderBytes);
  a.n_workers = n_workers, a.has_bias = dbias != nullptr;
  WorkerRows rows = {};
  for (int m = 0; m <= n_workers; ++m) rows.begin[m] = row_begin[m];
  WorkerBlocks share = {};
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  by_access(x_dtype, access, cols, [&](auto t, auto v, auto whole) {
    backward_launch<decltype(t), decltype(v)::value, decltype(whole)::value>(a, rows, row_begin, current_sms(), &share, cs);
  });
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_status(e);
  launch_after(norm_finalize_kernel, dim3((unsigned)ceil_div(cols, 32), (unsigned)n_workers, dbias ? 2u : 1u), 256, 0, cs,
               a.part, cols, dbias ? 2 : 1, a.w_bf16, share, dw, db);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
