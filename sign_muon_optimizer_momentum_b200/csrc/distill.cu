// Distillation from a teacher's top logits: the divergence of the student's
// softmax from the teacher's, per row and per worker, and the logits'
// gradient.
//
//   p = softmax(u / T) over the row's present entries, q = softmax(z / T)
//   row loss  T^2 sum_k p_k (log p_k - log q_{i_k})
//           = T^2 (sum_k p_k log p_k - sum_k p_k (z_{i_k} - max) / T + log S),
//             S = sum_v exp((z_v - max) / T)
//   gradient  c T (q - p) / n_m
//
// Three launches:
//   1. teacher   a warp a row: p by softmax over the entries, entries of the
//                same id put together, sum p log p, and whether the row counts;
//   2. rows      the logits: running maximum and sum, the row's loss, and the
//                gradient;
//   3. workers   the losses of each worker's rows, added in a fixed order.
// The second one reads the logits and writes the gradient, each once, and is
// bound by that: a block (for long rows a cluster of blocks) holds its row in
// shared memory from the pass that sums to the pass that writes.
#include "layers.cuh"

using namespace signmuon;

namespace {

constexpr int kMaxTop = 1024;
constexpr int kMaxVocab = 1 << 30;   // columns of a row, and rows of a call: ints count them
constexpr int kTeacherWarps = 4;
constexpr int kRowThreads = 512;           // of a block that reads its row twice
// Of a block that holds its rows (for the losses, that streams them) at most,
// and the chunks that a thread copies as one group.
constexpr int kHeldThreads = 384, kHeldBatch = 3;
constexpr int kStreamThreads = 512, kStreamBatch = 4;
constexpr int kShortWarps = 8, kShortCols = 1024;  // of a block of short rows; columns of one at most
constexpr int kLossThreads = 512;          // of a block that adds a worker's losses
constexpr int kWarpBatch = 8;              // vectors a lane loads at a time of a row that a warp has
constexpr int kDepth = 3;                  // groups under way where a row is not held
constexpr int kMaxCluster = 8;
constexpr int kSmSmem = 227 * 1024;
constexpr float kLog2e = 1.4426950408889634f;
// The divergence of a row is a difference of sums that fp32 gives to about 1e-6,
// and T^2 multiplies that.  Above kFineT rows of a divergence below kFineKl (a
// teacher that covers most of the vocabulary: T^2 times the divergence stays, the
// sums grow nearly equal) are taken again by left_row, so that a row's loss is off
// by 6e-5 at most, or by 2e-5 of itself.
constexpr float kFineT = 8.f, kFineKl = 1.f / 16;

// A teacher's entry: its id (-1: none) and the probability it holds.
struct Entry {
  int32_t id;
  float p;
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- teacher
// A warp a row, kPer entries a lane in registers.  Bound by the latency of its
// steps, one after the other (2048 rows of 64 entries: 4.1 us, 8192: 6.6; with
// a table of ids filled by atomicCAS, which takes the lanes one by one, 9.7 and
// 12.5).
template <int kPer>
__global__ void __launch_bounds__(kTeacherWarps * 32)
teacher_kernel(int64_t rows, int top, const void* __restrict__ ids, int wide, const void* __restrict__ logits, int bf16,
               int32_t vocab, float inv_t, Entry* __restrict__ entries, float* __restrict__ plogp, uint8_t* __restrict__ counts) {
  // Each warp: the ids, and a hash table of twice as many slots, to see whether
  // one comes twice; then, if one does, the entries.
  constexpr int kSlots = 64 * kPer;
  extern __shared__ Entry s_entries[];
  allow_next_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t row = (int64_t)blockIdx.x * kTeacherWarps + warp;
  if (row >= rows) return;
  Entry* mine = s_entries + warp * (32 * kPer);
  int32_t* s_id = reinterpret_cast<int32_t*>(mine);
  uint16_t* table = reinterpret_cast<uint16_t*>(s_id + 32 * kPer);
  int32_t id[kPer];
  float x[kPer], e[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int k = lane + 32 * j;
    id[j] = -1, x[j] = -INFINITY;
    if (k < top) {
      const int64_t v = load_id(ids, row * top + k, wide);
      x[j] = load_elem(logits, row * top + k, bf16);
      if (v >= 0 && v < vocab && x[j] != -INFINITY) id[j] = (int32_t)v;
    }
  }
  bool any = false, bad = false, twice = false;
  float top_u = -INFINITY;
  uint32_t open = 0;  // entries that are to be compared still
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    s_id[lane + 32 * j] = id[j];
    if (id[j] >= 0) top_u = fmaxf(top_u, x[j]), any = true, bad |= x[j] != x[j], open |= 1u << j;
  }
  // In turns: each writes itself into its id's slot.  One stays there, and is
  // done; one that finds another entry of its id there comes twice; the others
  // (with them, all of an id or none) try another hash.
  for (uint32_t odd = 2654435769u; __any_sync(0xffffffffu, open); odd *= 0x2c1b3c6du) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (open >> j & 1) table[(uint32_t)id[j] * odd >> 16 & (kSlots - 1)] = (uint16_t)(lane + 32 * j);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (open >> j & 1) {
        const int there = table[(uint32_t)id[j] * odd >> 16 & (kSlots - 1)];
        if (s_id[there] == id[j]) open &= ~(1u << j), twice |= there != lane + 32 * j;
      }
    __syncwarp();
  }
  any = __any_sync(0xffffffffu, any);
  // fmaxf drops a NaN: one among the entries makes the row NaN.
  top_u = __any_sync(0xffffffffu, bad) ? NAN : warp_max(top_u);
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    x[j] = (x[j] - top_u) * inv_t;
    e[j] = id[j] >= 0 ? expf(x[j]) : 0.f;
    sum += e[j];
  }
  sum = warp_sum(sum);
  const float log_sum = logf(sum), inv_sum = 1.f / sum;
  float h = 0.f;
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (id[j] >= 0) {
      e[j] *= inv_sum;
      if (e[j] != 0.f) h = fmaf(e[j], x[j] - log_sum, h);
    }
  h = warp_sum(h);
  if (lane == 0) plogp[row] = h, counts[row] = any;
  if (!__any_sync(0xffffffffu, twice)) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (lane + 32 * j < top) entries[row * top + lane + 32 * j] = {e[j] != 0.f ? id[j] : -1, e[j]};
    return;
  }
  // The first entry of an id holds all of the id's.
#pragma unroll
  for (int j = 0; j < kPer; ++j) mine[lane + 32 * j] = {id[j], e[j]};
  __syncwarp();
  for (int k = lane; k < top; k += 32) {
    const int32_t v = mine[k].id;
    float p = 0.f;
    bool first = true;
    for (int i = 0; i < top; ++i)
      if (mine[i].id == v) p += mine[i].p, first &= i >= k;
    entries[row * top + k] = {v >= 0 && first && p != 0.f ? v : -1, p};
  }
}

// ------------------------------------------------------------------- rows
struct RowArgs {
  const void* top_ids;
  const void* top_logits;
  int32_t ids_wide, top_bf16;
  const void* z;
  int64_t ld_z;
  void* dz;  // null: the losses alone
  int64_t ld_dz;
  Entry* entries;
  const float* plogp;
  const uint8_t* counts;
  float* row_loss;
  int64_t rows;
  int32_t vocab, top;
  float t, inv_t, grad_scale;
  float min_kl;  // divergence from which on fp32 does (-inf: always)
};

// A sum of 2^(c z) as s 2^e, c = log2(e) / T and e a whole number, at least c
// times the largest z so far.  c z - e is one fused multiply-add, rounded once
// and only to the size of the difference, and changing e multiplies s by a
// power of two.  An empty sum has e = -inf and s = 0.
// That holds while an ulp of c z is at most 1/2.  Logits below -kMaxExponent / c
// count nothing (a part of a row without others keeps that e, and the parts that
// have others are infinitely larger); a row whose largest is not above that, or
// is above kMaxExponent / c, is taken again by left_row.
constexpr float kMaxExponent = 1 << 22;
struct Soft {
  float e, s;
};
// Whether that is the sum (it is not if any of the row is NaN).
__device__ __forceinline__ bool soft_holds(Soft a) { return fabsf(a.e) < kMaxExponent && a.s > 0.f && a.s < INFINITY; }
__device__ __forceinline__ float soft_ref(float e) { return e == -INFINITY ? 0.f : -e; }  // added to c z
__device__ __forceinline__ void soft_raise(Soft& a, float top, float c) {
  const float e = fmaxf(ceilf(top * c), -kMaxExponent);
  if (e > a.e) {
    a.s *= a.e == -INFINITY ? 0.f : exp2_fast(a.e - e);
    a.e = e;
  }
}
__device__ __forceinline__ Soft soft_join(Soft a, Soft b) {
  const float e = fmaxf(a.e, b.e);
  return {e, (a.e == -INFINITY ? a.s : a.s * exp2_fast(a.e - e)) + (b.e == -INFINITY ? b.s : b.s * exp2_fast(b.e - e))};
}
__device__ __forceinline__ Soft warp_join(Soft a) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    a = soft_join(a, {__shfl_xor_sync(0xffffffffu, a.e, o), __shfl_xor_sync(0xffffffffu, a.s, o)});
  return a;
}
// log q of a logit, by way of half its size: c z may overflow where z / T does not.
__device__ __forceinline__ float soft_log(Soft a, float z, float c) {
  return (fmaf(z, 0.5f * c, -0.5f * a.e) - 0.5f * log2f(a.s)) * 1.3862943611198906f;
}

// Thread t's share, of `threads`, of the rows [begin, end) that count, 16 bytes at a time
// (counts starts on 16 bytes and has room to the next).
__device__ __forceinline__ int count_rows(const uint8_t* counts, int64_t begin, int64_t end, int t, int threads) {
  int n = 0;
#pragma unroll 4
  for (int64_t at = begin / 16 * 16 + t * 16; at < end; at += threads * 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(counts + at);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (at >= begin && at + 16 <= end) {
      n += __popc(w[0] | w[1] << 1 | w[2] << 2 | w[3] << 3);  // each byte is 0 or 1
    } else {
      for (int i = max((int)(begin - at), 0); i < min((int)(end - at), 16); ++i) n += counts[at + i];
    }
  }
  return n;
}

// -------------------------------------------------------------- rows left
// A row that fp32 does not give is left by the loop over rows, marked by this NaN
// (not one that arithmetic gives) as its loss, and taken when the loop is done:
// there it costs the others no registers.
constexpr uint32_t kLeft = 0x7fc0deadu;
__device__ __forceinline__ bool is_left(const RowArgs& a, int64_t row) { return __float_as_uint(a.row_loss[row]) == kLeft; }

// Threads that have a row together: a warp, or a block.
template <bool kWarp>
struct Team {
  __device__ __forceinline__ static int rank() { return kWarp ? threadIdx.x & 31 : threadIdx.x; }
  __device__ __forceinline__ static int size() { return kWarp ? 32 : blockDim.x; }
  __device__ __forceinline__ static void sync() {
    if constexpr (kWarp) __syncwarp();
    else __syncthreads();
  }
  // All get f over their values, joined in a fixed order by way of `sh`, a double
  // for each warp of a block.  (An array that the kernel has already: where the
  // dynamic shared memory starts behind the static arrays matters, 2048 x 50000
  // fp32 losses took 75 us from byte 448, 77 from 512 and 85 from 464.)
  template <typename F>
  __device__ __forceinline__ static double join(double v, double* sh, F f) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    if constexpr (!kWarp) {
      __syncthreads();
      if ((threadIdx.x & 31) == 0) sh[threadIdx.x / 32] = v;
      __syncthreads();
      v = sh[0];
      for (int i = 1; i < (int)blockDim.x / 32; ++i) v = f(v, sh[i]);
    }
    return v;
  }
  __device__ __forceinline__ static double sum(double v, double* sh) {
    return join(v, sh, [](double x, double y) { return x + y; });
  }
  __device__ __forceinline__ static double max(double v, double* sh) {
    return join(v, sh, [](double x, double y) { return fmax(x, y); });
  }
};

// A row from its definition in fp64, differences before products, with the
// entries as they were given.  The gradient may take the logits' place; `scale` is
// its factor.  The row's entries in the workspace are used up.  Bound by the fp64
// exponentials, one an element for the loss and one for the gradient: 2048 rows of
// 50000 bf16, all of them left, 893 us (losses alone 533), and 8192 of 512 at a high
// temperature 195, where fp32 does they take 107, 56 and 64.
template <typename T, bool kGrad, bool kWarp>
__device__ __forceinline__ void left_row(const RowArgs& a, int64_t row, double scale, double* sh) {
  using G = Team<kWarp>;
  const int t = G::rank(), n = G::size();
  const double inv_t = 1.0 / (double)a.t;
  const T* z = static_cast<const T*>(a.z) + row * a.ld_z;
  Entry* entries = a.entries + row * a.top;
  const auto logit = [&](int i) { return (double)load_elem(z, i, sizeof(T) == 2); };
  const auto entry = [&](int k, double& u) {  // its id, -1 if it is absent
    const int64_t id = load_id(a.top_ids, row * a.top + k, a.ids_wide);
    const float v = load_elem(a.top_logits, row * a.top + k, a.top_bf16);
    u = v;
    return id >= 0 && id < a.vocab && v != -INFINITY ? (int)id : -1;
  };
  double u, u_top = -INFINITY, su = 0.0, z_top = -INFINITY, sz = 0.0;
  for (int k = t; k < a.top; k += n)
    if (entry(k, u) >= 0) u_top = fmax(u_top, u);
  u_top = G::max(u_top, sh);
  for (int k = t; k < a.top; k += n)
    if (entry(k, u) >= 0) su += exp((u - u_top) * inv_t);
  su = G::sum(su, sh);
  for (int i = t; i < a.vocab; i += n) z_top = fmax(z_top, logit(i));
  z_top = G::max(z_top, sh);
  for (int i = t; i < a.vocab; i += n) sz += exp((logit(i) - z_top) * inv_t);
  sz = G::sum(sz, sh);
  const double log_su = log(su), log_sz = log(sz);
  double kl = 0.0, twice = 0.0;
  for (int k = t; k < a.top; k += n) {
    const int id = entry(k, u);
    if (id < 0) continue;
    const double x = (u - u_top) * inv_t, p = exp(x) / su, y = (logit(id) - z_top) * inv_t;
    if ((float)p == 0.f) continue;
    kl += p * ((x - log_su) - (y - log_sz));
    if (entries[k].id < 0) twice = 1.0;  // another entry holds this one's p
  }
  kl = G::sum(kl, sh);
  if (t == 0) a.row_loss[row] = (float)((double)a.t * a.t * kl);
  if constexpr (kGrad) {
    twice = G::max(twice, sh);
    for (int k = t; k < a.top; k += n) {
      const int id = entries[k].id;
      if (id < 0) continue;
      double q = exp((logit(id) - z_top) * inv_t) / sz;
      for (int j = twice > 0.0 ? 0 : k; j < (twice > 0.0 ? a.top : k + 1); ++j)
        if (entry(j, u) == id) q -= exp((u - u_top) * inv_t) / su;
      entries[k].p = (float)(q * scale);
    }
    G::sync();
    const double qs = scale / sz;
    T* dz = static_cast<T*>(a.dz) + row * a.ld_dz;
    for (int i = t; i < a.vocab; i += n) store_elem(dz, i, sizeof(T) == 2, (float)(exp((logit(i) - z_top) * inv_t) * qs));
    G::sync();
    for (int k = t; k < a.top; k += n)
      if (entries[k].id >= 0) store_elem(dz, entries[k].id, sizeof(T) == 2, entries[k].p);
  }
}

// The rows first, first + step, ... of a team that were left.
template <typename T, bool kGrad, bool kWarp>
__device__ __forceinline__ void left_rows(const RowArgs& a, const WorkerRows& workers, int64_t first, int64_t end, int64_t step,
                                          double* sh) {
  using G = Team<kWarp>;
  int worker = -1;
  double scale = 0.0;
  for (int64_t row = first; row < end; row += step) {
    if (!a.counts[row] || !is_left(a, row)) continue;
    G::sync();
    if (kGrad && (worker < 0 || workers.begin[worker + 1] <= row)) {
      while (workers.begin[++worker + 1] <= row) {}
      scale = (double)a.grad_scale * a.t /
              G::sum(count_rows(a.counts, workers.begin[worker], workers.begin[worker + 1], G::rank(), G::size()), sh);
    }
    left_row<T, kGrad, kWarp>(a, row, scale, sh);
  }
}

// ------------------------------------------------------------- short rows
// A warp a row, kE elements a lane in registers: one exponential an element, and
// no barrier a row.  (5927 rows of 586 bf16 with their gradient: 20 us, where a block
// a row, as below, took 33; 20000 rows of 193 fp32: 28 for 67 us.)
// (Blocks an SM: as many as the registers of the loop over rows allow.)
template <typename T, bool kGrad, int kE, bool kFine>
__global__ void __launch_bounds__(kShortWarps * 32, kE == 32 ? 2 : kGrad ? (kE == 4 ? 5 : 4) : (kE == 4 ? 8 : kE == 8 ? 6 : 5))
short_rows_kernel(const RowArgs a, const __grid_constant__ WorkerRows workers, int per_warp) {
  // The teacher's part of the gradient by column, zero but for a row's entries.
  __shared__ float s_sub[kGrad ? kShortWarps : 1][kGrad ? 32 * kE : 1];
  allow_next_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, n = a.vocab;
  const float c = a.inv_t * kLog2e;
  const int64_t first = ((int64_t)blockIdx.x * kShortWarps + warp) * per_warp;
  const int64_t last = first + per_warp < a.rows ? first + per_warp : a.rows;
  float* sub = s_sub[kGrad ? warp : 0];
  if constexpr (kGrad)
#pragma unroll
    for (int i = 0; i < kE; ++i) sub[lane + 32 * i] = 0.f;
  wait_for_kernel_before();
  // The rows that count of the worker that the block's first row belongs to.
  __shared__ int s_n;
  int worker = -1, first_worker = 0;
  if constexpr (kGrad) {
    const int64_t block_row = (int64_t)blockIdx.x * kShortWarps * per_warp;
    while (workers.begin[first_worker + 1] <= block_row) ++first_worker;
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    const int rows = __reduce_add_sync(0xffffffffu, count_rows(a.counts, workers.begin[first_worker], workers.begin[first_worker + 1],
                                                               threadIdx.x, kShortWarps * 32));
    if (lane == 0) atomicAdd(&s_n, rows);
    __syncthreads();
  }
  float scale = 0.f;
  bool left = false;
  for (int64_t row = first; row < last; ++row) {
    const T* z = static_cast<const T*>(a.z) + row * a.ld_z;
    T* dz = kGrad ? static_cast<T*>(a.dz) + row * a.ld_dz : nullptr;
    if (!a.counts[row]) {
      if (lane == 0) a.row_loss[row] = 0.f;
      if constexpr (kGrad)
#pragma unroll
        for (int i = 0; i < kE; ++i)
          if (lane + 32 * i < n) store_elem(dz, lane + 32 * i, sizeof(T) == 2, 0.f);
      continue;
    }
    float v[kE];
#pragma unroll
    for (int i = 0; i < kE; ++i) v[i] = lane + 32 * i < n ? load_elem(z, lane + 32 * i, sizeof(T) == 2) : -INFINITY;
    if constexpr (kGrad)
      if (worker < 0 || workers.begin[worker + 1] <= row) {
        while (workers.begin[++worker + 1] <= row) {}
        int rows = s_n;
        if (worker != first_worker)
          rows = __reduce_add_sync(0xffffffffu, count_rows(a.counts, workers.begin[worker], workers.begin[worker + 1], lane, 32));
        scale = a.grad_scale * a.t / (float)rows;
      }
    float top = v[0];
#pragma unroll
    for (int i = 1; i < kE; ++i) top = fmaxf(top, v[i]);
    top = warp_max(top);
    const float e = ceilf(top * c), ref = soft_ref(e);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kE; ++i) v[i] = exp2_fast(fmaf(v[i], c, ref)), s += v[i];
    const Soft soft = {e, warp_sum(s)};
    if (!soft_holds(soft)) {
      if (lane == 0) a.row_loss[row] = __uint_as_float(kLeft);
      left = true;
      continue;
    }
    // The entries, with their logits before the gradient may take their place.
    const Entry* entries = a.entries + row * a.top;
    float cross = 0.f;
    for (int k0 = lane; k0 < a.top; k0 += 128) {
      Entry entry[4];
      float logit[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) entry[j] = k0 + 32 * j < a.top ? entries[k0 + 32 * j] : Entry{-1, 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j) logit[j] = entry[j].id >= 0 ? load_elem(z, entry[j].id, sizeof(T) == 2) : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (entry[j].id >= 0) {
          cross = fmaf(entry[j].p, soft_log(soft, logit[j], c), cross);
          if constexpr (kGrad) sub[entry[j].id] = entry[j].p * scale;
        }
    }
    cross = warp_sum(cross);
    const float kl = lane == 0 || kFine ? a.plogp[row] - cross : 0.f;
    if (kFine && !(kl >= a.min_kl)) {
      if (lane == 0) a.row_loss[row] = __uint_as_float(kLeft);
      left = true;
      if constexpr (kGrad) {
        __syncwarp();
        for (int i = lane; i < n; i += 32) sub[i] = 0.f;
        __syncwarp();
      }
      continue;
    }
    if (lane == 0) a.row_loss[row] = a.t * a.t * kl;
    if constexpr (kGrad) {
      const float qs = scale / soft.s;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        const int col = lane + 32 * i;
        if (col < n) store_elem(dz, col, sizeof(T) == 2, fmaf(v[i], qs, -sub[col]));
        sub[col] = 0.f;
      }
      __syncwarp();
    }
  }
  if (left) {
    __syncwarp();
    left_rows<T, kGrad, true>(a, workers, first, last, 1, nullptr);
  }
}

// --------------------------------------------------- rows in shared memory
// A row is taken in chunks of 16 bytes that start on 16 bytes; its first chunk
// may begin before it (in the row before), its last is filled up with what is
// masked.  The chunks are split over the blocks of a cluster, and a block's
// over its threads, which each copy, read and write their own: no barrier but
// those of the sums.  For the gradient a block holds its part of the row; as
// soon as a thread has written the gradient of a batch of kBatch chunks it
// starts the copies of the next row's batch into the same place, which go on
// while the sums are joined and the other block of the SM computes.  For the
// losses alone a block holds the kDepth batches that come next.
//
// Bound by memory and by instructions about equally: 8192 rows of 50000 bf16 with
// their gradient in 349 us (floor 255; when it took 345, 289 with no exponential at all, 310 with one
// of the two), 513 of 131101 fp32 in 117 (floor 83; the same without exponentials:
// ten rounds of clusters for 9.3 of work).  Losses alone: 2048 rows of 50000 fp32 in
// 68 us (floor 64).
//
// With two exponentials an element (8.2 instructions an element without any
// bookkeeping) tests would cost time, so the batches that every thread has whole
// run without, at addresses that differ by constants (kThreads is the block's size
// where it is not 0), and what is left, and the ends of rows, chunk by chunk.
template <typename T>
struct Chunk;
template <>
struct Chunk<float> {
  static constexpr int kVec = 4;
  float4 r;
  __device__ __forceinline__ void clear() { r = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
  __device__ __forceinline__ void get(Pair (&v)[2]) const { v[0] = Pair(r.x, r.y), v[1] = Pair(r.z, r.w); }
  __device__ __forceinline__ float max() const { return fmaxf(fmaxf(r.x, r.y), fmaxf(r.z, r.w)); }
  // Keeps elements [lo, hi), the others are -inf.  (Not inlined: it would be
  // run under a false predicate by every chunk.)
  __device__ __noinline__ static float4 mask(float4 r, int lo, int hi) {
    r.x = 0 >= lo && 0 < hi ? r.x : -INFINITY, r.y = 1 >= lo && 1 < hi ? r.y : -INFINITY;
    r.z = 2 >= lo && 2 < hi ? r.z : -INFINITY, r.w = 3 >= lo && 3 < hi ? r.w : -INFINITY;
    return r;
  }
};
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int kVec = 8;
  uint4 r;
  __device__ __forceinline__ void clear() { r = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
  __device__ __forceinline__ void get(Pair (&v)[4]) const {
    v[0] = Pair(bf16_lo(r.x), bf16_hi(r.x)), v[1] = Pair(bf16_lo(r.y), bf16_hi(r.y));
    v[2] = Pair(bf16_lo(r.z), bf16_hi(r.z)), v[3] = Pair(bf16_lo(r.w), bf16_hi(r.w));
  }
  __device__ __forceinline__ static __nv_bfloat162 pair(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
  __device__ __forceinline__ float max() const {
    const float2 m = __bfloat1622float2(__hmax2(__hmax2(pair(r.x), pair(r.y)), __hmax2(pair(r.z), pair(r.w))));
    return fmaxf(m.x, m.y);
  }
  __device__ __noinline__ static uint4 mask(uint4 r, int lo, int hi) {
    uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * i < lo || 2 * i >= hi) w[i] = (w[i] & 0xffff0000u) | 0xff80u;
      if (2 * i + 1 < lo || 2 * i + 1 >= hi) w[i] = (w[i] & 0xffffu) | 0xff800000u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The elements of a row up to its first whole 16 bytes (head) and from body_end on
// are taken one at a time.
template <typename T>
struct RowSpan {
  static constexpr int kVec = 16 / sizeof(T);
  int head, body_end;
  __device__ RowSpan(const T* p, int n) {
    const int off = (int)(reinterpret_cast<uintptr_t>(p) % 16) / (int)sizeof(T);
    head = off ? min(kVec - off, n) : 0;
    body_end = head + (n - head) / kVec * kVec;
  }
};

// Losses alone, a warp a row at any address, kWarpBatch vectors a lane under way
// and no barrier.  Bound by memory where rows are many (8192 rows of 50000: fp32 239
// us, bf16 132; a block a row, as below, took 262 and 153), by latency else (4479
// of 6130 bf16 19 us for 33, 600 of 2000 8 for 13).
template <typename T>
__global__ void __launch_bounds__(kShortWarps * 32)
warp_losses_kernel(const RowArgs a) {
  constexpr int kVec = RowSpan<T>::kVec;
  allow_next_kernel();
  wait_for_kernel_before();
  const int lane = threadIdx.x & 31, n = a.vocab;
  const int64_t row = (int64_t)blockIdx.x * kShortWarps + threadIdx.x / 32;
  if (row >= a.rows) return;
  if (!a.counts[row]) {
    if (lane == 0) a.row_loss[row] = 0.f;
    return;
  }
  const float c = a.inv_t * kLog2e;
  const Pair cc(c, c);
  const T* z = static_cast<const T*>(a.z) + row * a.ld_z;
  const RowSpan<T> span(z, n);
  // The ends, fewer than 32 elements.
  const int ends = span.head + n - span.body_end;
  Soft soft = {-INFINITY, 0.f};
  if (lane < ends) {
    const float v = load_elem(z, lane < span.head ? lane : lane - span.head + span.body_end, sizeof(T) == 2);
    soft_raise(soft, v, c);
    soft.s += exp2_fast(fmaf(v, c, soft_ref(soft.e)));
  }
  __syncwarp();
  using Raw = decltype(Chunk<T>::r);
  const Raw* body = reinterpret_cast<const Raw*>(z + span.head);
  const int vecs = (span.body_end - span.head) / kVec;
  for (int at = lane; at - lane < vecs; at += 32 * kWarpBatch) {
    Chunk<T> x[kWarpBatch];
#pragma unroll
    for (int i = 0; i < kWarpBatch; ++i) {
      x[i].clear();
      if (at + 32 * i < vecs) x[i].r = __ldcs(body + at + 32 * i);
    }
    float top = x[0].max();
#pragma unroll
    for (int i = 1; i < kWarpBatch; ++i) top = fmaxf(top, x[i].max());
    soft_raise(soft, top, c);
    const Pair ref(soft_ref(soft.e), soft_ref(soft.e));
    Pair sum(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kWarpBatch; ++i) {
      Pair v[kVec / 2];
      x[i].get(v);
#pragma unroll
      for (int q = 0; q < kVec / 2; ++q) {
        const Pair e = fma(v[q], cc, ref);
        sum = sum + Pair(exp2_fast(e.lo()), exp2_fast(e.hi()));
      }
    }
    soft.s += sum.lo() + sum.hi();
  }
  __syncwarp();
  soft = warp_join(soft);
  if (!soft_holds(soft)) {
    left_row<T, false, true>(a, row, 0.0, nullptr);
    return;
  }
  const Entry* entries = a.entries + row * a.top;
  float cross = 0.f;
  for (int k0 = lane; k0 < a.top; k0 += 128) {
    Entry entry[4];
    float logit[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) entry[j] = k0 + 32 * j < a.top ? entries[k0 + 32 * j] : Entry{-1, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) logit[j] = entry[j].id >= 0 ? load_elem(z, entry[j].id, sizeof(T) == 2) : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (entry[j].id >= 0) cross = fmaf(entry[j].p, soft_log(soft, logit[j], c), cross);
  }
  cross = warp_sum(cross);
  const float kl = a.plogp[row] - cross;
  if (a.min_kl > 0.f && !(kl >= a.min_kl)) {
    left_row<T, false, true>(a, row, 0.0, nullptr);
    return;
  }
  if (lane == 0) a.row_loss[row] = a.t * a.t * kl;
}

// A thread's chunks of a row: q = 0 .. n - 1 at element q * stride of `at`,
// which may lie before the row (then the first chunk's first elements do).
struct Mine {
  int64_t at;     // element of the buffer where chunk 0 starts
  int col;        // its column
  int n;
  uint32_t ends;  // batches with an end of the row in this warp
};

// The rows first, first + step, ... that count.  A warp looks up 32 of them at
// a time.
struct RowWalk {
  int64_t base, step;  // row of bit 0
  uint32_t counts, rows;  // rows of the 32 that count, and that are there, from bit `at` on
  __device__ __forceinline__ RowWalk(const RowArgs& a, int64_t first, int64_t step) : base(first), step(step) { look(a); }
  __device__ __forceinline__ void look(const RowArgs& a) {
    const int64_t r = base + (threadIdx.x & 31) * step;
    rows = __ballot_sync(0xffffffffu, r < a.rows);
    counts = __ballot_sync(0xffffffffu, r < a.rows && a.counts[r]);
  }
  // The next row that counts (a.rows: none); skip(row) for those before it
  // that do not.
  template <typename F>
  __device__ __forceinline__ int64_t next(const RowArgs& a, F skip) {
    while (rows) {
      const int at = __ffs(rows) - 1;
      const uint32_t bit = 1u << at;
      const bool hit = counts & bit;
      const int64_t row = base + at * step;
      rows &= ~bit;
      if (!rows) {
        base += 32 * step;
        look(a);
      }
      if (hit) return row;
      skip(row);
    }
    return a.rows;
  }
};

template <typename T, bool kGrad, int kThreads>
__global__ void __launch_bounds__(kGrad ? kHeldThreads : kStreamThreads, 2)
held_rows_kernel(const RowArgs a, const __grid_constant__ WorkerRows workers, int slice) {
  constexpr int kVec = Chunk<T>::kVec, kBatch = kGrad ? kHeldBatch : kStreamBatch;
  constexpr int kMaxWarps = (kGrad ? kHeldThreads : kStreamThreads) / 32;
  // The block's chunks (for the losses kDepth batches), and the entries' logits.
  extern __shared__ __align__(16) uint8_t held[];
  __shared__ __align__(8) Soft s_soft[2][kMaxWarps];
  __shared__ Soft s_block[2][kMaxCluster];
  __shared__ float s_cross[kMaxWarps];
  __shared__ int s_n;
  allow_next_kernel();
  wait_for_kernel_before();
  const int threads = kThreads ? kThreads : blockDim.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = threads / 32;
  // Whole batches of every thread, and one more of what is left.
  const int full = slice / (kBatch * threads), batches = full + 1;
  Chunk<T>* const mine = reinterpret_cast<Chunk<T>*>(held) + threadIdx.x;
  float* const entry_z = reinterpret_cast<float*>(held + (size_t)(kGrad ? slice : kDepth * kBatch * threads) * 16);
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const int64_t step = gridDim.x / ranks;
  const int first = rank * slice, stride = threads * kVec;
  const float c = a.inv_t * kLog2e;
  const Pair cc(c, c);
  const T* const z_all = static_cast<const T*>(a.z);
  T* const dz_all = static_cast<T*>(a.dz);

  auto shift_of = [&](int64_t row) { return (int)(row * a.ld_z % kVec); };
  auto mine_of = [&](int64_t row) {
    const int shift = shift_of(row), chunk = first + threadIdx.x;
    const int end = min(first + slice, (a.vocab + shift + kVec - 1) / kVec);  // the row's chunks, and this block's
    Mine m;
    m.col = chunk * kVec - shift;
    m.at = row * a.ld_z + m.col;
    m.n = chunk < end ? (end - chunk + threads - 1) / threads : 0;
    // The whole batches of this warp that are not whole in this row: with its
    // first chunk, or its last, or after it.
    uint32_t ends = m.n > 0 && m.col < 0 ? 1u : 0u;
    if (m.n > 0 && m.col + (m.n - 1) * stride + kVec > a.vocab) ends |= 1u << min((m.n - 1) / kBatch, 31);
    if (m.n < full * kBatch) ends |= ~0u << min(m.n / kBatch, 31);
    m.ends = __reduce_or_sync(0xffffffffu, ends);
    return m;
  };
  auto plain = [&](const Mine& m, int b) { return b < full && !(m.ends >> min(b, 31) & 1); };
  auto whole = [&](int col) { return col >= 0 && col + kVec <= a.vocab; };
  // Copies of a batch (what a chunk has after the row's end is not read).
  auto fetch = [&](const Mine& m, int b, int slot) {
    Chunk<T>* to = mine + slot * kBatch * threads;
    const T* from = z_all + m.at + b * kBatch * stride;
    if (plain(m, b)) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) copy_async<16, true>(to + i * threads, from + i * stride, 16);
    } else {
#pragma unroll 1
      for (int i = 0; i < kBatch && b * kBatch + i < m.n; ++i)
        copy_async<16, false>(to + i * threads, from + i * stride,
                              min(a.vocab - (m.col + (b * kBatch + i) * stride), kVec) * (int)sizeof(T));
      __syncwarp();
    }
    copy_commit();
  };
  auto zero_row = [&](int64_t row) {
    if (rank == 0 && threadIdx.x == 0) a.row_loss[row] = 0.f;
    if (kGrad) {
      const Mine m = mine_of(row);
      T* dz = dz_all + row * a.ld_dz;
      for (int q = 0; q < m.n; ++q) {
        const int col = m.col + q * stride;
        if (col >= 0 && col + kVec <= a.vocab) {
          __stcs(reinterpret_cast<uint4*>(dz + col), make_uint4(0, 0, 0, 0));
        } else {
          for (int i = max(col, 0); i < min(col + kVec, a.vocab); ++i) store_elem(dz, i, sizeof(T) == 2, 0.f);
        }
      }
      __syncwarp();
    }
  };

  if (ranks > 1) cluster_sync();  // all blocks run before one writes to another
  // Rows of this block that count, two walks over them: `far` is the row whose
  // batches are fetched next, `row` the one at work.  The first one also does
  // what there is to do for the rows that do not count.
  RowWalk far_walk(a, blockIdx.x / ranks, step), walk = far_walk;
  int64_t far = far_walk.next(a, zero_row), row = walk.next(a, [](int64_t) {});
  Mine now = row < a.rows ? mine_of(row) : Mine{0, 0, 0, ~0u}, fetched = now;
  int ahead = 0;
  auto fetch_next = [&](int slot) {
    fetch(fetched, ahead, slot);
    if (++ahead == batches) {
      ahead = 0;
      far = far_walk.next(a, zero_row);
      fetched = far < a.rows ? mine_of(far) : Mine{0, 0, 0, ~0u};
    }
  };
  for (int b = 0; b < (kGrad ? batches : kDepth); ++b) fetch_next(b);
  int worker = -1, turn = 0, slot = 0;
  float scale = 0.f;
  bool left = false;
  // Each thread's first entry, a row ahead, so that nothing waits for it.
  const Entry none = {-1, 0.f};
  Entry entry_next = row < a.rows && (int)threadIdx.x < a.top ? a.entries[row * a.top + threadIdx.x] : none;
  while (row < a.rows) {
    const int64_t row_next = walk.next(a, [](int64_t) {});
    // The entries' logits, before the gradient may take their place.
    const Entry* entries = a.entries + row * a.top;
    const Entry entry = entry_next;
    float logit = 0.f;
    if (entry.id >= 0) logit = load_elem(a.z, row * a.ld_z + entry.id, sizeof(T) == 2);
    entry_next = row_next < a.rows && (int)threadIdx.x < a.top ? a.entries[row_next * a.top + threadIdx.x] : none;
    for (int k0 = threadIdx.x + threads; k0 < a.top; k0 += 4 * threads) {
      int id[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) id[i] = k0 + i * threads < a.top ? entries[k0 + i * threads].id : -1;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (id[i] >= 0) entry_z[k0 + i * threads] = load_elem(a.z, row * a.ld_z + id[i], sizeof(T) == 2);
    }
    const float plogp = threadIdx.x == 0 ? a.plogp[row] : 0.f;

    Soft soft = {-INFINITY, 0.f};
    for (int b = 0; b < batches; ++b) {
      // What may be on its way still: the batches after this one, for the
      // losses the kDepth - 1 that follow.
      if constexpr (kGrad) {
        const int out = full - b;
        if (out >= 3) copy_wait<3>();
        else if (out == 2) copy_wait<2>();
        else if (out == 1) copy_wait<1>();
        else copy_wait<0>();
      } else {
        copy_wait<kDepth - 1>();
      }
      const Chunk<T>* from = mine + (kGrad ? b : slot) * kBatch * threads;
      Chunk<T> x[kBatch];
      if (plain(now, b)) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) x[i] = from[i * threads];
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int col = now.col + (b * kBatch + i) * stride;
          x[i].clear();
          if (b * kBatch + i < now.n) x[i] = from[i * threads];
          if (b * kBatch + i < now.n && !whole(col)) x[i].r = Chunk<T>::mask(x[i].r, -col, a.vocab - col);
        }
        __syncwarp();
      }
      float top = x[0].max();
#pragma unroll
      for (int i = 1; i < kBatch; ++i) top = fmaxf(top, x[i].max());
      soft_raise(soft, top, c);
      const Pair ref(soft_ref(soft.e), soft_ref(soft.e));
      Pair sum(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        Pair v[kVec / 2];
        x[i].get(v);
#pragma unroll
        for (int q = 0; q < kVec / 2; ++q) {
          const Pair e = fma(v[q], cc, ref);
          sum = sum + Pair(exp2_fast(e.lo()), exp2_fast(e.hi()));
        }
      }
      soft.s += sum.lo() + sum.hi();
      if constexpr (!kGrad) {
        __syncwarp();
        fetch_next(slot);
        slot = slot == kDepth - 1 ? 0 : slot + 1;
      }
    }
    __syncwarp();
    soft = warp_join(soft);
    if (lane == 0) s_soft[turn][warp] = soft;
    __syncthreads();
    // Every warp joins the warps' parts, in the same order of lanes.
    soft = warp_join(lane < warps ? s_soft[turn][lane] : Soft{-INFINITY, 0.f});
    if (ranks > 1) {
      if (threadIdx.x < ranks) {
        uint32_t at;
        asm("mapa.shared::cluster.u32 %0, %1, %2;"
            : "=r"(at)
            : "r"((uint32_t)__cvta_generic_to_shared(&s_block[turn][rank])), "r"(threadIdx.x));
        asm volatile("st.shared::cluster.f32 [%0], %1;\n\tst.shared::cluster.f32 [%0+4], %2;" ::"r"(at), "f"(soft.e), "f"(soft.s)
                     : "memory");
      }
      cluster_sync();
      soft = s_block[turn][0];
      for (uint32_t i = 1; i < ranks; ++i) soft = soft_join(soft, s_block[turn][i]);
    }

    bool holds = soft_holds(soft);  // the same in all blocks of a cluster
    // Loss: sum p log q of the entries, a warp's part each.
    float cross = entry.id >= 0 ? entry.p * soft_log(soft, logit, c) : 0.f;
    for (int k = threadIdx.x + threads; k < a.top; k += threads)
      if (entries[k].id >= 0) cross = fmaf(entries[k].p, soft_log(soft, entry_z[k], c), cross);
    cross = warp_sum(cross);
    if (lane == 0) s_cross[warp] = cross;
    if (a.min_kl > 0.f) {
      __syncthreads();
      float kl = a.plogp[row];
      for (int w = 0; w < warps; ++w) kl -= s_cross[w];
      holds &= kl >= a.min_kl;
    }
    left |= !holds;
    if constexpr (kGrad) {
      if (worker < 0 || workers.begin[worker + 1] <= row) {
        // The rows that count of this row's worker.
        while (workers.begin[++worker + 1] <= row) {}
        const int n = __reduce_add_sync(0xffffffffu, count_rows(a.counts, workers.begin[worker], workers.begin[worker + 1], threadIdx.x, threads));
        if (threadIdx.x == 0) s_n = 0;
        __syncthreads();
        if (lane == 0) atomicAdd(&s_n, n);
        __syncthreads();
        scale = a.grad_scale * a.t / (float)s_n;
      }
      const float qs = scale / soft.s;
      const Pair ref(soft_ref(soft.e), soft_ref(soft.e)), qq(qs, qs);
      T* dz = dz_all + row * a.ld_dz + now.col;
      auto gradient = [&](const Chunk<T>& x, float (&o)[kVec]) {
        Pair v[kVec / 2];
        x.get(v);
#pragma unroll
        for (int q = 0; q < kVec / 2; ++q) {
          const Pair e = fma(v[q], cc, ref), g = Pair(exp2_fast(e.lo()), exp2_fast(e.hi())) * qq;
          o[2 * q] = g.lo(), o[2 * q + 1] = g.hi();
        }
      };
      if (!holds) now.n = 0, now.ends = ~0u;  // writes nothing
      for (int b = 0; b < batches; ++b, dz += kBatch * stride) {
        const Chunk<T>* from = mine + b * kBatch * threads;
        if (plain(now, b)) {
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            float o[kVec];
            gradient(from[i * threads], o);
            store_stream<T, kVec>(dz + i * stride, o);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < kBatch && b * kBatch + i < now.n; ++i) {
            const int col = now.col + (b * kBatch + i) * stride;
            float o[kVec];
            gradient(from[i * threads], o);
            if (whole(col)) {
              store_stream<T, kVec>(dz + i * stride, o);
            } else {
#pragma unroll
              for (int q = 0; q < kVec; ++q)
                if (col + q >= 0 && col + q < a.vocab) store_elem(dz, i * stride + q, sizeof(T) == 2, o[q]);
            }
          }
        }
        __syncwarp();
        fetch_next(b);
      }
      __syncthreads();
      // The entries' elements of this block's part of the row.
      const int shift = shift_of(row);
      auto fix = [&](Entry e, float z) {
        const int at = e.id >= 0 ? (e.id + shift) / kVec - first : -1;
        if (at >= 0 && at < slice && holds)
          store_elem(dz_all, row * a.ld_dz + e.id, sizeof(T) == 2, exp2_fast(fmaf(z, c, soft_ref(soft.e))) * qs - e.p * scale);
      };
      fix(entry, logit);
      for (int k = threadIdx.x + threads; k < a.top; k += threads) fix(entries[k], entry_z[k]);
    } else {
      __syncthreads();
    }
    if (rank == 0 && threadIdx.x == 0) {
      float x = 0.f;
      for (int w = 0; w < warps; ++w) x += s_cross[w];
      a.row_loss[row] = holds ? a.t * a.t * (plogp - x) : __uint_as_float(kLeft);
    }
    row = row_next;
    now = row < a.rows ? mine_of(row) : Mine{0, 0, 0, ~0u};
    turn ^= 1;
  }
  if (ranks > 1) cluster_sync();
  if (left && rank == 0) {
    __syncthreads();
    left_rows<T, kGrad, false>(a, workers, blockIdx.x / ranks, a.rows, step, reinterpret_cast<double*>(s_soft));
  }
}

// ------------------------------------------------------- rows of any address
// Where buffers do not start on 16 bytes, logits and gradient lie differently
// within them, or a row is too long for a cluster's shared memory: the second
// pass reads the row again.  Elements before the first and after the last
// whole 16 bytes are taken one at a time.  (2048 rows of 50000 with their gradient,
// one element past 16 bytes: bf16 142 us, fp32 269; on 16 bytes, held: 107 and 163.)
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
rows_kernel(const RowArgs a, const __grid_constant__ WorkerRows workers) {
  constexpr int kVec = RowSpan<T>::kVec;
  __shared__ __align__(8) Soft s_soft[kRowThreads / 32];
  __shared__ int s_n;
  __shared__ bool s_off;
  allow_next_kernel();
  wait_for_kernel_before();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, n = a.vocab;
  const float c = a.inv_t * kLog2e;
  int worker = -1;
  float scale = 0.f;
  bool left = false;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* z = static_cast<const T*>(a.z) + row * a.ld_z;
    T* dz = a.dz ? static_cast<T*>(a.dz) + row * a.ld_dz : nullptr;
    if (!a.counts[row]) {
      if (threadIdx.x == 0) a.row_loss[row] = 0.f;
      if (dz)
        for (int i = threadIdx.x; i < n; i += kRowThreads) store_elem(dz, i, sizeof(T) == 2, 0.f);
      continue;
    }
    const RowSpan<T> span(z, n);
    Soft soft = {-INFINITY, 0.f};
    auto add = [&](const auto& v) {
      float top = v[0];
      for (float x : v) top = fmaxf(top, x);
      soft_raise(soft, top, c);
      for (float x : v) soft.s += exp2_fast(fmaf(x, c, soft_ref(soft.e)));
    };
    for (int i = threadIdx.x; i < span.head + (n - span.body_end); i += kRowThreads) {
      const float v[1] = {load_elem(z, i < span.head ? i : i - span.head + span.body_end, sizeof(T) == 2)};
      add(v);
    }
#pragma unroll 2
    for (int i = span.head + threadIdx.x * kVec; i < span.body_end; i += kRowThreads * kVec) {
      float v[kVec];
      unpack(*reinterpret_cast<const typename RawVec<T, kVec>::type*>(z + i), v);
      add(v);
    }
    soft = warp_join(soft);
    __syncthreads();  // the row before is done with the shared values
    if (lane == 0) s_soft[warp] = soft;
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    soft = s_soft[0];
    for (int i = 1; i < kRowThreads / 32; ++i) soft = soft_join(soft, s_soft[i]);
    if (!soft_holds(soft)) {
      if (threadIdx.x == 0) a.row_loss[row] = __uint_as_float(kLeft);
      left = true;
      continue;
    }
    const Entry* entries = a.entries + row * a.top;
    if (warp == 0) {
      float x = 0.f;
      for (int k = lane; k < a.top; k += 32) {
        const Entry e = entries[k];
        if (e.id >= 0) x = fmaf(e.p, soft_log(soft, load_elem(z, e.id, sizeof(T) == 2), c), x);
      }
      const float kl = a.plogp[row] - warp_sum(x);
      const bool off = a.min_kl > 0.f && !(kl >= a.min_kl);
      if (lane == 0) a.row_loss[row] = off ? __uint_as_float(kLeft) : a.t * a.t * kl, s_off = off;
    }
    if (a.min_kl > 0.f) {
      __syncthreads();
      if (s_off) {
        left = true;
        continue;
      }
    }
    if (!dz) continue;
    if (worker < 0 || workers.begin[worker + 1] <= row) {
      // The rows of this row's worker that count.
      while (workers.begin[++worker + 1] <= row) {}
      const int cnt = __reduce_add_sync(0xffffffffu, count_rows(a.counts, workers.begin[worker], workers.begin[worker + 1], threadIdx.x, kRowThreads));
      if (lane == 0) atomicAdd(&s_n, cnt);
      __syncthreads();
      scale = a.grad_scale * a.t / (float)s_n;
    }
    const float qs = scale / soft.s, ref = soft_ref(soft.e);
    // Entries' logits are read before the gradient may overwrite them.
    float fix[kMaxTop / kRowThreads];
    for (int i = 0, k = threadIdx.x; k < a.top; ++i, k += kRowThreads) {
      const Entry e = entries[k];
      if (e.id >= 0) fix[i] = exp2_fast(fmaf(load_elem(z, e.id, sizeof(T) == 2), c, ref)) * qs - e.p * scale;
    }
    __syncthreads();
    const RowSpan<T> out(dz, n);
    if (out.head == span.head) {
      for (int i = threadIdx.x; i < span.head + (n - span.body_end); i += kRowThreads) {
        const int at = i < span.head ? i : i - span.head + span.body_end;
        store_elem(dz, at, sizeof(T) == 2, exp2_fast(fmaf(load_elem(z, at, sizeof(T) == 2), c, ref)) * qs);
      }
#pragma unroll 4
      for (int i = span.head + threadIdx.x * kVec; i < span.body_end; i += kRowThreads * kVec) {
        float v[kVec];
        unpack(*reinterpret_cast<const typename RawVec<T, kVec>::type*>(z + i), v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = exp2_fast(fmaf(v[j], c, ref)) * qs;
        store_stream<T, kVec>(dz + i, v);
      }
    } else {
      for (int i = threadIdx.x; i < n; i += kRowThreads)
        store_elem(dz, i, sizeof(T) == 2, exp2_fast(fmaf(load_elem(z, i, sizeof(T) == 2), c, ref)) * qs);
    }
    __syncthreads();
    for (int i = 0, k = threadIdx.x; k < a.top; ++i, k += kRowThreads) {
      const int id = entries[k].id;
      if (id >= 0) store_elem(dz, id, sizeof(T) == 2, fix[i]);
    }
  }
  if (left) {
    __syncthreads();
    if (a.dz) left_rows<T, true, false>(a, workers, blockIdx.x, a.rows, gridDim.x, reinterpret_cast<double*>(s_soft));
    else left_rows<T, false, false>(a, workers, blockIdx.x, a.rows, gridDim.x, reinterpret_cast<double*>(s_soft));
  }
}

// ---------------------------------------------------------------- workers
// A block a worker, in a fixed order; 2 us, bound by latency.
__global__ void __launch_bounds__(kLossThreads)
worker_loss_kernel(const float* row_loss, const uint8_t* counts, float* loss, const __grid_constant__ WorkerRows workers) {
  __shared__ double s_sum[kLossThreads / 32];
  __shared__ int64_t s_n[kLossThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, m = blockIdx.x;
  wait_for_kernel_before();
  double sum = 0.0;
  int64_t n = 0;
#pragma unroll 4
  for (int64_t i = workers.begin[m] + threadIdx.x; i < workers.begin[m + 1]; i += kLossThreads) sum += row_loss[i], n += counts[i];
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o), n += __shfl_xor_sync(0xffffffffu, n, o);
  if (lane == 0) s_sum[warp] = sum, s_n[warp] = n;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kLossThreads / 32; ++i) sum += s_sum[i], n += s_n[i];
    loss[m] = (float)(sum / (double)(n > 0 ? n : 1));
  }
}

// Clusters of this launch that the device holds (`guess` if it cannot say),
// kept for the last configuration asked for.
template <auto K>
int resident_clusters(cudaLaunchConfig_t cfg, int guess) {
  struct Known {
    int dev = -1, ranks = 0, threads = 0, n = 0;
    size_t smem = 0;
  };
  static thread_local Known known;
  const int dev = current_device(), ranks = (int)cfg.attrs[0].val.clusterDim.x, threads = (int)cfg.blockDim.x;
  if (known.dev != dev || known.ranks != ranks || known.threads != threads || known.smem != cfg.dynamicSmemBytes) {
    cfg.gridDim = dim3((unsigned)ranks);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, K, &cfg) != cudaSuccess) cudaGetLastError(), n = 0;
    if (n < 1) n = guess < 1 ? 1 : guess;
    known.dev = dev, known.ranks = ranks, known.threads = threads, known.smem = cfg.dynamicSmemBytes, known.n = n;
  }
  return known.n;
}

// Launches the pass over the logits.
template <typename T>
void launch_rows(const RowArgs& a, const WorkerRows& workers, cudaStream_t st) {
  constexpr int kVec = Chunk<T>::kVec;
  const int sms = current_sms();
  if (a.vocab <= kShortCols) {
    auto launch_one = [&](auto grad, auto per_lane, auto fine) {
      constexpr auto k = short_rows_kernel<T, decltype(grad)::value, decltype(per_lane)::value, decltype(fine)::value>;
      const int64_t most = (int64_t)sms * resident_blocks<k>(kShortWarps * 32, 0) * kShortWarps;
      const int per_warp = (int)ceil_div(a.rows, most);
      launch_after(k, dim3((unsigned)ceil_div(a.rows, (int64_t)per_warp * kShortWarps)), kShortWarps * 32, 0, st, a, workers,
                   per_warp);
    };
    auto launch = [&](auto grad, auto per_lane) {
      // (The test of a row's divergence costs the gradient's kernels up to 4 %.)
      if (!decltype(grad)::value || a.min_kl > 0.f) launch_one(grad, per_lane, std::true_type());
      else launch_one(grad, per_lane, std::bool_constant<!decltype(grad)::value>());
    };
    auto by_length = [&](auto grad) {
      if (a.vocab <= 128) launch(grad, std::integral_constant<int, 4>());
      else if (a.vocab <= 256) launch(grad, std::integral_constant<int, 8>());
      else if (a.vocab <= 512) launch(grad, std::integral_constant<int, 16>());
      else launch(grad, std::integral_constant<int, 32>());
    };
    if (a.dz) by_length(std::true_type());
    else by_length(std::false_type());
    return;  // the caller asks for the error
  }
  // Losses by a warp a row where rows are short, or so many that the SMs have
  // enough under way all the same: a warp alone reads 3 to 4 GB/s.
  if (!a.dz && (int64_t)a.vocab * (int64_t)sizeof(T) <= 8192 + 8192 * a.rows / (2 * sms)) {
    launch_after(warp_losses_kernel<T>, dim3((unsigned)ceil_div(a.rows, kShortWarps)), kShortWarps * 32, 0, st, a);
    return;  // the caller asks for the error
  }
  // More blocks than rows where rows are few.
  const int shift = a.ld_z % kVec ? kVec - 1 : 0;
  const int64_t chunks = ((int64_t)a.vocab + shift + kVec - 1) / kVec;
  int ranks = 1, threads = 0;
  while (ranks < kMaxCluster && a.rows * ranks * 2 <= sms && chunks >= 1024 * ranks) ranks *= 2;
  int64_t slice = 0, smem = 0, an_sm = 0;
  const auto plan = [&](int r) {
    const int batch = a.dz ? kHeldBatch : kStreamBatch, most = a.dz ? kHeldThreads : kStreamThreads;
    slice = ceil_div(chunks, r);
    const int64_t need = (int64_t)round_up((size_t)ceil_div(slice, batch), 32);
    if (a.dz) {
      // Blocks that an SM has shared memory and rows for, and their share of its
      // threads.  Eight at most (8000 rows of 3000 bf16, with six, eight, twelve: 50,
      // 46, 42 us; 5397 of 9487: 71, 66, 72; 2048 of 5000: 24, 21, 25).
      smem = slice * 16 + (int64_t)a.top * 4;
      an_sm = kSmSmem / (smem + 2048);
      const int64_t rows = ceil_div(a.rows * r, sms);
      an_sm = an_sm > rows ? rows : an_sm;
      an_sm = an_sm < 1 ? 1 : an_sm > 8 ? 8 : an_sm;
      threads = (int)(2 * most / an_sm / 32 * 32);
    } else {
      // Fewer threads a row, and more rows at a time, unless that leaves more SMs
      // without a row at the end: each row costs its bytes and the time of 64 KB
      // more (2048 rows of 50000, 128 or 512 threads: bf16 53 and 65 us, fp32 75
      // and 72; 924 of 13205 bf16: 16 and 26).
      threads = 256;
      int64_t least = INT64_MAX;
      for (int t = most; r == 1 && t >= 128; t /= 2) {
        const int64_t at_once = 2 * most / t, rounds = ceil_div(a.rows, at_once * sms);
        const int64_t cost = rounds * (at_once * chunks * 16 + 65536);
        if (cost < least) least = cost, threads = t;
      }
    }
    if (threads > most) threads = most;
    if (need < threads) threads = (int)need;
    if (!a.dz) smem = (int64_t)kDepth * batch * threads * 16 + (int64_t)a.top * 4;
    const int64_t room = kSmSmem / (smem + 2048), by_threads = 2 * most / threads;
    an_sm = room < by_threads ? room : by_threads;
    an_sm = an_sm < 1 ? 1 : an_sm > 32 ? 32 : an_sm;
  };
  // For the gradient a cluster of such a size holds a row that the SMs' shared
  // memory holds most of rows altogether, by two blocks an SM at least: that
  // decides the time (1371 rows of 80288 bf16: 112 us with 160 KB of rows an SM,
  // 133 with 120; 1000 of 131072: 126 with 197 KB, 147 with 131).
  if (a.dz) {
    int64_t most = -1;
    int best = ranks;
    for (int r = ranks; r <= kMaxCluster; r *= 2) {
      plan(r);
      if (smem + 2048 > kSmSmem) continue;
      const int64_t rows_held = an_sm == 1 && slice * 16 > 64 * 1024 ? slice / 2 : an_sm * slice;
      if (rows_held > most + most / 32) most = rows_held, best = r;
    }
    ranks = best;
  }
  plan(ranks);
  const bool apart = a.dz && (!aligned_to(a.dz, 16) || a.ld_dz % kVec != a.ld_z % kVec);
  if (aligned_to(a.z, 16) && !apart && smem + 1024 <= kSmSmem) {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem, cfg.stream = st;
    // A cluster, or a launch beside the kernel before (as launch_after's).  Not
    // both: a cluster that finds no place while that one still holds SMs would
    // be a second wave (513 rows of 131101 fp32: 174 us instead of 131).  And
    // no clusters of one block (5208 rows of 193 fp32: 45 us instead of 29).
    cudaLaunchAttribute attr;
    if (ranks > 1) {
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = (unsigned)ranks, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    } else {
      attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr.val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = &attr, cfg.numAttrs = 1;
    auto launch = [&](auto grad, auto block) {
      constexpr auto k = held_rows_kernel<T, decltype(grad)::value, decltype(block)::value>;
      resident_blocks<k>(32, 0);  // allows it the shared memory
      // Clusters that fit are fewer than the SMs would say, since a cluster
      // stays within a group of SMs; one that waits for its turn would come
      // last, with as many rows as the others had.
      int64_t units = ranks > 1 ? resident_clusters<k>(cfg, (int)(sms * an_sm / ranks)) : sms * an_sm;
      if (units > a.rows) units = a.rows;
      cfg.gridDim = dim3((unsigned)(units * ranks));
      cudaLaunchKernelEx(&cfg, k, a, workers, (int)slice);
    };
    auto by_block = [&](auto grad) {
      // (Sizes that long rows get have kernels of their own.)
      constexpr int kMost = decltype(grad)::value ? kHeldThreads : kStreamThreads;
      if (threads == kMost) launch(grad, std::integral_constant<int, kMost>());
      else if (threads == 256) launch(grad, std::integral_constant<int, 256>());
      else if (threads == 192) launch(grad, std::integral_constant<int, 192>());
      else if (threads == 128) launch(grad, std::integral_constant<int, 128>());
      else if constexpr (kMost == kHeldThreads) {
        if (threads == 96) launch(grad, std::integral_constant<int, 96>());
        else if (threads == 64) launch(grad, std::integral_constant<int, 64>());
        else launch(grad, std::integral_constant<int, 0>());
      } else {
        launch(grad, std::integral_constant<int, 0>());
      }
    };
    if (a.dz) by_block(std::true_type());
    else by_block(std::false_type());
    return;  // the caller asks for the error
  }
  const int64_t most = (int64_t)sms * 4;
  launch_after(rows_kernel<T>, dim3((unsigned)(a.rows < most ? a.rows : most)), kRowThreads, 0, st, a, workers);
}

struct Layout {
  size_t entries, plogp, counts, total;
};
Layout layout_of(int64_t rows, int top) {
  Layout l;
  l.entries = kWsHeaderBytes;
  l.plogp = l.entries + round_up((size_t)rows * top * sizeof(Entry), 256);
  l.counts = l.plogp + round_up((size_t)rows * 4, 256);
  l.total = l.counts + round_up((size_t)rows, 256);
  return l;
}

}  // namespace

extern "C" {

size_t signmuon_distill_workspace_bytes(int64_t rows, int top) {
  return rows < 0 || rows > kMaxVocab || top < 1 || top > kMaxTop ? 0 : layout_of(rows, top).total;
}

signmuon_status signmuon_distill_loss(int32_t vocab, int n_workers, const int64_t* row_begin, signmuon_dtype dtype,
                                      const void* logits, int64_t ld, int top, int ids_int64, const void* top_ids,
                                      signmuon_dtype top_dtype, const void* top_logits, float temperature,
                                      float grad_scale, float* loss, float* row_loss, void* dlogits, int64_t ld_d,
                                      void* workspace, size_t ws_bytes, void* stream) {
  if (vocab <= 0 || n_workers <= 0 || n_workers > SIGNMUON_MAX_WORKERS || !row_begin ||
      !valid_splits(row_begin, n_workers, row_begin[n_workers]) || !known_dtype(dtype) || !known_dtype(top_dtype) || top < 1 ||
      top > kMaxTop || ld < vocab || (dlogits && ld_d < vocab) || !loss || !(temperature >= 1e-6f && temperature <= 1e6f))
    return SIGNMUON_ERR_INVALID_ARG;
  const int64_t n = row_begin[n_workers];
  if (vocab > kMaxVocab || n > kMaxVocab) return SIGNMUON_ERR_UNSUPPORTED;
  if (n > 0 && (!logits || !top_ids || !top_logits || !row_loss)) return SIGNMUON_ERR_INVALID_ARG;
  const int zb = dtype_bytes(dtype);
  if (!aligned_to(logits, zb) || !aligned_to(dlogits, zb) || !aligned_to(top_ids, ids_int64 ? 8 : 4) ||
      !aligned_to(top_logits, dtype_bytes(top_dtype)) || !aligned_to(loss, 4) || !aligned_to(row_loss, 4))
    return SIGNMUON_ERR_ALIGNMENT;
  const Layout l = layout_of(n, top);
  const signmuon_status st = check_ws(workspace, ws_bytes, l.total);
  if (st) return st;
  const int64_t teacher_blocks = ceil_div(n, kTeacherWarps);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  RowArgs a = {};
  a.z = logits, a.ld_z = ld, a.dz = dlogits, a.ld_dz = ld_d;
  a.entries = reinterpret_cast<Entry*>(ws + l.entries);
  a.plogp = reinterpret_cast<float*>(ws + l.plogp);
  a.counts = ws + l.counts;
  a.row_loss = row_loss, a.rows = n, a.vocab = vocab, a.top = top;
  a.top_ids = top_ids, a.ids_wide = ids_int64 != 0, a.top_logits = top_logits, a.top_bf16 = top_dtype == SIGNMUON_BF16;
  a.t = temperature, a.inv_t = 1.f / temperature, a.grad_scale = grad_scale;
  a.min_kl = temperature > kFineT ? kFineKl : -INFINITY;
  WorkerRows workers = {};
  for (int m = 0; m <= n_workers; ++m) workers.begin[m] = row_begin[m];
  if (n) {
    auto teacher = [&](auto per) {
      constexpr int kPer = decltype(per)::value;
      constexpr size_t kSmem = kTeacherWarps * 32 * kPer * sizeof(Entry);
      resident_blocks<teacher_kernel<kPer>>(kTeacherWarps * 32, kSmem);  // allows it the shared memory
      teacher_kernel<kPer><<<(unsigned)teacher_blocks, kTeacherWarps * 32, kSmem, cs>>>(
          n, top, top_ids, ids_int64 != 0, top_logits, top_dtype == SIGNMUON_BF16, vocab, a.inv_t,
          reinterpret_cast<Entry*>(ws + l.entries), reinterpret_cast<float*>(ws + l.plogp), ws + l.counts);
    };
    if (top <= 32) teacher(std::integral_constant<int, 1>());
    else if (top <= 64) teacher(std::integral_constant<int, 2>());
    else if (top <= 128) teacher(std::integral_constant<int, 4>());
    else if (top <= 256) teacher(std::integral_constant<int, 8>());
    else if (top <= 512) teacher(std::integral_constant<int, 16>());
    else teacher(std::integral_constant<int, 32>());
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_status(e);
    if (dtype == SIGNMUON_F32) launch_rows<float>(a, workers, cs);
    else launch_rows<__nv_bfloat16>(a, workers, cs);
    if ((e = cudaGetLastError()) != cudaSuccess) return cuda_status(e);
  }
  launch_after(worker_loss_kernel, dim3((unsigned)n_workers), kLossThreads, 0, cs, row_loss, a.counts, loss, workers);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
