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
#include <cmath>

#include "layers.cuh"

using namespace signmuon;

namespace {

constexpr int kMaxTop = 1024;
constexpr int kTeacherWarps = 4;
constexpr int kRowThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;

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
__global__ void __launch_bounds__(kTeacherWarps * 32)
teacher_kernel(int64_t rows, int top, const void* __restrict__ ids, int wide, const void* __restrict__ logits, int bf16,
               int32_t vocab, float inv_t, Entry* __restrict__ entries, float* __restrict__ plogp, uint8_t* __restrict__ counts) {
  extern __shared__ Entry s_entries[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t row = (int64_t)blockIdx.x * kTeacherWarps + warp;
  if (row >= rows) return;
  Entry* mine = s_entries + warp * top;
  float top_u = -INFINITY;
  bool any = false, bad = false;
  for (int k = lane; k < top; k += 32) {
    const int64_t id = load_id(ids, row * top + k, wide);
    const float u = load_elem(logits, row * top + k, bf16);
    const bool in = id >= 0 && id < vocab && u != -INFINITY;
    mine[k] = {in ? (int32_t)id : -1, u};
    if (in) top_u = fmaxf(top_u, u), any = true, bad |= u != u;
  }
  any = __any_sync(0xffffffffu, any);
  // fmaxf drops a NaN: one among the entries makes the row NaN.
  top_u = __any_sync(0xffffffffu, bad) ? NAN : warp_max(top_u);
  float sum = 0.f;
  for (int k = lane; k < top; k += 32)
    if (mine[k].id >= 0) sum += expf((mine[k].p - top_u) * inv_t);
  sum = warp_sum(sum);
  const float log_sum = logf(sum), inv_sum = 1.f / sum;
  float h = 0.f;
  for (int k = lane; k < top; k += 32)
    if (mine[k].id >= 0) {
      const float x = (mine[k].p - top_u) * inv_t, p = expf(x) * inv_sum;
      if (p != 0.f) h = fmaf(p, x - log_sum, h);
      mine[k].p = p;
    }
  h = warp_sum(h);
  __syncwarp();
  // The first entry of an id holds all of the id's.
  for (int k = lane; k < top; k += 32) {
    Entry e = mine[k];
    if (e.id >= 0) {
      float p = 0.f;
      bool first = true;
      for (int j = 0; j < top; ++j) {
        const Entry o = mine[j];
        if (o.id == e.id) {
          p += o.p;
          first &= j >= k;
        }
      }
      e.id = first && p != 0.f ? e.id : -1;
      e.p = p;
    }
    entries[row * top + k] = e;
  }
  if (lane == 0) plogp[row] = h, counts[row] = any;
}

// ------------------------------------------------------------------- rows
struct RowArgs {
  const void* z;
  int64_t ld_z;
  void* dz;  // null: the losses alone
  int64_t ld_dz;
  const Entry* entries;
  const float* plogp;
  const uint8_t* counts;
  float* row_loss;
  int64_t rows;
  int32_t vocab, top, n_workers;
  float t, inv_t, grad_scale;
};

// Running maximum and sum of 2^((z - max) c).
struct Soft {
  float m, s;
};
__device__ __forceinline__ Soft soft_join(Soft a, Soft b, float c) {
  const float m = fmaxf(a.m, b.m);
  // An empty part has m = -inf and s = 0 and drops out.
  const float s = (a.m == -INFINITY ? a.s : a.s * exp2_fast((a.m - m) * c)) + (b.m == -INFINITY ? b.s : b.s * exp2_fast((b.m - m) * c));
  return {m, s};
}
template <int N>
__device__ __forceinline__ void soft_add(Soft& a, const float (&v)[N], float c) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
  if (m > a.m) {
    a.s = a.m == -INFINITY ? a.s : a.s * exp2_fast((a.m - m) * c);
    a.m = m;
  }
  // While nothing finite has come (m is -inf), differences are NaN unless
  // they are taken to 0; then every term is 2^-inf = 0.
  const float base = a.m == -INFINITY ? 0.f : a.m;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s += exp2_fast((v[i] - base) * c);
  a.s += s;
}

// Rows of any alignment: elements before the first and after the last whole
// 16 bytes are taken one at a time.
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

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
rows_kernel(const RowArgs a, const __grid_constant__ WorkerRows workers) {
  constexpr int kVec = RowSpan<T>::kVec;
  __shared__ Soft s_soft[kRowThreads / 32];
  __shared__ int s_n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, n = a.vocab;
  const float c = a.inv_t * kLog2e;
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
    for (int i = threadIdx.x; i < span.head + (n - span.body_end); i += kRowThreads) {
      float v[1] = {load_elem(z, i < span.head ? i : i - span.head + span.body_end, sizeof(T) == 2)};
      soft_add(soft, v, c);
    }
#pragma unroll 4
    for (int i = span.head + threadIdx.x * kVec; i < span.body_end; i += kRowThreads * kVec) {
      float v[kVec];
      unpack(*reinterpret_cast<const typename RawVec<T, kVec>::type*>(z + i), v);
      soft_add(soft, v, c);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
      soft = soft_join(soft, {__shfl_xor_sync(0xffffffffu, soft.m, o), __shfl_xor_sync(0xffffffffu, soft.s, o)}, c);
    __syncthreads();  // the row before is done with the shared values
    if (lane == 0) s_soft[warp] = soft;
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    soft = s_soft[0];
    for (int i = 1; i < kRowThreads / 32; ++i) soft = soft_join(soft, s_soft[i], c);
    const Entry* entries = a.entries + row * a.top;
    if (warp == 0) {
      float x = 0.f;
      for (int k = lane; k < a.top; k += 32) {
        const Entry e = entries[k];
        if (e.id >= 0) x = fmaf(e.p, (load_elem(z, e.id, sizeof(T) == 2) - soft.m) * a.inv_t, x);
      }
      x = warp_sum(x);
      if (lane == 0) a.row_loss[row] = a.t * a.t * (a.plogp[row] - x + logf(soft.s));
    }
    if (!dz) continue;
    // The rows of this worker that count.
    int m = 0;
    while (workers.begin[m + 1] <= row) ++m;
    int cnt = 0;
    for (int64_t i = workers.begin[m] + threadIdx.x; i < workers.begin[m + 1]; i += kRowThreads) cnt += a.counts[i];
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) atomicAdd(&s_n, cnt);
    __syncthreads();
    const float scale = a.grad_scale * a.t / (float)s_n, qs = scale / soft.s;
    // Entries' logits are read before the gradient may overwrite them.
    float fix[kMaxTop / kRowThreads];
    for (int i = 0, k = threadIdx.x; k < a.top; ++i, k += kRowThreads) {
      const Entry e = entries[k];
      if (e.id >= 0) fix[i] = exp2_fast((load_elem(z, e.id, sizeof(T) == 2) - soft.m) * c) * qs - e.p * scale;
    }
    __syncthreads();
    const RowSpan<T> out(dz, n);
    if (out.head == span.head) {
      for (int i = threadIdx.x; i < span.head + (n - span.body_end); i += kRowThreads) {
        const int at = i < span.head ? i : i - span.head + span.body_end;
        store_elem(dz, at, sizeof(T) == 2, exp2_fast((load_elem(z, at, sizeof(T) == 2) - soft.m) * c) * qs);
      }
#pragma unroll 4
      for (int i = span.head + threadIdx.x * kVec; i < span.body_end; i += kRowThreads * kVec) {
        float v[kVec];
        unpack(*reinterpret_cast<const typename RawVec<T, kVec>::type*>(z + i), v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = exp2_fast((v[j] - soft.m) * c) * qs;
        store_stream<T, kVec>(dz + i, v);
      }
    } else {
      for (int i = threadIdx.x; i < n; i += kRowThreads)
        store_elem(dz, i, sizeof(T) == 2, exp2_fast((load_elem(z, i, sizeof(T) == 2) - soft.m) * c) * qs);
    }
    __syncthreads();
    for (int i = 0, k = threadIdx.x; k < a.top; ++i, k += kRowThreads) {
      const int id = entries[k].id;
      if (id >= 0) store_elem(dz, id, sizeof(T) == 2, fix[i]);
    }
  }
}

// ---------------------------------------------------------------- workers
__global__ void __launch_bounds__(256)
worker_loss_kernel(const float* __restrict__ row_loss, const uint8_t* __restrict__ counts, float* __restrict__ loss,
                   const __grid_constant__ WorkerRows workers) {
  __shared__ double s_sum[8];
  __shared__ int64_t s_n[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, m = blockIdx.x;
  double sum = 0.0;
  int64_t n = 0;
  for (int64_t i = workers.begin[m] + threadIdx.x; i < workers.begin[m + 1]; i += 256) sum += row_loss[i], n += counts[i];
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o), n += __shfl_xor_sync(0xffffffffu, n, o);
  if (lane == 0) s_sum[warp] = sum, s_n[warp] = n;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) sum += s_sum[i], n += s_n[i];
    loss[m] = (float)(sum / (double)(n > 0 ? n : 1));
  }
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
  return rows < 0 || top < 1 || top > kMaxTop ? 0 : layout_of(rows, top).total;
}

signmuon_status signmuon_distill_loss(int32_t vocab, int n_workers, const int64_t* row_begin, signmuon_dtype dtype,
                                      const void* logits, int64_t ld, int top, int ids_int64, const void* top_ids,
                                      signmuon_dtype top_dtype, const void* top_logits, float temperature,
                                      float grad_scale, float* loss, float* row_loss, void* dlogits, int64_t ld_d,
                                      void* workspace, size_t ws_bytes, void* stream) {
  if (vocab <= 0 || n_workers <= 0 || n_workers > SIGNMUON_MAX_WORKERS || !row_begin ||
      !valid_splits(row_begin, n_workers, row_begin[n_workers]) || !known_dtype(dtype) || !known_dtype(top_dtype) || top < 1 ||
      top > kMaxTop || ld < vocab || (dlogits && ld_d < vocab) || !loss || !(temperature > 0.f) || std::isinf(temperature))
    return SIGNMUON_ERR_INVALID_ARG;
  const int64_t n = row_begin[n_workers];
  if (n > 0 && (!logits || !top_ids || !top_logits || !row_loss)) return SIGNMUON_ERR_INVALID_ARG;
  const int zb = dtype_bytes(dtype);
  if (!aligned_to(logits, zb) || !aligned_to(dlogits, zb) || !aligned_to(top_ids, ids_int64 ? 8 : 4) ||
      !aligned_to(top_logits, dtype_bytes(top_dtype)) || !aligned_to(loss, 4) || !aligned_to(row_loss, 4))
    return SIGNMUON_ERR_ALIGNMENT;
  const Layout l = layout_of(n, top);
  const signmuon_status st = check_ws(workspace, ws_bytes, l.total);
  if (st) return st;
  const int64_t teacher_blocks = ceil_div(n, kTeacherWarps);
  if (teacher_blocks > INT32_MAX) return SIGNMUON_ERR_UNSUPPORTED;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  RowArgs a = {};
  a.z = logits, a.ld_z = ld, a.dz = dlogits, a.ld_dz = ld_d;
  a.entries = reinterpret_cast<Entry*>(ws + l.entries);
  a.plogp = reinterpret_cast<float*>(ws + l.plogp);
  a.counts = ws + l.counts;
  a.row_loss = row_loss, a.rows = n, a.vocab = vocab, a.top = top, a.n_workers = n_workers;
  a.t = temperature, a.inv_t = 1.f / temperature, a.grad_scale = grad_scale;
  WorkerRows workers = {};
  for (int m = 0; m <= n_workers; ++m) workers.begin[m] = row_begin[m];
  if (n) {
    teacher_kernel<<<(unsigned)teacher_blocks, kTeacherWarps * 32, kTeacherWarps * top * sizeof(Entry), cs>>>(
        n, top, top_ids, ids_int64 != 0, top_logits, top_dtype == SIGNMUON_BF16, vocab, a.inv_t,
        reinterpret_cast<Entry*>(ws + l.entries), reinterpret_cast<float*>(ws + l.plogp), ws + l.counts);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_status(e);
    const int64_t most = (int64_t)current_sms() * 4;
    const unsigned grid = (unsigned)(n < most ? n : most);
    if (dtype == SIGNMUON_F32) rows_kernel<float><<<grid, kRowThreads, 0, cs>>>(a, workers);
    else rows_kernel<__nv_bfloat16><<<grid, kRowThreads, 0, cs>>>(a, workers);
    if ((e = cudaGetLastError()) != cudaSuccess) return cuda_status(e);
  }
  worker_loss_kernel<<<n_workers, 256, 0, cs>>>(row_loss, a.counts, loss, workers);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
