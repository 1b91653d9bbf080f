// Shared by the per-worker training operators (embedding.cu, layer_norm.cu,
// distill.cu): vector access to fp32 / bf16 rows, warp reductions, and the
// host-side checks of their entry points.
#pragma once

#include <atomic>
#include <type_traits>

#include "common.cuh"

namespace signmuon {

// ---------------------------------------------------------------------------
// Device: VEC consecutive elements of an fp32 or bf16 row as fp32.
// A row is read VEC elements at a time, VEC a power of two whose bytes
// (at most 16) divide the row's address and every element offset used.
// ---------------------------------------------------------------------------
template <typename T, int VEC>
struct RawVec;  // VEC elements as loaded, unconverted
template <> struct RawVec<float, 4> { using type = float4; };
template <> struct RawVec<float, 1> { using type = float; };
template <> struct RawVec<__nv_bfloat16, 8> { using type = uint4; };
template <> struct RawVec<__nv_bfloat16, 4> { using type = uint2; };
template <> struct RawVec<__nv_bfloat16, 2> { using type = uint32_t; };
template <> struct RawVec<__nv_bfloat16, 1> { using type = uint16_t; };

// The low / high bf16 of a word as fp32 (exact).
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void unpack(float4 r, float (&v)[4]) { v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w; }
__device__ __forceinline__ void unpack(float r, float (&v)[1]) { v[0] = r; }
__device__ __forceinline__ void unpack(uint4 r, float (&v)[8]) {
  v[0] = bf16_lo(r.x), v[1] = bf16_hi(r.x), v[2] = bf16_lo(r.y), v[3] = bf16_hi(r.y);
  v[4] = bf16_lo(r.z), v[5] = bf16_hi(r.z), v[6] = bf16_lo(r.w), v[7] = bf16_hi(r.w);
}
__device__ __forceinline__ void unpack(uint2 r, float (&v)[4]) {
  v[0] = bf16_lo(r.x), v[1] = bf16_hi(r.x), v[2] = bf16_lo(r.y), v[3] = bf16_hi(r.y);
}
__device__ __forceinline__ void unpack(uint32_t r, float (&v)[2]) { v[0] = bf16_lo(r), v[1] = bf16_hi(r); }
__device__ __forceinline__ void unpack(uint16_t r, float (&v)[1]) { v[0] = bf16_lo(r); }

// Two fp32 rounded (to nearest even) to a bf16 pair.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void pack(const float (&v)[4], float4& r) { r = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void pack(const float (&v)[1], float& r) { r = v[0]; }
__device__ __forceinline__ void pack(const float (&v)[8], uint4& r) {
  r = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void pack(const float (&v)[4], uint2& r) {
  r = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}
__device__ __forceinline__ void pack(const float (&v)[2], uint32_t& r) { r = pack_bf16(v[0], v[1]); }
__device__ __forceinline__ void pack(const float (&v)[1], uint16_t& r) {
  r = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
}

// Streamed rows are read once and written once: they pass L1 by and leave L2
// first.
template <typename T, int VEC>
__device__ __forceinline__ typename RawVec<T, VEC>::type load_stream(const T* p) {
  return __ldcs(reinterpret_cast<const typename RawVec<T, VEC>::type*>(p));
}
template <typename T, int VEC>
__device__ __forceinline__ void store_stream(T* p, const float (&v)[VEC]) {
  typename RawVec<T, VEC>::type r;
  pack(v, r);
  __stcs(reinterpret_cast<typename RawVec<T, VEC>::type*>(p), r);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  typename RawVec<T, VEC>::type r;
  pack(v, r);
  *reinterpret_cast<typename RawVec<T, VEC>::type*>(p) = r;
}

// Two fp32 in a register pair, and arithmetic on both with one instruction.
struct Pair {
  uint64_t v;
  __device__ __forceinline__ Pair() {}
  __device__ __forceinline__ Pair(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ float lo() const { return __uint_as_float((uint32_t)v); }
  __device__ __forceinline__ float hi() const { return __uint_as_float((uint32_t)(v >> 32)); }
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Asynchronous copies of 4 or 16 bytes to shared memory, of which only the
// first `valid` bytes are read and the others are zero; seen by the thread
// that issued them once its group is waited for.
template <int BYTES, bool kAll>
__device__ __forceinline__ void copy_async(void* smem, const void* global, int valid) {
  const uint32_t dst = (uint32_t)__cvta_generic_to_shared(smem);
  if constexpr (BYTES == 16 && kAll)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(global) : "memory");
  else if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(global), "r"(valid) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(global), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_elem(void* p, int64_t i, int bf16, float v) {
  if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(p)[i] = v;
}
__device__ __forceinline__ int64_t load_id(const void* ids, int64_t i, int wide) {
  return wide ? static_cast<const int64_t*>(ids)[i] : (int64_t) static_cast<const int32_t*>(ids)[i];
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A kernel that follows another one of the same call is launched while that
// one still runs (launch_after), which hides the launch itself: the first
// allows it when it starts, the second waits, before it reads or writes
// anything, until the first is done and its writes are seen.  What the first
// writes the second reads through plain pointers: const __restrict__ (or
// __ldg) would allow loads by the read-only path, or before the wait, of data
// that still changes.
__device__ __forceinline__ void allow_next_kernel() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------------------
// Host: a batch's rows by worker, as a kernel parameter.
// ---------------------------------------------------------------------------
struct WorkerRows {
  int64_t begin[SIGNMUON_MAX_WORKERS + 1];
};
struct WorkerBlocks {
  int32_t begin[SIGNMUON_MAX_WORKERS + 1];  // first block (of some launch) of each worker
};
struct WorkerPtrs {
  void* p[SIGNMUON_MAX_WORKERS];
};

// The worker that block b belongs to (workers without blocks are passed over).
__device__ __forceinline__ int worker_of_block(const WorkerBlocks& w, int n_workers, int b) {
  int lo = 0, hi = n_workers;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (w.begin[mid] <= b) lo = mid;
    else hi = mid;
  }
  return lo;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool known_dtype(signmuon_dtype t) { return t == SIGNMUON_F32 || t == SIGNMUON_BF16; }
inline int dtype_bytes(signmuon_dtype t) { return t == SIGNMUON_F32 ? 4 : 2; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// n_workers + 1 non-decreasing offsets from 0 to rows.
inline bool valid_splits(const int64_t* row_begin, int n_workers, int64_t rows) {
  if (!row_begin || n_workers <= 0 || n_workers > SIGNMUON_MAX_WORKERS) return false;
  if (row_begin[0] != 0 || row_begin[n_workers] != rows) return false;
  for (int m = 0; m < n_workers; ++m)
    if (row_begin[m + 1] < row_begin[m]) return false;
  return true;
}

inline signmuon_status check_ws(void* ws, size_t have, size_t need) {
  if (!ws || have < need) return SIGNMUON_ERR_WORKSPACE;
  return aligned_to(ws, 256) ? SIGNMUON_OK : SIGNMUON_ERR_ALIGNMENT;
}

// Columns a row may have (the grids of several kernels grow with them).
constexpr int kMaxCols = 1 << 20;

// The widest access (elements) for whole rows of `cols` elements: 16 bytes,
// for bf16 also 4 bytes, else one element; narrowed to what the address and
// the row stride of each buffer allow.
inline int vec_width(signmuon_dtype t, int64_t cols) {
  const int full = 16 / dtype_bytes(t);
  return cols % full == 0 ? full : (t == SIGNMUON_BF16 && cols % 2 == 0) ? 2 : 1;
}
inline int vec_narrow(int vec, signmuon_dtype t, const void* p, int64_t ld) {
  const int b = dtype_bytes(t);
  while (vec > 1 && (!aligned_to(p, (size_t)vec * b) || ld % vec)) vec = (t == SIGNMUON_BF16 && vec > 2) ? 2 : 1;
  return vec;
}

// What is asked of the device once and kept: a few driver queries cost as
// much as a small launch.
constexpr int kMaxDevices = 64;
inline int current_device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices ? dev : 0;
}
// SMs of the current device (148 on B200; 148 if the query fails).
inline int current_sms() {
  static std::atomic<int> known[kMaxDevices];
  const int dev = current_device();
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}
// Allows kernel K all the dynamic shared memory there is (227 KB less its
// static arrays), on this device, and gives the blocks of it that an SM holds.  `smem` is a function of K and `threads`.
template <auto K>
int resident_blocks(int threads, size_t smem) {
  static std::atomic<int> known[kMaxDevices][33];
  std::atomic<int>& slot = known[current_device()][threads / 32];
  int n = slot.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, K) == cudaSuccess)
      cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - (int)attr.sharedSizeBytes);
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, K, threads, smem) != cudaSuccess || n < 1) n = 1;
    slot.store(n, std::memory_order_relaxed);
  }
  return n;
}

// Launches a kernel that starts with wait_for_kernel_before().
template <typename... P, typename... A>
void launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid, cfg.blockDim = dim3((unsigned)threads), cfg.dynamicSmemBytes = smem, cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);  // its error is cudaGetLastError's
}

}  // namespace signmuon
