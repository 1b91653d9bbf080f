// Embedding lookup with scaling, and the table's gradient per worker.
//
//   forward    y[t] = s W[id_t]                     (0 for ids outside the table)
//   backward   G^(m)[v] = s sum_{t of worker m, id_t = v} dy[t]
//
// The lookup reads the rows that the ids name and writes y.  The gradient
// reads dy once and writes n_workers whole tables, nearly all zeros for a
// large vocabulary, so its floor is those writes.  It runs without atomics,
// in an order fixed by the ids:
//   1. sort   Each worker's (id, token) pairs are sorted by id in tiles of
//             kTile, a block a tile, in shared memory (stable counting passes
//             of up to 9 bits).  The other blocks of the launch meanwhile fill
//             the first rows of the tables with zeros: the sort is bound by
//             latency and takes few SMs, the fill is bound by HBM.
//   2. merge  Only for workers of more than one tile: each pair's place is its
//             place in its own run plus the smaller pairs of the other runs,
//             found by search, kFan runs at a time.
//   3. reduce A warp takes a chunk of consecutive sorted pairs (32, or 8 where
//             that leaves SMs without work) and a slab of columns, adds the rows of each run of equal ids in registers and
//             writes the runs that lie within the chunk.  What a run that
//             crosses a chunk's ends has there is left as a partial row.
//             Other blocks of the launch fill the tables' other rows with
//             zeros, those that no id names.
//   4. join   The chunk where such a run begins adds its partial rows and
//             writes the row; long runs (frequent tokens) by a whole block.
#include "layers.cuh"

using namespace signmuon;

namespace {

constexpr int64_t kMaxTokens = 1 << 30;  // of a backward call: places among them are ints
constexpr int kLookupThreads = 256;
constexpr int kLookupVecs = 4;       // vectors a lane loads of a row
constexpr int kAnyVecs = 4;          // the same, of a row at any address
constexpr int kSortThreads = 1024;
constexpr int kSortItems = 4;        // pairs a thread
constexpr int kTile = kSortThreads * kSortItems;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;
constexpr int64_t kFillBeside = 40 << 20;  // bytes that are filled in the time of a sort
constexpr int kFan = 32;             // runs merged at a time (one lane each)
constexpr int kMergeStage = 11264;   // keys of other runs that a block of the merge holds
constexpr int kMergeThreads = 256;
constexpr int kLongChunk = 32, kShortChunk = 8;  // sorted pairs a warp of the reduction takes
constexpr int kLaneCols = 8;         // columns of a lane's slab
constexpr int kSlab = 32 * kLaneCols;
constexpr int kReduceThreads = 256;
constexpr int kJoinChunks = 8;       // chunks (warps) a block of the join looks at
constexpr int kLongRun = 16;         // chunks from which a whole block adds a run

// ----------------------------------------------------------------- lookup
// lanes (a power of two) lanes take kLookupVecs vectors each of a token's
// row; blockIdx.y is the segment of rows that are longer than that.  Bound by
// memory: 32768 tokens of 4096 bf16 from 50000 rows in 61 us (floor 54).
template <typename TW, typename TY, int VEC>
__global__ void __launch_bounds__(kLookupThreads)
lookup_kernel(const TW* __restrict__ table, int64_t ld_table, int32_t vocab, int32_t cols, int64_t n_tokens,
              const void* __restrict__ ids, int wide, float scale, TY* __restrict__ y, int64_t ld_y, int lanes) {
  const int64_t token = (int64_t)blockIdx.x * (kLookupThreads / lanes) + threadIdx.x / lanes;
  if (token >= n_tokens) return;
  const int64_t id = load_id(ids, token, wide);
  const bool in = id >= 0 && id < vocab;
  const TW* src = table + (in ? id : 0) * ld_table;
  const int first = (blockIdx.y * lanes * kLookupVecs + threadIdx.x % lanes) * VEC;
  typename RawVec<TW, VEC>::type raw[kLookupVecs];
#pragma unroll
  for (int i = 0; i < kLookupVecs; ++i) {
    const int col = first + i * lanes * VEC;
    if (in && col < cols) raw[i] = __ldg(reinterpret_cast<const typename RawVec<TW, VEC>::type*>(src + col));
  }
#pragma unroll
  for (int i = 0; i < kLookupVecs; ++i) {
    const int col = first + i * lanes * VEC;
    if (col < cols) {
      float v[VEC];
      if (in) unpack(raw[i], v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = in ? v[j] * scale : 0.f;
      // Narrow stores share 32-byte sectors with others': those are left to L2
      // to put together.
      if (VEC * sizeof(TY) >= 8) store_stream<TY, VEC>(y + token * ld_y + col, v);
      else store_vec<TY, VEC>(y + token * ld_y + col, v);
    }
  }
}

// Rows of one type that are not all on 16 bytes.  y is written in whole 16
// bytes where they lie in the row; what goes there starts at the same place
// within 16 bytes all along a row of the table, so each is cut from two aligned
// vectors, by one shift that a row's lanes share.  Lanes with four vectors each
// (32 KB of loads under way an SM) are worth more than more warps with two.
// 65536 tokens of 1001 columns: bf16 42 us, fp32 83 us, where element by element
// they took 120 and 117 (1000 columns: 34 and 63); 131072 tokens of 33: 12 and 10
// for 26 and 25.
template <typename T>
__global__ void __launch_bounds__(kLookupThreads, 5)
lookup_any_kernel(const T* __restrict__ table, int64_t ld_table, int32_t vocab, int32_t cols, int64_t n_tokens,
                  const void* __restrict__ ids, int wide, float scale, T* __restrict__ y, int64_t ld_y, int lanes) {
  constexpr int kVec = 16 / sizeof(T), kWord = 4 / sizeof(T);  // elements of 16 bytes, and of 4
  const int64_t token = (int64_t)blockIdx.x * (kLookupThreads / lanes) + threadIdx.x / lanes;
  if (token >= n_tokens) return;
  const int64_t id = load_id(ids, token, wide);
  const bool in = id >= 0 && id < vocab;
  const T* src = table + (in ? id : 0) * ld_table;
  T* dst = y + token * ld_y;
  const int shift = (int)(reinterpret_cast<uintptr_t>(dst) % 16 / sizeof(T));  // of y's first vector before the row
  const int off = (int)((reinterpret_cast<uintptr_t>(src) / sizeof(T) - shift) % kVec);  // in the table's vectors
  const int first = blockIdx.y * lanes * kAnyVecs + threadIdx.x % lanes;
  const uint4* from = reinterpret_cast<const uint4*>(src - shift - off) + first;
  T* to = dst - shift + first * kVec;
  int col = first * kVec - shift;
  // The table's first and last rows, where a vector may reach over its ends.
  if (in && (id * ld_table < 2 * kVec || (vocab - 1 - id) * ld_table < 2 * kVec)) {
    for (int i = 0; i < kAnyVecs; ++i, col += lanes * kVec)
      for (int j = max(col, 0); j < min(col + kVec, cols); ++j)
        store_elem(dst, j, sizeof(T) == 2, load_elem(src, j, sizeof(T) == 2) * scale);
    return;
  }
  uint4 a[kAnyVecs], b[kAnyVecs];
#pragma unroll
  for (int i = 0; i < kAnyVecs; ++i) {
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    if (in && col + i * lanes * kVec < cols) {
      a[i] = __ldg(from + i * lanes);
      if (off) b[i] = __ldg(from + i * lanes + 1);
    }
  }
#pragma unroll
  for (int i = 0; i < kAnyVecs; ++i, col += lanes * kVec, to += lanes * kVec) {
    if (col >= cols) break;
    uint32_t w[8] = {a[i].x, a[i].y, a[i].z, a[i].w, b[i].x, b[i].y, b[i].z, b[i].w};
    const int words = off / kWord;
    if (words & 2)
#pragma unroll
      for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
    if (words & 1)
#pragma unroll
      for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
    if (off % kWord)
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 16);
    if (scale != 1.f) {
      typename RawVec<T, kVec>::type raw;
      memcpy(&raw, w, 16);
      float v[kVec];
      unpack(raw, v);
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = in ? v[j] * scale : 0.f;
      pack(v, raw);
      memcpy(w, &raw, 16);
    }
    if (col >= 0 && col + kVec <= cols) {
      *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (col + j >= 0 && col + j < cols) {
          if (sizeof(T) == 4) reinterpret_cast<uint32_t*>(to)[j] = w[j];
          else reinterpret_cast<uint16_t*>(to)[j] = (uint16_t)(w[j / kWord] >> j % kWord * 16);
        }
    }
  }
}

// ------------------------------------------------------------ sort and fill
struct Fill {
  WorkerPtrs grad;
  int64_t row_bytes;  // of a table's row
  int32_t rows;       // of a table; 0: nothing to fill
  int32_t head;       // rows that the sort's launch fills
  int32_t unit;       // rows that a warp of the reduction's launch fills (at most 32)
};

// Zeros from p on, by `threads` threads of which this is the t-th: the ends
// that are not whole 16 bytes two bytes at a time.
__device__ __forceinline__ void zero_bytes(uint8_t* p, int64_t bytes, int64_t t, int64_t threads) {
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int64_t head = min((int64_t)(-reinterpret_cast<uintptr_t>(p) & 15), bytes);
  const int64_t n16 = (bytes - head) / 16, tail = head + n16 * 16;
  uint4* q = reinterpret_cast<uint4*>(p + head);
  for (int64_t i = t; i < n16; i += threads) __stcs(q + i, zero);
  if (t < 8) {
    if (2 * t < head) *reinterpret_cast<uint16_t*>(p + 2 * t) = 0;
    if (tail + 2 * t < bytes) *reinterpret_cast<uint16_t*>(p + tail + 2 * t) = 0;
  }
}

// Blocks 0 .. tiles.begin[n_workers] - 1 sort a tile each, the rest fill.  (12 us
// for tiles of 4096 with two passes, the time that 40 MB of zeros take.)
// Keys are ids; an id outside the table gets the key `vocab` and sorts last.
__global__ void __launch_bounds__(kSortThreads)
sort_tiles_kernel(const __grid_constant__ WorkerRows rows, const __grid_constant__ WorkerBlocks tiles, int n_workers,
                  const void* __restrict__ ids, int wide, uint32_t vocab, int passes, int bits, uint32_t* __restrict__ out_key,
                  uint32_t* __restrict__ out_tok, const __grid_constant__ Fill fill) {
  extern __shared__ uint32_t s_key[];                                    // [kTile]
  uint16_t* s_tok = reinterpret_cast<uint16_t*>(s_key + kTile);          // [kTile]
  uint16_t* s_count = s_tok + kTile;                                     // [kSortWarps][kDigits]
  __shared__ uint32_t s_digit[kDigits];  // first place of each digit
  __shared__ uint32_t s_warp[kSortWarps];
  allow_next_kernel();
  const int n_tiles = tiles.begin[n_workers];
  if ((int)blockIdx.x >= n_tiles) {
    const int64_t t = (int64_t)(blockIdx.x - n_tiles) * kSortThreads + threadIdx.x;
    for (int m = 0; m < n_workers; ++m)
      zero_bytes(static_cast<uint8_t*>(fill.grad.p[m]), fill.head * fill.row_bytes, t, (int64_t)(gridDim.x - n_tiles) * kSortThreads);
    return;
  }
  const int m = worker_of_block(tiles, n_workers, blockIdx.x);
  const int64_t base = rows.begin[m] + (int64_t)(blockIdx.x - tiles.begin[m]) * kTile;
  const int n = (int)min((int64_t)kTile, rows.begin[m + 1] - base);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int first = warp * 32 * kSortItems + lane;  // this thread's items: first + 32 j
  // at[j]: the pair's token in the tile, and above it its rank among the warp's
  // pairs with the same digit (both at most 2^14).
  uint32_t key[kSortItems], at[kSortItems];
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const int i = first + 32 * j;
    int64_t id = -1;
    if (i < n) id = load_id(ids, base + i, wide);
    key[j] = id >= 0 && id < (int64_t)vocab ? (uint32_t)id : vocab;
    at[j] = i;
  }
  const uint32_t mask = (1u << bits) - 1, lower = (1u << lane) - 1;
  // Warps that have pairs (the last one's missing pairs have the last key).
  const int used = (n + 32 * kSortItems - 1) / (32 * kSortItems);
  uint16_t* count = s_count + warp * kDigits;
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * bits;
    if (warp < used) {
      for (int i = lane; i < kDigits / 2; i += 32) reinterpret_cast<uint32_t*>(count)[i] = 0;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kSortItems; ++j) {
        const uint32_t d = key[j] >> shift & mask;
        // The lanes with the same digit, bit by bit (4096 pairs: 10 us in all;
        // with __match_any_sync, which takes as long for each of the digits
        // that there are, 13).
        uint32_t peers = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < kDigitBits; ++i) {
          const bool set = d >> i & 1;
          const uint32_t with = __ballot_sync(0xffffffffu, set);
          peers &= set ? with : ~with;
        }
        const uint32_t seen = count[d], before = __popc(peers & lower);
        at[j] |= (seen + before) << 16;
        __syncwarp();
        if (before == 0) count[d] = (uint16_t)(seen + __popc(peers));
        __syncwarp();
      }
    }
    __syncthreads();
    // Counts to places: by digit, within a digit by warp.
    uint32_t total = 0;
    if (threadIdx.x < kDigits) {
      // (Warps without pairs have counts that nobody reads.)
      for (int w0 = 0; w0 < used; w0 += 8) {
        uint32_t c[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) c[w] = s_count[(w0 + w) * kDigits + threadIdx.x];
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          s_count[(w0 + w) * kDigits + threadIdx.x] = (uint16_t)total;
          total += w0 + w < used ? c[w] : 0;
        }
      }
    }
    uint32_t scan = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) s_warp[warp] = scan;
    __syncthreads();
    if (threadIdx.x < kDigits) {
      uint32_t below = lane < warp ? s_warp[lane] : 0;
      below = __reduce_add_sync(0xffffffffu, below);
      s_digit[threadIdx.x] = below + scan - total;
    }
    __syncthreads();
    if (warp < used)
#pragma unroll
      for (int j = 0; j < kSortItems; ++j) {
        const uint32_t d = key[j] >> shift & mask;
        const uint32_t to = s_digit[d] + count[d] + (at[j] >> 16);
        s_key[to] = key[j];
        s_tok[to] = (uint16_t)at[j];
      }
    __syncthreads();
    if (warp < used)
#pragma unroll
      for (int j = 0; j < kSortItems; ++j) key[j] = s_key[first + 32 * j], at[j] = s_tok[first + 32 * j];
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const int i = first + 32 * j;
    if (i < n) out_key[base + i] = key[j], out_tok[base + i] = (uint32_t)base + at[j];
  }
}

// ------------------------------------------------------------------ merge
// Runs of `run` sorted pairs of each worker, kFan at a time, to runs of
// kFan * run (run is kTile times a power of kFan).  Equal keys keep the runs'
// order.  A block has kMergeThreads pairs of one run, so what it looks for in
// another run lies between the places of its first and its last key there.
// Those are found first, by warps of 32 probes at a time, and the keys between
// them brought into shared memory, if they fit: the threads' searches then wait
// for no load.  (100003 tokens: 15 us for 25 runs, where two merges of eight
// runs each, searched in L2 from end to end, took 11 us each.)
__global__ void __launch_bounds__(kMergeThreads)
merge_kernel(const __grid_constant__ WorkerRows rows, const __grid_constant__ WorkerBlocks blocks, int n_workers, int run,
             const uint32_t* key, const uint32_t* tok, uint32_t* out_key, uint32_t* out_tok) {
  constexpr int kWarps = kMergeThreads / 32, kSearches = 2 * kFan / kWarps, kSide = 8;
  __shared__ uint32_t s_key[kMergeStage];
  // Of each run: the places of the block's first and behind its last key, from
  // the run's start; where the keys between are in s_key.
  __shared__ int s_edge[2 * kFan], s_at[kFan + 1];
  allow_next_kernel();
  wait_for_kernel_before();
  const int m = worker_of_block(blocks, n_workers, blockIdx.x);
  const int n = (int)(rows.begin[m + 1] - rows.begin[m]);  // at most kMaxTokens in all
  const int p0 = (blockIdx.x - blocks.begin[m]) * kMergeThreads, p = p0 + threadIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  key += rows.begin[m];
  const int mine = p0 / run, group = mine / kFan * kFan, own = mine - group;
  const int runs = min(kFan, (n + run - 1) / run - group);
  const uint32_t edge[2] = {key[p0], key[min(p0 + kMergeThreads, n) - 1]}, k = p < n ? key[p] : edge[1];
  const uint32_t t = p < n ? tok[rows.begin[m] + p] : 0;
  // What goes before a pair: keys below its own, and in earlier runs equal ones.
  int at[kSearches];
#pragma unroll
  for (int q = 0; q < kSearches; ++q) at[q] = 0;
  int step = run;
  do {
    step = (step + 31) / 32;
    uint32_t seen[kSearches];
#pragma unroll
    for (int q = 0; q < kSearches; ++q) {
      const int i = (warp * kSearches + q) / 2;
      seen[q] = ~0u;
      if (i < runs && i != own) {
        const int begin = (group + i) * run, probe = at[q] + (lane + 1) * step;
        if (probe <= min(run, n - begin)) seen[q] = key[begin + probe - 1];
      }
    }
#pragma unroll
    for (int q = 0; q < kSearches; ++q) {
      const int i = (warp * kSearches + q) / 2;
      at[q] += __popc(__ballot_sync(0xffffffffu, seen[q] < edge[q % 2] + (i < own ? 1u : 0u))) * step;
    }
  } while (step > 1);
  if (lane == 0)
#pragma unroll
    for (int q = 0; q < kSearches; ++q) s_edge[warp * kSearches + q] = at[q];
  __syncthreads();
  if (warp == 0) {
    int scan = s_edge[2 * lane + 1] - s_edge[2 * lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    s_at[lane + 1] = scan;
    if (lane == 0) s_at[0] = 0;
  }
  __syncthreads();
  // kSide searches side by side, without branches: one alone would wait for
  // each of its loads.
  int before = 0;
  auto search = [&](int i0, int i1, int first, auto in_shared) {
    for (; i0 < i1; i0 += kSide) {
      const uint32_t* from[kSide];
      int len[kSide], to[kSide], most = 0;
#pragma unroll
      for (int q = 0; q < kSide; ++q) {
        const int i = i0 + q;
        len[q] = s_at[i + 1] - s_at[i], to[q] = 0;
        if constexpr (decltype(in_shared)::value) from[q] = s_key + (s_at[i] - s_at[first]);
        else from[q] = key + (group + min(i, runs - 1)) * run + s_edge[2 * i];
        before += s_edge[2 * i];
        most = max(most, len[q]);
      }
      for (int s = most ? 1 << (31 - __clz(most)) : 0; s; s /= 2) {
#pragma unroll
        for (int q = 0; q < kSide; ++q) {
          const int probe = to[q] + s;
          if (probe <= len[q] && from[q][probe - 1] < k + (i0 + q < own ? 1u : 0u)) to[q] = probe;
        }
      }
#pragma unroll
      for (int q = 0; q < kSide; ++q) before += to[q];
    }
  };
  // As many runs at a time, in kSides, as s_key holds.
  for (int first = 0, last; first < runs; first = last) {
    for (last = first; last < runs && s_at[last + kSide] - s_at[first] <= kMergeStage;) last += kSide;
    if (last == first) {
      last += kSide;
      search(first, last, first, std::false_type());
      continue;
    }
    __syncthreads();
    for (int i = first + warp; i < min(last, runs); i += kWarps) {
      const uint32_t* from = key + (group + i) * run + s_edge[2 * i];
      uint32_t* to = s_key + (s_at[i] - s_at[first]);
      const int len = s_at[i + 1] - s_at[i];
#pragma unroll 8
      for (int j = lane; j < len; j += 32) to[j] = from[j];
    }
    __syncthreads();
    search(first, last, first, std::true_type());
  }
  if (p < n) {
    const int64_t place = rows.begin[m] + (int64_t)group * run + (p - mine * run) + before;
    out_key[place] = k;
    out_tok[place] = t;
  }
}

// ----------------------------------------------------------------- reduce
// Bound by memory: 100003 rows of 999 fp32 in 72 us (5.6 TB/s); eight workers'
// 32768 rows of 768 bf16 and what is left of eight tables of 50000 rows to fill in
// 101 us (6.2 TB/s).
struct ReduceArgs {
  const uint32_t* key;
  const uint32_t* tok;
  const void* dy;
  int64_t ld_dy;
  // [chunks][2][slabs][2][32 lanes] of four floats: what the run from the chunk
  // before, and the one into the next, have here, as the lanes hold it.
  float4* part;
  uint32_t vocab;
  int32_t chunk;  // pairs of a chunk
  int32_t cols, slabs, n_workers, accumulate;
  int32_t n_blocks;  // of the reduction; further blocks of its launch fill
  float scale;
  __device__ __forceinline__ float4* partial(int chunk_, int which, int slab) const {
    return part + (((int64_t)chunk_ * 2 + which) * slabs + slab) * 64 + (threadIdx.x & 31);
  }
};

// One chunk of a worker's sorted pairs.
struct Chunk {
  int64_t begin;   // of the pairs
  int n;           // pairs in the table (the others sort last)
  uint32_t key;    // this lane's
  uint32_t ends;   // bit j: a run ends at pair j
  bool from_before, into_next;
};
__device__ __forceinline__ Chunk chunk_at(const ReduceArgs& a, const WorkerRows& rows, const WorkerBlocks& chunks, int m,
                                          int chunk) {
  Chunk c;
  const int lane = threadIdx.x & 31;
  const int last = a.chunk - 1;
  c.begin = rows.begin[m] + (int64_t)(chunk - chunks.begin[m]) * a.chunk;
  const int64_t end = rows.begin[m + 1];
  const bool in = lane <= last && c.begin + lane < end;
  c.key = in ? a.key[c.begin + lane] : a.vocab;
  // The neighbours' keys; vocab where there is none, which equals no key here.
  uint32_t edge = a.vocab;
  if (lane == 0 && c.begin > rows.begin[m]) edge = a.key[c.begin - 1];
  if (lane == last && c.begin + a.chunk < end) edge = a.key[c.begin + a.chunk];
  c.n = __popc(__ballot_sync(0xffffffffu, c.key < a.vocab));
  uint32_t after = __shfl_down_sync(0xffffffffu, c.key, 1);
  if (lane == last) after = edge;
  c.ends = __ballot_sync(0xffffffffu, c.key < a.vocab && c.key != after);
  const uint32_t joins = __ballot_sync(0xffffffffu, c.key < a.vocab && c.key == edge);
  c.from_before = joins & 1u;
  c.into_next = joins >> last & 1u;
  return c;
}

// First of the sorted keys [lo, hi) that is above `key` (kAbove) or not below
// it, by a warp, 32 probes at a time.
template <bool kAbove>
__device__ __forceinline__ int64_t find_key(const uint32_t* keys, int64_t lo, int64_t hi, uint32_t key) {
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) / 32, probe = lo + (threadIdx.x & 31) * step + step - 1;
    const bool below = probe < hi && (kAbove ? keys[probe] <= key : keys[probe] < key);
    lo = min(hi, lo + __popc(__ballot_sync(0xffffffffu, below)) * step);
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// Fills the u-th `unit` rows of those that the sort's launch left, of all tables
// in turn, where no id names them.
__device__ __forceinline__ void fill_rest(const ReduceArgs& a, const WorkerRows& rows, const Fill& fill, int64_t u) {
  const int per_table = (fill.rows - fill.head + fill.unit - 1) / fill.unit, lane = threadIdx.x & 31;
  const int m = (int)(u / per_table);
  if (m >= a.n_workers) return;
  const uint32_t first = fill.head + (uint32_t)(u % per_table) * fill.unit;
  const uint32_t last = min(first + fill.unit, (uint32_t)fill.rows);
  uint32_t named = last - first < 32 ? ~0u << (last - first) : 0u;  // rows that are not to be filled
  const int64_t end = rows.begin[m + 1];
  for (int64_t at = find_key<false>(a.key, rows.begin[m], end, first); at < end; at += 32) {
    const uint32_t key = at + lane < end ? a.key[at + lane] : a.vocab;
    named |= __reduce_or_sync(0xffffffffu, key < last ? 1u << (key - first) : 0u);
    const uint32_t far = __shfl_sync(0xffffffffu, key, 31);
    if (far >= last) break;
    // Past the rest of a long run at once.
    if (far == __shfl_sync(0xffffffffu, key, 0)) at = find_key<true>(a.key, at + 32, end, far) - 32;
  }
  uint8_t* table = static_cast<uint8_t*>(fill.grad.p[m]);
  while (~named) {
    const int begin = __ffs(~named) - 1;
    const uint32_t after = named >> begin;
    const int n = after ? __ffs(after) - 1 : 32 - begin;
    zero_bytes(table + (int64_t)(first + begin) * fill.row_bytes, n * fill.row_bytes, lane, 32);
    named |= (n == 32 ? ~0u : (1u << n) - 1) << begin;
  }
}

template <typename TG, int VEC>
__device__ __forceinline__ void write_grad(TG* row, int col0, int cols, int accumulate, float scale, const float (&acc)[kLaneCols]) {
#pragma unroll
  for (int c = 0; c < kLaneCols / VEC; ++c) {
    const int col = col0 + c * 32 * VEC;
    if (col < cols) {
      float v[VEC];
      if (accumulate) unpack(*reinterpret_cast<const typename RawVec<TG, VEC>::type*>(row + col), v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = accumulate ? fmaf(acc[c * VEC + j], scale, v[j]) : acc[c * VEC + j] * scale;
      store_vec<TG, VEC>(row + col, v);
    }
  }
}

template <typename TD, typename TG, int VEC>
__global__ void __launch_bounds__(kReduceThreads)
reduce_kernel(const ReduceArgs a, const __grid_constant__ WorkerRows rows, const __grid_constant__ WorkerBlocks chunks,
              const __grid_constant__ Fill fill) {
  constexpr int kVecs = kLaneCols / VEC, kBatch = 4;
  allow_next_kernel();
  wait_for_kernel_before();
  if ((int)blockIdx.x >= a.n_blocks) {
    fill_rest(a, rows, fill, (int64_t)(blockIdx.x - a.n_blocks) * (kReduceThreads / 32) + threadIdx.x / 32);
    return;
  }
  const int lane = threadIdx.x & 31, slab = blockIdx.x % a.slabs;
  const int chunk = blockIdx.x / a.slabs * (kReduceThreads / 32) + threadIdx.x / 32;
  if (chunk >= chunks.begin[a.n_workers]) return;
  const int m = worker_of_block(chunks, a.n_workers, chunk);
  const Chunk c = chunk_at(a, rows, chunks, m, chunk);
  const uint32_t tok = lane < c.n ? a.tok[c.begin + lane] : 0;
  const int col0 = slab * kSlab + lane * VEC, cols = a.cols;
  const TD* dy = static_cast<const TD*>(a.dy);
  TG* table = static_cast<TG*>(fill.grad.p[m]);
  float acc[kLaneCols] = {};
  bool first = true;
  auto write_part = [&](int which) {
    float4* p = a.partial(chunk, which, slab);
    p[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    p[32] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  };
  for (int j0 = 0; j0 < c.n; j0 += kBatch) {
    typename RawVec<TD, VEC>::type raw[kBatch][kVecs];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint32_t row = __shfl_sync(0xffffffffu, tok, min(j0 + j, 31));
      const TD* p = dy + (int64_t)row * a.ld_dy;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const int col = col0 + i * 32 * VEC;
        if (j0 + j < c.n && col < cols) raw[j][i] = load_stream<TD, VEC>(p + col);
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint32_t key = __shfl_sync(0xffffffffu, c.key, min(j0 + j, 31));
      if (j0 + j < c.n) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
          if (col0 + i * 32 * VEC < cols) {
            float v[VEC];
            unpack(raw[j][i], v);
#pragma unroll
            for (int q = 0; q < VEC; ++q) acc[i * VEC + q] += v[q];
          }
        if (c.ends >> (j0 + j) & 1) {
          if (first && c.from_before) write_part(0);
          else write_grad<TG, VEC>(table + (int64_t)key * cols, col0, cols, a.accumulate, a.scale, acc);
          first = false;
#pragma unroll
          for (int i = 0; i < kLaneCols; ++i) acc[i] = 0.f;
        }
      }
    }
  }
  if (c.into_next) write_part(first && c.from_before ? 0 : 1);
}

// ------------------------------------------------------------------- join
// Bound by latency (a search, loads of partial rows in batches of eight): 6 us for
// eight workers' 4096 tokens, 14 for 100003 tokens of which the most frequent id has
// a thirteenth.
template <typename TG, int VEC>
__global__ void __launch_bounds__(kJoinChunks * 32)
join_kernel(const ReduceArgs a, const __grid_constant__ WorkerRows rows, const __grid_constant__ WorkerBlocks chunks,
            const __grid_constant__ WorkerPtrs grad) {
  __shared__ int s_follow[kJoinChunks];
  __shared__ uint32_t s_key[kJoinChunks];
  __shared__ int s_worker[kJoinChunks];
  __shared__ float s_acc[kJoinChunks][kSlab];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, cols = a.cols;
  const int chunk0 = blockIdx.x * kJoinChunks, chunk = chunk0 + warp, slab = blockIdx.y;
  const int col0 = slab * kSlab + lane * VEC;
  int follow = 0, m = 0;
  uint32_t key = 0;
  wait_for_kernel_before();
  if (chunk < chunks.begin[a.n_workers]) {
    m = worker_of_block(chunks, a.n_workers, chunk);
    const Chunk c = chunk_at(a, rows, chunks, m, chunk);
    key = __shfl_sync(0xffffffffu, c.key, a.chunk - 1);
    // A run that begins here (this chunk is not all one run from before) and
    // goes on: how many chunks it goes on in.
    if (c.into_next && (c.ends || !c.from_before)) {
      // By the first keys of the 32 chunks after the next, or else by search.
      const int64_t begin = c.begin + a.chunk, end = rows.begin[m + 1], probe = begin + (int64_t)(1 + lane) * a.chunk;
      const uint32_t same = __ballot_sync(0xffffffffu, probe < end && a.key[probe] == key);
      follow = same != 0xffffffffu ? __ffs(~same)
                                   : (int)((find_key<true>(a.key, begin + 1, end, key) - begin + a.chunk - 1) / a.chunk);
    }
  }
  // Adds the partial rows of chunk + i for i = from, from + step, ... <= n.
  auto add = [&](int at, int from, int step, int n, float (&acc)[kLaneCols]) {
    constexpr int kBatch = 8;
    for (int i0 = from; i0 <= n; i0 += kBatch * step) {
      float4 p[kBatch][2];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j * step;
        if (i <= n) {
          const float4* q = a.partial(at + i, i == 0 ? 1 : 0, slab);
          p[j][0] = q[0], p[j][1] = q[32];
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (i0 + j * step <= n) {
          acc[0] += p[j][0].x, acc[1] += p[j][0].y, acc[2] += p[j][0].z, acc[3] += p[j][0].w;
          acc[4] += p[j][1].x, acc[5] += p[j][1].y, acc[6] += p[j][1].z, acc[7] += p[j][1].w;
        }
    }
  };
  const bool is_long = follow >= kLongRun;
  if (lane == 0) s_follow[warp] = is_long ? follow : 0, s_key[warp] = key, s_worker[warp] = m;
  if (follow && !is_long) {
    float acc[kLaneCols] = {};
    add(chunk, 0, 1, follow, acc);
    write_grad<TG, VEC>(static_cast<TG*>(grad.p[m]) + (int64_t)key * cols, col0, cols, a.accumulate, a.scale, acc);
  }
  __syncthreads();
  for (int w = 0; w < kJoinChunks; ++w) {
    if (!s_follow[w]) continue;
    float acc[kLaneCols] = {};
    add(chunk0 + w, warp, kJoinChunks, s_follow[w], acc);
#pragma unroll
    for (int q = 0; q < kLaneCols; ++q) s_acc[warp][q * 32 + lane] = acc[q];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int q = 0; q < kLaneCols; ++q) {
        acc[q] = 0.f;
        for (int i = 0; i < kJoinChunks; ++i) acc[q] += s_acc[i][q * 32 + lane];
      }
      write_grad<TG, VEC>(static_cast<TG*>(grad.p[s_worker[w]]) + (int64_t)s_key[w] * cols, col0, cols, a.accumulate,
                          a.scale, acc);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------- host
struct BackwardLayout {
  size_t key[2], tok[2], part, total;
};
int64_t chunks_of(const int64_t* row_begin, int n_workers, int chunk) {
  int64_t n = 0;
  for (int m = 0; m < n_workers; ++m) n += ceil_div(row_begin[m + 1] - row_begin[m], chunk);
  return n;
}
// Short chunks where long ones make fewer than 8 warps an SM: a warp's loads of
// rows wait for one another.
int chunk_pairs(int32_t cols, int n_workers, const int64_t* row_begin) {
  return chunks_of(row_begin, n_workers, kLongChunk) * ceil_div(cols, kSlab) < 8 * (int64_t)current_sms() ? kShortChunk
                                                                                                      : kLongChunk;
}
BackwardLayout backward_layout(int32_t cols, int n_workers, const int64_t* row_begin) {
  const size_t n = round_up((size_t)row_begin[n_workers] * 4, 256);
  BackwardLayout l;
  l.key[0] = kWsHeaderBytes;
  l.key[1] = l.key[0] + n;
  l.tok[0] = l.key[1] + n;
  l.tok[1] = l.tok[0] + n;
  l.part = l.tok[1] + n;
  l.total = l.part + round_up((size_t)chunks_of(row_begin, n_workers, chunk_pairs(cols, n_workers, row_begin)) * 2 * ceil_div(cols, kSlab) * kSlab * 4, 256);
  return l;
}

// Blocks of `per` rows for each worker.
WorkerBlocks blocks_of(const int64_t* row_begin, int n_workers, int64_t per) {
  WorkerBlocks b = {};
  for (int m = 0; m < n_workers; ++m) b.begin[m + 1] = b.begin[m] + (int32_t)ceil_div(row_begin[m + 1] - row_begin[m], per);
  return b;
}

template <int VEC>
using Width = std::integral_constant<int, VEC>;

// f(first type, second type, width) for a width that both types have.
template <typename F>
void by_types(signmuon_dtype a, signmuon_dtype b, int vec, F f) {
  using bf16 = __nv_bfloat16;
  if (a == SIGNMUON_F32 && b == SIGNMUON_F32) vec == 4 ? f(float(), float(), Width<4>()) : f(float(), float(), Width<1>());
  else if (a == SIGNMUON_F32) vec == 4 ? f(float(), bf16(), Width<4>()) : f(float(), bf16(), Width<1>());
  else if (b == SIGNMUON_F32) vec == 4 ? f(bf16(), float(), Width<4>()) : f(bf16(), float(), Width<1>());
  else if (vec == 8) f(bf16(), bf16(), Width<8>());
  else if (vec == 2) f(bf16(), bf16(), Width<2>());
  else f(bf16(), bf16(), Width<1>());
}
// The widest access that both buffers allow.
int common_width(signmuon_dtype ta, const void* a, int64_t lda, signmuon_dtype tb, const void* b, int64_t ldb, int32_t cols) {
  if (ta == tb) return vec_narrow(vec_narrow(vec_width(ta, cols), ta, a, lda), tb, b, ldb);
  const bool four = cols % 4 == 0 && lda % 4 == 0 && ldb % 4 == 0 && aligned_to(a, 4 * dtype_bytes(ta)) &&
                    aligned_to(b, 4 * dtype_bytes(tb));
  return four ? 4 : 1;
}

}  // namespace

extern "C" {

signmuon_status signmuon_embedding_forward(signmuon_shape table_shape, signmuon_dtype table_dtype, const void* table,
                                           int64_t ld_table, int64_t n_tokens, int ids_int64, const void* ids,
                                           float scale, signmuon_dtype y_dtype, void* y, int64_t ld_y, void* stream) {
  const int32_t cols = table_shape.cols;
  if (cols > kMaxCols) return SIGNMUON_ERR_UNSUPPORTED;
  if (table_shape.rows <= 0 || cols <= 0 || n_tokens < 0 || !known_dtype(table_dtype) || !known_dtype(y_dtype) || !table ||
      ld_table < cols || ld_y < cols || (n_tokens > 0 && (!ids || !y)))
    return SIGNMUON_ERR_INVALID_ARG;
  if (!aligned_to(table, dtype_bytes(table_dtype)) || !aligned_to(y, dtype_bytes(y_dtype)) || !aligned_to(ids, ids_int64 ? 8 : 4))
    return SIGNMUON_ERR_ALIGNMENT;
  const int vec = common_width(table_dtype, table, ld_table, y_dtype, y, ld_y, cols);
  const int full = 16 / dtype_bytes(y_dtype);
  const bool any = table_dtype == y_dtype && vec < full;
  const int64_t vecs = any ? ceil_div(cols + full - 1, full) : ceil_div(cols, vec);  // of a row at most
  int lanes = 1;
  while (lanes < 32 && lanes * (any ? kAnyVecs : 1) < vecs) lanes *= 2;
  const int64_t blocks = ceil_div(n_tokens, kLookupThreads / lanes);
  const int segments = (int)ceil_div(vecs, (int64_t)lanes * (any ? kAnyVecs : kLookupVecs));
  if (blocks > INT32_MAX) return SIGNMUON_ERR_UNSUPPORTED;
  if (!n_tokens) return SIGNMUON_OK;
  if (any) {
    auto launch = [&](auto t) {
      using T = decltype(t);
      lookup_any_kernel<T><<<dim3((unsigned)blocks, (unsigned)segments), kLookupThreads, 0, static_cast<cudaStream_t>(stream)>>>(
          static_cast<const T*>(table), ld_table, table_shape.rows, cols, n_tokens, ids, ids_int64 != 0, scale,
          static_cast<T*>(y), ld_y, lanes);
    };
    if (table_dtype == SIGNMUON_F32) launch(float());
    else launch(__nv_bfloat16());
    return cuda_status(cudaGetLastError());
  }
  by_types(table_dtype, y_dtype, vec, [&](auto tw, auto ty, auto v) {
    using TW = decltype(tw);
    using TY = decltype(ty);
    constexpr int kVec = decltype(v)::value;
    if constexpr (!std::is_same_v<TW, TY> || kVec * sizeof(TW) == 16)
      lookup_kernel<TW, TY, kVec><<<dim3((unsigned)blocks, (unsigned)segments), kLookupThreads, 0, static_cast<cudaStream_t>(stream)>>>(
          static_cast<const TW*>(table), ld_table, table_shape.rows, cols, n_tokens, ids, ids_int64 != 0, scale,
          static_cast<TY*>(y), ld_y, lanes);
  });
  return cuda_status(cudaGetLastError());
}

static bool valid_backward_shape(signmuon_shape s, int n_workers, const int64_t* row_begin) {
  return s.rows > 0 && s.cols > 0 && n_workers > 0 && n_workers <= SIGNMUON_MAX_WORKERS && row_begin &&
         valid_splits(row_begin, n_workers, row_begin[n_workers]);
}

size_t signmuon_embedding_backward_workspace_bytes(signmuon_shape table_shape, int n_workers, const int64_t* row_begin) {
  if (!valid_backward_shape(table_shape, n_workers, row_begin) || row_begin[n_workers] > kMaxTokens) return 0;
  return backward_layout(table_shape.cols, n_workers, row_begin).total;
}

signmuon_status signmuon_embedding_backward(signmuon_shape table_shape, int n_workers, const int64_t* row_begin,
                                            int ids_int64, const void* ids, signmuon_dtype dy_dtype, const void* dy,
                                            int64_t ld_dy, float scale, int accumulate, signmuon_dtype grad_dtype,
                                            void* const* grad, void* workspace, size_t ws_bytes, void* stream) {
  const int32_t cols = table_shape.cols;
  if (!valid_backward_shape(table_shape, n_workers, row_begin) || !known_dtype(dy_dtype) || !known_dtype(grad_dtype) ||
      !grad || ld_dy < cols)
    return SIGNMUON_ERR_INVALID_ARG;
  const int64_t n = row_begin[n_workers];
  if (cols > kMaxCols || n > kMaxTokens) return SIGNMUON_ERR_UNSUPPORTED;
  if (n > 0 && (!ids || !dy)) return SIGNMUON_ERR_INVALID_ARG;
  if (!aligned_to(ids, ids_int64 ? 8 : 4) || !aligned_to(dy, dtype_bytes(dy_dtype))) return SIGNMUON_ERR_ALIGNMENT;
  Fill fill = {};
  int vec = 8;
  for (int m = 0; m < n_workers; ++m) {
    if (!grad[m]) return SIGNMUON_ERR_INVALID_ARG;
    if (!aligned_to(grad[m], dtype_bytes(grad_dtype))) return SIGNMUON_ERR_ALIGNMENT;
    fill.grad.p[m] = grad[m];
    const int v = common_width(dy_dtype, dy, ld_dy, grad_dtype, grad[m], cols, cols);
    if (v < vec) vec = v;
  }
  const BackwardLayout l = backward_layout(cols, n_workers, row_begin);
  const signmuon_status st = check_ws(workspace, ws_bytes, l.total);
  if (st) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* key[2] = {reinterpret_cast<uint32_t*>(ws + l.key[0]), reinterpret_cast<uint32_t*>(ws + l.key[1])};
  uint32_t* tok[2] = {reinterpret_cast<uint32_t*>(ws + l.tok[0]), reinterpret_cast<uint32_t*>(ws + l.tok[1])};
  WorkerRows rows = {};
  int64_t longest = 0;
  for (int m = 0; m <= n_workers; ++m) {
    rows.begin[m] = row_begin[m];
    if (m && row_begin[m] - row_begin[m - 1] > longest) longest = row_begin[m] - row_begin[m - 1];
  }

  // Sort (keys 0 .. rows) and fill.
  int key_bits = 1;
  while (key_bits < 31 && (table_shape.rows >> key_bits)) ++key_bits;
  const int passes = (key_bits + kDigitBits - 1) / kDigitBits, bits = (key_bits + passes - 1) / passes;
  const WorkerBlocks tiles = blocks_of(row_begin, n_workers, kTile);
  // The sort's launch fills what it has the time for (kFillBeside bytes), the
  // reduction's the rest.
  fill.rows = accumulate ? 0 : table_shape.rows;
  fill.row_bytes = (int64_t)cols * dtype_bytes(grad_dtype);
  const int64_t head = kFillBeside / (fill.row_bytes * n_workers) + 1;
  fill.head = (int32_t)(n == 0 || head > fill.rows ? fill.rows : head);
  int64_t fill_blocks = ceil_div(fill.head * fill.row_bytes * n_workers, 65536);
  if (fill_blocks > 2 * current_sms()) fill_blocks = 2 * current_sms();
  const int64_t grid = tiles.begin[n_workers] + fill_blocks;
  if (!grid) return SIGNMUON_OK;
  constexpr size_t kSmem = (size_t)kTile * 6 + kSortWarps * kDigits * 2;
  resident_blocks<sort_tiles_kernel>(kSortThreads, kSmem);  // allows it the shared memory
  sort_tiles_kernel<<<(unsigned)grid, kSortThreads, kSmem, cs>>>(rows, tiles, n_workers, ids, ids_int64 != 0,
                                                                (uint32_t)table_shape.rows, passes, bits, key[0], tok[0], fill);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_status(e);
  if (!n) return SIGNMUON_OK;

  int at = 0;
  for (int64_t run = kTile; run < longest; run *= kFan, at ^= 1) {
    const WorkerBlocks blocks = blocks_of(row_begin, n_workers, kMergeThreads);
    launch_after(merge_kernel, dim3((unsigned)blocks.begin[n_workers]), kMergeThreads, 0, cs, rows, blocks, n_workers, (int)run,
                 key[at], tok[at], key[at ^ 1], tok[at ^ 1]);
    if ((e = cudaGetLastError()) != cudaSuccess) return cuda_status(e);
  }

  const int chunk = chunk_pairs(cols, n_workers, row_begin);
  const WorkerBlocks chunks = blocks_of(row_begin, n_workers, chunk);
  const int n_chunks = chunks.begin[n_workers];
  ReduceArgs a = {};
  a.key = key[at], a.tok = tok[at], a.dy = dy, a.ld_dy = ld_dy, a.part = reinterpret_cast<float4*>(ws + l.part);
  a.vocab = (uint32_t)table_shape.rows, a.chunk = chunk, a.cols = cols, a.n_workers = n_workers, a.accumulate = accumulate != 0, a.scale = scale;
  a.slabs = (int32_t)ceil_div(cols, kSlab);
  const int64_t reduce_blocks = ceil_div(n_chunks, kReduceThreads / 32) * a.slabs;
  // Up to 32 rows a warp, fewer while there are fewer than 32 warps an SM.
  int64_t unit = ((int64_t)fill.rows - fill.head) * n_workers / (32 * current_sms());
  fill.unit = (int32_t)(unit < 1 ? 1 : unit > 32 ? 32 : unit);
  const int64_t rest = ceil_div((int64_t)fill.rows - fill.head, fill.unit) * n_workers;
  if (reduce_blocks + ceil_div(rest, kReduceThreads / 32) > INT32_MAX) return SIGNMUON_ERR_UNSUPPORTED;
  a.n_blocks = (int32_t)reduce_blocks;
  const unsigned blocks = (unsigned)(reduce_blocks + ceil_div(rest, kReduceThreads / 32));
  by_types(dy_dtype, grad_dtype, vec, [&](auto td, auto tg, auto v) {
    launch_after(reduce_kernel<decltype(td), decltype(tg), decltype(v)::value>, dim3(blocks), kReduceThreads, 0, cs, a, rows,
                 chunks, fill);
    if ((e = cudaGetLastError()) != cudaSuccess) return;
    launch_after(join_kernel<decltype(tg), decltype(v)::value>,
                 dim3((unsigned)ceil_div(n_chunks, kJoinChunks), (unsigned)a.slabs), kJoinChunks * 32, 0, cs, a, rows, chunks,
                 fill.grad);
    e = cudaGetLastError();
  });
  return cuda_status(e);
}

}  // extern "C"
