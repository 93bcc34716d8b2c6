// Tokens into the experts' order and back:
//   moe_sort          a stable counting sort of the T x k expert numbers,
//   moe_dispatch      Y[pos[t][s]] = w[t][s] X[t],
//   moe_combine       Y[t] = sum_s w[t][s] X[pos[t][s]],
//   moe_combine_grad  dX[pos[t][s]] = w[t][s] dY[t],  dw[t][s] = sum_c dY[t][c] X[pos[t][s]][c].
//
// The copies are bound by memory.  All three go token by token, so that a token's
// row is read (or written) once, whatever k is: reading X by sorted row instead
// would read it k times.  Sums are fp32 and in the order of the slots; nothing is
// added atomically, so results do not change from run to run.  4096 tokens x 8 of 4096
// bfloat16: dispatch 46 us (5.7 TB/s), combine 51.6 (5.8); the gradient of 3001 x 6 rows of 2050
// binary16 30 (5.3); the sort 8.5 of 32768 entries, 3 of 128.
//
// The sort: a wave takes 64 entries at a time, finds the lanes with the same expert by a ballot
// for every bit of its number, and counts them in its own row of LDS; a scan over experts and
// waves gives every wave its first row of each expert.  More than 1024 entries go over
// several workgroups, whose counts a first launch leaves in the workspace.
#include "lm_common.h"
#include "lm_launch.h"

namespace lasg {

namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / kWave;
constexpr int kMostChunks = 256;   // workgroups of the two-launch sort

struct SortArgs {
  SortCall c;
  int per_wave;   // entries of a wave, a multiple of 64
  int chunks;
};

// The lanes with the same key as this one, among all 64 (`bits`: of the largest key).
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
  uint64_t same = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool set = key >> b & 1;
    const uint64_t with = __ballot(set);
    same &= set ? with : ~with;
  }
  return same;
}

// Key of entry i: its expert, or `experts` for none (also past the end).
__device__ __forceinline__ int key_of(const SortCall& c, int64_t i) {
  if (i >= c.entries) return c.experts;
  const int e = c.ids[i];
  return e >= 0 && e < c.experts ? e : c.experts;
}

// Exclusive sums over the experts of count[], one to 1024 of them, by 1024 threads.
__device__ __forceinline__ int exclusive_sum(int x, int* part) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  int sum = x;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int y = __shfl_up(sum, d);
    if (lane >= d) sum += y;
  }
  if (lane == kWave - 1) part[wave] = sum;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) before += w < wave ? part[w] : 0;
  return before + sum - x;
}

// One entry a lane: its key, and the lanes of the wave with the same.
struct Entry {
  int key;
  uint64_t same;
  __device__ __forceinline__ Entry(const SortCall& c, int64_t i, int bits)
      : key(key_of(c, i)), same(same_key(key, bits)) {}
  // Counted by expert into the wave's own `count`.
  __device__ __forceinline__ void count(const SortCall& c, int* count) const {
    if (key < c.experts && __builtin_ctzll(same) == (int)threadIdx.x % kWave)
      count[key] += __popcll(same);
  }
  // Its row; `next`: the next row of every expert for this wave.
  __device__ __forceinline__ void place(const SortCall& c, int64_t i, int* next) const {
    const int rank = __popcll(same & ((1ull << threadIdx.x % kWave) - 1));
    int row = -1;
    if (key < c.experts) row = next[key] + rank;
    if (i < c.entries) c.pos[i] = row;
    if (row >= 0) {
      c.src[row] = (int)i;
      if (rank == 0) next[key] = row + __popcll(same);
    }
  }
};

__device__ __forceinline__ int bits_of(int experts) { return 32 - __builtin_clz(experts); }

}  // namespace

// First launch of the sort of many entries: every chunk's counts.  (EXPERTS: room in LDS.)
template <int EXPERTS>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs p) {
  __shared__ int count[kSortWaves * EXPERTS];
  const SortCall& c = p.c;
  for (int x = threadIdx.x; x < kSortWaves * c.experts; x += kSortThreads) count[x] = 0;
  __syncthreads();
  const int wave = threadIdx.x / kWave;
  const int64_t first = ((int64_t)blockIdx.x * kSortWaves + wave) * p.per_wave;
  const int lane = threadIdx.x % kWave, bits = bits_of(c.experts);
  for (int64_t i = first + lane; i < first + p.per_wave && i - lane < c.entries; i += kWave)
    Entry(c, i, bits).count(c, count + wave * c.experts);
  __syncthreads();
  if ((int)threadIdx.x < c.experts) {
    int sum = 0;
    for (int w = 0; w < kSortWaves; ++w) sum += count[w * c.experts + threadIdx.x];
    static_cast<int*>(c.ws)[(int64_t)blockIdx.x * c.experts + threadIdx.x] = sum;
  }
}

// Second launch, or the only one where all entries are one workgroup's.
template <int EXPERTS>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortArgs p) {
  __shared__ int next[kSortWaves * EXPERTS], part[kSortWaves];
  const SortCall& c = p.c;
  const int e = threadIdx.x, wave = threadIdx.x / kWave, bits = bits_of(c.experts);
  for (int x = threadIdx.x; x < kSortWaves * c.experts; x += kSortThreads) next[x] = 0;
  __syncthreads();
  const int64_t first = ((int64_t)blockIdx.x * kSortWaves + wave) * p.per_wave;
  const int64_t mine = first + threadIdx.x % kWave, end = first + p.per_wave;
  const Entry held(c, mine, bits);   // the first of a lane's entries, mostly the only one
  held.count(c, next + wave * c.experts);
  for (int64_t i = mine + kWave; i < end && i - mine + first < c.entries; i += kWave)
    Entry(c, i, bits).count(c, next + wave * c.experts);
  // This expert's entries: of all chunks, and of those before this one.
  int total = 0, before = 0;
  if (p.chunks > 1 && e < c.experts) {
    const int* counts = static_cast<const int*>(c.ws) + e;
#pragma unroll 8
    for (int x = 0; x < p.chunks; ++x) {
      const int n = counts[(int64_t)x * c.experts];
      total += n;
      before += x < (int)blockIdx.x ? n : 0;
    }
  }
  __syncthreads();
  if (p.chunks == 1 && e < c.experts)
    for (int w = 0; w < kSortWaves; ++w) total += next[w * c.experts + e];
  const int begin = exclusive_sum(e < c.experts ? total : 0, part);
  int all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) all += part[w];
  if (e < c.experts) {
    int row = begin + before;
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = next[w * c.experts + e];
      next[w * c.experts + e] = row;
      row += n;
    }
    if (blockIdx.x == 0) c.offsets[e] = begin;
  }
  if (blockIdx.x == 0 && e == 0) c.offsets[c.experts] = all;
  __syncthreads();
  held.place(c, mine, next + wave * c.experts);
  for (int64_t i = mine + kWave; i < end && i - mine + first < c.entries; i += kWave)
    Entry(c, i, bits).place(c, i, next + wave * c.experts);
  for (int64_t r = all + (int64_t)blockIdx.x * kSortThreads + threadIdx.x; r < c.entries;
       r += (int64_t)p.chunks * kSortThreads)
    c.src[r] = -1;
}

size_t sort_workspace_bytes(int64_t entries, int experts) {
  return entries <= kSortThreads ? 256 : (size_t)kMostChunks * experts * sizeof(int);
}

namespace {

template <int EXPERTS>
hipError_t launch_sorts(const SortArgs& p, hipStream_t s) {
  if (p.chunks > 1) {
    sort_count_kernel<EXPERTS><<<p.chunks, kSortThreads, 0, s>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  sort_place_kernel<EXPERTS><<<p.chunks, kSortThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sort(const SortCall& c, hipStream_t s) {
  SortArgs p{c, kWave, 1};
  const int64_t n = c.entries;
  if (n > kSortThreads) {
    int64_t chunks = (n + kSortThreads - 1) / kSortThreads;
    if (chunks > kMostChunks) chunks = kMostChunks;
    const int64_t waves = chunks * kSortWaves;
    p.per_wave = (int)((n + waves * kWave - 1) / (waves * kWave) * kWave);
    p.chunks = (int)((n + (int64_t)p.per_wave * kSortWaves - 1) / ((int64_t)p.per_wave * kSortWaves));
  }
  return c.experts <= 128 ? launch_sorts<128>(p, s) : launch_sorts<1024>(p, s);
}

// ---------------------------------------------------------------------- copies and sums by token

namespace {

// 16 bytes of a row as fp32 numbers, and back, rounded to nearest even.
template <int TYPE>
struct Row16 {
  static constexpr int N = 8, SIZE = 2;
  static __device__ __forceinline__ void wide(u32x4 v, float (&x)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const uint16_t b = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
      x[e] = TYPE == GEMM_TYPE_F16 ? LmF16::value(b) : LmBF16::value(b);
    }
  }
  static __device__ __forceinline__ u32x4 narrow(const float (&x)[N]) {
    uint16_t h[N];
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] = TYPE == GEMM_TYPE_F16 ? LmF16::bits(x[e]) : LmBF16::bits(x[e]);
    return __builtin_bit_cast(u32x4, h);
  }
};
template <>
struct Row16<GEMM_TYPE_F32> {
  static constexpr int N = 4, SIZE = 4;
  static __device__ __forceinline__ void wide(u32x4 v, float (&x)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = __builtin_bit_cast(float, (uint32_t)v[e]);
  }
  static __device__ __forceinline__ u32x4 narrow(const float (&x)[N]) {
    return __builtin_bit_cast(u32x4, f32x4{x[0], x[1], x[2], x[3]});
  }
};

// How a call's rows lie: NARROW ones have fewer values than a piece and are stored one by one;
// rows of WHOLE 128-byte lines are loaded past the caches where nobody else reads them
// (combine of 4096 x 8 rows of 4096 bfloat16 56 -> 52 us; rows of 2050 values, whose
// neighbours share lines, 31 -> 37).
enum Rows { NARROW, ANY, WHOLE };

// A thread's piece of a row: N values from column `col`.  The last piece of a row is its
// last N values: those that it shares with the piece before come out the same there.
template <int TYPE, Rows ROWS>
struct Piece {
  typedef Row16<TYPE> R;
  int col;      // where it begins
  int shared;   // values at its front that the piece before has too
  bool inside;  // whether there is one
  __device__ __forceinline__ Piece(int at, int cols) {
    const int want = at * R::N;
    inside = want < cols;
    col = ROWS == NARROW ? 0 : want < cols - R::N ? want : cols - R::N;
    shared = ROWS == NARROW || !inside ? 0 : want - col;
  }
  // ONCE: nobody else reads this row.
  template <bool ONCE = false>
  __device__ __forceinline__ u32x4 get(const void* base, int64_t row, int ld, int cols) const {
    const uint8_t* p = static_cast<const uint8_t*>(base) + row * ld * R::SIZE;
    if constexpr (ROWS == NARROW) return load16_row(p, 0, cols * R::SIZE);
    p += (int64_t)col * R::SIZE;
    if constexpr (ONCE && ROWS == WHOLE)
      return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
    return load16(p);
  }
  // (Past the caches too: the rows of a long call do not fit them.  dispatch of 4096 x 8 rows
  // of 4096 bfloat16 with its sort 63 -> 54 us.)
  __device__ __forceinline__ void put(void* base, int64_t row, int ld, int cols, u32x4 v) const {
    if (!inside) return;
    uint8_t* p = static_cast<uint8_t*>(base) + row * ld * R::SIZE;
    if constexpr (ROWS == NARROW) {
#pragma unroll
      for (int e = 0; e < R::N; ++e)
        if (e < cols) {
          if constexpr (R::SIZE == 4)
            reinterpret_cast<uint32_t*>(p)[e] = v[e % 4];
          else
            reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(v[e / 2 % 4] >> (16 * (e & 1)));
        }
    } else {
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p + (int64_t)col * R::SIZE));
    }
  }
};

constexpr int kCopyThreads = 512;   // at most
constexpr int kSlots = 8;   // slots that are on their way together

struct ExchangeArgs {
  ExchangeCall c;
  int segments;   // workgroups that a row takes, a piece a thread
  int64_t items;  // tokens x segments
};

// The rows and weights of up to 64 slots of a token, a slot a lane: row -1 for none.  (Held
// in scalar registers, those of eight slots spilled.)
struct Slots {
  int row;
  float w;
  __device__ __forceinline__ Slots(const ExchangeCall& c, int64_t token) {
    const int slot = threadIdx.x % kWave;
    const int64_t at = token * c.top_k + slot;
    const int r = slot < c.top_k ? c.pos[at] : -1;
    row = r >= 0 && r < c.rows ? r : -1;
    w = row >= 0 && c.w != nullptr ? c.w[at] : 1.0f;
  }
  __device__ __forceinline__ int row_of(int slot) const {
    return __builtin_amdgcn_readlane(row, slot);
  }
  __device__ __forceinline__ float weight_of(int slot) const {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), slot));
  }
};

}  // namespace

template <int TYPE, Rows ROWS>
__global__ void __launch_bounds__(kCopyThreads) dispatch_kernel(ExchangeArgs p) {
  typedef Row16<TYPE> R;
  const ExchangeCall& c = p.c;
  for (int64_t item = blockIdx.x; item < p.items; item += gridDim.x) {
    const int64_t token = item / p.segments;
    const int segment = (int)(item - token * p.segments);
    const Piece<TYPE, ROWS> piece(segment * blockDim.x + threadIdx.x, c.cols);
    const Slots slots(c, token);
    const u32x4 v = piece.get(c.tok, token, c.ldtok, c.cols);
    float x[R::N];
    R::wide(v, x);
    for (int slot = 0; slot < c.top_k; ++slot) {
      const int row = slots.row_of(slot);
      if (row < 0) continue;
      u32x4 out = v;
      if (c.w != nullptr) {
        const float w = slots.weight_of(slot);
        float y[R::N];
#pragma unroll
        for (int e = 0; e < R::N; ++e) y[e] = w * x[e];
        out = R::narrow(y);
      }
      piece.put(c.out, row, c.ldout, c.cols, out);
    }
  }
}

template <int TYPE, Rows ROWS>
__global__ void __launch_bounds__(kCopyThreads) combine_kernel(ExchangeArgs p) {
  typedef Row16<TYPE> R;
  const ExchangeCall& c = p.c;
  for (int64_t item = blockIdx.x; item < p.items; item += gridDim.x) {
    const int64_t token = item / p.segments;
    const int segment = (int)(item - token * p.segments);
    const Piece<TYPE, ROWS> piece(segment * blockDim.x + threadIdx.x, c.cols);
    const Slots slots(c, token);
    float sum[R::N] = {};
    for (int first = 0; first < c.top_k; first += kSlots) {
      u32x4 v[kSlots];
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        const int row = slots.row_of(first + u);
        if (row >= 0) v[u] = piece.template get<true>(c.sorted, row, c.ldsorted, c.cols);
      }
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        if (slots.row_of(first + u) < 0) continue;
        const float w = slots.weight_of(first + u);
        float x[R::N];
        R::wide(v[u], x);
#pragma unroll
        for (int e = 0; e < R::N; ++e) sum[e] = __builtin_fmaf(w, x[e], sum[e]);
      }
    }
    piece.put(c.out, token, c.ldout, c.cols, R::narrow(sum));
  }
}

// One workgroup a token, since dw sums over its whole row.
template <int TYPE, Rows ROWS>
__global__ void __launch_bounds__(kCopyThreads) combine_grad_kernel(ExchangeArgs p) {
  typedef Row16<TYPE> R;
  const ExchangeCall& c = p.c;
  __shared__ float part[kCopyThreads / kWave][kSlots];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  for (int64_t token = blockIdx.x; token < c.tokens; token += gridDim.x) {
    const Slots slots(c, token);
    for (int first = 0; first < c.top_k; first += kSlots) {
      float dot[kSlots] = {};
      for (int segment = 0; segment < p.segments; ++segment) {
        const Piece<TYPE, ROWS> piece(segment * blockDim.x + threadIdx.x, c.cols);
        u32x4 v[kSlots];
        if (c.dw != nullptr) {
#pragma unroll
          for (int u = 0; u < kSlots; ++u) {
            const int row = slots.row_of(first + u);
            if (row >= 0) v[u] = piece.template get<true>(c.sorted, row, c.ldsorted, c.cols);
          }
        }
        float dy[R::N];
        R::wide(piece.get(c.tok, token, c.ldtok, c.cols), dy);
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
          const int row = slots.row_of(first + u);
          if (row < 0) continue;
          if (c.out != nullptr) {
            const float w = slots.weight_of(first + u);
            float y[R::N];
#pragma unroll
            for (int e = 0; e < R::N; ++e) y[e] = w * dy[e];
            piece.put(c.out, row, c.ldout, c.cols, R::narrow(y));
          }
          if (c.dw != nullptr && piece.inside) {
            float x[R::N];
            R::wide(v[u], x);
#pragma unroll
            for (int e = 0; e < R::N; ++e)   // (a value of two pieces counts once)
              if (e >= piece.shared) dot[u] = __builtin_fmaf(dy[e], x[e], dot[u]);
          }
        }
      }
      if (c.dw == nullptr) continue;
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        float sum = dot[u];
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) sum += __shfl_xor(sum, d);
        if (lane == 0) part[wave][u] = sum;
      }
      __syncthreads();
      const int u = threadIdx.x;
      if (u < kSlots && first + u < c.top_k) {
        float sum = 0.0f;
#pragma unroll
        for (int x = 0; x < kCopyThreads / kWave; ++x)
          if (x < (int)blockDim.x / kWave) sum += part[x][u];
        c.dw[token * c.top_k + first + u] = sum;
      }
      __syncthreads();
    }
  }
}

namespace {

unsigned grid_of(int64_t items) { return (unsigned)(items < (1 << 22) ? items : 1 << 22); }

}  // namespace

// A piece a thread, as few workgroups a row as hold it: a row of 2050 values takes five waves, not
// two workgroups of four (the second for one piece).
#define LASG_LAUNCH(kernel, rows, items)                                                \
  switch (c.type) {                                                                     \
    case GEMM_TYPE_F32:                                                                 \
      kernel<GEMM_TYPE_F32, rows><<<grid_of(items), threads, 0, s>>>(p);                \
      break;                                                                            \
    case GEMM_TYPE_F16:                                                                 \
      kernel<GEMM_TYPE_F16, rows><<<grid_of(items), threads, 0, s>>>(p);                \
      break;                                                                            \
    default: kernel<GEMM_TYPE_BF16, rows><<<grid_of(items), threads, 0, s>>>(p);        \
  }
#define LASG_BY_TYPE(kernel, whole, items)                                              \
  const int n = c.type == GEMM_TYPE_F32 ? 4 : 8;                                        \
  const int pieces = (int)(((int64_t)c.cols + n - 1) / n);                              \
  const int segments = (pieces + kCopyThreads - 1) / kCopyThreads;                      \
  const int each = segments > 0 ? (pieces + segments - 1) / segments : 1;               \
  const unsigned threads = (unsigned)(each + kWave - 1) / kWave * kWave;                \
  const ExchangeArgs p{c, segments, (int64_t)c.tokens * segments};                      \
  if (c.cols < n) {                                                                     \
    LASG_LAUNCH(kernel, NARROW, items)                                                  \
  } else if (whole) {                                                                   \
    LASG_LAUNCH(kernel, WHOLE, items)                                                   \
  } else {                                                                              \
    LASG_LAUNCH(kernel, ANY, items)                                                     \
  }                                                                                     \
  return hipGetLastError()

namespace {

// Whether every sorted row that is read is whole 128-byte lines.
bool whole_lines(const ExchangeCall& c) {
  const int64_t size = c.type == GEMM_TYPE_F32 ? 4 : 2;
  return c.cols * size % 128 == 0 && c.ldsorted * size % 128 == 0 &&
         reinterpret_cast<uintptr_t>(c.sorted) % 128 == 0;
}

}  // namespace

hipError_t launch_dispatch(const ExchangeCall& c, hipStream_t s) {
  LASG_BY_TYPE(dispatch_kernel, false, p.items);
}
hipError_t launch_combine(const ExchangeCall& c, hipStream_t s) {
  LASG_BY_TYPE(combine_kernel, whole_lines(c), p.items);
}
hipError_t launch_combine_grad(const ExchangeCall& c, hipStream_t s) {
  LASG_BY_TYPE(combine_grad_kernel, whole_lines(c), (int64_t)c.tokens);
}

#undef LASG_BY_TYPE
#undef LASG_LAUNCH

}  // namespace lasg
