// The norm of many tensors taken together, and their scaling by what clips it
// (bfp8_layer.h).  Memory-bound: the norm reads every value once, the scaling
// reads and writes it once.

#include <algorithm>

#include "layer.h"

namespace bfp8 {
namespace {

// Tensors of one launch: passed by value, so that no table has to be copied to
// the device.  Arguments lie in host memory, where each cache line that a kernel
// touches first costs it a trip: the chunks' bounds are together, and what belongs to a
// job is one line.
struct BatchJob {
  const void* g;
  void* out;
  int64_t rows, cols, ldg, ldo;
  int64_t per_row;  // vectors that cover a row wherever it starts
  int64_t fill;     // up to the line
};
constexpr int kJobs = 58;
struct GradBatch {
  int n;
  unsigned first[kJobs + 1];  // first chunk of each job
  BatchJob job[kJobs];
};
static_assert(sizeof(BatchJob) == 64 && sizeof(GradBatch) + 64 <= 4096, "kernel arguments");

// Vectors of a chunk: 2, 4 and 8 a thread took 186, 188 and 196 us for 101 million
// float32 values, and 50 to 51 for 50 million in bf16.
constexpr int kThreads = 256, kUnroll = 4, kChunk = kThreads * kUnroll;

// A vector is 16 bytes at a 16-byte boundary of memory: vector k of a row that
// starts `lead` elements past one holds columns k N - lead .. + N - 1, those of
// them that the row has.  So rows may start anywhere.
template <typename T>
struct Vector {
  static constexpr int N = 16 / sizeof(T);
  uint32_t w[4];
  __device__ __forceinline__ void load(const T* p) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  }
  __device__ __forceinline__ void load_part(const T* row, int64_t c, int64_t cols) {
    if (c >= 0 && c + N <= cols) return load(row + c);
    auto bits = [&](int i) -> uint32_t {
      if (c + i < 0 || c + i >= cols) return 0u;
      if constexpr (N == 8) return row[c + i];
      else return __float_as_uint(row[c + i]);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = N == 8 ? bits(2 * i) | bits(2 * i + 1) << 16 : bits(i);
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (N == 8)
      return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    else
      return __uint_as_float(w[i]);
  }
  __device__ __forceinline__ void scale(float c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (N == 8) w[i] = pack_bf16x2(get(2 * i) * c, get(2 * i + 1) * c);
      else w[i] = __float_as_uint(get(i) * c);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    store_once(p, make_uint4(w[0], w[1], w[2], w[3]));
  }
  __device__ __forceinline__ void store_part(T* row, int64_t c, int64_t cols) const {
    if (c >= 0 && c + N <= cols && (reinterpret_cast<uintptr_t>(row + c) & 15) == 0)
      return store(row + c);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (c + i < 0 || c + i >= cols) continue;
      if constexpr (N == 8) row[c + i] = static_cast<T>(w[i >> 1] >> (16 * (i & 1)));
      else row[c + i] = __uint_as_float(w[i]);
    }
  }
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0; }
};

template <typename T>
__device__ __forceinline__ int lead_of(const T* p) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / static_cast<int>(sizeof(T));
}

// One chunk of a job: the first element of a dense one that has all its vectors
// (most are), or null.
template <typename T>
__device__ __forceinline__ const T* whole_chunk(const GradBatch& b, int j, int64_t base) {
  const T* p = static_cast<const T*>(b.job[j].g);
  const int64_t c = base * Vector<T>::N - lead_of(p);
  return b.job[j].rows == 1 && c >= 0 && c + kChunk * Vector<T>::N <= b.job[j].cols ? p + c : nullptr;
}

// Row, first column and first element of the row of vector `at` of job j.
template <typename T>
__device__ __forceinline__ const T* place(const GradBatch& b, int j, int64_t at, int64_t& row,
                                          int64_t& c) {
  row = b.job[j].rows == 1 ? 0 : at / b.job[j].per_row;
  const T* p = static_cast<const T*>(b.job[j].g) + row * b.job[j].ldg;
  c = (at - row * b.job[j].per_row) * Vector<T>::N - lead_of(p);
  return p;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) v += __shfl_xor(v, m);
  return v;
}

// The sum of squares of this workgroup's chunks, in float64: a float32 square
// would overflow past 1.8e19 and vanish below 1e-23.
template <typename T>
__global__ __launch_bounds__(kThreads) void grad_square_kernel(GradBatch b, double* partial) {
  __shared__ double parts[kThreads / 64];
  constexpr int N = Vector<T>::N;
  double sum[2] = {0.0, 0.0};
  int j = 0;
  for (unsigned chunk = blockIdx.x; chunk < b.first[b.n]; chunk += gridDim.x) {
    while (chunk >= b.first[j + 1]) ++j;
    const int64_t base = static_cast<int64_t>(chunk - b.first[j]) * kChunk;
    Vector<T> v[kUnroll];
    if (const T* p = whole_chunk<T>(b, j, base)) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) v[u].load(p + (u * kThreads + threadIdx.x) * N);
    } else {
      const int64_t count = b.job[j].rows * b.job[j].per_row;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t at = base + u * kThreads + threadIdx.x;
        v[u].clear();
        if (at >= count) continue;
        int64_t row, c;
        const T* q = place<T>(b, j, at, row, c);
        v[u].load_part(q, c, b.job[j].cols);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const double x = v[u].get(i);
        sum[i & 1] = fma(x, x, sum[i & 1]);
      }
  }
  const double all = wave_sum(sum[0] + sum[1]);
  if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = all;
  __syncthreads();
  if (threadIdx.x == 0) partial[blockIdx.x] = (parts[0] + parts[1]) + (parts[2] + parts[3]);
}

// The norm from all partial sums, by one workgroup of kThreads; the same order
// and so the same bits wherever it is done.
__device__ __forceinline__ float norm_of(const double* partial, int64_t n, double* parts) {
  double sum = 0.0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < n; i += kThreads) sum += partial[i];
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = sum;
  __syncthreads();
  return static_cast<float>(sqrt((parts[0] + parts[1]) + (parts[2] + parts[3])));
}

__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const double* partial, int64_t n, float* norm) {
  __shared__ double parts[kThreads / 64];
  const float v = norm_of(partial, n, parts);
  if (threadIdx.x == 0) norm[0] = v;
}

__device__ __forceinline__ float factor_of(float norm, float max_norm) {
  return norm > max_norm ? max_norm / norm : norm <= max_norm ? 1.0f : norm;  // NaN stays NaN
}

// Scales by max_norm over the norm: a given one, or (OWN) that of `partial`'s n
// sums, which every workgroup adds up for itself and the first one writes down.
template <typename T, bool OWN>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(GradBatch b, float* norm, float max_norm,
                                                              const double* partial, int64_t n) {
  __shared__ double parts[kThreads / 64];
  constexpr int N = Vector<T>::N;
  float v;
  if (OWN) {
    v = norm_of(partial, n, parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) norm[0] = v;
  } else {
    v = norm[0];
  }
  const float c = factor_of(v, max_norm);
  // Last chunks first, which the norm read last, and results past the caches:
  // what is left of the gradients in the last-level cache is read from there
  // (225 -> 194 us for 101 million float32 values, 59 -> 50 for 50 million in bf16).
  int j = b.n - 1;
  const unsigned last = b.first[b.n] - 1;
  for (unsigned turn = blockIdx.x; turn <= last; turn += gridDim.x) {
    const unsigned chunk = last - turn;
    while (chunk < b.first[j]) --j;
    if (c == 1.0f && b.job[j].out == b.job[j].g) continue;  // in place, and nothing to change
    const int64_t base = static_cast<int64_t>(chunk - b.first[j]) * kChunk;
    Vector<T> x[kUnroll];
    const T* p = whole_chunk<T>(b, j, base);
    T* o = static_cast<T*>(b.job[j].out);
    if (p != nullptr) o += p - static_cast<const T*>(b.job[j].g);
    if (p != nullptr && lead_of(o) == 0) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) x[u].load(p + (u * kThreads + threadIdx.x) * N);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        x[u].scale(c);
        x[u].store(o + (u * kThreads + threadIdx.x) * N);
      }
      continue;
    }
    const int64_t count = b.job[j].rows * b.job[j].per_row, cols = b.job[j].cols;
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = base + u * kThreads + threadIdx.x;
      if (at >= count) break;
      int64_t row, col;
      const T* q = place<T>(b, j, at, row, col);
      x[0].load_part(q, col, cols);
      x[0].scale(c);
      x[0].store_part(static_cast<T*>(b.job[j].out) + row * b.job[j].ldo, col, cols);
    }
  }
}

int64_t vectors_per_row(const bfp8_grad_job& j) {
  const int64_t size = j.dt == BFP8_IN_F32 ? 4 : 2, per = 16 / size;
  // the worst lead of any row
  int64_t lead = per - 1;
  if (j.rows == 1 || j.ldg * size % 16 == 0)
    lead = static_cast<int64_t>(reinterpret_cast<uintptr_t>(j.g) & 15) / size;
  return (j.cols + lead + per - 1) / per;
}
int64_t chunks_of(const bfp8_grad_job& j) {
  return j.rows == 0 || j.cols == 0 ? 0 : (j.rows * vectors_per_row(j) + kChunk - 1) / kChunk;
}

constexpr unsigned kMaxGroups = 1024;  // workgroups of a norm launch: one partial sum each
constexpr unsigned kMaxScaleGroups = 1u << 20;
// Sums that every workgroup of the scaling adds up for itself; more of them (and
// none) get a launch of their own.
constexpr int64_t kOwnSums = 2 * kMaxGroups;

void add_job(GradBatch& b, const bfp8_grad_job& j, int64_t chunks) {
  b.job[b.n] = BatchJob{j.g, j.out, j.rows, j.cols, j.ldg, j.ldo, vectors_per_row(j), 0};
  b.first[b.n + 1] = b.first[b.n] + static_cast<unsigned>(chunks);
  ++b.n;
}

void clear(GradBatch& b) {
  b.n = 0;
  b.first[0] = 0;
}

// The jobs as launches of up to kJobs tensors of one type and fewer than 2^31
// chunks: calls f(batch, its type, workgroups), first for bf16 jobs, then for fp32.
template <typename F>
bfp8_status for_batches(const bfp8_grad_job* jobs, int64_t n, unsigned most, F&& f) {
  for (int f32 = 0; f32 < 2; ++f32) {
    GradBatch b;
    clear(b);
    for (int64_t i = 0; i <= n; ++i) {
      const bool mine = i < n && (jobs[i].dt == BFP8_IN_F32) == (f32 == 1);
      const int64_t chunks = mine ? chunks_of(jobs[i]) : 0;
      const bool full = b.n == kJobs || b.first[b.n] + chunks >= (int64_t(1) << 31);
      if (b.n > 0 && (full || i == n)) {
        const bfp8_status st = f(b, f32 == 1, std::min(b.first[b.n], most));
        if (st != BFP8_OK) return st;
        clear(b);
      }
      if (chunks > 0) add_job(b, jobs[i], chunks);
    }
  }
  return BFP8_OK;
}

}  // namespace

size_t grad_norm_workspace(const bfp8_grad_job* jobs, int64_t n) {
  size_t groups = 0;
  for_batches(jobs, n, kMaxGroups, [&](const GradBatch&, bool, unsigned g) {
    groups += g;
    return BFP8_OK;
  });
  return groups * sizeof(double);
}

bfp8_status launch_grad_clip(const bfp8_grad_job* jobs, int64_t n, float* norm, float max_norm,
                             hipStream_t stream) {
  return for_batches(jobs, n, kMaxScaleGroups, [&](const GradBatch& b, bool f32, unsigned groups) {
    return launch(f32 ? grad_scale_kernel<float, false> : grad_scale_kernel<uint16_t, false>,
                  dim3(groups), dim3(kThreads), stream, b, norm, max_norm, nullptr, int64_t(0));
  });
}

// The partial sums; n_sums receives their number.
static bfp8_status launch_squares(const bfp8_grad_job* jobs, int64_t n, double* partial,
                                  int64_t& n_sums, hipStream_t stream) {
  n_sums = 0;
  return for_batches(jobs, n, kMaxGroups, [&](const GradBatch& b, bool f32, unsigned groups) {
    double* p = partial + n_sums;
    n_sums += groups;
    return launch(f32 ? grad_square_kernel<float> : grad_square_kernel<uint16_t>, dim3(groups),
                  dim3(kThreads), stream, b, p);
  });
}

bfp8_status launch_grad_norm(const bfp8_grad_job* jobs, int64_t n, float* norm, double* partial,
                             hipStream_t stream) {
  int64_t n_sums;
  const bfp8_status st = launch_squares(jobs, n, partial, n_sums, stream);
  if (st != BFP8_OK) return st;
  return launch(grad_norm_kernel, dim3(1), dim3(kThreads), stream, partial, n_sums, norm);
}

bfp8_status launch_grad_norm_clip(const bfp8_grad_job* jobs, int64_t n, float* norm, float max_norm,
                                  double* partial, hipStream_t stream) {
  int64_t n_sums;
  bfp8_status st = launch_squares(jobs, n, partial, n_sums, stream);
  if (st != BFP8_OK) return st;
  if (n_sums == 0 || n_sums > kOwnSums) {
    st = launch(grad_norm_kernel, dim3(1), dim3(kThreads), stream, partial, n_sums, norm);
    return st != BFP8_OK ? st : launch_grad_clip(jobs, n, norm, max_norm, stream);
  }
  return for_batches(jobs, n, kMaxScaleGroups, [&](const GradBatch& b, bool f32, unsigned groups) {
    return launch(f32 ? grad_scale_kernel<float, true> : grad_scale_kernel<uint16_t, true>,
                  dim3(groups), dim3(kThreads), stream, b, norm, max_norm, partial, n_sums);
  });
}

}  // namespace bfp8
