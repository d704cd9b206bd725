// The norm of many tensors taken together, and their scaling by what clips it
// (bfp8_layer.h).  Memory-bound: the norm reads every value once, the scaling
// reads and writes it once.

#include <algorithm>

#include "layer.h"

namespace bfp8 {
namespace {

// Tensors of one launch: passed by value, so that no table has to be copied to
// the device (28 bytes to spare below 4 KiB of arguments).
constexpr int kJobs = 48;
struct GradBatch {
  const void* g[kJobs];
  void* out[kJobs];
  int64_t rows[kJobs], cols[kJobs], ldg[kJobs], ldo[kJobs];
  int64_t per_row[kJobs];         // vectors that cover a row wherever it starts
  unsigned first[kJobs + 1];      // first chunk of each job
  int f32;                        // of all jobs of the launch
  int n;
};

constexpr int kThreads = 256, kUnroll = 8, kChunk = kThreads * kUnroll;  // vectors

// A vector is 16 bytes at a 16-byte boundary of memory: vector k of a row that
// starts `lead` elements past one holds columns k N - lead .. + N - 1, those of
// them that the row has.  So rows may start anywhere.
template <typename T>
struct Vector {
  static constexpr int N = 16 / sizeof(T);
  float v[N];
  __device__ __forceinline__ void load(const T* row, int64_t c, int64_t cols) {
    if (c >= 0 && c + N <= cols) {
      if constexpr (N == 8) {
        Load8<T>::run(row + c, v, 8);
      } else {
        const float4 u = *reinterpret_cast<const float4*>(row + c);
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = 0.0f;
        if (c + i >= 0 && c + i < cols) {
          if constexpr (N == 8) v[i] = bf16_bits_to_f32(row[c + i]);
          else v[i] = row[c + i];
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* row, int64_t c, int64_t cols, bool aligned) const {
    if (aligned && c >= 0 && c + N <= cols) {
      if constexpr (N == 8) store8(row + c, v, 8);
      else *reinterpret_cast<float4*>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (c + i < 0 || c + i >= cols) continue;
        if constexpr (N == 8) row[c + i] = static_cast<uint16_t>(pack_bf16x2(v[i], 0.0f));
        else row[c + i] = v[i];
      }
    }
  }
};

// Row and first column of vector `at` of job j.
template <typename T>
__device__ __forceinline__ const T* place(const GradBatch& b, int j, int64_t at, int64_t& row,
                                          int64_t& c) {
  row = b.rows[j] == 1 ? 0 : at / b.per_row[j];
  const T* p = static_cast<const T*>(b.g[j]) + row * b.ldg[j];
  const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / static_cast<int>(sizeof(T));
  c = (at - row * b.per_row[j]) * Vector<T>::N - lead;
  return p;
}

// The sum of squares of this workgroup's chunks, in float64: a float32 square
// would overflow past 1.8e19 and vanish below 1e-23.
template <typename T>
__global__ __launch_bounds__(kThreads) void grad_square_kernel(GradBatch b, double* partial) {
  __shared__ double parts[kThreads / 64];
  double sum = 0.0;
  int j = 0;
  for (unsigned chunk = blockIdx.x; chunk < b.first[b.n]; chunk += gridDim.x) {
    while (chunk >= b.first[j + 1]) ++j;
    const int64_t base = static_cast<int64_t>(chunk - b.first[j]) * kChunk + threadIdx.x;
    const int64_t count = b.rows[j] * b.per_row[j], cols = b.cols[j];
    Vector<T> v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = base + u * kThreads;
      int64_t row, c = -Vector<T>::N;  // past the job: no element
      const T* p = static_cast<const T*>(b.g[j]);
      if (at < count) p = place<T>(b, j, at, row, c);
      v[u].load(p, c, cols);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int i = 0; i < Vector<T>::N; ++i) {
        const double x = v[u].v[i];
        sum = fma(x, x, sum);
      }
  }
#pragma unroll
  for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m);
  if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) partial[blockIdx.x] = (parts[0] + parts[1]) + (parts[2] + parts[3]);
}

__global__ __launch_bounds__(1024) void grad_norm_kernel(const double* partial, int64_t n, float* norm) {
  __shared__ double parts[16];
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) sum += partial[i];
#pragma unroll
  for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m);
  if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < 16; ++w) sum += parts[w];
    norm[0] = static_cast<float>(sqrt(sum));
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(GradBatch b, const float* norm,
                                                              float max_norm) {
  const float n = norm[0];
  const float c = n > max_norm ? max_norm / n : n <= max_norm ? 1.0f : n;  // NaN stays NaN
  int j = 0;
  for (unsigned chunk = blockIdx.x; chunk < b.first[b.n]; chunk += gridDim.x) {
    while (chunk >= b.first[j + 1]) ++j;
    if (c == 1.0f && b.out[j] == b.g[j]) continue;  // in place, and nothing to change
    const int64_t base = static_cast<int64_t>(chunk - b.first[j]) * kChunk + threadIdx.x;
    const int64_t count = b.rows[j] * b.per_row[j], cols = b.cols[j];
    Vector<T> v[kUnroll];
    int64_t rows[kUnroll], at_c[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = base + u * kThreads;
      rows[u] = 0, at_c[u] = -Vector<T>::N;
      const T* p = static_cast<const T*>(b.g[j]);
      if (at < count) p = place<T>(b, j, at, rows[u], at_c[u]);
      v[u].load(p, at_c[u], cols);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      T* p = static_cast<T*>(b.out[j]) + rows[u] * b.ldo[j];
#pragma unroll
      for (int i = 0; i < Vector<T>::N; ++i) v[u].v[i] *= c;
      const bool aligned = (reinterpret_cast<uintptr_t>(p + at_c[u]) & 15) == 0;
      v[u].store(p, at_c[u], cols, aligned);
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

// The jobs as launches of up to kJobs tensors of one type and fewer than 2^31
// chunks: calls f(batch, workgroups), first for bf16 jobs and then for fp32.
template <typename F>
bfp8_status for_batches(const bfp8_grad_job* jobs, int64_t n, unsigned most, F&& f) {
  for (int f32 = 0; f32 < 2; ++f32) {
    GradBatch b;
    b.n = 0;
    b.f32 = f32;
    b.first[0] = 0;
    for (int64_t i = 0; i <= n; ++i) {
      const bool mine = i < n && (jobs[i].dt == BFP8_IN_F32) == (f32 == 1);
      const int64_t chunks = mine ? chunks_of(jobs[i]) : 0;
      const bool full = b.n == kJobs || (mine && b.first[b.n] + chunks >= (int64_t(1) << 31));
      if (b.n > 0 && (full || i == n)) {
        const bfp8_status st = f(b, std::min(b.first[b.n], most));
        if (st != BFP8_OK) return st;
        b.n = 0;
      }
      if (chunks == 0) continue;
      const bfp8_grad_job& j = jobs[i];
      b.g[b.n] = j.g;
      b.out[b.n] = j.out;
      b.rows[b.n] = j.rows;
      b.cols[b.n] = j.cols;
      b.ldg[b.n] = j.ldg;
      b.ldo[b.n] = j.ldo;
      b.per_row[b.n] = vectors_per_row(j);
      b.first[b.n + 1] = b.first[b.n] + static_cast<unsigned>(chunks);
      ++b.n;
    }
  }
  return BFP8_OK;
}

}  // namespace

size_t grad_norm_workspace(const bfp8_grad_job* jobs, int64_t n) {
  size_t groups = 0;
  for_batches(jobs, n, kMaxGroups, [&](const GradBatch&, unsigned g) {
    groups += g;
    return BFP8_OK;
  });
  return groups * sizeof(double);
}

bfp8_status launch_grad_norm(const bfp8_grad_job* jobs, int64_t n, float* norm, double* partial,
                             hipStream_t stream) {
  int64_t at = 0;
  const bfp8_status st = for_batches(jobs, n, kMaxGroups, [&](const GradBatch& b, unsigned groups) {
    double* p = partial + at;
    at += groups;
    return b.f32 ? launch(grad_square_kernel<float>, dim3(groups), dim3(kThreads), stream, b, p)
                 : launch(grad_square_kernel<uint16_t>, dim3(groups), dim3(kThreads), stream, b, p);
  });
  if (st != BFP8_OK) return st;
  return launch(grad_norm_kernel, dim3(1), dim3(1024), stream, partial, at, norm);
}

bfp8_status launch_grad_clip(const bfp8_grad_job* jobs, int64_t n, const float* norm,
                             float max_norm, hipStream_t stream) {
  return for_batches(jobs, n, 1u << 20, [&](const GradBatch& b, unsigned groups) {
    return b.f32 ? launch(grad_scale_kernel<float>, dim3(groups), dim3(kThreads), stream, b, norm, max_norm)
                 : launch(grad_scale_kernel<uint16_t>, dim3(groups), dim3(kThreads), stream, b, norm, max_norm);
  });
}

}  // namespace bfp8
