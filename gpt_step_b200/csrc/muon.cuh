// Newton-Schulz orthogonalisation of weight-shaped matrices on tcgen05.
//
// For each matrix M of a batch, X = M / (|M|_F + 1e-7), taken with the smaller
// dimension as its n rows (m columns), goes through `steps` rounds of
//   A = X X^T,   P = a I + b A + c A A,   X <- P X,
// (a, b, c) = (3.4445, -4.7750, 2.0315): every singular value s becomes
// a s + b s^3 + c s^5, which takes any s in (0, 1] to about 0.7 .. 1.2 in five
// rounds and leaves the singular vectors as they are.
//
// Numbers. The small singular values grow by up to a^5 = 485, and so does every
// rounding error that lies along them. With bf16 operands the result is 1% (a
// flat spectrum) to 4% (a falling one) off; fp16 operands have three more bits
// at the same tensor rate and their range is enough, because every element of X,
// A, P is bounded (1.21, 1.46, 16): they are held times 2^10. X is held as two fp16
// numbers (hi + lo, 22 bits) in all but the last two rounds: the tensor cores see hi
// alone, and a lo, its part in the term a X along which the growth happens, is added
// in fp32, for no more matrix instructions. Five rounds then end 0.10 to 0.13% off on spectra
// that are flat or fall like 1/k (0.5% without lo) and 0.15 to 0.21% on steeper ones (1/k^2,
// e^(-k/20); 2% and 1.5% without), beside the 0.17% of the bf16 result's own rounding. lo
// needs its fp16: with e4m3, half the bytes and 3% less time for large matrices, eight rounds on
// the steep spectra ended 0.6 to 0.9% off, the result's rounding included, instead of 0.22 to 0.38%.
// From eight rounds on the fp32 sums of P X count too: what they leave grows by up to 3.44 a
// round (1,536 rows, e^(-k/20): 0.27% after five rounds, 0.38% after eight, 2.4% after ten).
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace muon {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScale = 1024.f, kInvScale = 1.f / 1024.f;
constexpr int kMaxSteps = 16;
constexpr int kMaxDim = 16384;

// ---------------------------------------------------------------------------
// |M|_F: fp64 partial sums of squares, `parts` a matrix
// ---------------------------------------------------------------------------
template <typename T>
GPT2_DEV float load1(const T* p) { return (float)*p; }
template <>
GPT2_DEV float load1<bf16>(const bf16* p) { return __bfloat162float(*p); }

template <typename T>
__global__ void __launch_bounds__(256) ns_sumsq_kernel(const T* __restrict__ x, long stride, long count, int vec,
                                                       double* __restrict__ part) {
  pdl_begin();
  __shared__ double red[8];
  const T* m = x + (size_t)blockIdx.y * stride;
  double s = 0.0;
  const long step = (long)gridDim.x * 256;
  long done = 0;
  if (vec) {
    constexpr int E = 16 / sizeof(T);
    const long nv = count / E;
    for (long i = blockIdx.x * 256L + threadIdx.x; i < nv; i += step) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(m) + i);
      const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const double v = load1(e + j);
        s += v * v;
      }
    }
    done = nv * E;
  }
  for (long i = done + blockIdx.x * 256L + threadIdx.x; i < count; i += step) {
    const double v = load1(m + i);
    s += v * v;
  }
  s = warp_sum_d(s);
  if (lane_id() == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) s += red[w];
    part[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = s;
  }
}

// ---------------------------------------------------------------------------
// X = M / (|M|_F + 1e-7), times 2^10, as hi and lo [batch][n][ld] fp16, padding 0;
// and the counters of the rounds at 0. A thread forms 8 columns of a row; tall matrices
// come through shared memory, 64 x 64 at a time.
// ---------------------------------------------------------------------------
GPT2_DEV uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// hi and lo of eight values
GPT2_DEV void split8(const float* f, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_half2(f[2 * i], f[2 * i + 1]);
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    l[i] = pack_half2(f[2 * i] - v.x, f[2 * i + 1] - v.y);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Eight neighbouring elements, in 16-byte loads if `vec`; those from `valid` on are 0.
template <typename T>
GPT2_DEV void load8(const T* p, int valid, bool vec, float (&f)[8]) {
  if (vec && valid >= 8) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int q = 0; q < 8; q += E) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(p + q));
      const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int j = 0; j < E; ++j) f[q + j] = load1(e + j);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = q < valid ? load1(p + q) : 0.f;
  }
}

template <typename T, bool TALL>
__global__ void __launch_bounds__(256) ns_convert_kernel(const T* __restrict__ x, long stride, int rows, int cols,
                                                         const double* __restrict__ part, int parts,
                                                         __half* __restrict__ hi, __half* __restrict__ lo, int ld,
                                                         int vec, uint32_t* __restrict__ count) {
  pdl_begin();
  __shared__ float tile[TALL ? 64 : 1][65];
  __shared__ float mul_s;
  const int z = blockIdx.y;
  if (threadIdx.x < 32) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 32) s += part[(size_t)z * parts + i];
    s = warp_sum_d(s);
    if (threadIdx.x == 0) mul_s = (float)((double)kScale / (sqrt(s) + 1e-7));
    if (blockIdx.x == 0 && threadIdx.x < 3) count[z * 3 + threadIdx.x] = 0;
  }
  __syncthreads();
  const float mul = mul_s;
  const int n = TALL ? cols : rows, m = TALL ? rows : cols;
  const T* src = x + (size_t)z * stride;
  auto put = [&](int r, int c, float (&f)[8]) {
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] *= mul;
    uint4 h, l;
    split8(f, h, l);
    const size_t at = ((size_t)z * n + r) * ld + c;
    *reinterpret_cast<uint4*>(hi + at) = h;
    *reinterpret_cast<uint4*>(lo + at) = l;
  };
  if (!TALL) {
    const int per_row = ld / 8;
    const long units = (long)n * per_row;
#pragma unroll 4
    for (long u = blockIdx.x * 256L + threadIdx.x; u < units; u += gridDim.x * 256L) {
      const int r = (int)(u / per_row), c = (int)(u - (long)r * per_row) * 8;
      float f[8];
      load8(src + (size_t)r * cols + c, m - c, vec, f);
      put(r, c, f);
    }
  } else {
    // tiles of 64 columns of X (rows of M) x 64 rows of X
    const int tr = (n + 63) / 64;
    const long tiles = (long)tr * (ld / 64);
    for (long t = blockIdx.x; t < tiles; t += gridDim.x) {
      const int r0 = (int)(t % tr) * 64, c0 = (int)(t / tr) * 64;
      // 8 threads a row of M, 32 rows at a time
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = threadIdx.x / 8 + 32 * h, r = (threadIdx.x % 8) * 8;
        float f[8];
        load8(src + (size_t)(c0 + c) * cols + r0 + r, c0 + c < m ? n - r0 - r : 0, vec, f);
#pragma unroll
        for (int q = 0; q < 8; ++q) tile[c][r + q] = f[q];
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = threadIdx.x / 8 + 32 * h, c = (threadIdx.x % 8) * 8;
        float f[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = tile[c + q][r];
        if (r0 + r < n) put(r0 + r, c0 + c, f);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// shared by the kernels of the rounds
// ---------------------------------------------------------------------------
constexpr int BK = 64;   // fp16 elements of a 128-byte swizzle row

// fp16 x fp16 -> fp32
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
struct Work {
  int n, m, ld_x, ld_a, parts;
  size_t x0, x1, lo, a, q, part, count, total;
};

inline bool plan(int batch, int rows, int cols, Work* w) {
  if (batch <= 0 || batch > 65535 || rows <= 0 || cols <= 0 || rows > kMaxDim || cols > kMaxDim) return false;
  w->n = std::min(rows, cols);
  w->m = std::max(rows, cols);
  w->ld_x = (w->m + 63) / 64 * 64;
  w->ld_a = (w->n + 63) / 64 * 64;
  const long count = (long)rows * cols;
  w->parts = (int)std::max(1L, std::min((count + 8191) / 8192, std::max(1L, 148L * 8 / batch)));
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t r = o; o += (bytes + 255) / 256 * 256; return r; };
  const size_t xb = (size_t)batch * w->n * w->ld_x * 2, ab = (size_t)batch * w->n * w->ld_a * 2;
  w->x0 = take(xb);
  w->x1 = take(xb);
  w->lo = take(xb);
  w->a = take(ab);
  w->q = take(ab);
  w->part = take((size_t)batch * w->parts * 8);
  w->count = take((size_t)batch * 3 * 4);
  w->total = o;
  return true;
}

// X of the batch into the workspace. have_parts: it holds the partial sums of squares already.
template <typename T>
cudaError_t prepare_x(const Work& w, char* base, const T* x, long x_stride, int batch, int rows, int cols,
                      bool have_parts, cudaStream_t s) {
  double* part = reinterpret_cast<double*>(base + w.part);
  const int vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (batch == 1 || (x_stride * sizeof(T)) % 16 == 0);
  if (!have_parts) {
    const cudaError_t e = launch_pdl(ns_sumsq_kernel<T>, dim3(w.parts, batch), dim3(256), 0, s, x, x_stride,
                                     (long)rows * cols, vec, part);
    if (e != cudaSuccess) return e;
  }
  __half* hi = reinterpret_cast<__half*>(base + w.x0);
  __half* lo = reinterpret_cast<__half*>(base + w.lo);
  uint32_t* count = reinterpret_cast<uint32_t*>(base + w.count);
  const bool tall = rows > cols;
  const int vec_rows = vec && (cols * sizeof(T)) % 16 == 0;   // every row of M begins on 16 bytes
  const long work = tall ? (long)((w.n + 63) / 64) * (w.ld_x / 64) : ((long)w.n * w.ld_x / 8 + 255) / 256;
  const int grid = (int)std::min(work, std::max(1L, 148L * 8 / batch));
  return launch_pdl(tall ? ns_convert_kernel<T, true> : ns_convert_kernel<T, false>, dim3(grid, batch), dim3(256), 0, s,
                    x, x_stride, rows, cols, (const double*)part, w.parts, hi, lo, w.ld_x, vec_rows, count);
}

}  // namespace muon
