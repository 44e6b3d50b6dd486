// Newton-Schulz orthogonalisation of weight-shaped matrices on tcgen05.
//
// For each matrix M of a batch, X = M / (|M|_F + 1e-7), taken with the smaller
// dimension as its n rows (m columns), goes through `steps` rounds of
//   A = X X^T,   Q = b A + c A A,   X <- a X + Q X,
// (a, b, c) = (3.4445, -4.7750, 2.0315): every singular value s becomes
// a s + b s^3 + c s^5, which takes any s in (0, 1] to about 0.7 .. 1.2 in five
// rounds and leaves the singular vectors as they are.
//
// Numbers. The small singular values grow by up to a^5 = 485, and so does every
// rounding error that lies along them. With bf16 operands the result is 1% (a
// flat spectrum) to 4% (a falling one) off; fp16 operands have three more bits
// at the same tensor rate and their range is enough, because every element of X,
// A, Q is bounded (1.21, 1.46, 12): they are held times 2^10. The term a X, along
// which the growth happens, is added in fp32 from X held as two fp16 numbers
// (hi + lo, 22 bits) in all but the last two rounds; the tensor cores see hi
// alone. That ends 0.1% off for either spectrum (0.5% without lo) for no more
// matrix instructions, below the 0.17% of the bf16 result's own rounding.
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
// X = M / (|M|_F + 1e-7), times 2^10, as hi and lo [batch][n][ld] fp16;
// 64 x 64 tiles through shared memory, transposed for tall matrices
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) ns_convert_kernel(const T* __restrict__ x, long stride, int rows, int cols,
                                                         const double* __restrict__ part, int parts,
                                                         __half* __restrict__ hi, __half* __restrict__ lo, int ld) {
  pdl_begin();
  __shared__ float tile[64][65];
  __shared__ float mul;
  if (threadIdx.x < 32) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 32) s += part[(size_t)blockIdx.z * parts + i];
    s = warp_sum_d(s);
    if (threadIdx.x == 0) mul = (float)((double)kScale / (sqrt(s) + 1e-7));
  }
  const bool tall = rows > cols;
  const int n = tall ? cols : rows, m = tall ? rows : cols;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;   // of X
  const T* src = x + (size_t)blockIdx.z * stride;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  for (int i = ty; i < 64; i += 4) {
    // the inner index runs along the stored rows of M either way
    const int xr = tall ? r0 + tx : r0 + i, xc = tall ? c0 + i : c0 + tx;
    float v = 0.f;
    if (xr < n && xc < m) v = load1(src + (tall ? (size_t)xc * cols + xr : (size_t)xr * cols + xc));
    if (tall) tile[tx][i] = v;
    else tile[i][tx] = v;
  }
  __syncthreads();
  const float mu = mul;
  for (int i = ty; i < 64; i += 4) {
    const int xr = r0 + i, xc = c0 + tx;
    if (xr >= n || xc >= ld) continue;
    const float v = tile[i][tx] * mu;
    const __half h = __float2half_rn(v);
    const size_t at = ((size_t)blockIdx.z * n + xr) * ld + xc;
    hi[at] = h;
    lo[at] = __float2half_rn(v - __half2float(h));
  }
}

// ---------------------------------------------------------------------------
// the three products
// ---------------------------------------------------------------------------
enum Mode : int { GRAM = 0, POLY = 1, APPLY = 2, LAST = 3 };

constexpr int BM = 128, BN = 128, BK = 64, STAGES = 3;
constexpr int kStageBytes = (BM + BN) * BK * 2;
constexpr int kSmem = STAGES * kStageBytes + 1024 + 256;
constexpr int kThreads = 192;

struct Params {
  int n, m, ld_x, ld_a;      // X is [n][m], its rows ld_x apart; A, Q are [n][n], rows ld_a apart
  int nkb;                   // 64-wide blocks of the reduction
  __half* out;               // GRAM: A, POLY: Q, APPLY: the next X's hi
  const __half* aux;         // POLY: A, APPLY and LAST: X's hi
  __half* lo;                // APPLY: X's lo, read (use_lo) and written (put_lo); LAST: read
  bf16* result;              // LAST: [rows][cols], transposed back for tall matrices
  long result_stride;
  int rows, cols;
  int use_lo, put_lo;
  int* err;
};

GPT2_DEV void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// fp16 x fp16 -> fp32
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

GPT2_DEV uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

GPT2_DEV void load_half32(const __half* p, float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 u = *reinterpret_cast<const uint4*>(p + 8 * j);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[h]));
      v[8 * j + 2 * h] = f.x;
      v[8 * j + 2 * h + 1] = f.y;
    }
  }
}

GPT2_DEV void store_half32(__half* p, const float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(p + 8 * j) =
        make_uint4(pack_half2(v[8 * j], v[8 * j + 1]), pack_half2(v[8 * j + 2], v[8 * j + 3]),
                   pack_half2(v[8 * j + 4], v[8 * j + 5]), pack_half2(v[8 * j + 6], v[8 * j + 7]));
}

// One 128 x 128 output tile a CTA: warp 0 brings operands in by TMA, warp 1
// issues the MMAs, warps 2..5 run the epilogue. A and Q are symmetric: their
// tiles below the diagonal are computed and written to both places.
template <int MODE>
__global__ void __launch_bounds__(kThreads, 2)
    ns_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                   const Params p) {
  extern __shared__ __align__(1024) uint8_t ns_smem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ns_smem) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * kStageBytes);
  uint64_t* empty = full + STAGES;
  uint64_t* done = empty + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  constexpr bool SYM = MODE == GRAM || MODE == POLY;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    mbar_init(smem_u32(done), 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_begin();

  int ti, tj;
  if (SYM) {
    // tile index -> (ti, tj), tj <= ti
    ti = (int)((sqrtf(8.f * blockIdx.x + 1.f) - 1.f) * 0.5f);
    while ((ti + 1) * (ti + 2) / 2 <= (int)blockIdx.x) ++ti;
    while (ti * (ti + 1) / 2 > (int)blockIdx.x) --ti;
    tj = blockIdx.x - ti * (ti + 1) / 2;
  } else {
    const int num_m = (p.n + BM - 1) / BM;
    ti = blockIdx.x % num_m;
    tj = blockIdx.x / num_m;
  }
  const int z = blockIdx.y;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = 0; kb < p.nkb; ++kb) {
        if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1, p.err)) break;
        const uint32_t fb = smem_u32(&full[stage]);
        mbar_arrive_expect_tx(fb, kStageBytes);
        const uint32_t sa = smem_u32(smem + stage * kStageBytes), sb = sa + BM * BK * 2;
        tma_load_3d(sa, &tm_a, fb, kb * BK, ti * BM, z);
        if (SYM) {
          tma_load_3d(sb, &tm_b, fb, kb * BK, tj * BN, z);
        } else {
          for (int j = 0; j < BN / 64; ++j) tma_load_3d(sb + j * 8192, &tm_b, fb, tj * BN + 64 * j, kb * BK, z);
        }
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f16_f32(BM, BN, !SYM);
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = 0; kb < p.nkb; ++kb) {
        if (!mbar_wait(smem_u32(&full[stage]), phase, p.err)) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + stage * kStageBytes), sb = sa + BM * BK * 2;
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
          const uint64_t ad = smem_desc_sw128(sa + kk * 32, 16, 1024);
          const uint64_t bd = SYM ? smem_desc_sw128(sb + kk * 32, 16, 1024)
                                  : smem_desc_sw128(sb + kk * 2048, 8192, 1024);
          tc_mma_bf16(tmem, ad, bd, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
        }
        tc_commit(smem_u32(&empty[stage]));
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
      }
      tc_commit(smem_u32(done));
      mbar_wait(smem_u32(done), 0, p.err);
    }
  } else if (mbar_wait(smem_u32(done), 0, p.err)) {
    tc_fence_after();
    const int q = warp & 3;
    const int row = ti * BM + q * 32 + lane;
    const bool row_ok = row < p.n;
    const int ld = SYM ? p.ld_a : p.ld_x;
    const size_t zrow = ((size_t)z * p.n + row) * ld;
#pragma unroll 1
    for (int c = 0; c < BN; c += 32) {
      const int col = tj * BN + c;
      if (col >= ld) break;                 // ld is a multiple of 64
      float v[32];
      tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + c, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= MODE == POLY ? kC * kInvScale : kInvScale;
      if (MODE != GRAM && row_ok) {
        constexpr float f = MODE == POLY ? kB : kA;
        float x[32];
        load_half32(p.aux + zrow + col, x);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = fmaf(f, x[i], v[i]);
        if (MODE >= APPLY && p.use_lo) {
          load_half32(p.lo + zrow + col, x);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = fmaf(f, x[i], v[i]);
        }
      }
      if (MODE == LAST) {
        const bool tall = p.rows > p.cols;
        bf16* res = p.result + (size_t)z * p.result_stride;
        if (row_ok) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (col + i < p.m)
              res[tall ? (size_t)(col + i) * p.cols + row : (size_t)row * p.cols + col + i] =
                  __float2bfloat16_rn(v[i] * kInvScale);
        }
        continue;
      }
      if (row_ok) {
        store_half32(p.out + zrow + col, v);
        if (MODE == APPLY && p.put_lo) {
          float l[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) l[i] = v[i] - __half2float(__float2half_rn(v[i]));
          store_half32(p.lo + zrow + col, l);
        }
      }
      if (SYM && ti != tj && row < ld) {
        // the mirror image; rows n .. ld - 1 are 0 and become its padding
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (col + i < p.n) p.out[((size_t)z * p.n + col + i) * ld + row] = __float2half_rn(v[i]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, BN);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
struct Work {
  int n, m, ld_x, ld_a, parts;
  size_t x0, x1, lo, a, q, part, total;
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
  w->total = o;
  return true;
}

// [batch][rows][ld] fp16; boxes of 64 columns x box_rows rows of one matrix
inline bool map_3d(CUtensorMap* m, const __half* base, int ld, int rows, int batch, uint32_t box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)ld, (cuuint64_t)rows, (cuuint64_t)batch};
  cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * rows * 2};
  cuuint32_t box[3] = {64, box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t launch_gemm(const CUtensorMap& a, const CUtensorMap& b, const Params& p, int tiles, int batch,
                        cudaStream_t s) {
  static PerDeviceOnce once;
  const cudaError_t e = smem_optin(once, ns_gemm_kernel<MODE>, kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(ns_gemm_kernel<MODE>, dim3(tiles, batch), dim3(kThreads), kSmem, s, a, b, p);
}

// out[b] = the orthogonalised x[b], bf16 [rows][cols]; matrices x_stride, out_stride
// elements apart. have_parts: the workspace holds the partial sums of squares already.
template <typename T>
int orthogonalize(const T* x, long x_stride, bf16* out, long out_stride, int batch, int rows, int cols, int steps,
                  void* ws, size_t ws_bytes, int* err, cudaStream_t s, bool have_parts = false) {
  Work w;
  if (!plan(batch, rows, cols, &w) || ws_bytes < w.total || (reinterpret_cast<uintptr_t>(ws) & 255))
    return GPT2_ERR_ARG;
  if (steps < 1 || steps > kMaxSteps) return GPT2_ERR_ARG;
  char* base = static_cast<char*>(ws);
  __half* xh[2] = {reinterpret_cast<__half*>(base + w.x0), reinterpret_cast<__half*>(base + w.x1)};
  __half* lo = reinterpret_cast<__half*>(base + w.lo);
  __half* a = reinterpret_cast<__half*>(base + w.a);
  __half* q = reinterpret_cast<__half*>(base + w.q);
  double* part = reinterpret_cast<double*>(base + w.part);

  CUtensorMap mx_rows[2], mx_cols[2], ma, mq;
  for (int i = 0; i < 2; ++i)
    if (!map_3d(&mx_rows[i], xh[i], w.ld_x, w.n, batch, BM) || !map_3d(&mx_cols[i], xh[i], w.ld_x, w.n, batch, 64))
      return GPT2_ERR_CUDA;
  if (!map_3d(&ma, a, w.ld_a, w.n, batch, BM) || !map_3d(&mq, q, w.ld_a, w.n, batch, BM)) return GPT2_ERR_CUDA;

  const int vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (x_stride * sizeof(T)) % 16 == 0;
  cudaError_t e = cudaSuccess;
  if (!have_parts)
    e = launch_pdl(ns_sumsq_kernel<T>, dim3(w.parts, batch), dim3(256), 0, s, x, x_stride, (long)rows * cols, vec, part);
  if (e == cudaSuccess)
    e = launch_pdl(ns_convert_kernel<T>, dim3(w.ld_x / 64, (w.n + 63) / 64, batch), dim3(256), 0, s, x, x_stride, rows,
                   cols, (const double*)part, w.parts, xh[0], lo, w.ld_x);
  const int nt = (w.n + BM - 1) / BM, mt = (w.m + BN - 1) / BN;
  Params p{};
  p.n = w.n; p.m = w.m; p.ld_x = w.ld_x; p.ld_a = w.ld_a;
  p.rows = rows; p.cols = cols; p.err = err;
  for (int i = 0; i < steps && e == cudaSuccess; ++i) {
    const int cur = i & 1;
    p.nkb = w.ld_x / 64;
    p.out = a;
    e = launch_gemm<GRAM>(mx_rows[cur], mx_rows[cur], p, nt * (nt + 1) / 2, batch, s);
    if (e != cudaSuccess) break;
    p.nkb = w.ld_a / 64;
    p.out = q; p.aux = a;
    e = launch_gemm<POLY>(ma, ma, p, nt * (nt + 1) / 2, batch, s);
    if (e != cudaSuccess) break;
    p.aux = xh[cur]; p.lo = lo;
    p.use_lo = i < steps - 2; p.put_lo = i + 1 < steps - 2;
    p.out = xh[cur ^ 1];
    p.result = out; p.result_stride = out_stride;
    e = i + 1 < steps ? launch_gemm<APPLY>(mq, mx_cols[cur], p, nt * mt, batch, s)
                      : launch_gemm<LAST>(mq, mx_cols[cur], p, nt * mt, batch, s);
  }
  return e == cudaSuccess ? GPT2_OK : GPT2_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// the optimizer's elementwise passes
// ---------------------------------------------------------------------------
// Momentum: mom = mu mom + g', u = g' + mu mom with g' = g * gscale; u takes the
// gradient's place and its sum of squares goes to part[matrix][block]. A step
// flagged non-finite leaves mom alone.
__global__ void __launch_bounds__(256) momentum_kernel(float* __restrict__ g, float* __restrict__ mom, long stride,
                                                       long count4, float mu, const float* __restrict__ gscale,
                                                       const int* __restrict__ skip, double* __restrict__ part) {
  pdl_begin();
  __shared__ double red[8];
  const float gs = *gscale;
  const bool off = *skip != 0;
  float4* g4 = reinterpret_cast<float4*>(g + (size_t)blockIdx.y * stride);
  float4* m4 = reinterpret_cast<float4*>(mom + (size_t)blockIdx.y * stride);
  double s = 0.0;
  if (!off)
    for (long i = blockIdx.x * 256L + threadIdx.x; i < count4; i += (long)gridDim.x * 256) {
      float4 gv = g4[i], mv = m4[i];
      float* gp = &gv.x;
      float* mp = &mv.x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float gg = gp[j] * gs;
        mp[j] = mu * mp[j] + gg;
        gp[j] = gg + mu * mp[j];
        s += (double)gp[j] * gp[j];
      }
      m4[i] = mv;
      g4[i] = gv;
    }
  s = warp_sum_d(s);
  if (lane_id() == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) s += red[w];
    part[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = s;
  }
}

// w -= lr (adj o + wd w), the bf16 copy, and g = 0; a flagged step only clears g.
__global__ void __launch_bounds__(256) apply_kernel(float* __restrict__ w, bf16* __restrict__ wb, float* __restrict__ g,
                                                    const bf16* __restrict__ o, long stride, long count4, float lr,
                                                    float adj, float wd, const int* __restrict__ skip) {
  pdl_begin();
  const bool off = *skip != 0;
  const size_t base = (size_t)blockIdx.y * stride;
  float4* g4 = reinterpret_cast<float4*>(g + base);
  float4* w4 = reinterpret_cast<float4*>(w + base);
  uint2* b4 = reinterpret_cast<uint2*>(wb + base);
  const uint2* o4 = reinterpret_cast<const uint2*>(o) + (size_t)blockIdx.y * count4;
  for (long i = blockIdx.x * 256L + threadIdx.x; i < count4; i += (long)gridDim.x * 256) {
    g4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (off) continue;
    const uint2 ov = o4[i];
    float4 wv = w4[i];
    const float2 lo = unpack_bf16x2(ov.x), hi = unpack_bf16x2(ov.y);
    wv.x -= lr * (adj * lo.x + wd * wv.x);
    wv.y -= lr * (adj * lo.y + wd * wv.y);
    wv.z -= lr * (adj * hi.x + wd * wv.z);
    wv.w -= lr * (adj * hi.y + wd * wv.w);
    w4[i] = wv;
    b4[i] = make_uint2(pack_bf16x2(wv.x, wv.y), pack_bf16x2(wv.z, wv.w));
  }
}

constexpr int kUpdateLaunches = 3 + 3 * 5;   // momentum, convert, five rounds of three products, apply

// Muon's update of a batch of fp32 weights (matrices `stride` elements apart,
// rows * cols a multiple of 4): the orthogonalised momentum scaled to the
// root-mean-square of an AdamW step, 0.2 sqrt(max(rows, cols)).
inline size_t update_workspace(int batch, int rows, int cols) {
  Work w;
  if (!plan(batch, rows, cols, &w)) return 0;
  return w.total + (size_t)batch * rows * cols * 2;
}

inline int update(float* w, bf16* wb, float* g, float* mom, long stride, int batch, int rows, int cols, float lr,
                  float mu, float wd, const float* gscale, const int* skip, void* ws, size_t ws_bytes, int* err,
                  cudaStream_t s) {
  Work wk;
  if (!plan(batch, rows, cols, &wk) || ws_bytes < update_workspace(batch, rows, cols)) return GPT2_ERR_ARG;
  const long count = (long)rows * cols;
  if (count % 4 || stride % 4) return GPT2_ERR_ARG;
  char* base = static_cast<char*>(ws);
  bf16* o = reinterpret_cast<bf16*>(base + wk.total);
  if (launch_pdl(momentum_kernel, dim3(wk.parts, batch), dim3(256), 0, s, g, mom, stride, count / 4, mu, gscale, skip,
                 reinterpret_cast<double*>(base + wk.part)) != cudaSuccess)
    return GPT2_ERR_CUDA;
  const int st = orthogonalize<float>(g, stride, o, count, batch, rows, cols, 5, ws, wk.total, err, s, true);
  if (st != GPT2_OK) return st;
  const float adj = 0.2f * sqrtf((float)std::max(rows, cols));
  return launch_pdl(apply_kernel, dim3(wk.parts, batch), dim3(256), 0, s, w, wb, g, (const bf16*)o, stride, count / 4,
                    lr, adj, wd, skip) == cudaSuccess
             ? GPT2_OK
             : GPT2_ERR_CUDA;
}

}  // namespace muon
