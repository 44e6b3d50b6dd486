// Newton-Schulz for matrices whose smaller dimension is at most 128, in one
// launch: a matrix stays on chip from its first read to the result.
//
// A cluster of nc CTAs takes one matrix X [n <= 128 rows, m columns]; each holds
// w = 64 ceil(m / (64 nc)) <= 256 columns (384 where it is alone) in shared memory as
// hi and lo fp16. The columns stand in blocks of 64: a block is 128 rows of 128 bytes in
// the 128-byte swizzle, which is the K-major tile of X that X X^T wants and, read the
// other way, the MN-major tile that P X wants. A round is three products with their
// accumulators in tensor memory (128 x 128 twice, 128 x w) and three passes of registers
// between tensor and shared memory. Only X X^T needs the other CTAs: each sends its partial
// sum's columns to the CTA that adds them up (fp32, in the order of the ranks), which sends
// the sum to all as fp16. Every CTA forms A A and P for itself.
//
// What bounds it is latency: 15 dependent steps. On the device a CTA alone takes 3.1 us a
// round at 128 columns, 4.4 at 256, 5.7 at 384; a cluster of eight at 2,048 columns 10 us.
// 1 x 128 x 128: 22 us (as separate launches, two passes over M and three products a round,
// 104 us); 1 x 128 x 2,048: 60 us; 16 of them 122 us. A result stored one bf16 a thread, its
// own row each, took 20 us more than rows out of shared memory.
#pragma once
#include "gemm2sm.cuh"
#include "muon.cuh"

namespace muon {
namespace small {

constexpr int kThreads = 512;              // four warps a tensor-memory lane quarter: 32 columns each of 128
constexpr int kBlock = 128 * 128;          // bytes of 64 columns
constexpr int kMaxW = 256, kMaxCtas = 8;   // columns a CTA of a cluster
constexpr int kMaxW1 = 384;                // and of a CTA alone, which keeps no partial sums
constexpr int kStage = 128 * 128 * 4;      // the partial sums sent to this CTA
constexpr int kMinSmem = 120 * 1024;       // one CTA an SM: tensor memory is taken whole

inline int smem_bytes(int w, int nc) {
  const int need = 2 * (w / 64) * kBlock + 2 * kBlock + (nc > 1 ? kStage : 0) + 1024 + 256;
  return need > kMinSmem ? need : kMinSmem;
}

struct Args {
  long x_stride, out_stride;
  int rows, cols, n, m, w, steps, vec, vec_out;
  int* err;
};

// Byte offset of row r's 16-byte chunk j (0 .. 7) in a block.
GPT2_DEV uint32_t at_chunk(int r, int j) { return (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4)); }

GPT2_DEV void unpack8(uint4 u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
GPT2_DEV uint4 pack8(const float* f) {
  return make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
}
GPT2_DEV void fence_proxy_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
GPT2_DEV void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
GPT2_DEV void st_cluster_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
GPT2_DEV void st_cluster_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) ns_small_kernel(const T* __restrict__ x, bf16* __restrict__ out,
                                                               const Args a) {
  extern __shared__ __align__(1024) uint8_t small_smem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(small_smem) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bar;
  __shared__ uint32_t tmem_slot;
  __shared__ double red[kThreads / 32], sums[kMaxCtas];
  uint32_t nc, rank;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(nc));
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int wb = a.w / 64;                         // blocks of this CTA's columns
  uint8_t* s_hi = smem;
  uint8_t* s_lo = s_hi + wb * kBlock;
  uint8_t* s_p = s_lo + wb * kBlock;               // A, then P
  float* s_stage = reinterpret_cast<float*>(s_p + 2 * kBlock);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (nc > 1) gemm2::cluster_sync();               // the others' shared memory exists
  pdl_begin();

  // ---- X: read once, raw fp32 into the room of its hi and lo; the norm; hi and lo ----
  const bool tall = a.rows > a.cols;
  const T* src = x + (size_t)(blockIdx.x / nc) * a.x_stride;
  const int c0 = rank * a.w;
  const int wc = max(0, min(a.w, a.m - c0));       // this CTA's real columns
  const int units = wb * 8 * 128;                  // chunks of 8 columns of a row
  // neighbouring threads along M's stored rows
  auto unit_at = [&](int i, int& r, int& ch) {
    r = tall ? i & 127 : i / (wb * 8);
    ch = tall ? i >> 7 : i - r * (wb * 8);
  };
  double ss = 0.0;
#pragma unroll 4
  for (int i = threadIdx.x; i < units; i += kThreads) {
    int r, ch;
    unit_at(i, r, ch);
    float f[8];
    if (a.vec) {
      // whole 16-byte pieces of a stored row of X
      constexpr int E = 16 / sizeof(T);
      const T* p = src + (size_t)r * a.cols + c0 + ch * 8;
#pragma unroll
      for (int q = 0; q < 8; q += E) {
        const bool ok = r < a.n && ch * 8 + q < wc;
        const uint4 u = ok ? __ldg(reinterpret_cast<const uint4*>(p + q)) : make_uint4(0u, 0u, 0u, 0u);
        const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int j = 0; j < E; ++j) f[q + j] = load1(e + j);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int c = ch * 8 + q;
        f[q] = r < a.n && c < wc ? load1(src + (tall ? (size_t)(c0 + c) * a.cols + r : (size_t)r * a.cols + c0 + c)) : 0.f;
      }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) ss += (double)f[q] * f[q];
    const uint32_t o = (ch >> 3) * kBlock + at_chunk(r, ch & 7);
    *reinterpret_cast<float4*>(s_hi + o) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(s_lo + o) = make_float4(f[4], f[5], f[6], f[7]);
  }
  ss = warp_sum_d(ss);
  if (lane == 0) red[warp] = ss;
  __syncthreads();
  if (threadIdx.x < nc) {
    double s = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) s += red[w];
    st_cluster_f64(gemm2::mapa_shared(smem_u32(&sums[rank]), threadIdx.x), s);
  }
  if (nc > 1) gemm2::cluster_sync();
  else __syncthreads();
  double total = 0.0;
  for (uint32_t i = 0; i < nc; ++i) total += sums[i];
  const float mul = (float)((double)kScale / (sqrt(total) + 1e-7));
#pragma unroll 2
  for (int i = threadIdx.x; i < units; i += kThreads) {   // the thread's own units again
    int r, ch;
    unit_at(i, r, ch);
    const uint32_t o = (ch >> 3) * kBlock + at_chunk(r, ch & 7);
    const float4 lo4 = *reinterpret_cast<const float4*>(s_hi + o), hi4 = *reinterpret_cast<const float4*>(s_lo + o);
    const float f[8] = {lo4.x * mul, lo4.y * mul, lo4.z * mul, lo4.w * mul,
                        hi4.x * mul, hi4.y * mul, hi4.z * mul, hi4.w * mul};
    uint4 hi, lo;
    split8(f, hi, lo);
    *reinterpret_cast<uint4*>(s_hi + o) = hi;
    *reinterpret_cast<uint4*>(s_lo + o) = lo;
  }

  // ---- the rounds ------------------------------------------------------------------
  // A A leaves its columns before P X takes them
  const uint32_t d_gram = tmem, d_poly = tmem + 128, d_x = tmem + 128;
  const int q4 = warp & 3, group = warp >> 2;
  const int row = q4 * 32 + lane;
  const uint32_t t_row = (uint32_t)(q4 * 32) << 16;
  const uint32_t hi32 = smem_u32(s_hi), p32 = smem_u32(s_p);
  uint32_t phase = 0;
  // one thread issues a product once everything it reads is in shared memory
  auto product = [&](auto&& issue) {
    fence_proxy_all();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
      tc_fence_after();
      issue();
      tc_commit(smem_u32(&bar));
    }
    mbar_wait(smem_u32(&bar), phase, a.err);   // gave up: flagged, and the rounds run out without it
    phase ^= 1;
    tc_fence_after();
  };
  for (int it = 0; it < a.steps; ++it) {
    const bool use_lo = it < a.steps - 2, put_lo = it + 1 < a.steps - 2, last = it + 1 == a.steps;
    // A = X X^T
    product([&] {
      constexpr uint32_t idesc = idesc_f16_f32(128, 128, false);
      for (int kb = 0; kb < wb; ++kb)
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t d = smem_desc_sw128(hi32 + kb * kBlock + kk * 32, 16, 1024);
          tc_mma_bf16(d_gram, d, d, idesc, (kb | kk) ? 1u : 0u);
        }
    });
    if (nc == 1) {
      {
        const int c = group * 32;
        float v[32];
        tmem_ld32(d_gram + t_row + c, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= kInvScale;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(s_p + (c >> 6) * kBlock + at_chunk(row, ((c & 63) >> 3) + j)) = pack8(v + 8 * j);
      }
    } else {
      // columns [k span, ..) of the partial sum go to rank k: stage[source][4 columns][row]
      const int span = 128 / nc;
      {
        const int c = group * 32;
        float v[32];
        tmem_ld32(d_gram + t_row + c, v);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const int to = (c + i) / span, in = (c + i) - to * span;
          st_cluster_v4(gemm2::mapa_shared(smem_u32(s_stage + (((int)rank * span + in) / 4 * 128 + row) * 4), to),
                        make_uint4(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                                   __float_as_uint(v[i + 3])));
        }
      }
      gemm2::cluster_sync();
      for (int u = threadIdx.x; u < 128 * (span / 8); u += kThreads) {
        const int r = u & 127, ch = u >> 7;
        float f[8] = {};
#pragma unroll 4
        for (uint32_t k = 0; k < nc; ++k) {
          const float4* p = reinterpret_cast<const float4*>(s_stage) + ((int)k * span / 4 + ch * 2) * 128 + r;
          const float4 x0 = p[0], x1 = p[128];
          f[0] += x0.x; f[1] += x0.y; f[2] += x0.z; f[3] += x0.w;
          f[4] += x1.x; f[5] += x1.y; f[6] += x1.z; f[7] += x1.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= kInvScale;
        const uint4 h = pack8(f);
        const int col = rank * span + ch * 8;
        const uint32_t o = p32 + (col >> 6) * kBlock + at_chunk(r, (col & 63) >> 3);
        for (uint32_t k = 0; k < nc; ++k) st_cluster_v4(gemm2::mapa_shared(o, k), h);
      }
      fence_proxy_all();
      gemm2::cluster_sync();
    }
    // P = a I + b A + c A A, in A's place
    product([&] {
      constexpr uint32_t idesc = idesc_f16_f32(128, 128, false);
      for (int kb = 0; kb < 2; ++kb)
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t d = smem_desc_sw128(p32 + kb * kBlock + kk * 32, 16, 1024);
          tc_mma_bf16(d_poly, d, d, idesc, (kb | kk) ? 1u : 0u);
        }
    });
    {
      const int c = group * 32;
      float v[32];
      tmem_ld32(d_poly + t_row + c, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4* p = reinterpret_cast<uint4*>(s_p + (c >> 6) * kBlock + at_chunk(row, ((c & 63) >> 3) + j));
        float f[8];
        unpack8(*p, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[i] = fmaf(kB, f[i], kC * kInvScale * v[8 * j + i]);
          if (c + 8 * j + i == row && row < a.n) f[i] += kA * kScale;
        }
        *p = pack8(f);
      }
    }
    // X <- P X (+ a lo)
    product([&] {
      for (int c = 0; c < a.w; c += 256) {         // at most 256 columns an instruction
        const uint32_t idesc = idesc_f16_f32(128, min(256, a.w - c), true);
        for (int kb = 0; kb < 2; ++kb)
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_bf16(d_x + c, smem_desc_sw128(p32 + kb * kBlock + kk * 32, 16, 1024),
                        smem_desc_sw128(hi32 + (c >> 6) * kBlock + (kb * 64 + kk * 16) * 128, kBlock, 1024), idesc,
                        (kb | kk) ? 1u : 0u);
      }
    });
#pragma unroll 1
    for (int c = group * 32; c < a.w; c += 128) {
      float v[32];
      tmem_ld32(d_x + t_row + c, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t o = (c >> 6) * kBlock + at_chunk(row, ((c & 63) >> 3) + j);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * j + i] *= kInvScale;
        if (use_lo) {
          float f[8];
          unpack8(*reinterpret_cast<const uint4*>(s_lo + o), f);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[8 * j + i] = fmaf(kA, f[i], v[8 * j + i]);
        }
        if (!last) {
          uint4 hi, lo;
          split8(v + 8 * j, hi, lo);
          *reinterpret_cast<uint4*>(s_hi + o) = hi;
          if (put_lo) *reinterpret_cast<uint4*>(s_lo + o) = lo;
        }
      }
      if (last) {
        bf16* res = out + (size_t)(blockIdx.x / nc) * a.out_stride;
        if (tall) {      // a warp's lanes lie along the stored rows
          if (row < a.n)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c + i < wc) res[(size_t)(c0 + c + i) * a.cols + row] = __float2bfloat16_rn(v[i] * kInvScale);
        } else {         // into the chunk's own slot, to leave by whole rows
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_bf16x2(v[8 * j + 2 * i] * kInvScale, v[8 * j + 2 * i + 1] * kInvScale);
            *reinterpret_cast<uint4*>(s_hi + (c >> 6) * kBlock + at_chunk(row, ((c & 63) >> 3) + j)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  }
  if (!tall) {
    // stored one element a thread they took 20 us of a 128 x 128 matrix's 39 us
    bf16* res = out + (size_t)(blockIdx.x / nc) * a.out_stride + c0;
    __syncthreads();
    if (a.vec_out) {
      for (int i = threadIdx.x; i < units; i += kThreads) {
        int r, ch;
        unit_at(i, r, ch);
        if (r < a.n && ch * 8 < wc)
          *reinterpret_cast<uint4*>(res + (size_t)r * a.cols + ch * 8) =
              *reinterpret_cast<const uint4*>(s_hi + (ch >> 3) * kBlock + at_chunk(r, ch & 7));
      }
    } else {
      for (int i = threadIdx.x; i < a.n * wc; i += kThreads) {
        const int r = i / wc, c = i - r * wc;
        res[(size_t)r * a.cols + c] =
            *reinterpret_cast<const bf16*>(s_hi + (c >> 6) * kBlock + at_chunk(r, (c & 63) >> 3) + (c & 7) * 2);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (nc > 1) gemm2::cluster_sync();   // nobody leaves while its shared memory is written to
}

// CTAs a matrix, as few as hold it: joining the partial sums costs a round more than
// the columns that another CTA would take off this one.
inline int ctas(int m) {
  if (m <= kMaxW1) return 1;
  int nc = 2;
  while (nc < kMaxCtas && m > kMaxW * nc) nc *= 2;
  return nc;
}
inline bool fits(int n, int m) { return n <= 128 && m <= kMaxCtas * kMaxW; }

template <typename T>
int run(const T* x, long x_stride, bf16* out, long out_stride, int batch, int rows, int cols, int steps, int* err,
        cudaStream_t s) {
  Args a{};
  a.x_stride = x_stride; a.out_stride = out_stride; a.rows = rows; a.cols = cols;
  a.n = std::min(rows, cols); a.m = std::max(rows, cols); a.steps = steps; a.err = err;
  a.vec = rows <= cols && (reinterpret_cast<uintptr_t>(x) & 15) == 0 && ((long)cols * sizeof(T)) % 16 == 0 &&
          (batch == 1 || (x_stride * sizeof(T)) % 16 == 0);
  a.vec_out = (reinterpret_cast<uintptr_t>(out) & 15) == 0 && cols % 8 == 0 && (batch == 1 || out_stride % 8 == 0);
  const int nc = ctas(a.m);
  a.w = (a.m + 64 * nc - 1) / (64 * nc) * 64;
  static PerDeviceOnce once;
  if (smem_optin(once, ns_small_kernel<T>, std::max(smem_bytes(kMaxW, 2), smem_bytes(kMaxW1, 1))) != cudaSuccess) return GPT2_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(batch * nc));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(a.w, nc);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = nc;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ns_small_kernel<T>, x, out, (const Args)a) == cudaSuccess ? GPT2_OK : GPT2_ERR_CUDA;
}

}  // namespace small
}  // namespace muon
