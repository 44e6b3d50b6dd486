// Orthogonalisation as a call, and Muon's update of fp32 weights with it.
#pragma once
#include "muon.cuh"
#include "muon_pair.cuh"
#include "muon_small.cuh"

namespace muon {

// out[b] = the orthogonalised x[b], bf16 [rows][cols]; matrices x_stride, out_stride
// elements apart. have_parts: the workspace holds the partial sums of squares.
// *launches (may be null) grows by the kernels launched.
template <typename T>
int orthogonalize(const T* x, long x_stride, bf16* out, long out_stride, int batch, int rows, int cols, int steps,
                  void* ws, size_t ws_bytes, int* err, cudaStream_t s, bool have_parts = false,
                  int* launches = nullptr) {
  Work w;
  if (!plan(batch, rows, cols, &w) || ws_bytes < w.total || (reinterpret_cast<uintptr_t>(ws) & 255))
    return GPT2_ERR_ARG;
  if (steps < 1 || steps > kMaxSteps) return GPT2_ERR_ARG;
  const bool on_chip = small::fits(w.n, w.m);
  if (launches) *launches += on_chip ? 1 : have_parts ? 2 : 3;
  if (on_chip)
    return small::run(x, x_stride, out, out_stride, batch, rows, cols, steps, err, s);
  char* base = static_cast<char*>(ws);
  if (prepare_x(w, base, x, x_stride, batch, rows, cols, have_parts, s) != cudaSuccess) return GPT2_ERR_CUDA;
  return pair::rounds(w, base, out, out_stride, batch, rows, cols, steps, err, s);
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
                  cudaStream_t s, int* launches) {
  Work wk;
  if (!plan(batch, rows, cols, &wk) || ws_bytes < update_workspace(batch, rows, cols)) return GPT2_ERR_ARG;
  const long count = (long)rows * cols;
  if (count % 4 || stride % 4) return GPT2_ERR_ARG;
  char* base = static_cast<char*>(ws);
  bf16* o = reinterpret_cast<bf16*>(base + wk.total);
  if (launch_pdl(momentum_kernel, dim3(wk.parts, batch), dim3(256), 0, s, g, mom, stride, count / 4, mu, gscale, skip,
                 reinterpret_cast<double*>(base + wk.part)) != cudaSuccess)
    return GPT2_ERR_CUDA;
  const int st = orthogonalize<float>(g, stride, o, count, batch, rows, cols, 5, ws, wk.total, err, s, true, launches);
  *launches += 2;
  if (st != GPT2_OK) return st;
  const float adj = 0.2f * sqrtf((float)std::max(rows, cols));
  return launch_pdl(apply_kernel, dim3(wk.parts, batch), dim3(256), 0, s, w, wb, g, (const bf16*)o, stride, count / 4,
                    lr, adj, wd, skip) == cudaSuccess
             ? GPT2_OK
             : GPT2_ERR_CUDA;
}

}  // namespace muon
