// Post-training losses over the head's logits, each with its gradient:
// the clipped policy loss with a KL term and the paired preference loss.
//
// Both reach the logits through one number per row, the log-probability of the
// row's token over the V real ids,
//   lp = z[t] - lse(z[0 .. V-1]),      d lp / d z[j] = [j == t] - p[j],
// so a row's gradient is dz[j] = g ([j == t] - p[j]) with a scalar g that the
// loss decides, exactly 0 for padded ids and for rows left out. Sums run in
// base 2 on y = z log2(e): a row is kept as (c, S) with sum_j 2^y[j] = 2^c S,
// every term one FFMA and one ex2, and lp = (y[t] - c - log2 S) ln 2.
#pragma once
#include "kernels.cuh"

namespace pt {

constexpr int kRowThreads = 256;
constexpr int kUnroll = 4;

// Running (c, S) over the real columns of one 8-wide chunk.
GPT2_DEV void row_accumulate(uint4 u, int col0, int V, float& c, float& s) {
  float f[8];
  k::bf16x8_to_f32(u, f);
  if (col0 + 8 > V) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col0 + j >= V) f[j] = -INFINITY;
  }
  float lm = f[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) lm = fmaxf(lm, f[j]);
  lm *= k::kLog2eF;
  if (lm > c) {
    s *= ex2_approx(c - lm);
    c = lm;
  }
  // nothing but -inf so far: no term to add (a NaN still has to reach the sum)
  const float base = c == -INFINITY ? 0.f : c;
  float acc = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) acc += ex2_approx(fmaf(f[j], k::kLog2eF, -base));
  s += acc;
}

// (c, S) of one logits row over its real columns, the same in every thread of
// the CTA. With `part` (the logits GEMM's row partials, same base-2 form) the
// row itself is not read.
GPT2_DEV void row_stats(const uint4* zr, int V, const float2* part, int slots, float& c, float& s) {
  constexpr int W = kRowThreads / 32;
  __shared__ float2 red[W];
  c = -INFINITY;
  s = 0.f;
  if (part != nullptr) {
    for (int i = threadIdx.x; i < slots; i += kRowThreads) {
      const float2 v = __ldcs(part + i);
      k::ce_combine(c, s, v.x, v.y);
    }
  } else {
    const int nv = (V + 7) / 8;   // chunks that hold real ids
    for (int i0 = threadIdx.x; i0 < nv; i0 += kRowThreads * kUnroll) {
      uint4 u[kUnroll];
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) {
        const int i = i0 + q * kRowThreads;
        u[q] = i < nv ? __ldcg(zr + i) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) {
        const int i = i0 + q * kRowThreads;
        if (i < nv) row_accumulate(u[q], i * 8, V, c, s);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    k::ce_combine(c, s, __shfl_xor_sync(0xffffffffu, c, o), __shfl_xor_sync(0xffffffffu, s, o));
  if (lane_id() == 0) red[threadIdx.x >> 5] = make_float2(c, s);
  __syncthreads();
  c = -INFINITY;
  s = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) k::ce_combine(c, s, red[w].x, red[w].y);
}

GPT2_DEV float row_logp(float zt, float c, float s) {
  return (fmaf(zt, k::kLog2eF, -c) - log2f(s)) * k::kLn2F;
}

// dst[j] = g ([j == t] - 2^(y[j] - c) / S) over a row's real columns, 0 behind
// them; dst may be the row itself.
GPT2_DEV void row_gradient(const uint4* zr, uint4* dst, int t, int V, int Vp, float c, float s, float g) {
  const int nv = Vp / 8;
  const float gs = -g / s;
  for (int i0 = threadIdx.x; i0 < nv; i0 += kRowThreads * kUnroll) {
    uint4 u[kUnroll];
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
      const int i = i0 + q * kRowThreads;
      u[q] = i * 8 < V ? __ldcg(zr + i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
      const int i = i0 + q * kRowThreads;
      if (i >= nv) continue;
      const int c0 = i * 8;
      float f[8];
      k::bf16x8_to_f32(u[q], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = ex2_approx(fmaf(f[j], k::kLog2eF, -c)) * gs;
      if (c0 + 8 > V) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c0 + j >= V) f[j] = 0.f;
      }
      if ((unsigned)(t - c0) < 8u) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += c0 + j == t ? g : 0.f;
      }
      __stcs(dst + i, make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                 pack_bf16x2(f[6], f[7])));
    }
  }
}

GPT2_DEV void row_zero(uint4* dst, int Vp) {
  for (int i = threadIdx.x; i < Vp / 8; i += kRowThreads) __stcs(dst + i, make_uint4(0u, 0u, 0u, 0u));
}

struct PolicyArgs {
  const bf16* logits;
  const int32_t* targets;
  const float *old_logp, *ref_logp, *adv, *weight;   // ref_logp, weight may be null
  bf16* dlogits;                                     // may be null (loss only) or the logits
  float *logps, *losses;                             // logps may be null
  const float2* part;                                // row partials of the logits GEMM, or null
  int slots, V, Vp, ignore_index;
  float clip_low, clip_high, kl_coef, dscale;
  int* err;
};

// One CTA per row: pass 1 for (c, S), the row's loss and g, pass 2 for the gradient.
__global__ void __launch_bounds__(kRowThreads) policy_loss_kernel(const PolicyArgs a) {
  pdl_begin();
  const int row = blockIdx.x;
  const size_t off = (size_t)row * a.Vp;
  const uint4* zr = reinterpret_cast<const uint4*>(a.logits + off);
  uint4* dr = a.dlogits ? reinterpret_cast<uint4*>(a.dlogits + off) : nullptr;
  const int t = a.targets[row];
  const bool in_range = t >= 0 && t < a.V;
  if (t == a.ignore_index || !in_range) {
    if (threadIdx.x == 0) {
      if (t != a.ignore_index) atomicOr(a.err, DEVERR_TOKEN_RANGE);
      a.losses[row] = 0.f;
      if (a.logps) a.logps[row] = 0.f;
    }
    if (dr) row_zero(dr, a.Vp);
    return;
  }
  const float old_lp = a.old_logp[row], adv = a.adv[row];
  const float ref = a.ref_logp ? a.ref_logp[row] : 0.f;
  const float w = a.weight ? a.weight[row] : 1.f;
  const float zt = __bfloat162float(a.logits[off + t]);   // before any thread may overwrite it
  float c, s;
  row_stats(zr, a.V, a.part ? a.part + (size_t)row * a.slots : nullptr, a.slots, c, s);
  const float lp = row_logp(zt, c, s);
  const float r = expf(lp - old_lp);
  // r A and its clipped form; an advantage of 0 gives 0 for any ratio
  const float free_s = adv == 0.f ? 0.f : r * adv;
  const float cut_s = fminf(fmaxf(r, 1.f - a.clip_low), 1.f + a.clip_high) * adv;
  const bool active = free_s <= cut_s;
  float loss = active ? -free_s : -cut_s;
  float g = active ? -free_s : 0.f;
  if (a.ref_logp) {
    // e^d - d - 1 without the cancellation of small d
    const float d = ref - lp, em = expm1f(d);
    loss += a.kl_coef * (em - d);
    g -= a.kl_coef * em;
  }
  g *= w * a.dscale;
  if (threadIdx.x == 0) {
    a.losses[row] = w * loss;
    if (a.logps) a.logps[row] = lp;
  }
  if (!dr) return;
  if (g == 0.f && isfinite(lp)) row_zero(dr, a.Vp);
  else row_gradient(zr, dr, t, a.V, a.Vp, c, s, g);
}

struct RowArgs {
  const bf16* logits;
  const int32_t* targets;
  float* logps;
  float2* stats;            // (c, S) per row, or null
  const float2* part;
  const float* tgt_val;     // the target's logit per row where the logits are not stored, or null
  const int32_t* seq_start; // only rows seq_start[0] .. seq_start[n_seq] - 1, or null: all rows
  int n_seq, slots, V, Vp, ignore_index;
  int* err;
};

// One CTA per row: lp (0 for a row left out) and the row's (c, S).
__global__ void __launch_bounds__(kRowThreads) row_logp_kernel(const RowArgs a) {
  pdl_begin();
  const int row = blockIdx.x;
  if (a.seq_start && (row < a.seq_start[0] || row >= a.seq_start[a.n_seq])) return;
  const size_t off = (size_t)row * a.Vp;
  const int t = a.targets[row];
  const bool in_range = t >= 0 && t < a.V;
  if (t == a.ignore_index || !in_range) {
    if (threadIdx.x == 0) {
      if (t != a.ignore_index) atomicOr(a.err, DEVERR_TOKEN_RANGE);
      a.logps[row] = 0.f;
    }
    return;
  }
  const float zt = a.tgt_val ? a.tgt_val[row] : __bfloat162float(a.logits[off + t]);
  float c, s;
  row_stats(a.logits ? reinterpret_cast<const uint4*>(a.logits + off) : nullptr, a.V,
            a.part ? a.part + (size_t)row * a.slots : nullptr, a.slots, c, s);
  if (threadIdx.x == 0) {
    a.logps[row] = row_logp(zt, c, s);
    if (a.stats) a.stats[row] = make_float2(c, s);
  }
}

struct PairArgs {
  const float* logps;
  const int32_t* targets;
  const int32_t* seq_start;   // [2 P + 1] row offsets, or null: sequences of seq_len rows
  const float* ref_logp;      // [2 P] or null
  float* seq_logps;           // [2 P] or null
  float* losses;              // [P]
  float* coef;                // [2 P]: g of the sequence's kept rows
  int N, seq_len, V, ignore_index, kind, average;
  float beta, smoothing, dscale;
  int* err;
};

GPT2_DEV double softplus_d(double x) { return fmax(x, 0.0) + log1p(exp(-fabs(x))); }

// One CTA per pair. Sequence 2p is the chosen one, 2p + 1 the rejected one. The
// sums over a sequence and the difference of the two run in 64 bits: a margin
// of a few units is left of sums of thousands.
__global__ void __launch_bounds__(kRowThreads) pair_kernel(const PairArgs a) {
  pdl_begin();
  constexpr int W = kRowThreads / 32;
  __shared__ double red[2][W];
  __shared__ int cnt[2][W];
  const int p = blockIdx.x;
  bool bad = false;
  for (int h = 0; h < 2; ++h) {
    int b, e;
    if (a.seq_start) {
      b = a.seq_start[2 * p + h];
      e = a.seq_start[2 * p + h + 1];
    } else {
      b = (2 * p + h) * a.seq_len;
      e = b + a.seq_len;
    }
    if (b < 0 || e < b || e > a.N) {
      bad = true;
      b = e = 0;
    }
    double s = 0.0;
    int n = 0;
    for (int i = b + threadIdx.x; i < e; i += kRowThreads) {
      const int t = a.targets[i];
      if (t != a.ignore_index && t >= 0 && t < a.V) {
        s += (double)a.logps[i];
        ++n;
      }
    }
    s = warp_sum_d(s);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane_id() == 0) {
      red[h][threadIdx.x >> 5] = s;
      cnt[h][threadIdx.x >> 5] = n;
    }
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  double gap[2], share[2];
  for (int h = 0; h < 2; ++h) {
    double s = 0.0;
    int n = 0;
    for (int w = 0; w < W; ++w) {
      s += red[h][w];
      n += cnt[h][w];
    }
    share[h] = a.average ? 1.0 / (n > 0 ? n : 1) : 1.0;
    s *= share[h];
    if (a.seq_logps) a.seq_logps[2 * p + h] = (float)s;
    gap[h] = s - (a.ref_logp ? (double)a.ref_logp[2 * p + h] : 0.0);
  }
  const double delta = gap[0] - gap[1], b = a.beta, eps = a.smoothing;
  double loss, dd;
  if (a.kind == 0) {
    loss = (1.0 - eps) * softplus_d(-b * delta) + eps * softplus_d(b * delta);
    dd = -b * ((1.0 - eps) / (1.0 + exp(b * delta)) - eps / (1.0 + exp(-b * delta)));
  } else {
    const double off = delta - 0.5 / b;
    loss = off * off;
    dd = 2.0 * off;
  }
  if (bad) {   // bounds that are not bounds: no loss, no gradient, flagged
    atomicOr(a.err, DEVERR_TOKEN_RANGE);
    loss = dd = 0.0;
  }
  a.losses[p] = (float)loss;
  a.coef[2 * p] = (float)(dd * share[0] * a.dscale);
  a.coef[2 * p + 1] = (float)(-dd * share[1] * a.dscale);
}

struct PairGradArgs {
  const bf16* logits;
  const int32_t* targets;
  const int32_t* seq_start;
  const float2* stats;
  const float* coef;
  bf16* dlogits;
  int n_seq, seq_len, V, Vp, ignore_index;
};

// The sequence that holds `row`, or -1: the last one that begins at or before it.
GPT2_DEV int find_sequence(const int32_t* start, int n_seq, int row) {
  int lo = 0, hi = n_seq;   // start[lo] <= row is looked for in [0, n_seq)
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= row) lo = mid + 1;
    else hi = mid;
  }
  return (lo > 0 && row < start[lo]) ? lo - 1 : -1;
}

// One CTA per row: its gradient, from the pair's coefficient and the row's (c, S).
__global__ void __launch_bounds__(kRowThreads) pair_grad_kernel(const PairGradArgs a) {
  pdl_begin();
  const int row = blockIdx.x;
  const int seq = a.seq_start ? find_sequence(a.seq_start, a.n_seq, row) : row / a.seq_len;
  if (seq < 0 || seq >= a.n_seq) return;   // behind the last sequence: left as it was
  const size_t off = (size_t)row * a.Vp;
  uint4* dr = reinterpret_cast<uint4*>(a.dlogits + off);
  const int t = a.targets[row];
  if (t == a.ignore_index || t < 0 || t >= a.V) {
    row_zero(dr, a.Vp);
    return;
  }
  const float2 st = a.stats[row];
  row_gradient(reinterpret_cast<const uint4*>(a.logits + off), dr, t, a.V, a.Vp, st.x, st.y, a.coef[seq]);
}

// acc += factor * rows * sum(losses), *mean_out = factor * sum(losses) (fp64 sums).
__global__ void scaled_loss_kernel(const float* __restrict__ losses, int n, double factor, double rows,
                                   double* __restrict__ acc, float* __restrict__ mean_out) {
  pdl_begin();
  __shared__ double red[32];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) s += (double)losses[i];
  s = warp_sum_d(s);
  if (lane_id() == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = threadIdx.x < (blockDim.x >> 5) ? red[threadIdx.x] : 0.0;
    s = warp_sum_d(s);
    if (threadIdx.x == 0) {
      acc[0] += s * factor * rows;
      *mean_out = (float)(s * factor);
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline bool logits_ok(const void* logits, int N, int V, int Vp) {
  return N > 0 && V > 0 && V <= Vp && Vp % 8 == 0 && aligned16(logits);
}

inline int policy_loss(const PolicyArgs& a, int N, cudaStream_t s) {
  launch_pdl(policy_loss_kernel, dim3(N), dim3(kRowThreads), 0, s, a);
  return cudaGetLastError() == cudaSuccess ? GPT2_OK : GPT2_ERR_CUDA;
}

inline int row_logps(const RowArgs& a, int N, cudaStream_t s) {
  launch_pdl(row_logp_kernel, dim3(N), dim3(kRowThreads), 0, s, a);
  return cudaGetLastError() == cudaSuccess ? GPT2_OK : GPT2_ERR_CUDA;
}

// Workspace: a row's (c, S), then a sequence's coefficient.
inline size_t preference_workspace(int N, int P) { return (size_t)N * 8 + (size_t)P * 8; }

}  // namespace pt
