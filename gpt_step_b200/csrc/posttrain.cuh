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
#include <type_traits>

#include "kernels.cuh"

namespace pt {

constexpr int kPairThreads = 256;
constexpr uint32_t kNegInf2 = 0xFF80FF80u;   // two bf16 -inf

// (c, S) of a row split over `G` warps, from each lane's own pair.
template <int G>
GPT2_DEV void combine_stats(float& c, float& s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    k::ce_combine(c, s, __shfl_xor_sync(0xffffffffu, c, o), __shfl_xor_sync(0xffffffffu, s, o));
  if (G > 1) {
    __shared__ float2 red[G];
    if (lane_id() == 0) red[threadIdx.x >> 5] = make_float2(c, s);
    __syncthreads();
    const float2 v = lane_id() < G ? red[lane_id()] : make_float2(-INFINITY, 0.f);
    c = v.x;
    s = v.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      k::ce_combine(c, s, __shfl_xor_sync(0xffffffffu, c, o), __shfl_xor_sync(0xffffffffu, s, o));
  }
}

// Columns of the 8-wide chunk at `col0` that are no real ids become -inf.
GPT2_DEV void mask_chunk(uint4& u, int col0, int V) {
  if (col0 + 8 <= V) return;
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (col0 + 2 * j >= V) w[j] = kNegInf2;
    else if (col0 + 2 * j + 1 >= V) w[j] = (w[j] & 0xFFFFu) | (kNegInf2 & 0xFFFF0000u);
  }
  u = make_uint4(w[0], w[1], w[2], w[3]);
}

GPT2_DEV __nv_bfloat162 as_bf2(uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); }

// max over a chunk; NaN only where every value is
GPT2_DEV __nv_bfloat162 chunk_max(uint4 u) {
  return __hmax2(__hmax2(as_bf2(u.x), as_bf2(u.y)), __hmax2(as_bf2(u.z), as_bf2(u.w)));
}
GPT2_DEV float2 bf2_to_f2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// 2^(y - c) of a chunk's values, paired fp32 arithmetic.
GPT2_DEV void chunk_exp(uint4 u, float c, float2 (&e)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  const float2 l2 = make_float2(k::kLog2eF, k::kLog2eF), nc = make_float2(-c, -c);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 y = f2_fma(bf2_to_f2(w[j]), l2, nc);
    e[j] = make_float2(ex2_approx(y.x), ex2_approx(y.y));
  }
}

// A row held by the 32 G lanes of its warps, R chunks a lane (chunk i on lane i
// mod 32 G): read once, its softmax and gradient from registers.
template <int G, int R>
struct HeldRow {
  uint4 u[R];
  int at;                                        // this lane's first chunk
  GPT2_DEV HeldRow() : at(G == 1 ? (int)lane_id() : (int)threadIdx.x) {}

  GPT2_DEV void load(const uint4* zr, int V) {
    const int nv = (V + 7) / 8;
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int i = at + q * 32 * G;
      u[q] = i < nv ? __ldcs(zr + i) : make_uint4(kNegInf2, kNegInf2, kNegInf2, kNegInf2);
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int i = at + q * 32 * G;
      if (i == nv - 1) mask_chunk(u[q], i * 8, V);
    }
  }

  // max first, then one sum: no rescaling
  GPT2_DEV void stats(float& c, float& s) const {
    __nv_bfloat162 m2 = chunk_max(u[0]);
#pragma unroll
    for (int q = 1; q < R; ++q) m2 = __hmax2(m2, chunk_max(u[q]));
    const float2 mf = __bfloat1622float2(m2);
    // the lanes of a warp share one c, so that their sums add up
    c = warp_max(fmaxf(mf.x, mf.y)) * k::kLog2eF;
    const float base = c == -INFINITY ? 0.f : c;
    float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float2 e[4];
      chunk_exp(u[q], base, e);
      acc0 = f2_add(acc0, f2_add(e[0], e[1]));
      acc1 = f2_add(acc1, f2_add(e[2], e[3]));
    }
    s = warp_sum((acc0.x + acc0.y) + (acc1.x + acc1.y));
    if (G > 1) combine_warps<G>(c, s);
  }

  // dst = g ([j == t] - 2^(y - c) / S), 0 behind the real columns
  GPT2_DEV void gradient(uint4* dst, int t, int V, int Vp, float c, float s, float g) {
    const float gs = -g / s;
    const float2 gs2 = make_float2(gs, gs);
    const int nv = Vp / 8;
    // what is held over the reduction is the packed row, not its unpacked values
    // (kept in fp32 by the compiler they took 248 registers a thread at R = 18)
#pragma unroll
    for (int q = 0; q < R; ++q)
      asm volatile("" : "+r"(u[q].x), "+r"(u[q].y), "+r"(u[q].z), "+r"(u[q].w));
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int i = at + q * 32 * G;
      if (i >= nv) break;
      store_chunk(dst + i, u[q], i * 8, t, V, c, gs2, g);
    }
  }

  template <int GG>
  static GPT2_DEV void combine_warps(float& c, float& s) {
    __shared__ float2 red[GG];
    if (lane_id() == 0) red[threadIdx.x >> 5] = make_float2(c, s);
    __syncthreads();
    c = red[0].x;
    s = red[0].y;
#pragma unroll
    for (int w = 1; w < GG; ++w) k::ce_combine(c, s, red[w].x, red[w].y);
  }

  static GPT2_DEV void store_chunk(uint4* dst, uint4 z, int col0, int t, int V, float c, float2 gs2, float g) {
    if (col0 >= V) {
      __stcs(dst, make_uint4(0u, 0u, 0u, 0u));
      return;
    }
    float2 e[4];
    chunk_exp(z, c, e);
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = f2_mul(e[j], gs2);
    if (col0 + 8 > V || (unsigned)(t - col0) < 8u) {
      // the target's chunk, and the last one, whose padded columns get exactly 0
      float* f = &e[0].x;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = col0 + j >= V ? 0.f : f[j] + (col0 + j == t ? g : 0.f);
    }
    __stcs(dst, make_uint4(pack_bf16x2(e[0].x, e[0].y), pack_bf16x2(e[1].x, e[1].y), pack_bf16x2(e[2].x, e[2].y),
                           pack_bf16x2(e[3].x, e[3].y)));
  }
};

// A row too long for registers: streamed twice by the CTA's G warps, the second
// time out of L2.
template <int G>
struct StreamedRow {
  static constexpr int kThreads = 32 * G, kUnroll = 4;
  const uint4* zr;

  GPT2_DEV void load(const uint4* p, int) { zr = p; }

  GPT2_DEV void stats_of(int V, float& c, float& s) const {
    c = -INFINITY;
    s = 0.f;
    const int nv = (V + 7) / 8;
    for (int i0 = threadIdx.x; i0 < nv; i0 += kThreads * kUnroll) {
      uint4 u[kUnroll];
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) {
        const int i = i0 + q * kThreads;
        u[q] = i < nv ? __ldcg(zr + i) : make_uint4(kNegInf2, kNegInf2, kNegInf2, kNegInf2);
        if (i == nv - 1) mask_chunk(u[q], i * 8, V);
      }
      __nv_bfloat162 m2 = chunk_max(u[0]);
#pragma unroll
      for (int q = 1; q < kUnroll; ++q) m2 = __hmax2(m2, chunk_max(u[q]));
      const float2 mf = __bfloat1622float2(m2);
      const float lm = fmaxf(mf.x, mf.y) * k::kLog2eF;
      if (lm > c) {
        s *= ex2_approx(c - lm);
        c = lm;
      }
      const float base = c == -INFINITY ? 0.f : c;
      float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) {
        float2 e[4];
        chunk_exp(u[q], base, e);
        acc0 = f2_add(acc0, f2_add(e[0], e[1]));
        acc1 = f2_add(acc1, f2_add(e[2], e[3]));
      }
      s += (acc0.x + acc0.y) + (acc1.x + acc1.y);
    }
    combine_stats<G>(c, s);
  }

  GPT2_DEV void gradient(uint4* dst, int t, int V, int Vp, float c, float s, float g) const {
    const float gs = -g / s;
    const float2 gs2 = make_float2(gs, gs);
    const int nv = Vp / 8;
    for (int i0 = threadIdx.x; i0 < nv; i0 += kThreads * kUnroll) {
      uint4 u[kUnroll];
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) {
        const int i = i0 + q * kThreads;
        u[q] = i * 8 < V ? __ldcs(zr + i) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) {
        const int i = i0 + q * kThreads;
        if (i < nv) HeldRow<1, 1>::store_chunk(dst + i, u[q], i * 8, t, V, c, gs2, g);
      }
    }
  }
};

// How a kernel's CTA holds its rows: R > 0: R chunks a lane of G warps; R == 0:
// streamed by G warps. Several one-warp rows share a CTA of four warps.
template <int G, int R>
struct RowShape {
  static constexpr int kRows = G == 1 ? 4 : 1;
  static constexpr int kThreads = 32 * G * kRows;
  // registers: the held chunks and about 50 more
  static constexpr int kMinCtas = R > 0 ? 65536 / (kThreads * (4 * R + 50)) : 1;
  static GPT2_DEV int row() { return G == 1 ? blockIdx.x * kRows + (threadIdx.x >> 5) : blockIdx.x; }
  static GPT2_DEV bool first() { return G == 1 ? lane_id() == 0 : threadIdx.x == 0; }
  static GPT2_DEV int lane() { return G == 1 ? lane_id() : threadIdx.x; }
  static GPT2_DEV void zero(uint4* dst, int Vp) {
    for (int i = lane(); i < Vp / 8; i += 32 * G) __stcs(dst + i, make_uint4(0u, 0u, 0u, 0u));
  }
};

// (c, S) of a row from the logits GEMM's row partials (the same base-2 form).
template <int G>
GPT2_DEV void part_stats(const float2* part, int slots, int lane, float& c, float& s) {
  c = -INFINITY;
  s = 0.f;
  for (int i = lane; i < slots; i += 32 * G) {
    const float2 v = __ldcs(part + i);
    k::ce_combine(c, s, v.x, v.y);
  }
  combine_stats<G>(c, s);
}

GPT2_DEV float row_logp(float zt, float c, float s) {
  return (fmaf(zt, k::kLog2eF, -c) - log2f(s)) * k::kLn2F;
}

struct PolicyArgs {
  const bf16* logits;
  const int32_t* targets;
  const float *old_logp, *ref_logp, *adv, *weight;   // ref_logp, weight may be null
  bf16* dlogits;                                     // may be null (loss only) or the logits
  float *logps, *losses;                             // logps may be null
  const float2* part;                                // row partials of the logits GEMM, or null
  int N, slots, V, Vp, ignore_index;
  float clip_low, clip_high, kl_coef, dscale;
  int* err;
};

// The row's loss and g = dscale dloss/dlp.
GPT2_DEV void policy_row(const PolicyArgs& a, float lp, float old_lp, float adv, float ref, float w, float& loss,
                         float& g) {
  const float r = expf(lp - old_lp);
  // r A and its clipped form; an advantage of 0 gives 0 for any ratio
  const float free_s = adv == 0.f ? 0.f : r * adv;
  const float cut_s = fminf(fmaxf(r, 1.f - a.clip_low), 1.f + a.clip_high) * adv;
  const bool active = free_s <= cut_s;
  loss = active ? -free_s : -cut_s;
  g = active ? -free_s : 0.f;
  if (a.ref_logp) {
    // e^d - d - 1 without the cancellation of small d
    const float d = ref - lp, em = expm1f(d);
    loss += a.kl_coef * (em - d);
    g -= a.kl_coef * em;
  }
  loss *= w;
  g *= w * a.dscale;
}

GPT2_DEV void policy_left_out(const PolicyArgs& a, int row, int t, bool first) {
  if (!first) return;
  if (t != a.ignore_index) atomicOr(a.err, DEVERR_TOKEN_RANGE);
  a.losses[row] = 0.f;
  if (a.logps) a.logps[row] = 0.f;
}

GPT2_DEV bool row_kept(int t, int V, int ignore_index) { return t != ignore_index && t >= 0 && t < V; }

// A row: its softmax, the loss and g, the gradient. PART: (c, S) come from the
// logits GEMM's partials and the row is read for the gradient alone.
template <int G, int R, bool PART>
__global__ void __launch_bounds__(RowShape<G, R>::kThreads, RowShape<G, R>::kMinCtas)
    policy_loss_kernel(const PolicyArgs a) {
  using Shape = RowShape<G, R>;
  pdl_begin();
  const int row = Shape::row();
  if (row >= a.N) return;
  const size_t off = (size_t)row * a.Vp;
  const uint4* zr = reinterpret_cast<const uint4*>(a.logits + off);
  uint4* dr = a.dlogits ? reinterpret_cast<uint4*>(a.dlogits + off) : nullptr;
  const int t = a.targets[row];
  if (!row_kept(t, a.V, a.ignore_index)) {
    policy_left_out(a, row, t, Shape::first());
    if (dr) Shape::zero(dr, a.Vp);
    return;
  }
  std::conditional_t<(R > 0), HeldRow<G, R ? R : 1>, StreamedRow<G>> held;
  held.load(zr, a.V);
  const float old_lp = a.old_logp[row], adv = a.adv[row];
  const float ref = a.ref_logp ? a.ref_logp[row] : 0.f;
  const float w = a.weight ? a.weight[row] : 1.f;
  const float zt = __bfloat162float(a.logits[off + t]);   // before any thread may overwrite it
  float c, s, loss, g;
  if constexpr (PART) part_stats<G>(a.part + (size_t)row * a.slots, a.slots, Shape::lane(), c, s);
  else if constexpr (R > 0) held.stats(c, s);
  else held.stats_of(a.V, c, s);
  const float lp = row_logp(zt, c, s);
  policy_row(a, lp, old_lp, adv, ref, w, loss, g);
  if (Shape::first()) {
    a.losses[row] = loss;
    if (a.logps) a.logps[row] = lp;
  }
  if (!dr) return;
  if (g == 0.f && isfinite(lp)) Shape::zero(dr, a.Vp);
  else held.gradient(dr, t, a.V, a.Vp, c, s, g);
}

GPT2_DEV void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
GPT2_DEV void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Long rows, persistent: a row stands in shared memory, every chunk in a slot of
// the thread that works on it, so a chunk's slot takes the next row's chunk as
// soon as its gradient is formed, with no barrier between; the copy of a row runs
// under the gradient and the stores of the one before. The sum takes the target's
// logit as its reference: 2^(y - y_t) needs no pass for the maximum, and a row
// where that overflows is summed again from its maximum.
template <int G>
__global__ void __launch_bounds__(32 * G, 32 / G) policy_long_kernel(const PolicyArgs a) {
  constexpr int kT = 32 * G;
  extern __shared__ __align__(128) uint4 slots[];
  __shared__ float red[2][G];
  __shared__ float red_m[G];
  pdl_begin();
  const int stride = gridDim.x, nvr = (a.V + 7) / 8, nv = a.Vp / 8;
  const int lane = lane_id(), warp = threadIdx.x >> 5;
  auto kept_at = [&](long r) { return r < a.N && row_kept(a.targets[r], a.V, a.ignore_index); };
  // the first kept row of r, r + stride, ..., or one past the last row
  auto scan = [&](long r) {
    for (; r < a.N; r += 32L * stride) {
      const uint32_t hit = __ballot_sync(0xffffffffu, kept_at(r + (long)lane * stride));
      if (hit) return r + (long)(__ffs(hit) - 1) * stride;
    }
    return r;
  };
  auto skip = [&](long from, long to) {
    for (long r = from; r < to && r < a.N; r += stride) {
      policy_left_out(a, (int)r, a.targets[r], threadIdx.x == 0);
      if (a.dlogits) RowShape<G, 0>::zero(reinterpret_cast<uint4*>(a.dlogits + (size_t)r * a.Vp), a.Vp);
    }
  };
  const uint32_t slot0 = smem_u32(slots);
  long row = scan(blockIdx.x);
  if (row < a.N) {
    const uint4* zr = reinterpret_cast<const uint4*>(a.logits + (size_t)row * a.Vp);
    for (int i = threadIdx.x; i < nvr; i += kT) cp_async16(slot0 + i * 16, zr + i);
  }
  skip(blockIdx.x, row);
  int flip = 0;
  while (row < a.N) {
    const size_t off = (size_t)row * a.Vp;
    const int t = a.targets[row];
    const float zt = __bfloat162float(a.logits[off + t]);   // before any thread may overwrite it
    const float old_lp = a.old_logp[row], adv = a.adv[row];
    const float ref = a.ref_logp ? a.ref_logp[row] : 0.f;
    const float w = a.weight ? a.weight[row] : 1.f;
    const long next = scan(row + stride);
    cp_async_wait();
    if ((nvr - 1) % kT == (int)threadIdx.x) mask_chunk(slots[nvr - 1], (nvr - 1) * 8, a.V);
    auto sum_from = [&](float c) {
      float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll 4
      for (int i = threadIdx.x; i < nvr; i += kT) {
        float2 e[4];
        chunk_exp(slots[i], c, e);
        acc0 = f2_add(acc0, f2_add(e[0], e[1]));
        acc1 = f2_add(acc1, f2_add(e[2], e[3]));
      }
      const float p = warp_sum((acc0.x + acc0.y) + (acc1.x + acc1.y));
      if (lane == 0) red[flip][warp] = p;
      __syncthreads();
      const float v = lane < G ? red[flip][lane] : 0.f;
      flip ^= 1;
      return warp_sum(v);
    };
    float c = zt * k::kLog2eF, s = sum_from(c);
    if (!(s < 3e38f)) {   // (the same in every thread)
      __nv_bfloat162 m2 = as_bf2(kNegInf2);
      for (int i = threadIdx.x; i < nvr; i += kT) m2 = __hmax2(m2, chunk_max(slots[i]));
      const float2 mf = __bfloat1622float2(m2);
      const float m = warp_max(fmaxf(mf.x, mf.y));
      if (lane == 0) red_m[warp] = m;
      __syncthreads();
      c = warp_max(lane < G ? red_m[lane] : -INFINITY) * k::kLog2eF;
      s = sum_from(c);
    }
    const float lp = row_logp(zt, c, s);
    float loss, g;
    policy_row(a, lp, old_lp, adv, ref, w, loss, g);
    if (threadIdx.x == 0) {
      a.losses[row] = loss;
      if (a.logps) a.logps[row] = lp;
    }
    uint4* dr = a.dlogits ? reinterpret_cast<uint4*>(a.dlogits + off) : nullptr;
    const uint4* zn = next < a.N ? reinterpret_cast<const uint4*>(a.logits + (size_t)next * a.Vp) : nullptr;
    const bool none = !dr || (g == 0.f && isfinite(lp));
    const float gs = -g / s;
    const float2 gs2 = make_float2(gs, gs);
#pragma unroll 4
    for (int i = threadIdx.x; i < nvr; i += kT) {
      if (!none) HeldRow<1, 1>::store_chunk(dr + i, slots[i], i * 8, t, a.V, c, gs2, g);
      if (zn) cp_async16(slot0 + i * 16, zn + i);
    }
    if (dr)
      for (int i = (none ? 0 : nvr) + threadIdx.x; i < nv; i += kT) __stcs(dr + i, make_uint4(0u, 0u, 0u, 0u));
    skip(row + stride, next);
    row = next;
  }
}

struct RowArgs {
  const bf16* logits;
  const int32_t* targets;
  float* logps;
  float2* stats;            // (c, S) per row, or null
  const float2* part;
  const float* tgt_val;     // the target's logit per row where the logits are not stored, or null
  const int32_t* seq_start; // only rows seq_start[0] .. seq_start[n_seq] - 1, or null: all rows
  int N, n_seq, slots, V, Vp, ignore_index;
  int* err;
};

// A row's lp (0 for a row left out) and (c, S).
template <int G, int R, bool PART>
__global__ void __launch_bounds__(RowShape<G, R>::kThreads) row_logp_kernel(const RowArgs a) {
  using Shape = RowShape<G, R>;
  pdl_begin();
  const int row = Shape::row();
  if (row >= a.N) return;
  if (a.seq_start && (row < a.seq_start[0] || row >= a.seq_start[a.n_seq])) return;
  const size_t off = (size_t)row * a.Vp;
  const int t = a.targets[row];
  const bool in_range = t >= 0 && t < a.V;
  if (t == a.ignore_index || !in_range) {
    if (Shape::first()) {
      if (t != a.ignore_index) atomicOr(a.err, DEVERR_TOKEN_RANGE);
      a.logps[row] = 0.f;
    }
    return;
  }
  float c, s;
  const float zt = a.tgt_val ? a.tgt_val[row] : __bfloat162float(a.logits[off + t]);
  if constexpr (PART) {
    part_stats<G>(a.part + (size_t)row * a.slots, a.slots, Shape::lane(), c, s);
  } else {
    std::conditional_t<(R > 0), HeldRow<G, R ? R : 1>, StreamedRow<G>> held;
    held.load(reinterpret_cast<const uint4*>(a.logits + off), a.V);
    if constexpr (R > 0) held.stats(c, s);
    else held.stats_of(a.V, c, s);
  }
  if (Shape::first()) {
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
__global__ void __launch_bounds__(kPairThreads) pair_kernel(const PairArgs a) {
  pdl_begin();
  constexpr int W = kPairThreads / 32;
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
    for (int i = b + threadIdx.x; i < e; i += kPairThreads) {
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
  int N, n_seq, seq_len, V, Vp, ignore_index;
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

// A row's gradient, from the pair's coefficient and the row's (c, S).
template <int G>
__global__ void __launch_bounds__(RowShape<G, 0>::kThreads) pair_grad_kernel(const PairGradArgs a) {
  using Shape = RowShape<G, 0>;
  pdl_begin();
  const int row = Shape::row();
  if (row >= a.N) return;
  const int seq = a.seq_start ? find_sequence(a.seq_start, a.n_seq, row) : row / a.seq_len;
  if (seq < 0 || seq >= a.n_seq) return;   // behind the last sequence: left as it was
  const size_t off = (size_t)row * a.Vp;
  uint4* dr = reinterpret_cast<uint4*>(a.dlogits + off);
  const int t = a.targets[row];
  if (t == a.ignore_index || t < 0 || t >= a.V) {
    Shape::zero(dr, a.Vp);
    return;
  }
  const float2 st = a.stats[row];
  const uint4* zr = reinterpret_cast<const uint4*>(a.logits + off);
  const float g = a.coef[seq], gs = -g / st.y;
  const float2 gs2 = make_float2(gs, gs);
  const int nv = a.Vp / 8;
  constexpr int kStep = 32 * G, kUnroll = 4;
  for (int i0 = Shape::lane(); i0 < nv; i0 += kStep * kUnroll) {
    uint4 u[kUnroll];
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
      const int i = i0 + q * kStep;
      u[q] = i * 8 < a.V ? __ldcs(zr + i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
      const int i = i0 + q * kStep;
      if (i < nv) HeldRow<1, 1>::store_chunk(dr + i, u[q], i * 8, t, a.V, st.x, gs2, g);
    }
  }
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

template <int V>
using Int = std::integral_constant<int, V>;

// Calls f(G, R) with the shape that holds a row of Vp columns, or (0, 0).
template <typename F>
int with_shape(int Vp, F&& f) {
  const int nv = Vp / 8;
  if (nv <= 4 * 32) return f(Int<1>{}, Int<4>{});
  if (nv <= 10 * 32) return f(Int<1>{}, Int<10>{});
  if (nv <= 18 * 32) return f(Int<1>{}, Int<18>{});
  if (nv <= 9 * 128) return f(Int<4>{}, Int<9>{});
  if (nv <= 16 * 128) return f(Int<4>{}, Int<16>{});
  if (nv <= 16 * 256) return f(Int<8>{}, Int<16>{});
  return f(Int<0>{}, Int<0>{});
}

constexpr int kLongMax = 112 * 1024;   // shared memory of one of two CTAs an SM

template <int G, int R, typename... KArgs, typename Args>
int launch_rows(void (*kern)(KArgs...), int N, cudaStream_t s, const Args& a) {
  using Shape = RowShape<G, R>;
  const int grid = (N + Shape::kRows - 1) / Shape::kRows;
  return launch_pdl(kern, dim3(grid), dim3(Shape::kThreads), 0, s, a) == cudaSuccess ? GPT2_OK : GPT2_ERR_CUDA;
}

template <int G>
int launch_long(const PolicyArgs& a, cudaStream_t s) {
  static PerDeviceOnce once;
  if (smem_optin(once, policy_long_kernel<G>, kLongMax * (G / 16)) != cudaSuccess) return GPT2_ERR_CUDA;
  const int grid = std::min(a.N, device_sm_count() * (32 / G));
  return launch_pdl(policy_long_kernel<G>, dim3(grid), dim3(32 * G), (a.V + 7) / 8 * 16, s, a) == cudaSuccess
             ? GPT2_OK
             : GPT2_ERR_CUDA;
}

inline int policy_loss(const PolicyArgs& a, cudaStream_t s) {
  if (a.part) return launch_rows<8, 0>(policy_loss_kernel<8, 0, true>, a.N, s, a);
  return with_shape(a.Vp, [&](auto g, auto r) {
    constexpr int G = decltype(g)::value, R = decltype(r)::value;
    if constexpr (G > 0) {
      return launch_rows<G, R>(policy_loss_kernel<G, R, false>, a.N, s, a);
    } else {
      const int bytes = (a.V + 7) / 8 * 16;
      if (bytes <= kLongMax) return launch_long<16>(a, s);
      if (bytes <= 2 * kLongMax) return launch_long<32>(a, s);
      return launch_rows<16, 0>(policy_loss_kernel<16, 0, false>, a.N, s, a);
    }
  });
}

inline int row_logps(const RowArgs& a, cudaStream_t s) {
  if (a.part) return launch_rows<1, 0>(row_logp_kernel<1, 0, true>, a.N, s, a);
  return with_shape(a.Vp, [&](auto g, auto r) {
    constexpr int G = decltype(g)::value, R = decltype(r)::value;
    if constexpr (G > 0) return launch_rows<G, R>(row_logp_kernel<G, R, false>, a.N, s, a);
    else return launch_rows<8, 0>(row_logp_kernel<8, 0, false>, a.N, s, a);
  });
}

inline int pair_losses(const PairArgs& a, int P, cudaStream_t s) {
  return launch_pdl(pair_kernel, dim3(P), dim3(kPairThreads), 0, s, a) == cudaSuccess ? GPT2_OK : GPT2_ERR_CUDA;
}

inline int pair_gradients(const PairGradArgs& a, cudaStream_t s) {
  if (a.Vp <= 4608) return launch_rows<1, 0>(pair_grad_kernel<1>, a.N, s, a);
  if (a.Vp <= 16384) return launch_rows<4, 0>(pair_grad_kernel<4>, a.N, s, a);
  return launch_rows<8, 0>(pair_grad_kernel<8>, a.N, s, a);
}

// Workspace: a row's (c, S), then a sequence's coefficient.
inline size_t preference_workspace(int N, int P) { return (size_t)N * 8 + (size_t)P * 8; }

}  // namespace pt
