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

// (c, S) joined with another. Where both maxima are -inf the sums hold no numbers, 0 or, of
// values that are all NaN, a NaN that must not be lost.
GPT2_DEV void join_stats(float& c, float& s, float oc, float os) {
  const float m = fmaxf(c, oc);
  s = m == -INFINITY ? s + os : s * ex2_approx(c - m) + os * ex2_approx(oc - m);
  c = m;
}

// (c, S) of a row split over `G` warps, from each lane's own pair.
template <int G>
GPT2_DEV void combine_stats(float& c, float& s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    join_stats(c, s, __shfl_xor_sync(0xffffffffu, c, o), __shfl_xor_sync(0xffffffffu, s, o));
  if (G > 1) {
    __shared__ float2 red[G];
    if (lane_id() == 0) red[threadIdx.x >> 5] = make_float2(c, s);
    __syncthreads();
    const float2 v = lane_id() < G ? red[lane_id()] : make_float2(-INFINITY, 0.f);
    c = v.x;
    s = v.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      join_stats(c, s, __shfl_xor_sync(0xffffffffu, c, o), __shfl_xor_sync(0xffffffffu, s, o));
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

// 2^y on the fp32 pipe, relative error below 1.7e-7: y = n + f with n its nearest integer
// (the low bits of y + 1.5 x 2^23), 2^f a polynomial of degree 5 on [-1/2, 1/2] with value 1
// at 0 (weighted least squares of the relative error), n added to its exponent bits. y is
// held in [-127, 127]; at -127, and so at -inf, the bits are those of 0. A NaN comes out
// above 10^38, as an overflow does.
GPT2_DEV float2 exp2_poly(float2 y) {
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;\n\tmin.NaN.f32 %0, %0, 0f42FE0000;" : "+f"(y.x));
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;\n\tmin.NaN.f32 %0, %0, 0f42FE0000;" : "+f"(y.y));
  auto both = [](float v) { return make_float2(v, v); };
  const float2 t = f2_add(y, both(12582912.f)), n = f2_add(t, both(-12582912.f)), f = f2_fma(n, both(-1.f), y);
  float2 p = f2_fma(both(1.326472731e-03f), f, both(9.671512991e-03f));
  p = f2_fma(p, f, both(5.550733581e-02f));
  p = f2_fma(p, f, both(2.402224243e-01f));
  p = f2_fma(p, f, both(6.931470037e-01f));
  p = f2_fma(p, f, both(1.f));
  return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23)));
}

// 2^(y - c) of a chunk's values, paired fp32 arithmetic; MIX: a quarter of them on the fp32
// pipe (overflows and NaN as there).
template <bool MIX = false>
GPT2_DEV void chunk_exp(uint4 u, float c, float2 (&e)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  const float2 l2 = make_float2(k::kLog2eF, k::kLog2eF), nc = make_float2(-c, -c);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 y = f2_fma(bf2_to_f2(w[j]), l2, nc);
    e[j] = MIX && j == 3 ? exp2_poly(y) : make_float2(ex2_approx(y.x), ex2_approx(y.y));
  }
}

// Two values rounded to bf16 on the fp32 pipe: x (2^16 + 1) - (x (2^16 + 1) - x) is x
// rounded to 8 bits (Dekker's splitting), its upper half the bf16. The conversion
// instruction shares the pipe of ex2, which is what bounds these kernels next to memory.
// For values below 2^111.
GPT2_DEV uint32_t round_bf16x2(float2 x) {
  const float2 c = f2_mul(x, make_float2(65537.f, 65537.f));
  const float2 d = f2_fma(x, make_float2(-1.f, -1.f), c);
  const float2 h = f2_fma(d, make_float2(-1.f, -1.f), c);
  return __byte_perm(__float_as_uint(h.x), __float_as_uint(h.y), 0x7632);
}

// A row's gradient g ([j == t] - 2^(y - c) / S), 0 behind the real columns, by chunks.
struct RowGradient {
  int V, t, t_chunk, edge;       // edge: the chunk with the last real column and padded ones, or -1
  float c, g, gs;

  GPT2_DEV RowGradient(int V_, int t_, float c_, float s, float g_)
      : V(V_), t(t_), t_chunk(t_ >> 3), edge((V_ & 7) ? V_ >> 3 : -1), c(c_), g(g_), gs(-g_ / s) {}
  // Whether no value (none exceeds |g|) leaves the range of round_bf16x2.
  GPT2_DEV bool rounds() const { return fabsf(g) < 1e30f; }

  template <bool ROUNDS>
  GPT2_DEV void store(uint4* dst, uint4 z, int i) const {
    float2 e[4];
    chunk_exp(z, c, e);
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = f2_mul(e[j], make_float2(gs, gs));
    if (i == t_chunk || i == edge) {
      float* f = &e[0].x;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = i * 8 + j >= V ? 0.f : f[j] + (i * 8 + j == t ? g : 0.f);
    }
    __stcs(dst + i, ROUNDS ? make_uint4(round_bf16x2(e[0]), round_bf16x2(e[1]), round_bf16x2(e[2]), round_bf16x2(e[3]))
                           : make_uint4(pack_bf16x2(e[0].x, e[0].y), pack_bf16x2(e[1].x, e[1].y),
                                        pack_bf16x2(e[2].x, e[2].y), pack_bf16x2(e[3].x, e[3].y)));
  }
};

// Columns from c0 on (a multiple of 8) of a gradient row, 0.
GPT2_DEV void zero_row(uint4* dst, int c0, int Vp, int lane, int lanes) {
  for (int i = c0 / 8 + lane; i < Vp / 8; i += lanes) __stcs(dst + i, make_uint4(0u, 0u, 0u, 0u));
}

// (c, S) of a row read from global memory by the CTA's G warps, with its running maximum.
template <int G>
GPT2_DEV void streamed_stats(const uint4* zr, int V, float& c, float& s) {
  constexpr int kThreads = 32 * G, kUnroll = 4;
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

// A row's gradient from its (c, S), read from and written to global memory (dst may be the row).
GPT2_DEV void streamed_gradient(const uint4* zr, uint4* dst, int t, int V, int Vp, float c, float s, float g, int lane,
                                int lanes) {
  constexpr int kUnroll = 4;
  const RowGradient grad(V, t, c, s, g);
  const int nvr = (V + 7) / 8;
  if (!grad.rounds()) {
    for (int i = lane; i < nvr; i += lanes) grad.store<false>(dst, __ldcs(zr + i), i);
    zero_row(dst, nvr * 8, Vp, lane, lanes);
    return;
  }
  for (int i0 = lane; i0 < nvr; i0 += lanes * kUnroll) {
    uint4 u[kUnroll];
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
      const int i = i0 + q * lanes;
      u[q] = i < nvr ? __ldcs(zr + i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
      const int i = i0 + q * lanes;
      if (i < nvr) grad.store<true>(dst, u[q], i);
    }
  }
  zero_row(dst, nvr * 8, Vp, lane, lanes);
}

// (c, S) of a row from the logits GEMM's row partials (the same base-2 form).
template <int G>
GPT2_DEV void part_stats(const float2* part, int slots, int lane, float& c, float& s) {
  c = -INFINITY;
  s = 0.f;
  for (int i = lane; i < slots; i += 32 * G) {
    const float2 v = __ldcs(part + i);
    join_stats(c, s, v.x, v.y);
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

// r held in [lo, hi]; a NaN stays one.
GPT2_DEV float clip_nan(float r, float lo, float hi) {
  asm("max.NaN.f32 %0, %0, %1;\n\tmin.NaN.f32 %0, %0, %2;" : "+f"(r) : "f"(lo), "f"(hi));
  return r;
}

// The row's loss and g = dscale dloss/dlp.
GPT2_DEV void policy_row(const PolicyArgs& a, float lp, float old_lp, float adv, float ref, float w, float& loss,
                         float& g) {
  const float r = expf(lp - old_lp);
  // r A and its clipped form; an advantage of 0 gives 0 for any ratio, but does not hide that
  // the row has no log-probability
  const bool none = adv == 0.f && !isnan(lp);
  const float free_s = none ? 0.f : r * adv;
  const float cut_s = none ? 0.f : clip_nan(r, 1.f - a.clip_low, 1.f + a.clip_high) * adv;
  const bool active = !(free_s > cut_s);   // a NaN goes on into the loss and the gradient
  loss = active ? -free_s : -cut_s;
  g = active ? -free_s : 0.f;
  if (a.ref_logp) {
    // e^d - d - 1 without the cancellation of small d, and +inf where d is
    const float d = ref - lp, em = expm1f(d);
    loss += a.kl_coef * (em - fminf(d, 3.402823466e38f));
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

GPT2_DEV void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
GPT2_DEV void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The rows of a CTA, in windows of 32, row k of the window with lane k. Of every gridDim.x
// rows a CTA takes one, each time 0.38 of the way further on: with a fixed place, sequences
// whose length divides the grid would give all their prompts (rows left out) to the same
// CTAs. A window's targets, and with them the targets' logits, are read 32 at a time.
struct RowWindows {
  const int32_t* targets;
  const bf16* logits;
  long begin, end, base;            // rows of interest; the window's first row number without the turn
  int V, Vp, ignore_index;
  uint32_t grid, place, lane_turn, turn32, hits;
  long row;                         // this lane's row and its target and logit
  int t;
  float zt;

  GPT2_DEV RowWindows(const int32_t* tg, const bf16* z, long b, long e, int v, int vp, int ign)
      : targets(tg), logits(z), begin(b), end(e), V(v), Vp(vp), ignore_index(ign), hits(0), row(0), t(0), zt(0.f) {
    grid = gridDim.x;
    const uint32_t turn = (uint32_t)(0.382f * grid);
    lane_turn = lane_id() * turn % grid;
    turn32 = 32 * turn % grid;
    base = 0;
    place = blockIdx.x;
  }
  GPT2_DEV bool more() const { return base < end; }
  // Reads the next window; the lanes whose row is of interest but left out.
  GPT2_DEV uint32_t load() {
    uint32_t at = place + lane_turn;
    if (at >= grid) at -= grid;
    row = base + (long)lane_id() * grid + at;
    const bool in = row >= begin && row < end;
    t = in ? targets[row] : -1;
    const bool kept = in && row_kept(t, V, ignore_index);
    zt = kept ? __bfloat162float(logits[(size_t)row * Vp + t]) : 0.f;
    hits = __ballot_sync(0xffffffffu, kept);
    base += 32L * grid;
    place += turn32;
    if (place >= grid) place -= grid;
    return __ballot_sync(0xffffffffu, in && !kept);
  }
};

// A row in shared memory: every 16-byte chunk has a slot that belongs to the thread that
// works on it, so a slot takes the next row's chunk as soon as this row is done with it,
// without a barrier, and copies run under the arithmetic and the stores. The sum takes the
// target's logit as its reference, c = y_t, which needs no pass for the maximum; a row
// whose sum passes kSumMax (a log-probability below -41) is summed again from its maximum,
// long before the sum, or the gradient's factor g / S, leaves the range of fp32.
constexpr float kSumMax = 1e18f;

template <int G>
struct RowPipe {
  static constexpr int kThreads = 32 * G;
  uint4* slots;
  uint32_t slot0;
  int nvr;                       // chunks that hold real ids
  float (*red)[G];               // [2][G]: two sums in flight
  int flip;

  GPT2_DEV void prefetch(const uint4* zr) const {
    for (int i = threadIdx.x; i < nvr; i += kThreads) cp_async16(slot0 + i * 16, zr + i);
  }
  // Waits for this thread's chunks of the row.
  GPT2_DEV void arrive(int V) const {
    cp_async_wait();
    if ((nvr - 1) % kThreads == (int)threadIdx.x) mask_chunk(slots[nvr - 1], (nvr - 1) * 8, V);
  }
  GPT2_DEV float sum_all(float v) {
    v = warp_sum(v);
    if (G == 1) return v;
    if (lane_id() == 0) red[flip][threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane_id() < G ? red[flip][lane_id()] : 0.f;
    flip ^= 1;
    return warp_sum(v);
  }
  // sum of 2^(y - c); with `zn` the slots take the next row on the way. MIX: a sum from
  // kSumMax on stands for an overflow or a NaN too.
  template <bool MIX>
  GPT2_DEV float sum_from(float c, const uint4* zn) {
    float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
    auto add = [&](uint4 u) {
      float2 e[4];
      chunk_exp<MIX>(u, c, e);
      acc0 = f2_add(acc0, f2_add(e[0], e[1]));
      acc1 = f2_add(acc1, f2_add(e[2], e[3]));
    };
    int i = threadIdx.x;
    for (; i + 3 * kThreads < nvr; i += 4 * kThreads) {   // four chunks in flight
      uint4 u[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) u[q] = slots[i + q * kThreads];
#pragma unroll
      for (int q = 0; q < 4; ++q) add(u[q]);
      if (zn) {
#pragma unroll
        for (int q = 0; q < 4; ++q) cp_async16(slot0 + (i + q * kThreads) * 16, zn + i + q * kThreads);
      }
    }
    for (; i < nvr; i += kThreads) {
      add(slots[i]);
      if (zn) cp_async16(slot0 + i * 16, zn + i);
    }
    return sum_all((acc0.x + acc0.y) + (acc1.x + acc1.y));
  }
};

// The policy loss: a row is read from memory once and its gradient written once, which is
// what bounds it. 19,456 x 50,257 with a quarter of the rows left out: 598 to 627 us by box, 5.7 TB/s of
// the bytes it cannot do without (0.87 of the measured copy rate); the ex2 pipe is 49% busy
// beside it, at 1.75 of them an element. Measured before: the row read twice, the second
// time out of L2, 727 us (eight CTAs an SM bring more rows than L2 holds); held in registers
// by 512 threads 678 us; in shared memory by one bulk copy a row, with a pass for the
// maximum, 657 us. 16,384 x 4,353: 54 us, 0.72; there a row is short and its fixed part
// (reductions, exponentials of the ratio) counts.
template <int G>
__global__ void __launch_bounds__(32 * G, 32 / G) policy_loss_kernel(const PolicyArgs a) {
  extern __shared__ __align__(128) uint4 row_slots[];
  __shared__ float red[2][G];
  __shared__ float red_m[G];
  pdl_begin();
  const int lane = lane_id();
  RowPipe<G> pipe{row_slots, smem_u32(row_slots), (a.V + 7) / 8, red, 0};
  RowWindows win(a.targets, a.logits, 0, a.N, a.V, a.Vp, a.ignore_index);
  float l_old = 0.f, l_adv = 0.f, l_ref = 0.f, l_w = 1.f;   // of the lane's row
  // The next kept row's lane in the window, -1 behind the last; rows left out on the way are finished.
  auto advance = [&]() {
    while (win.hits == 0) {
      if (!win.more()) return -1;
      for (uint32_t miss = win.load(); miss; miss &= miss - 1) {
        const long r = __shfl_sync(0xffffffffu, win.row, __ffs(miss) - 1);
        policy_left_out(a, (int)r, a.targets[r], threadIdx.x == 0);
        if (a.dlogits) zero_row(reinterpret_cast<uint4*>(a.dlogits + (size_t)r * a.Vp), 0, a.Vp, threadIdx.x, 32 * G);
      }
      if (win.hits >> lane & 1) {
        l_old = a.old_logp[win.row];
        l_adv = a.adv[win.row];
        if (a.ref_logp) l_ref = a.ref_logp[win.row];
        if (a.weight) l_w = a.weight[win.row];
      }
    }
    const int j = __ffs(win.hits) - 1;
    win.hits &= win.hits - 1;
    return j;
  };
  // a row's numbers, from the lane that has them
  struct Row { long row; int t; float zt, old_lp, adv, ref, w; };
  auto take = [&](int j) {
    Row r;
    r.row = __shfl_sync(0xffffffffu, win.row, j);
    r.t = __shfl_sync(0xffffffffu, win.t, j);
    r.zt = __shfl_sync(0xffffffffu, win.zt, j);
    r.old_lp = __shfl_sync(0xffffffffu, l_old, j);
    r.adv = __shfl_sync(0xffffffffu, l_adv, j);
    r.ref = __shfl_sync(0xffffffffu, l_ref, j);
    r.w = __shfl_sync(0xffffffffu, l_w, j);
    return r;
  };
  int j = advance();
  if (j < 0) return;
  Row cur = take(j);
  pipe.prefetch(reinterpret_cast<const uint4*>(a.logits + (size_t)cur.row * a.Vp));
  while (j >= 0) {
    const long row = cur.row;
    const size_t off = (size_t)row * a.Vp;
    const int t = cur.t;
    const float zt = cur.zt;
    pipe.arrive(a.V);
    float c = zt * k::kLog2eF, s = pipe.template sum_from<true>(c, nullptr);
    if (!(s < kSumMax)) {   // (the same in every thread)
      __nv_bfloat162 m2 = as_bf2(kNegInf2);
      for (int i = threadIdx.x; i < pipe.nvr; i += 32 * G) m2 = __hmax2(m2, chunk_max(row_slots[i]));
      const float2 mf = __bfloat1622float2(m2);
      float m = warp_max(fmaxf(mf.x, mf.y));
      if (G > 1) {
        if (lane == 0) red_m[threadIdx.x >> 5] = m;
        __syncthreads();
        m = warp_max(lane < G ? red_m[lane] : -INFINITY);
      }
      c = m * k::kLog2eF;
      s = pipe.template sum_from<false>(c, nullptr);
    }
    const float lp = row_logp(zt, c, s);
    float loss, g;
    policy_row(a, lp, cur.old_lp, cur.adv, cur.ref, cur.w, loss, g);
    if (threadIdx.x == 0) {
      a.losses[row] = loss;
      if (a.logps) a.logps[row] = lp;
    }
    j = advance();
    if (j >= 0) cur = take(j);
    uint4* dr = a.dlogits ? reinterpret_cast<uint4*>(a.dlogits + off) : nullptr;
    const uint4* zn = j >= 0 ? reinterpret_cast<const uint4*>(a.logits + (size_t)cur.row * a.Vp) : nullptr;
    const bool none = !dr || (g == 0.f && isfinite(lp));
    if (none) {
      if (zn) pipe.prefetch(zn);
    } else if (const RowGradient grad(a.V, t, c, s, g); !grad.rounds()) {
      for (int i = threadIdx.x; i < pipe.nvr; i += 32 * G) grad.template store<false>(dr, row_slots[i], i);
      if (zn) pipe.prefetch(zn);
    } else {
      constexpr int kT = 32 * G;
      int i = threadIdx.x;
      for (; i + kT < pipe.nvr; i += 2 * kT) {   // two chunks in flight
        const uint4 u0 = row_slots[i], u1 = row_slots[i + kT];
        grad.template store<true>(dr, u0, i);
        grad.template store<true>(dr, u1, i + kT);
        if (zn) {
          cp_async16(pipe.slot0 + i * 16, zn + i);
          cp_async16(pipe.slot0 + (i + kT) * 16, zn + i + kT);
        }
      }
      if (i < pipe.nvr) {
        grad.template store<true>(dr, row_slots[i], i);
        if (zn) cp_async16(pipe.slot0 + i * 16, zn + i);
      }
    }
    if (dr) zero_row(dr, none ? 0 : pipe.nvr * 8, a.Vp, threadIdx.x, 32 * G);
  }
}

// A row a CTA, from global memory: rows too long for shared memory (read a second time
// for the gradient, out of L2), and with PART rows whose (c, S) the logits GEMM's
// epilogue has left, which are read for the gradient alone.
template <int G, bool PART>
__global__ void __launch_bounds__(32 * G) policy_streamed_kernel(const PolicyArgs a) {
  pdl_begin();
  const int row = blockIdx.x;
  const size_t off = (size_t)row * a.Vp;
  const uint4* zr = reinterpret_cast<const uint4*>(a.logits + off);
  uint4* dr = a.dlogits ? reinterpret_cast<uint4*>(a.dlogits + off) : nullptr;
  const int t = a.targets[row];
  if (!row_kept(t, a.V, a.ignore_index)) {
    policy_left_out(a, row, t, threadIdx.x == 0);
    if (dr) zero_row(dr, 0, a.Vp, threadIdx.x, 32 * G);
    return;
  }
  // read by all threads before (the sums' barrier) one of them writes: the logits, and the
  // inputs if an output takes their place
  const float zt = __bfloat162float(a.logits[off + t]);
  const float old_lp = a.old_logp[row], adv = a.adv[row];
  const float ref = a.ref_logp ? a.ref_logp[row] : 0.f, w = a.weight ? a.weight[row] : 1.f;
  float c, s, loss, g;
  if (PART) part_stats<G>(a.part + (size_t)row * a.slots, a.slots, threadIdx.x, c, s);
  else streamed_stats<G>(zr, a.V, c, s);
  const float lp = row_logp(zt, c, s);
  policy_row(a, lp, old_lp, adv, ref, w, loss, g);
  if (threadIdx.x == 0) {
    a.losses[row] = loss;
    if (a.logps) a.logps[row] = lp;
  }
  if (!dr) return;
  if (g == 0.f && isfinite(lp)) zero_row(dr, 0, a.Vp, threadIdx.x, 32 * G);
  else streamed_gradient(zr, dr, t, a.V, a.Vp, c, s, g, threadIdx.x, 32 * G);
}

// The rows that the sequences cut up: from the first bound to the last, or all where those are no bounds.
struct RowSpan {
  long begin, end;
  GPT2_DEV RowSpan(const int32_t* start, int n_seq, int N) : begin(start[0]), end(start[n_seq]) {
    if (begin < 0 || end < begin || end > N) {
      begin = 0;
      end = N;
    }
  }
  // Pair p's three bounds, and whether they are bounds.
  GPT2_DEV int4 bounds(const int32_t* start, int p) const {
    const int32_t a = start[2 * p], b = start[2 * p + 1], c = start[2 * p + 2];
    return make_int4(a, b, c, begin <= a && a <= b && b <= c && c <= end);
  }
};

struct RowArgs {
  const bf16* logits;
  const int32_t* targets;
  float* logps;
  float2* stats;            // (c, S) per row, or null
  const float2* part;
  const float* tgt_val;     // the target's logit per row where the logits are not stored, or null
  const int32_t* seq_start; // only the rows of its span, or null: all rows
  int N, n_seq, slots, V, Vp, ignore_index;
  int* err;
};

// Rows' lp (0 for rows left out) and (c, S); rows outside the sequences are passed over.
// With all exponentials on it the ex2 pipe is 60% busy here, in bursts between a row's
// arrivals: a quarter of them on the fp32 pipe takes the preference loss of 9 pairs of 1,024 x 50,257 from
// 747 us to 735, half of them to 765. The policy loss sums the same way, for the same bits
// (19,456 x 50,257: 622 us against 626, 16,384 x 4,353: 54.2 against 53.7); a quarter of its
// gradient's exponentials too would cost it 30 us.
template <int G>
__global__ void __launch_bounds__(32 * G, 32 / G) row_logp_kernel(const RowArgs a) {
  extern __shared__ __align__(128) uint4 row_slots[];
  __shared__ float red[2][G];
  pdl_begin();
  RowPipe<G> pipe{row_slots, smem_u32(row_slots), (a.V + 7) / 8, red, 0};
  long begin = 0, end = a.N;
  if (a.seq_start) {
    const RowSpan span(a.seq_start, a.n_seq, a.N);
    begin = span.begin;
    end = span.end;
  }
  RowWindows win(a.targets, a.logits, begin, end, a.V, a.Vp, a.ignore_index);
  auto advance = [&]() {
    while (win.hits == 0) {
      if (!win.more()) return -1;
      if (win.load() >> lane_id() & 1) {
        if (win.t != a.ignore_index) atomicOr(a.err, DEVERR_TOKEN_RANGE);
        a.logps[win.row] = 0.f;
      }
    }
    const int j = __ffs(win.hits) - 1;
    win.hits &= win.hits - 1;
    return j;
  };
  int j = advance();
  if (j < 0) return;
  long row = __shfl_sync(0xffffffffu, win.row, j);
  float zt = __shfl_sync(0xffffffffu, win.zt, j);
  pipe.prefetch(reinterpret_cast<const uint4*>(a.logits + (size_t)row * a.Vp));
  while (j >= 0) {
    j = advance();
    const long next = __shfl_sync(0xffffffffu, win.row, max(j, 0));
    const float zt_next = __shfl_sync(0xffffffffu, win.zt, max(j, 0));
    const uint4* zn = j >= 0 ? reinterpret_cast<const uint4*>(a.logits + (size_t)next * a.Vp) : nullptr;
    pipe.arrive(a.V);
    float c = zt * k::kLog2eF, s = pipe.template sum_from<true>(c, zn);
    if (!(s < kSumMax))   // (the same in every thread) the slots have moved on
      streamed_stats<G>(reinterpret_cast<const uint4*>(a.logits + (size_t)row * a.Vp), a.V, c, s);
    if (threadIdx.x == 0) {
      a.logps[row] = row_logp(zt, c, s);
      if (a.stats) a.stats[row] = make_float2(c, s);
    }
    row = next;
    zt = zt_next;
  }
}

// The same a row a CTA: rows too long for shared memory, and with PART rows whose (c, S)
// the logits GEMM's epilogue has left (the target's logit too where none are stored).
template <int G, bool PART>
__global__ void __launch_bounds__(32 * G) row_logp_streamed_kernel(const RowArgs a) {
  pdl_begin();
  const int row = blockIdx.x;
  if (a.seq_start) {
    const RowSpan span(a.seq_start, a.n_seq, a.N);
    if (row < span.begin || row >= span.end) return;
  }
  const size_t off = (size_t)row * a.Vp;
  const int t = a.targets[row];
  if (!row_kept(t, a.V, a.ignore_index)) {
    if (threadIdx.x == 0) {
      if (t != a.ignore_index) atomicOr(a.err, DEVERR_TOKEN_RANGE);
      a.logps[row] = 0.f;
    }
    return;
  }
  const float zt = a.tgt_val ? a.tgt_val[row] : __bfloat162float(a.logits[off + t]);
  float c, s;
  if (PART) part_stats<G>(a.part + (size_t)row * a.slots, a.slots, threadIdx.x, c, s);
  else streamed_stats<G>(reinterpret_cast<const uint4*>(a.logits + off), a.V, c, s);
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
  float2* coef;               // [P], or null where pair_grad_kernel forms them itself
  int N, n_pairs, seq_len, V, ignore_index, kind, average;
  float beta, smoothing, dscale;
  int* err;
};

// The preference loss reads the logits twice, in row_logp_kernel and pair_grad_kernel: no
// row's gradient is known before all rows of its pair are. A pair of the largest case (two
// sequences of 1,024 x 50,257) is more than L2 holds. Nine such pairs: 723 us, 4.4 TB/s of
// the bytes needed once and 6.1 TB/s of those moved; eight pairs of up to 2 x 1,024 x 4,353:
// 56 us. One cooperative launch with grid barriers between the steps, and groups of pairs
// that L2 holds, measured 921 and 100 us.

// The coefficients g of pair p's two sequences, 2p the chosen one and 2p + 1 the rejected
// one, by a CTA of T threads (the same in all of them); with `put` the pair's loss and its
// sequences' log-probabilities are written too. The sums over a sequence and the difference
// of the two run in 64 bits: a margin of a few units is left of sums of thousands.
template <int T>
GPT2_DEV float2 pair_of(const PairArgs& a, int p, bool put) {
  constexpr int W = T / 32;
  __shared__ double red[2][W];
  __shared__ int cnt[2][W];
  __shared__ float2 coef;
  bool bad = false;
  int4 at{};
  if (a.seq_start) {
    at = RowSpan(a.seq_start, 2 * a.n_pairs, a.N).bounds(a.seq_start, p);
    bad = !at.w;
    if (bad) at = make_int4(0, 0, 0, 0);
  }
  for (int h = 0; h < 2; ++h) {
    const long b = a.seq_start ? (h ? at.y : at.x) : (2L * p + h) * a.seq_len;
    const long e = a.seq_start ? (h ? at.z : at.y) : b + a.seq_len;
    double s = 0.0;
    int n = 0;
#pragma unroll 8
    for (long i = b + threadIdx.x; i < e; i += T) s += (double)a.logps[i];   // 0 for rows left out
    if (a.average)
      for (long i = b + threadIdx.x; i < e; i += T) n += row_kept(a.targets[i], a.V, a.ignore_index);
    s = warp_sum_d(s);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane_id() == 0) {
      red[h][threadIdx.x >> 5] = s;
      cnt[h][threadIdx.x >> 5] = n;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
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
      if (put && a.seq_logps) a.seq_logps[2 * p + h] = (float)s;
      gap[h] = s - (a.ref_logp ? (double)a.ref_logp[2 * p + h] : 0.0);
    }
    const double delta = gap[0] - gap[1], b = a.beta, eps = a.smoothing;
    double loss, dd;
    if (a.kind == 0) {
      // softplus(+-x) and sigma(+-x) from one exponential
      const double x = b * delta, e = exp(-fabs(x)), big = 1.0 / (1.0 + e), small = e * big;
      const double l = put ? log1p(e) : 0.0, up = fmax(-x, 0.0) + l, down = fmax(x, 0.0) + l;   // softplus(-x), softplus(x)
      loss = (1.0 - eps) * up + (eps > 0.0 ? eps * down : 0.0);   // (down may be infinite)
      dd = -b * (x > 0 ? (1.0 - eps) * small - eps * big : (1.0 - eps) * big - eps * small);
    } else {
      const double off = delta - 0.5 / b;
      loss = off * off;
      dd = 2.0 * off;
    }
    if (bad) {   // bounds that are not bounds: no loss, no gradient, flagged
      atomicOr(a.err, DEVERR_TOKEN_RANGE);
      loss = dd = 0.0;
    }
    coef = make_float2((float)(dd * share[0] * a.dscale), (float)(-dd * share[1] * a.dscale));
    if (put) {
      a.losses[p] = (float)loss;
      if (a.coef) a.coef[p] = coef;
    }
  }
  __syncthreads();
  const float2 out = coef;
  __syncthreads();   // the shared memory is free again
  return out;
}

__global__ void __launch_bounds__(kPairThreads) pair_kernel(const PairArgs a) {
  pdl_begin();
  pair_of<kPairThreads>(a, blockIdx.x, true);
}

struct PairGradArgs {
  const bf16* logits;
  const int32_t* targets;
  const int32_t* seq_start;
  const float2* stats;
  bf16* dlogits;
  int N, n_seq, seq_len, V, Vp, ignore_index;
};

// The sequence that holds `row`: the last one that begins at or before it. kOutside for rows
// in front of the first and behind the last, kNone where bounds that are not bounds let none be found.
constexpr int kOutside = -1, kNone = -2;
GPT2_DEV int find_sequence(const int32_t* start, int n_seq, int N, int row) {
  const RowSpan span(start, n_seq, N);
  int lo = 0, hi = n_seq;   // start[lo] <= row is looked for in [0, n_seq)
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= row) lo = mid + 1;
    else hi = mid;
  }
  if (row < span.begin || row >= span.end) return kOutside;
  const int s = max(lo - 1, 0);
  const int4 b = span.bounds(start, s >> 1);
  return b.w && row >= (s & 1 ? b.y : b.x) && row < (s & 1 ? b.z : b.y) ? s : kNone;
}

// The rows' gradients from their (c, S): a warp a row where G is 1 (four a CTA), else the
// CTA's G warps. OWN: the first n_seq / 2 CTAs take the pairs, and every other CTA adds up
// its rows' pair for itself, a few thousand log-probabilities out of L2, instead of waiting
// for a launch between (pa.coef otherwise holds the coefficients). Rows in descending order:
// the last ones of row_logp_kernel's pass are still in L2 (9 pairs of 1,024 x 50,257: 723 us
// against 733).
template <int G, bool OWN>
__global__ void __launch_bounds__(G == 1 ? 128 : 32 * G) pair_grad_kernel(const PairGradArgs a, const PairArgs pa) {
  constexpr int kRows = G == 1 ? 4 : 1, T = G == 1 ? 128 : 32 * G;
  __shared__ int pair_s[kRows];
  __shared__ float2 coef_s[kRows];
  pdl_begin();
  const int P = OWN ? a.n_seq / 2 : 0;
  if ((int)blockIdx.x < P) {
    pair_of<T>(pa, blockIdx.x, true);
    return;
  }
  const int w = G == 1 ? threadIdx.x >> 5 : 0, lane = G == 1 ? lane_id() : threadIdx.x;
  const long row = (long)(gridDim.x - 1 - blockIdx.x) * kRows + w;
  int seq = kOutside, t = 0;
  bool kept = false;
  if (row < a.N) {
    seq = a.seq_start ? find_sequence(a.seq_start, a.n_seq, a.N, (int)row) : (int)(row / a.seq_len);
    if (seq >= a.n_seq) seq = kOutside;
    t = a.targets[row];
    kept = seq >= 0 && row_kept(t, a.V, a.ignore_index);
  }
  float2 c = make_float2(0.f, 0.f);
  if (OWN) {
    if (lane == 0) pair_s[w] = kept ? seq >> 1 : -1;
    __syncthreads();
    for (int i = 0; i < kRows; ++i) {     // uniform in the CTA
      const int p = pair_s[i];
      if (p < 0) continue;
      int same = -1;
      for (int j = 0; j < i; ++j)
        if (pair_s[j] == p) same = j;
      const float2 ci = same >= 0 ? coef_s[same] : pair_of<T>(pa, p, false);
      if (threadIdx.x == 0) coef_s[i] = ci;
      __syncthreads();
    }
    c = coef_s[w];
  }
  if (seq == kOutside) return;   // left as it was
  const size_t off = (size_t)row * a.Vp;
  uint4* dr = reinterpret_cast<uint4*>(a.dlogits + off);
  if (!kept) {
    zero_row(dr, 0, a.Vp, lane, 32 * G);
    return;
  }
  if (!OWN) c = pa.coef[seq >> 1];
  const float2 st = a.stats[row];
  streamed_gradient(reinterpret_cast<const uint4*>(a.logits + off), dr, t, a.V, a.Vp, st.x, st.y, seq & 1 ? c.y : c.x,
                    lane, 32 * G);
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

constexpr int kSmemSm = 227 * 1024, kSmemCta = 1024 + 512;   // of an SM; a CTA's own share beside its row

template <int V>
using Int = std::integral_constant<int, V>;

// Calls f(G) with the fewest warps for one row of V ids in shared memory that keep 32 warps
// an SM at work on the rows it holds: f(0) where one row does not fit.
template <typename F>
int with_warps(int V, F&& f) {
  const int bytes = (V + 7) / 8 * 16 + kSmemCta;
  if (bytes * 32 <= kSmemSm) return f(Int<1>{});
  if (bytes * 16 <= kSmemSm) return f(Int<2>{});
  if (bytes * 8 <= kSmemSm) return f(Int<4>{});
  if (bytes * 4 <= kSmemSm) return f(Int<8>{});
  if (bytes * 2 <= kSmemSm) return f(Int<16>{});
  if (bytes <= kSmemSm) return f(Int<32>{});
  return f(Int<0>{});
}

template <int G, typename Args>
int launch_pipe(void (*kern)(Args), const Args& a, PerDeviceOnce& once, cudaStream_t s) {
  if (smem_optin(once, kern, kSmemSm - kSmemCta) != cudaSuccess) return GPT2_ERR_CUDA;
  const int bytes = (a.V + 7) / 8 * 16;
  const int per_sm = std::min(32 / G, kSmemSm / (bytes + kSmemCta));
  const int grid = std::min(a.N, device_sm_count() * per_sm);
  return launch_pdl(kern, dim3(grid), dim3(32 * G), bytes, s, a) == cudaSuccess ? GPT2_OK : GPT2_ERR_CUDA;
}

inline int launched(cudaError_t e) { return e == cudaSuccess ? GPT2_OK : GPT2_ERR_CUDA; }

inline int policy_loss(const PolicyArgs& a, cudaStream_t s) {
  if (a.part) return launched(launch_pdl(policy_streamed_kernel<8, true>, dim3(a.N), dim3(256), 0, s, a));
  return with_warps(a.V, [&](auto g) {
    constexpr int G = decltype(g)::value;
    if constexpr (G > 0) {
      static PerDeviceOnce once;
      return launch_pipe<G>(policy_loss_kernel<G>, a, once, s);
    } else {
      return launched(launch_pdl(policy_streamed_kernel<16, false>, dim3(a.N), dim3(512), 0, s, a));
    }
  });
}

inline int row_logps(const RowArgs& a, cudaStream_t s) {
  if (a.part) return launched(launch_pdl(row_logp_streamed_kernel<1, true>, dim3(a.N), dim3(32), 0, s, a));
  return with_warps(a.V, [&](auto g) {
    constexpr int G = decltype(g)::value;
    if constexpr (G > 0) {
      static PerDeviceOnce once;
      return launch_pipe<G>(row_logp_kernel<G>, a, once, s);
    } else {
      return launched(launch_pdl(row_logp_streamed_kernel<16, false>, dim3(a.N), dim3(512), 0, s, a));
    }
  });
}

// What follows the rows' log-probabilities: the pairs' losses, and with a.dlogits the
// gradients. Times of a whole call on the device (captured), and from the host one by one.
//
// A row a warp where rows are many and short, else a row a CTA. 512 rows of 1,024 ids 7.8 us
// against 6.7, 1,024 of 2,048 11.0 against 9.5; 1,536 of 2,048 11.8 against 12.9, 4,096 of
// 4,608 25.2 against 28.9; the long end of the rule: 1,536 of 6,144 19.4 against 18.5, 2,048
// of 6,144 21.0 either way, 4,096 of 8,192 37.7 against 39.0, 8,192 of 12,288 107 against 106.
//
// A pair's coefficient is formed in the gradient's launch where N rows add up no more than
// 8 MB of log-probabilities however the pairs divide them (all in one pair: N / rows CTAs
// times N), a launch of its own otherwise. From the host a launch costs 2 us: 256 rows of
// 1,000 ids 11.6 us against 13.6, 1,206 of 8,449 17.8 against 19.0; on the device 1,536 of 2,048 11.8 us
// against 12.6, and above the bound 4,096 of 1,024 13.4 against 12.0, with nearly all rows in
// one of 4 pairs 16.1 against 13.5 (8,192 of 5,120, 256 MB: 79 against 61). A row a warp and
// longer rows take the launch (2,048 of 4,608 22.3 against 18.4), as do rows over 16,384 ids
// (2 of 2 x 200 x 30,000 29.0 against 27.8).
inline int pairs(PairGradArgs a, PairArgs pa, float2* coef, cudaStream_t s, int* launches = nullptr) {
  const int P = pa.n_pairs = a.n_seq / 2;
  const int rows = a.N > 1024 && a.Vp <= std::min(3L * a.N, 10240L) ? 4 : 1;   // a CTA's
  if (a.dlogits && a.Vp <= (rows == 4 ? 2048 : 16384) && (long)a.N * a.N / rows <= 1 << 21) {
    if (launches) *launches += 1;
    pa.coef = nullptr;
    return rows == 4
               ? launched(launch_pdl(pair_grad_kernel<1, true>, dim3(P + (a.N + 3) / 4), dim3(128), 0, s, a, pa))
               : launched(launch_pdl(pair_grad_kernel<4, true>, dim3(P + a.N), dim3(128), 0, s, a, pa));
  }
  if (launches) *launches += a.dlogits ? 2 : 1;
  pa.coef = coef;
  const int st = launched(launch_pdl(pair_kernel, dim3(P), dim3(kPairThreads), 0, s, pa));
  if (st != GPT2_OK || !a.dlogits) return st;
  return rows == 4 ? launched(launch_pdl(pair_grad_kernel<1, false>, dim3((a.N + 3) / 4), dim3(128), 0, s, a, pa))
                   : launched(launch_pdl(pair_grad_kernel<8, false>, dim3(a.N), dim3(256), 0, s, a, pa));
}

// Workspace: the rows' (c, S), then the pairs' coefficients.
inline size_t preference_workspace(int N, int P) { return (size_t)N * 8 + (size_t)P * 8; }

}  // namespace pt
