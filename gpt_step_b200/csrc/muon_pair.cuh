// All Newton-Schulz rounds of a batch of matrices in one cooperative launch on CTA
// pairs (cta_group::2), output tiles of 256 x BN.
//
// A round is three products: A = X X^T, P = a I + b A + c A A, X <- P X (+ a lo, see
// muon.cuh). The tiles of all of them stand in one list, ordered by round, product,
// matrix, and pair k takes tiles k, k + pairs, ... A tile waits only for its own
// matrix's previous product (a counter of finished tiles in global memory), so the
// last wave of one product runs beside the first of the next, and 15 launches with
// their fills and drains are one. The wait ends: every tile waits only for earlier
// ones, every pair works in order, and the launch is cooperative, so all are resident.
//
// Inside a pair: a TMA warp, an issuing warp, a warp that looks whether the next tiles'
// inputs are finished, and eight epilogue warps; two accumulators in tensor memory, so that
// a tile's epilogue runs under the next tile's main loop. A and P are symmetric: only tiles
// that touch or lie below the diagonal are computed, and a chunk below it is staged a second
// time turned over and stored to its mirror image. The a I of P stands in P's fp16 values:
// rounding P near 0.7 costs less than rounding P - a I near -2.8, and the last product then
// reads nothing but lo.
//
// What bounds it: large matrices the tensor pipe, not all of the time (16 x 1,536 x 6,144:
// 4.36 to 4.5 ms, 0.86 PFLOP/s of the products with symmetric ones counted half, 0.62 of what a
// GEMM sustains under the power limit; diagonal tiles computed whole are 6% of it, the rest has
// not been taken apart); 768 rows the
// shared memory, whose bandwidth the operands take whole at the full tensor rate (64 bytes a
// clock in and out) and an APPLY tile's hi, lo and aux boxes half as much again (tile 6.4 us
// against 4.5 of main loop; 12 x 2,304 x 768: 458 us); small ones the
// latency of a product, 5 to 7 us: loads and MMA 1.8, epilogue 2, its stores in memory and
// seen by the next product 1.5 (3 x 333 x 517: 117 us). Measured and rejected, against 124 us
// and 461 us of the kernel as it was then: results
// by 16-byte stores out of the boxes (3 x 333 x 517 145 us, 12 x 2,304 x 768 500 us), by
// 32-byte stores of a row a lane (144, 575), sixteen epilogue warps with a box each (139,
// 483), three launches a round (146, 483).
#pragma once
#include "gemm2sm.cuh"
#include "muon.cuh"

namespace muon {
namespace pair {

constexpr int kEpiWarps = 8, kThreads = 32 * (3 + kEpiWarps), kTileM = 256;
constexpr int kWarpBytes = 8192;                    // an epilogue warp's 32 x 32 boxes: two for each of two outputs
constexpr int kSignals = 2 * kEpiWarps;             // a tile's epilogue warps

template <int BN>
struct Cfg {
  static constexpr int kStages = BN == 256 ? 5 : 6;
  static constexpr int kABytes = 128 * BK * 2, kBBytes = BN / 2 * BK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kSmem = kStages * kStageBytes + kEpiWarps * kWarpBytes + 2048;
};

enum Product : int { GRAM = 0, POLY = 1, APPLY = 2 };

struct Maps {
  CUtensorMap a_x[2], b_x[2], c_x[2];   // X by rows of 128, by rows of BN / 2, by 64 x 64 columns
  CUtensorMap a_a, b_a, a_p;            // A by rows (both operands), P by rows
  CUtensorMap out_x[2], out_lo, out_a, out_p, out;   // boxes of 32 x 32
};

struct Params {
  int n, m, ld_x, ld_a, batch, steps;
  int tiles_m, sym, full;               // row tiles; tiles of a symmetric product, of the last one
  const __half *lo, *a;
  uint32_t* count;                      // [batch][3] signals of finished tiles
  bf16* result;
  long result_stride;
  int rows, cols, tma_out;              // tma_out: its rows are whole 16-byte pieces
  int* err;
};

GPT2_DEV void load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
GPT2_DEV void store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}

// One tile of the list.
struct Tile {
  int round, product, z, ti, tj;
};

template <int BN>
GPT2_DEV Tile tile_at(const Params& p, int t) {
  Tile r;
  const int gram = p.batch * p.sym, per_round = 2 * gram + p.batch * p.full;
  r.round = t / per_round;
  int i = t - r.round * per_round;
  r.product = i < gram ? GRAM : i < 2 * gram ? POLY : APPLY;
  i -= r.product * gram;
  const int per = r.product == APPLY ? p.full : p.sym;
  r.z = i / per;
  i -= r.z * per;
  if (r.product == APPLY) {
    r.tj = i / p.tiles_m;
    r.ti = i - r.tj * p.tiles_m;
  } else {
    // row tile ti has (ti + 1) * kTileM / BN column tiles, as far as the matrix goes
    constexpr int W = kTileM / BN;
    r.ti = 0;
    while (W * (r.ti + 1) * (r.ti + 2) / 2 <= i) ++r.ti;
    r.tj = i - W * r.ti * (r.ti + 1) / 2;
  }
  return r;
}

// Waits until the products that `t` reads are finished: false if it gave up. `idle`:
// sleep between looks.
GPT2_DEV bool wait_inputs(const Params& p, const Tile& t, bool idle) {
  if (t.round == 0 && t.product == GRAM) return true;
  const uint32_t* c = p.count + t.z * 3;
  uint32_t want;
  if (t.product == GRAM) {
    c += APPLY;
    want = (uint32_t)(t.round * p.full * kSignals);
  } else {
    c += t.product - 1;
    want = (uint32_t)((t.round + 1) * p.sym * kSignals);
  }
  unsigned long long t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(c) : "memory");
    if (v >= want) return true;
    if ((it & 63u) == 63u) {
      if (*(volatile int*)p.err & DEVERR_TIMEOUT) return false;
      const unsigned long long now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kWaitLimitNs) {
        atomicOr(p.err, DEVERR_TIMEOUT);
        return false;
      }
    }
    if (idle) __nanosleep(64);
  }
}

GPT2_DEV bool is_ready(uint32_t at, uint32_t k) {
  uint32_t v;
  asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v > k;
}

// Waits until the count at a shared-memory address exceeds k: false if it gave up.
GPT2_DEV bool wait_ready(uint32_t at, uint32_t k, int* err) {
  unsigned long long t0 = 0;
  for (uint32_t it = 0;; ++it) {
    if (is_ready(at, k)) return true;
    if ((it & 1023u) == 1023u) {
      if (*(volatile int*)err & DEVERR_TIMEOUT) return false;
      const unsigned long long now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kWaitLimitNs) {
        atomicOr(err, DEVERR_TIMEOUT);
        return false;
      }
    }
  }
}

// 16-byte chunk j of row r in a 32 x 32 box of 64-byte rows, 64-byte swizzle.
GPT2_DEV uint32_t box_at(int r, int j) { return (uint32_t)(r * 64 + ((j ^ ((r >> 1) & 3)) << 4)); }

// A lane's 32 values (its row) down a column of the box: the box turned over.
GPT2_DEV void stage_turned(uint8_t* box, int lane, const uint32_t (&w)[16]) {
  const uint32_t at = smem_u32(box) + (lane & 7) * 2;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    asm volatile(
        "{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tst.shared.b16 [%0], lo;\n\tst.shared.b16 [%1], hi;\n\t}" ::"r"(
            at + box_at(2 * i, lane >> 3)),
        "r"(at + box_at(2 * i + 1, lane >> 3)), "r"(w[i])
        : "memory");
  }
}

// Whether the phase has completed, without waiting.
GPT2_DEV bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

template <int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ns_rounds_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using C = Cfg<BN>;
  constexpr int S = C::kStages;
  extern __shared__ __align__(1024) uint8_t pair_smem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pair_smem) + 1023) & ~uintptr_t(1023));
  uint8_t* epi = smem + S * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + kEpiWarps * kWarpBytes);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  uint32_t* ready_slot = tmem_slot + 1;                // tiles of this CTA whose inputs are finished

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = gemm2::cluster_rank();
  const bool leader = rank == 0;
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
  const int total = p.steps * p.batch * (2 * p.sym + p.full);

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), kSignals);
    }
    *ready_slot = 0;
    mbar_init(smem_u32(done), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    gemm2::tmem_alloc2(smem_u32(tmem_slot), 2 * BN);
    gemm2::tmem_relinquish2();
  }
  tc_fence_before();
  gemm2::cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot, ready = smem_u32(ready_slot);

  if (warp == 2) {
    // looks ahead of the loads: a tile's inputs are usually finished before its turn
    if (lane == 0) {
      uint32_t k = 0;
      for (int t = cid; t < total; t += ncl) {
        if (!wait_inputs(p, tile_at<BN>(p, t), true)) break;
        ++k;
        asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(ready), "r"(k) : "memory");
      }
    }
  } else if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, k = 0;
      bool ok = true;
      for (int t = cid; t < total && ok; t += ncl, ++k) {
        const Tile tl = tile_at<BN>(p, t);
        const int cur = tl.round & 1;
        const CUtensorMap* ma = tl.product == GRAM ? &maps.a_x[cur] : tl.product == POLY ? &maps.a_a : &maps.a_p;
        const CUtensorMap* mb = tl.product == GRAM ? &maps.b_x[cur] : tl.product == POLY ? &maps.b_a : &maps.c_x[cur];
        const int nkb = (tl.product == GRAM ? p.ld_x : p.ld_a) / BK;
        const int m0 = tl.ti * kTileM + 128 * rank, n0 = tl.tj * BN + BN / 2 * rank;
        // (a tile that has to wait is seen sooner here than through the looking-ahead warp)
        if (!is_ready(ready, k) && !wait_inputs(p, tl, false)) break;
        asm volatile("fence.proxy.async;" ::: "memory");   // the loads come after the wait
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1, p.err)) { ok = false; break; }
          const uint32_t fb = gemm2::mapa_shared(smem_u32(&full[stage]), 0);
          if (leader) mbar_arrive_expect_tx(smem_u32(&full[stage]), 2 * C::kStageBytes);
          const uint32_t sa = smem_u32(smem + stage * C::kStageBytes), sb = sa + C::kABytes;
          load_3d(sa, ma, fb, kb * BK, m0, tl.z);
          if (tl.product != APPLY) {
            load_3d(sb, mb, fb, kb * BK, n0, tl.z);
          } else {
#pragma unroll
            for (int j = 0; j < BN / 128; ++j) load_3d(sb + j * 8192, mb, fb, n0 + 64 * j, kb * BK, tl.z);
          }
          if (++stage == S) { stage = 0; phase ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = cid; t < total && ok; t += ncl, ++it) {
        const Tile tl = tile_at<BN>(p, t);
        const int nkb = (tl.product == GRAM ? p.ld_x : p.ld_a) / BK;
        const bool mn = tl.product == APPLY;
        const uint32_t idesc = idesc_f16_f32(kTileM, BN, mn);
        const int acc = it & 1;
        if (!mbar_wait(smem_u32(&tempty[acc]), ((it >> 1) & 1) ^ 1, p.err)) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * BN;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(smem_u32(&full[stage]), phase, p.err)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * C::kStageBytes), sb = sa + C::kABytes;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            gemm2::tc_mma2_bf16(d, smem_desc_sw128(sa + kk * 32, 16, 1024),
                                mn ? smem_desc_sw128(sb + kk * 2048, 8192, 1024)
                                   : smem_desc_sw128(sb + kk * 32, 16, 1024),
                                idesc, (kb | kk) ? 1u : 0u);
          gemm2::tc_commit2_mc(smem_u32(&empty[stage]), 0x3);
          if (++stage == S) { stage = 0; phase ^= 1; }
        }
        gemm2::tc_commit2_mc(smem_u32(&tfull[acc]), 0x3);
      }
      gemm2::tc_commit2_mc(smem_u32(done), 0x1);
      mbar_wait(smem_u32(done), 0, p.err);
    }
  } else {
    constexpr int kCols = BN / 2;                   // of a warp
    const int q = warp & 3, part = (warp - 3) >> 2; // tensor-memory lane quarter, half of the columns
    uint8_t* wbuf = epi + (warp - 3) * kWarpBytes;
    uint32_t nstore = 0;
    const uint32_t te0 = gemm2::mapa_shared(smem_u32(&tempty[0]), 0), te1 = gemm2::mapa_shared(smem_u32(&tempty[1]), 0);
    const bool tall = p.rows > p.cols;
    uint32_t* pending = nullptr;                    // the counter of a tile stored but not signalled
    // What this warp stored is in memory (with `newer`, but for the latest group): say so.
    // The wait makes the stores visible to this thread, the release to whoever acquires the
    // count and, behind its proxy fence, to its loads.
    auto signal = [&](bool newer) {
      if (newer) gemm::bulk_wait_all<1>();
      else gemm::bulk_wait_all<0>();
      asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(pending) : "memory");
      pending = nullptr;
    };
    int it = 0;
    for (int t = cid; t < total; t += ncl, ++it) {
      const Tile tl = tile_at<BN>(p, t);
      const int z = tl.z, acc = it & 1;
      const bool sym = tl.product != APPLY, last = !sym && tl.round + 1 == p.steps;
      const bool put_lo = !sym && tl.round + 1 < p.steps - 2;
      const bool mirror = sym && (tl.tj + 1) * BN <= tl.ti * kTileM;
      const bool turn = last && tall;               // the result is stored by columns of X
      const CUtensorMap* mo = tl.product == GRAM   ? &maps.out_a
                              : tl.product == POLY ? &maps.out_p
                              : last               ? &maps.out
                                                   : &maps.out_x[(tl.round & 1) ^ 1];
      const int ld = sym ? p.ld_a : p.ld_x;
      const int row0 = tl.ti * kTileM + 128 * rank + q * 32, row = row0 + lane;
      const int n0 = tl.tj * BN + part * kCols;
      const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16) + acc * BN + part * kCols;
      // POLY adds b A, APPLY a lo
      const __half* aux = tl.product == POLY ? p.a : !sym && tl.round < p.steps - 2 ? p.lo : nullptr;
      const float aux_f = tl.product == POLY ? kB : kA;
      const float mul = tl.product == POLY ? kC * kInvScale : last ? kInvScale * kInvScale : kInvScale;
      uint4 ah[4];
      // a chunk's aux, coalesced: lane l loads 16-byte piece l & 3 of rows (l >> 2) + 8 i
      auto fetch_aux = [&](int n) {
        if (n >= ld) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = row0 + (lane >> 2) + 8 * i;
          const size_t at = ((size_t)z * p.n + rr) * ld + n + 8 * (lane & 3);
          ah[i] = rr < p.n ? __ldcg(reinterpret_cast<const uint4*>(aux + at)) : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      if (aux) {                   // under the tile's main loop
        int ok = 1;
        if (lane == 0) ok = wait_ready(ready, it, p.err);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        __syncwarp();
        if (!ok) break;
        fetch_aux(n0);
      }
      if (!mbar_wait(smem_u32(&tfull[acc]), (it >> 1) & 1, p.err)) break;
      tc_fence_after();
      uint32_t vr[32];
      tmem_ld32_async(t_row, vr);
#pragma unroll 1
      for (int c = 0; c < kCols; c += 32) {
        const int n = n0 + c;
        tmem_wait_ld();
        if (n >= ld) break;        // ld is a multiple of 64: whole chunks, the same in the warp
        float2 v[16];              // paired fp32 arithmetic: two columns an instruction
#pragma unroll
        for (int i = 0; i < 16; ++i)
          v[i] = f2_mul(make_float2(__uint_as_float(vr[2 * i]), __uint_as_float(vr[2 * i + 1])), make_float2(mul, mul));
        uint8_t* box = wbuf + (nstore & 1) * 2048;
        uint8_t* box2 = box + 4096;
        ++nstore;
        // the stores from these boxes two chunks ago have read them
        if (lane == 0) gemm::bulk_wait_read<1>();
        __syncwarp();
        if (aux) {                 // turned into one row a lane through the box
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(box + box_at((lane >> 2) + 8 * i, lane & 3)) = ah[i];
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 u = *reinterpret_cast<const uint4*>(box + box_at(lane, j));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&w[h]));
              v[4 * j + h] = f2_fma(make_float2(aux_f, aux_f), g, v[4 * j + h]);
            }
          }
          __syncwarp();
          if (c + 32 < kCols) fetch_aux(n + 32);
        }
        if (c + 32 < kCols) tmem_ld32_async(t_row + c + 32, vr);
        if (tl.product == POLY && row0 == n) {     // the chunk on the diagonal
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (2 * i == lane && row < p.n) v[i].x += kA * kScale;
            if (2 * i + 1 == lane && row < p.n) v[i].y += kA * kScale;
          }
        }
        uint32_t w[16];
        if (last) {
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[i].x, v[i].y);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack_half2(v[i].x, v[i].y);
        }
        // (each form once: a launch pays for the instructions it brings in, 0.4 us of 117 here)
        if (!turn) gemm::stage_row(box, lane, w);
        if (mirror || turn) stage_turned(turn ? box : box2, lane, w);
        if (put_lo) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            w[i] = pack_half2(v[i].x - h.x, v[i].y - h.y);
          }
          gemm::stage_row(box2, lane, w);
        }
        if (last && !p.tma_out) {  // rows at any alignment: a warp stores one row's columns at a time
          bf16* res = p.result + (size_t)z * p.result_stride;
          __syncwarp();
          const int r0 = turn ? n : row0, c0 = turn ? row0 : n;
#pragma unroll 4
          for (int r = 0; r < 32 && r0 + r < p.rows; ++r)
            if (c0 + lane < p.cols)
              res[(size_t)(r0 + r) * p.cols + c0 + lane] =
                  *reinterpret_cast<const bf16*>(box + box_at(r, lane >> 3) + (lane & 7) * 2);
          if (lane == 0) gemm::bulk_commit();
          continue;
        }
        gemm::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (row0 < p.n && (!last || n < p.m)) {
            store_3d(mo, smem_u32(box), turn ? row0 : n, turn ? n : row0, z);
            if (put_lo) store_3d(&maps.out_lo, smem_u32(box2), n, row0, z);
          }
          // the mirror image; its rows n .. ld - 1 are the padding columns, and 0
          if (mirror && row0 < ld && n < p.n) store_3d(mo, smem_u32(box2), row0, n, z);
          gemm::bulk_commit();
          if (pending) signal(true);
        }
      }
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        gemm2::mbar_arrive_remote(acc ? te1 : te0);
        if (pending) signal(false);                // a tile without chunks of its own came in between
        if (!last) {
          pending = p.count + z * 3 + tl.product;
          // at once if the next tile is not there yet, else under its first chunk
          const int nx = it + 1;
          if (!mbar_test(smem_u32(&tfull[nx & 1]), (nx >> 1) & 1)) signal(false);
        }
      }
    }
    if (lane == 0) {
      if (pending) signal(false);
      gemm::bulk_wait_all<0>();
    }
  }

  tc_fence_before();
  gemm2::cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    gemm2::tmem_dealloc2(tmem, 2 * BN);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
// [batch][rows][cols] (row stride ld, matrices `apart`) of 16-bit elements; boxes of
// box_x columns x box_y rows of one matrix, 128-byte swizzle at 64 columns, else 64-byte
inline bool map_3d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, long cols, long ld, long rows, long apart,
                   int batch, int box_x, int box_y) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
  cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)apart * 2};
  cuuint32_t box[3] = {(cuuint32_t)box_x, (cuuint32_t)box_y, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, dt, 3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_x == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN>
int launch(const Maps& maps, const Params& p, cudaStream_t s) {
  using C = Cfg<BN>;
  static PerDeviceOnce once;
  static int most[PerDeviceOnce::kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= PerDeviceOnce::kMaxDevices) return GPT2_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (device_sm_count() / 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;   // all pairs resident: tiles wait for one another
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = once.run([&] {
    const cudaError_t e1 = cudaFuncSetAttribute(reinterpret_cast<const void*>(ns_rounds_kernel<BN>),
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    return e1 != cudaSuccess ? e1 : cudaOccupancyMaxActiveClusters(&most[dev], ns_rounds_kernel<BN>, &cfg);
  });
  if (e != cudaSuccess || most[dev] < 1) return GPT2_ERR_CUDA;
  const int widest = p.batch * std::max(p.sym, p.full);
  cfg.gridDim = dim3(2 * std::min(widest, most[dev]));
  return cudaLaunchKernelEx(&cfg, ns_rounds_kernel<BN>, maps, p) == cudaSuccess ? GPT2_OK : GPT2_ERR_CUDA;
}

// The rounds on X in the workspace (prepare_x).
template <int BN>
int rounds_bn(const Work& w, char* base, bf16* out, long out_stride, int batch, int rows, int cols, int steps, int* err,
              cudaStream_t s) {
  __half* xh[2] = {reinterpret_cast<__half*>(base + w.x0), reinterpret_cast<__half*>(base + w.x1)};
  __half* lo = reinterpret_cast<__half*>(base + w.lo);
  __half* a = reinterpret_cast<__half*>(base + w.a);
  __half* q = reinterpret_cast<__half*>(base + w.q);
  Maps m;
  auto x_map = [&](CUtensorMap* t, const __half* of, int box_x, int box_y) {
    return map_3d(t, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, of, w.ld_x, w.ld_x, w.n, (long)w.n * w.ld_x, batch, box_x, box_y);
  };
  auto a_map = [&](CUtensorMap* t, const __half* of, int box_x, int box_y) {
    return map_3d(t, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, of, w.ld_a, w.ld_a, w.n, (long)w.n * w.ld_a, batch, box_x, box_y);
  };
  bool ok = true;
  for (int i = 0; i < 2; ++i)
    ok = ok && x_map(&m.a_x[i], xh[i], 64, 128) && x_map(&m.b_x[i], xh[i], 64, BN / 2) &&
         x_map(&m.c_x[i], xh[i], 64, 64) && x_map(&m.out_x[i], xh[i], 32, 32);
  ok = ok && a_map(&m.a_a, a, 64, 128) && a_map(&m.b_a, a, 64, BN / 2) && a_map(&m.a_p, q, 64, 128) &&
       x_map(&m.out_lo, lo, 32, 32) && a_map(&m.out_a, a, 32, 32) && a_map(&m.out_p, q, 32, 32);
  if (!ok) return GPT2_ERR_CUDA;
  const long apart = batch > 1 ? out_stride : (long)rows * cols;
  Params p{};
  // the result leaves by TMA where its rows are whole 16-byte pieces
  p.tma_out = (reinterpret_cast<uintptr_t>(out) & 15) == 0 && cols % 8 == 0 && apart % 8 == 0 &&
              map_3d(&m.out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, out, cols, cols, rows, apart, batch, 32, 32);
  if (!p.tma_out) m.out = m.out_a;
  p.n = w.n; p.m = w.m; p.ld_x = w.ld_x; p.ld_a = w.ld_a; p.batch = batch; p.steps = steps;
  p.tiles_m = (w.n + kTileM - 1) / kTileM;
  const int tn = (w.n + BN - 1) / BN;
  constexpr int W = kTileM / BN;
  p.sym = W * p.tiles_m * (p.tiles_m + 1) / 2 - (W * p.tiles_m - tn);   // the last row tile ends with the matrix
  p.full = p.tiles_m * ((w.m + BN - 1) / BN);
  p.lo = lo; p.a = a; p.count = reinterpret_cast<uint32_t*>(base + w.count);
  p.result = out; p.result_stride = out_stride; p.rows = rows; p.cols = cols; p.err = err;
  return launch<BN>(m, p, s);
}

// Tile width: 256, the tensor pipe's better rate, unless a product of the batch then has
// fewer tiles than there are pairs: with 128 an epilogue warp has half as much to do per
// tile, and latency is what counts (1 x 129 x 129: 92 us against 104, 3 x 333 x 517: 122
// against 152, 6 x 1,536 x 384 with 72 tiles: 180 against 198; above, 12 x 768 x 768
// with 108 tiles: 228 us at 256 against 258).
inline int rounds(const Work& w, char* base, bf16* out, long out_stride, int batch, int rows, int cols, int steps,
                  int* err, cudaStream_t s) {
  const long wide = (long)batch * ((w.n + 255) / 256) * ((w.m + 255) / 256);
  return wide >= device_sm_count() / 2
             ? rounds_bn<256>(w, base, out, out_stride, batch, rows, cols, steps, err, s)
             : rounds_bn<128>(w, base, out, out_stride, batch, rows, cols, steps, err, s);
}

}  // namespace pair
}  // namespace muon
