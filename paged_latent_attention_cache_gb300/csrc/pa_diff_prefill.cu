// Differential attention, prefill: any number of new tokens per sequence
// (include/pa_diff.h), on the tensor cores (tcgen05, TMEM, TMA).
//
// A work unit is up to 128 query rows of one kv head: tpc consecutive tokens
// of one sequence x the kv head's grp heads. Its two softmax maps run on the
// two CTAs of a cluster, CTA r with map r: the accumulator of one map is 128 x
// vhs f32, half of a TMEM at vhs 256, so both maps of a unit do not fit one SM
// together with their scores, and each map streams keys of its own anyway.
// The CTAs run apart until the end, where they exchange halves of their
// normalized outputs through distributed shared memory: CTA r takes the
// difference of value channels [r vg / 2, (r + 1) vg / 2), the sums of squares
// of the norm are exchanged the same way, and each writes its channels once.
// Nothing but the output leaves the chip.
//
// Inside a CTA, per tile of 128 keys:
//   warp 8    TMA: key and value rows of the tile through the block table,
//             a ring of stages
//   warp 9    QK^T (S: 128 x 128 f32 in TMEM), PV (A = P from TMEM, O: 128 x vg)
//   warps 0-7 softmax: two threads per row, 64 columns each, held in registers:
//             S is read from TMEM once and is free for the next QK^T before
//             the exponentials start; P (16 bit) goes to one of two buffers
// TMEM columns: O vg <= 256 | S 128 | P 2 x 64.
//
// Bound: per tile and map the MMAs take 128 * 128 * (hs + vhs) / 4096 cycles
// (1536 at 128 / 256, 768 at 64 / 128) and the exponentials 16384 / 16 per SM.
//
// P and the rotated query are rounded to the dtype for the products, as in
// the other prefill kernels; two parts each (as decode takes) would double the
// tensor time here.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "pa_diff_internal.h"
#include "pa_tc_cluster.cuh"

namespace pa {
namespace diff {
namespace {

using namespace pa::tc;

constexpr int kN = 128;             // keys of a tile
constexpr int kSoftWarps = 8;
constexpr int kSoft = kSoftWarps * 32;
constexpr int kProdWarp = 8, kMmaWarp = 9;
constexpr int kPreThreads = 320;
constexpr int kBox = kN * 128;      // bytes of a 64-channel slab of 128 rows
constexpr int kMaxStages = 8;
constexpr size_t kSmemMax = 225 * 1024;

struct PreBars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t s_full, s_free, p_full[2], pv_done[2];
  uint64_t q_tma, q_full, drain;
  uint32_t tmem_base;
  int bad, abort;
};

struct PreArgs {
  Params P;           // what the shared helpers read
  int hs;
  const float* lambda_vectors;
  const void* norm_weight;
  float lambda_init, norm_eps;
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void st_peer4(uint32_t raddr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(raddr), "f"(a), "f"(b),
               "f"(c), "f"(d)
               : "memory");
}
__device__ __forceinline__ void st_peer(uint32_t raddr, float a) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(raddr), "f"(a) : "memory");
}

// The rotation of one query row in place in its swizzled slabs (16-byte chunk
// c of row r at c ^ (r & 7)), by two threads (`part` 0 and 1), in f32, rounded
// once.
template <typename T>
__device__ __noinline__ void rotate_row(uint8_t* q_s, int row, int part, const Params& P,
                                        int64_t pos) {
  auto at = [&](int d0) -> uint4* {
    return reinterpret_cast<uint4*>(q_s + (d0 >> 6) * kBox + row * 128 +
                                    ((((d0 >> 3) & 7) ^ (row & 7)) << 4));
  };
  const int half = P.rd >> 1;
  const T* crow = reinterpret_cast<const T*>(P.cos_cache) + pos * half;
  const T* srow = reinterpret_cast<const T*>(P.sin_cache) + pos * half;
  if (P.interleaved) {
    for (int d0 = P.ro + part * 8; d0 < P.ro + P.rd; d0 += 16) {
      float a[8], none[8];
      unpack8<T>(*at(d0), a);
      rope8<T>(a, none, d0, P.ro, P.rd, 1, crow, srow);
      *at(d0) = pack8<T>(a);
    }
    return;
  }
  for (int d0 = P.ro + part * 8; d0 < P.ro + half; d0 += 16) {
    float a[8], b[8], na[8], nb[8];
    unpack8<T>(*at(d0), a);
    unpack8<T>(*at(d0 + half), b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      na[e] = a[e];
      nb[e] = b[e];
    }
    rope8<T>(na, b, d0, P.ro, P.rd, 0, crow, srow);
    rope8<T>(nb, a, d0 + half, P.ro, P.rd, 0, crow, srow);
    *at(d0) = pack8<T>(na);
    *at(d0 + half) = pack8<T>(nb);
  }
}

template <typename T, bool CAP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPreThreads, 1)
diff_prefill_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const __grid_constant__ CUtensorMap qmap, const __grid_constant__ PreArgs A) {
  const Params& P = A.P;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Work work;
  __shared__ PreBars bars_s;
  __shared__ float s_max[2][kRows];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint8_t* q_s = smem;
  uint8_t* k_s = smem + P.q_bytes;  // stage: key slabs, then value slabs, kN rows each
  // in the query's place, once the last QK^T is done: the halves' sums, and
  // [CTA * 2 + half] sums of squares, the peer's too
  float (*s_sum)[kRows] = reinterpret_cast<float (*)[kRows]>(q_s);
  float (*s_ss)[kRows] = s_sum + 2;
  PreBars* bars = &bars_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slabs = P.slabs, vslabs = P.vslabs, vg = P.vg, stages = P.stages;
  const int kvh = P.kvh, grp = P.grp, vhs = P.vhs;
  const int map = (int)cluster_rank();
  const int pair = blockIdx.x >> 1;
  const int unit = pair / kvh, gk = pair - unit * kvh;

  if (warp == 0) {
    if (!P.early) grid_dep_wait();
    Work w = prefill_group_warp(P, unit, P.tpc);
    if (w.status == 0) {
      const int64_t pos_hi = w.pos + w.ntok - 1;
      const bool bad_ctx = w.past < 0 || pos_hi >= (int64_t)P.max_blocks * P.bs || w.t < 0 ||
                           w.t + w.ntok > P.num_tokens;
      const bool bad_pos = P.rd > 0 && pos_hi >= P.cos_rows;
      const int64_t lo_key = P.window >= 0 ? max((int64_t)0, w.pos - P.window) : 0;
      w.t_begin = lo_key / kN;
      w.t_end = pos_hi / kN + 1;
      if (bad_ctx || bad_pos) {
        if (lane == 0 && gk == 0 && map == 0)
          raise_flag(P.err_flags, bad_ctx ? PA_DEVERR_CONTEXT : PA_DEVERR_POSITION);
        const int nt = w.t < 0 ? 0 : (int)max((int64_t)0, min((int64_t)w.ntok, P.num_tokens - w.t));
        if (map == 0)
          for (int i = lane; i < nt * grp * vhs; i += 32) {
            const int tt = i / (grp * vhs), rem = i - tt * grp * vhs;
            reinterpret_cast<T*>(P.out)[((w.t + tt) * P.H + gk * grp) * (int64_t)vhs + rem] =
                Half<T>::from_f32(0.f);
          }
        w.status = 2;
      }
    }
    if (lane == 0) work = w;
  } else if (warp == 1 && lane == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1);
      mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    mbar_init(smem_u32(&bars->s_full), 1);
    mbar_init(smem_u32(&bars->s_free), kSoft);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->p_full[i]), kSoft);
      mbar_init(smem_u32(&bars->pv_done[i]), 1);
    }
    mbar_init(smem_u32(&bars->q_tma), 1);
    mbar_init(smem_u32(&bars->q_full), kSoft);
    mbar_init(smem_u32(&bars->drain), 1);
    bars->bad = 0;
    bars->abort = 0;
    fence_barrier_init();
  } else if (warp == kProdWarp && lane == 0) {
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
    prefetch_tmap(&qmap);
  } else if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  if (warp != 0 && !P.early) grid_dep_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const uint32_t col_s = vg, col_p = vg + kN;
  volatile int* abort = &bars->abort;
  const Work W = work;
  const bool run = W.status == 0;
  const int ntok = W.ntok, rows = run ? ntok * grp : 0;
  const int n = run ? (int)max((int64_t)0, W.t_end - W.t_begin) : 0;

  // what the softmax threads carry to the epilogue
  const int half = warp >> 2, row = (warp & 3) * 32 + lane;
  const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  const bool live = warp < kSoftWarps && (warp & 3) * 32 < rows;
  float coef = 0.f;
  bool ok = true;

  if (run) {
    const int64_t t = W.t, pos = W.pos, t_begin = W.t_begin;
    const int64_t pos_hi = pos + ntok - 1;
    const int64_t lo = P.window >= 0 ? max((int64_t)0, pos - P.window) : 0;
    const int64_t lo_hi = P.window >= 0 ? max((int64_t)0, pos_hi - P.window) : 0;

    if (warp < kSoftWarps) {
      // =================== softmax ===================
      const int64_t pos_r = row < rows ? pos + row / grp : -1;
      const int64_t lo_r = P.window >= 0 ? max((int64_t)0, pos_r - P.window) : 0;
      float lam = 0.f;
      if (map == 1) {
        float d0 = 0.f, d1 = 0.f;
        const float* lv = A.lambda_vectors;
        for (int d = lane; d < A.hs; d += 32) {
          d0 = fmaf(lv[d], lv[A.hs + d], d0);
          d1 = fmaf(lv[2 * A.hs + d], lv[3 * A.hs + d], d1);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          d0 += __shfl_xor_sync(0xffffffffu, d0, o);
          d1 += __shfl_xor_sync(0xffffffffu, d1, o);
        }
        lam = expf(d0) - expf(d1) + A.lambda_init;
      }
      ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->q_tma), 0, abort, P.err_flags));
      if (ok && row < rows && P.rd > 0) rotate_row<T>(q_s, row, half, P, pos_r);
      fence_proxy_async();
      mbar_arrive(smem_u32(&bars->q_full));

      float m_used = -INFINITY, l = 0.f;
      const float sl = CAP ? 1.f : P.scale_log2;
      // Every warp goes through all n tiles and meets its partner of the
      // quadrant twice in each; after a wait that gave up (ok false) it does
      // nothing else.
      for (int k = 0; k < n; ++k) {
        const int pb = k & 1;
        const int64_t j0 = (t_begin + k) * kN;
        const bool edge = j0 < lo_hi || j0 + kN - 1 > pos;
        if (ok)
          ok = __all_sync(0xffffffffu,
                          wait_bar(smem_u32(&bars->s_full), k & 1, abort, P.err_flags));
        uint32_t s0[32], s1[32];
        if (live && ok) {
          tc_fence_after();
          tmem_ld32_nowait(lane_addr + col_s + half * 64, s0);
          tmem_ld32_nowait(lane_addr + col_s + half * 64 + 32, s1);
          tmem_wait_ld();
          reg_fence(s0);
          reg_fence(s1);
          tc_fence_before();
        }
        if (ok) mbar_arrive(smem_u32(&bars->s_free));  // the next QK^T may overwrite S
        if (edge && ok) {  // zero the value rows of keys no row of the unit sees
          uint8_t* vst = k_s + (k % stages) * P.stage_bytes + P.k_bytes;
          for (int i = tid; i < kN * vslabs * 8; i += kSoft) {
            const int rr = (i >> 3) & (kN - 1);
            const int64_t j = j0 + rr;
            if (j < lo || j > pos_hi)
              *reinterpret_cast<uint4*>(vst + (i >> 10) * kBox + rr * 128 + (i & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
        }
        if (k >= 2 && ok)
          ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->pv_done[pb]),
                                                ((k - 2) >> 1) & 1, abort, P.err_flags));
        float factor = 1.f;
        bool rescale = false;
        if (live && ok) {
          if (edge) {
            const int c0 = (int)min((int64_t)kN, max((int64_t)0, lo_r - j0)) - half * 64;
            const int c1 = (int)max((int64_t)-1, min((int64_t)(kN - 1), pos_r - j0)) - half * 64;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (e < c0 || e > c1) s0[e] = __float_as_uint(-INFINITY);
              if (e + 32 < c0 || e + 32 > c1) s1[e] = __float_as_uint(-INFINITY);
            }
          }
          float v0 = -INFINITY, v1 = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            v0 = fmaxf(v0, __uint_as_float(s0[e]));
            v1 = fmaxf(v1, __uint_as_float(s1[e]));
          }
          s_max[half][row] = fmaxf(v0, v1);
        }
        if (live) named_sync(1 + (warp & 3), 64);
        if (live && ok) {
          const float vmax = fmaxf(s_max[0][row], s_max[1][row]);
          const float mt = !CAP ? vmax * sl
                           : vmax == -INFINITY ? -INFINITY
                                               : P.cap_out * tanh_ex2(vmax * P.cap_in);
          if (m_used == -INFINITY) {
            m_used = mt;  // (nothing but zeros was added before a first visible key)
          } else if (mt > m_used + kRescaleLog2) {
            factor = ex2(m_used - mt);
            m_used = mt;
            l *= factor;
            rescale = true;
          }
          const float mu = m_used == -INFINITY ? 0.f : m_used;
          const ExpArgs E{sl, mu, P.cap_in, P.cap_out, 0.f, 0.f, 0.f, 0.f, 0.f};
          uint32_t pk[16];
          const uint32_t dst = lane_addr + col_p + pb * 64 + half * 32;
          l += exp_chunk<T, CAP ? 2 : 0>(s0, pk, E);
          tmem_st16(dst, pk);
          l += exp_chunk<T, CAP ? 2 : 0>(s1, pk, E);
          tmem_st16(dst + 16, pk);
          if (__any_sync(0xffffffffu, rescale)) {
            // (k >= 1) each half scales half of O, once the PV before has added to it
            ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->pv_done[(k - 1) & 1]),
                                                  ((k - 1) >> 1) & 1, abort, P.err_flags));
            if (ok) {
              tc_fence_after();
#pragma unroll 1
              for (int c = half * (vg >> 1); c < (half + 1) * (vg >> 1); c += 16) {
                uint32_t r[16];
                tmem_ld16(lane_addr + c, r);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  r[e] = __float_as_uint(__uint_as_float(r[e]) * factor);
                tmem_st16(lane_addr + c, r);
              }
            }
          }
          tmem_wait_st();
          tc_fence_before();
        }
        if (live) named_sync(1 + (warp & 3), 64);  // before s_max is used again
        if (ok) mbar_arrive(smem_u32(&bars->p_full[pb]));
      }
      grid_dep_launch();
      if (live) s_sum[half][row] = l;
      named_sync(5, kSoft);
      ok = __all_sync(0xffffffffu, ok && !*abort);
      if (ok && n > 0)
        ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->pv_done[(n - 1) & 1]),
                                              ((n - 1) >> 1) & 1, abort, P.err_flags));
      tc_fence_after();
      const float lt = s_sum[0][row] + s_sum[1][row];
      coef = lt > 0.f ? (map == 0 ? 1.f : lam) / lt : 0.f;
    } else if (warp == kProdWarp) {
      // =================== TMA producer ===================
      if (lane == 0) {
        const uint32_t qb = smem_u32(&bars->q_tma);
        mbar_expect_tx(qb, (uint32_t)(slabs * grp * P.tpc * 128));
        for (int slab = 0; slab < slabs; ++slab)
          tma_load_4d(smem_u32(q_s) + slab * kBox, &qmap, slab * 64, map, gk * grp, (int)t, qb);
      }
      int dirty_from = 0;
      if (P.early && P.own_slots) dirty_from = (int)max((int64_t)0, W.past / kN - t_begin);
      bool waited = !P.early;
      const int nsub = kN / P.box_rows;
      const int32_t* bt = P.block_table + (int64_t)W.b * P.max_blocks;
      const int sh = __ffs(P.bs) - 1;
      int issued = 0, stage = 0;
      uint32_t par = 1;
      for (int k = 0; k < n; ++k) {
        if (!waited && k >= dirty_from) {
          grid_dep_wait();
          waited = true;
        }
        int y = (int)P.num_slots;  // out of range: TMA fills zeros
        if (lane < nsub) {
          const int64_t key0 = (t_begin + k) * kN + (int64_t)lane * P.box_rows;
          if (key0 <= pos_hi && key0 + P.box_rows - 1 >= lo) {
            const int32_t phys = bt[key0 >> sh];
            if (phys >= 0 && phys < P.num_blocks) {
              y = (int)((int64_t)phys * P.bs + (key0 & (int64_t)(P.bs - 1)));
            } else {
              bars->bad = 1;
              raise_flag(P.err_flags, PA_DEVERR_BLOCK);
            }
          }
        }
        if (k >= stages) {
          bool okw = true;
          if (lane == 0) okw = wait_bar(smem_u32(&bars->empty[stage]), par, abort, P.err_flags);
          if (!__shfl_sync(0xffffffffu, okw ? 1 : 0, 0)) break;
        }
        if (lane == 0) mbar_expect_tx(smem_u32(&bars->full[stage]), (uint32_t)P.stage_bytes);
        __syncwarp();
        if (lane < nsub) {
          const uint32_t full = smem_u32(&bars->full[stage]);
          const uint32_t dst0 = smem_u32(k_s + stage * P.stage_bytes) + lane * P.box_rows * 128;
#pragma unroll 1
          for (int slab = 0; slab < slabs; ++slab)
            tma_load_3d(dst0 + slab * kBox, &kmap, slab * 64, 2 * gk + map, y, full);
#pragma unroll 1
          for (int slab = 0; slab < vslabs; ++slab)
            tma_load_3d(dst0 + P.k_bytes + slab * kBox, &vmap, slab * 64, gk, y, full);
        }
        issued = k + 1;
        if (++stage == stages) {
          stage = 0;
          par ^= 1;
        }
        __syncwarp();
      }
      if (!waited) grid_dep_wait();
      if (*abort && lane == 0) {
        drain_wait(smem_u32(&bars->q_tma), 0, P.err_flags);
        for (int st = 0; st < stages && st < issued; ++st)
          drain_wait(smem_u32(&bars->full[st]), ((issued - 1 - st) / stages) & 1, P.err_flags);
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // =================== MMA issuer ===================
      if (lane == 0) {
        constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
        constexpr uint32_t id_qk = idesc_f16(kBf16, kRows, kN, false);
        const uint32_t id_pv = idesc_f16(kBf16, kRows, vg, true);
        const int nk = P.hs >> 4;
        const uint64_t q_desc = sdesc(smem_u32(q_s), 16, 1024);
        const uint32_t k_base = smem_u32(k_s);
        bool go = wait_bar(smem_u32(&bars->q_full), 0, abort, P.err_flags);
        if (go) {
          tc_fence_after();
          int kq = 0, kp = 0, sq = 0, sp = 0;
          uint32_t fpar = 0;
          const uint64_t t0 = globaltimer();
          uint32_t spins = 0;
          while (kp < n) {
            bool progressed = false;
            // QK^T of the next tile first: the softmax warps wait for it, and
            // it runs while they turn the tile before into probabilities
            if (kq < n && kq <= kp + 1 &&
                (kq == 0 || mbar_test_wait(smem_u32(&bars->s_free), (kq - 1) & 1)) &&
                mbar_test_wait(smem_u32(&bars->full[sq]), fpar)) {
              tc_fence_after();
              const uint64_t kd = sdesc(k_base + sq * P.stage_bytes, 16, 1024);
              for (int kk = 0; kk < nk; ++kk) {
                const uint32_t o = (uint32_t)(kk >> 2) * (kBox >> 4) + (uint32_t)(kk & 3) * 2;
                mma_ss(tmem + col_s, q_desc + o, kd + o, id_qk, kk > 0 ? 1u : 0u);
              }
              tc_commit(smem_u32(&bars->s_full));
              ++kq;
              if (++sq == stages) {
                sq = 0;
                fpar ^= 1;
              }
              progressed = true;
            }
            if (kp < kq && mbar_test_wait(smem_u32(&bars->p_full[kp & 1]), (kp >> 1) & 1)) {
              tc_fence_after();
              const uint64_t vd = sdesc(k_base + sp * P.stage_bytes + P.k_bytes, kBox, 1024);
              const uint32_t pa = tmem + col_p + (kp & 1) * 64;
#pragma unroll
              for (int kk = 0; kk < kN / 16; ++kk)
                mma_ts(tmem, pa + kk * 8, vd + (uint64_t)(kk * 128), id_pv,
                       (kp > 0 || kk > 0) ? 1u : 0u);
              tc_commit(smem_u32(&bars->pv_done[kp & 1]));
              tc_commit(smem_u32(&bars->empty[sp]));
              ++kp;
              if (++sp == stages) sp = 0;
              progressed = true;
            }
            if (progressed) {
              spins = 0;
              continue;
            }
            if ((++spins & 15u) == 0) {
              if (*abort) break;
              if (globaltimer() - t0 > kWaitLimitNs * 4) {
                *abort = 1;
                raise_flag(P.err_flags, PA_DEVERR_TIMEOUT);
                break;
              }
            }
          }
        }
        tc_commit(smem_u32(&bars->drain));
        drain_wait(smem_u32(&bars->drain), 0, P.err_flags);
      }
      __syncwarp();
    }
  } else {
    if (P.early) grid_dep_wait();
    grid_dep_launch();
  }

  // =================== epilogue ===================
  // The cluster barriers are met by every thread of both CTAs, whatever the
  // unit's state. First: nobody uses the rings any more.
  const int cols = vg >> 2;  // columns a thread sends, and columns it finishes
  cluster_sync_all();
  if (live && ok && n > 0) {
    const uint32_t peer = map_peer(smem_u32(k_s), 1 - map);
    const int c0 = half * cols;  // within the peer's half of the channels
#pragma unroll 1
    for (int c = 0; c < cols; c += 16) {
      uint32_t r[16];
      tmem_ld16(lane_addr + (1 - map) * (vg >> 1) + c0 + c, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int ch = ((c0 + c) >> 2) + e;
        st_peer4(peer + row * vg * 2 + ((ch ^ (row & 7)) << 4), __uint_as_float(r[4 * e]) * coef,
                 __uint_as_float(r[4 * e + 1]) * coef, __uint_as_float(r[4 * e + 2]) * coef,
                 __uint_as_float(r[4 * e + 3]) * coef);
      }
    }
  }
  cluster_sync_all();
  float x[64], ss = 0.f;
  if (live && ok && n > 0) {
#pragma unroll
    for (int c = 0; c < 64; c += 16) {
      if (c < cols) {
        uint32_t r[16];
        tmem_ld16(lane_addr + map * (vg >> 1) + half * cols + c, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ch = ((half * cols + c) >> 2) + e;
          const float4 p =
              *reinterpret_cast<const float4*>(k_s + row * vg * 2 + ((ch ^ (row & 7)) << 4));
          const float pv[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float own = __uint_as_float(r[4 * e + i]) * coef;
            const float d = map == 0 ? own - pv[i] : pv[i] - own;
            x[c + 4 * e + i] = d;
            ss = fmaf(d, d, ss);
          }
        }
      }
    }
    s_ss[map * 2 + half][row] = ss;
    st_peer(map_peer(smem_u32(&s_ss[map * 2 + half][row]), 1 - map), ss);
  }
  cluster_sync_all();
  if (live && ok && n > 0 && row < rows) {
    ss = (s_ss[0][row] + s_ss[1][row]) + (s_ss[2][row] + s_ss[3][row]);
    const float inv =
        bars->bad ? 0.f : (1.f - A.lambda_init) / sqrtf(ss / (float)vhs + A.norm_eps);
    const int ch0 = map * (vg >> 1) + half * cols;
    T* dst = reinterpret_cast<T*>(P.out) +
             ((W.t + row / grp) * P.H + gk * grp + row % grp) * (int64_t)vhs + ch0;
    const T* nw = reinterpret_cast<const T*>(A.norm_weight) + ch0;
#pragma unroll
    for (int c = 0; c < 64; c += 8) {
      if (c < cols && ch0 + c < vhs) {
        float w[8], o[8];
        unpack8<T>(*reinterpret_cast<const uint4*>(nw + c), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = bars->bad ? 0.f : x[c + e] * inv * w[e];
        *reinterpret_cast<uint4*>(dst + c) = pack8<T>(o);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
cudaError_t encode(CUtensorMap* map, bool bf16, const void* base, int rank, const cuuint64_t* dims,
                   const cuuint64_t* str, const cuuint32_t* box) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             (cuuint32_t)rank, const_cast<void*>(base), dims, str, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <typename T, bool CAP>
cudaError_t launch(const Geometry& g, const DiffArgs& a, const PreArgs& A, int64_t units) {
  static std::atomic<bool> configured[64];
  auto kern = diff_prefill_kernel<T, CAP>;
  cudaError_t e = once_per_device(configured, g.device, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  });
  if (e != cudaSuccess) return e;
  const Params& P = A.P;
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const cuuint64_t slots = (cuuint64_t)g.num_blocks * g.bs, hb = (cuuint64_t)g.hs * 2;
  CUtensorMap kmap, vmap, qmap;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)g.hs, (cuuint64_t)(2 * g.kvh), slots};
    const cuuint64_t str[2] = {hb, hb * 2 * g.kvh};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)P.box_rows};
    if ((e = encode(&kmap, bf16, a.key_cache, 3, dims, str, box)) != cudaSuccess) return e;
  }
  {
    const cuuint64_t dims[3] = {(cuuint64_t)g.vhs, (cuuint64_t)g.kvh, slots};
    const cuuint64_t str[2] = {(cuuint64_t)g.vhs * 2, (cuuint64_t)g.vhs * 2 * g.kvh};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)P.box_rows};
    if ((e = encode(&vmap, bf16, a.value_cache, 3, dims, str, box)) != cudaSuccess) return e;
  }
  {  // query [T][H][2][hs]: boxes of 64 channels x one map x grp heads x tpc tokens
    const cuuint64_t dims[4] = {(cuuint64_t)g.hs, 2, (cuuint64_t)g.H, (cuuint64_t)a.num_tokens};
    const cuuint64_t str[3] = {hb, 2 * hb, 2 * hb * g.H};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)P.grp, (cuuint32_t)P.tpc};
    if ((e = encode(&qmap, bf16, a.query, 4, dims, str, box)) != cudaSuccess) return e;
  }
  const size_t smem = 1024 + (size_t)P.q_bytes + (size_t)P.stages * P.stage_bytes;
  return launch_pdl(kern, dim3((unsigned)(units * g.kvh * 2)), dim3(kPreThreads), smem, a.stream,
                    kmap, vmap, qmap, A);
}

}  // namespace

cudaError_t launch_prefill(const Geometry& g, const DiffArgs& a) {
  PreArgs A{};
  Params& P = A.P;
  const int grp = g.H / g.kvh;
  P.out = a.out;
  P.cos_cache = a.cos_cache;
  P.sin_cache = a.sin_cache;
  P.cumseq = a.cumseq;
  P.past = a.past;
  P.block_table = a.block_table;
  P.err_flags = a.err_flags;
  P.num_tokens = a.num_tokens;
  P.num_slots = (int64_t)g.num_blocks * g.bs;
  P.num_seqs = a.num_seqs;
  P.pf_begin = P.seq_begin = a.seq_begin;
  P.pf_end = P.seq_end = a.seq_end;
  P.H = g.H;
  P.hs = g.hs;
  P.vhs = g.vhs;
  P.ro = g.ro;
  P.rd = g.rd;
  P.interleaved = g.interleaved;
  P.cos_rows = g.cos_rows;
  P.bs = g.bs;
  P.num_blocks = g.num_blocks;
  P.max_blocks = g.max_blocks;
  P.scale_log2 = g.scale * kLog2e;
  P.cap_in = g.softcap > 0.f ? g.scale / g.softcap : 0.f;
  P.cap_out = g.softcap * kLog2e;
  P.window = g.window;
  P.box_rows = g.bs < kN ? g.bs : kN;
  P.early = (g.flags & PA_FLAG_AFTER_WRITE) ? 1 : 0;
  P.own_slots = (g.flags & PA_FLAG_OWN_SLOTS) ? 1 : 0;
  P.kvh = g.kvh;
  P.grp = grp;
  P.tpc = kRows / grp;
  P.slabs = (g.hs + 63) / 64;
  P.vslabs = (g.vhs + 63) / 64;
  P.vg = 64 * P.vslabs;
  P.q_bytes = P.slabs * kBox;
  P.k_bytes = P.slabs * kBox;
  P.stage_bytes = (P.slabs + P.vslabs) * kBox;
  P.stages = (int)((kSmemMax - 1024 - P.q_bytes) / P.stage_bytes);
  if (P.stages > kMaxStages) P.stages = kMaxStages;
  A.hs = g.hs;
  A.lambda_vectors = a.lambda_vectors;
  A.norm_weight = a.norm_weight;
  A.lambda_init = a.lambda_init;
  A.norm_eps = a.norm_eps;
  const int64_t units = (a.num_tokens + P.tpc - 1) / P.tpc + (a.seq_end - a.seq_begin);
  const bool cap = g.softcap > 0.f;
  if (g.dtype == PA_DTYPE_BF16)
    return cap ? launch<__nv_bfloat16, true>(g, a, A, units)
               : launch<__nv_bfloat16, false>(g, a, A, units);
  return cap ? launch<__half, true>(g, a, A, units) : launch<__half, false>(g, a, A, units);
}

}  // namespace diff
}  // namespace pa
