// Flash backward over a sliding window with sinks (head dims 64 and 128).
//
// Gradient of out = softmax(scale q k^T + mask) v, the mask letting the query at
// position p see the key at position t iff t <= p and (p - t < window or t <
// sinks).  As in the causal fused backward (attn_bwd_fused.cu, where the step's
// products, TMEM columns and shared memory are set out) a CTA owns a key tile of
// one KV head and walks the query tiles that see it: per step S^T = K Q^T and
// dP^T = V dO^T, then dV += P^T dO, dK += dS^T Q, and dQ = dS K added into an
// fp32 accumulator by TMA reduce-add.
//
// What differs:
//
//  * Tiles are runs of positions (WinTiles), in every token order, so the query
//    tiles that see a key tile are one run of tiles: from its own to the window's
//    end behind it, or to the sequence's where it holds a sink.  They are walked
//    from the last to the first, for each query head of the group.
//  * In edge tiles a key is seen by a run of columns: masked by column bits, and
//    32 columns that see none of a warp's keys cost no exponential.  (Walked
//    position by position the masks took longer than the rest of the step: the
//    64-head layer's backward at 16384 tokens, window 2048, 3.12 -> 2.33 ms.)
//  * A unit with far more steps than the rest (a sink's tile) comes in parts:
//    each walks some of its steps and writes dk, dv as fp32 to a buffer of its
//    own; the last kernel adds a tile's parts in order.
//  * Units are taken over by cluster launch control, longest first, not dealt
//    out beforehand (SMs do not keep the same pace).
//
// Bound (D = 128): no single unit.  A step takes about 4,850 clocks, of which the
// issuing thread spends 3,900 handing over 40 products, at 100 clocks instead of
// the tensor core's 64, and waits 900 for dQ's columns, which dP needs next.
// Meanwhile shared memory moves 480 KB (128 bytes a clock), the SM 128 KB to and
// from L2, half of it the fp32 adds (they alone run at 25 bytes a clock and SM at
// most), whose tile lies in dO's space until they are read; and long runs are at
// the power limit.  So products handed over faster (by a whole warp, see the
// issuer) gained nothing at D = 128 (window 1024, 32 heads: 376 -> 387 us; window
// 2048, 64 heads on 8: 2,360 -> 2,350), and it keeps its one thread.  At D = 64
// dQ has columns and staging of its own: dP is formed before dQ, and no space
// waits for the adds (8192 tokens, 32 heads, window 1024: 286 -> 278 us; with the
// whole warp 262).  A unit's end and start take 5,000 clocks more (9,000 before
// its first Q was loaded ahead of K and dV, dK left through V's space: window 128
// without sinks, 2 x 8192 tokens, 32 heads: 271 -> 256 us).  Measured: 16384
// tokens, 64 heads on 8, D = 128, window 2048, 4 sinks: 2,350 us, 1,230 TF/s over
// the tiles it takes (1,100 over the pairs seen).
#include "common.cuh"
#include "internal.h"

namespace cpattn {
namespace {

// warps 0-7 element-wise (two column halves), 8 TMA producer, 9 MMA issuer,
// 10 dQ reducer, 11 idle, 12-15 dQ read-out.  setmaxnreg moves registers from
// warpgroup 2 (producer, MMA, reducer) and warpgroup 3 (read-out) to the
// element-wise warpgroups.
constexpr int kThreadsF = 512;
constexpr int kRegsLaunchF = 128;  // 65536 / 512
constexpr int kRegsEw = 152;
constexpr int kRegsWg2 = 112;
constexpr int kRegsWg3 = 96;
static_assert(256 * kRegsEw + 128 * kRegsWg2 + 128 * kRegsWg3 <= kThreadsF * kRegsLaunchF, "register split");
// a warpgroup's share is set with setmaxnreg.inc when it grows from the launch
// count and .dec when it shrinks (either one in the other direction is invalid)
template <int N>
__device__ __forceinline__ void regs_to() {
  static_assert(N % 8 == 0 && N >= 24 && N <= 256, "setmaxnreg range");
  if constexpr (N > kRegsLaunchF) regs_inc<N>();
  else if constexpr (N < kRegsLaunchF) regs_dec<N>();
}
constexpr int kRows = 128;      // key rows per unit, query rows per step

template <int D>
struct FCfg {
  static constexpr int TILE = kRows * D * 2;  // D/64 boxes of 128 rows x 128 B
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = TILE;
  static constexpr int OFF_Q = 2 * TILE;   // stage s at OFF_Q + s*TILE
  static constexpr int OFF_DO = 4 * TILE;  // stage s at OFF_DO + s*TILE
  static constexpr int OFF_DS = 6 * TILE;  // dS as two query halves x 128 key rows x 128 B
  static constexpr int DS_BYTES = 2 * kRows * 128;
  // D = 64 leaves room for dQ by itself: two tiles of TMEM columns and two
  // staging tiles (at D = 128 it takes dP's columns, and the dS and dO spaces)
  static constexpr bool APART = D == 64;
  static constexpr int NDQ = APART ? 2 : 1;  // dQ tiles in TMEM, by step (1 or 2)
  static constexpr int OFF_STG = OFF_DS + DS_BYTES;
  static constexpr int STG_BYTES = APART ? kRows * D * 4 : 0;
  static constexpr int OFF_VEC = OFF_STG + 2 * STG_BYTES;  // stage s: lse[128] then delta[128] (fp32)
  static constexpr int VEC_BYTES = 2 * kRows * 4;
  static constexpr int OFF_BAR = OFF_VEC + 2 * VEC_BYTES;
  static constexpr int OFF_MISC = OFF_BAR + 320;  // TMEM address, abort flag, StepInfo[2] at +32
  static constexpr int OFF_U = OFF_MISC + 64;     // BwdUnit[2]
  static constexpr int OFF_CLC = OFF_U + 2 * (int)sizeof(BwdUnit);  // answer of the launch control, 16 bytes
  static constexpr int SMEM = OFF_CLC + 16;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(TILE % 1024 == 0 && OFF_DS % 1024 == 0, "swizzled tiles need 1024-byte alignment");
  // TMEM columns
  static constexpr int T_S = 0;
  static constexpr int T_DP = 128;
  static constexpr int T_DV = 256;
  static constexpr int T_DK = 256 + D;
  static constexpr int T_DQ = APART ? T_DK + D : T_DP;  // of step j at T_DQ + (j % NDQ) * D
  static_assert(T_DK + D + (APART ? NDQ * D : 0) <= 512, "TMEM budget");
};

// what the producer publishes with each Q stage: the query tile's first
// position (its complement where the window cuts some pair of the step) and
// whether it is the last step of its unit
struct StepInfo {
  int qpos, last, pad[2];
};

struct FBars {
  uint64_t k_full, k_empty, v_full, v_empty;
  uint64_t q_full[2], q_empty[2], do_full[2], do_empty[2];
  uint64_t s_full, p_full, dp_full, dst_full, dss_full, dq_free, staged, staged_ds, ds_free;
  uint64_t dv_full, dk_full, done;
  // per dQ tile.  (One dq_full for both of APART's tiles would not do: two of them may be formed before the read-out
  // looks for the first, and the barrier, two phases on, would show it the parity of a phase that is not complete.)
  uint64_t dq_full[2];
  uint64_t dq_free2[2], staged2[2], stg_empty[2];  // APART
  uint64_t clc, unit_full[2], unit_empty[2];  // the next unit's number has come; units published, read
};
static_assert(sizeof(FBars) <= 320, "barrier area");
// who reads a unit: the MMA issuer, the reducer, 8 element-wise and 4 read-out warps
constexpr int kUnitReaders = 14;

// this thread's bulk async-groups, all but the newest N, have read their sources
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// P for this thread's 64 query columns of one step: scores from TMEM (t_s),
// p = exp2(s * scale*log2e - lse*log2e), zero outside columns lo .. hi (EDGE
// steps only), kept in fp32 for dS and stored back to TMEM (t_pk) as packed
// bf16.  (Rows past a tile's end come with lse = inf and give zeros.)
template <bool EDGE>
__device__ __forceinline__ void ew_p(uint32_t t_s, uint32_t t_pk, const float* lse_s, uint64_t sl2x2, float (&p)[64],
                                     int lo, int hi) {
  auto below = [](int x) { return x <= 0 ? 0u : (x >= 32 ? 0xffffffffu : (1u << x) - 1u); };
  uint32_t sv[2][32];
  tmem_ld32(t_s, sv[0]);
  tmem_ld32(t_s + 32, sv[1]);
  tmem_ld_wait();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t see = EDGE ? below(hi + 1 - 32 * h) & ~below(lo - 32 * h) : 0xffffffffu;
    uint32_t pk[16];
    if (EDGE && !__any_sync(0xffffffffu, see != 0)) {
#pragma unroll
      for (int c = 0; c < 32; ++c) p[32 * h + c] = 0.f;
#pragma unroll
      for (int c = 0; c < 16; ++c) pk[c] = 0u;
    } else {
      const uint64_t* nl2 = reinterpret_cast<const uint64_t*>(lse_s + 32 * h);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        float p0, p1;
        f2unpack(f2fma(f2pack_u(sv[h][c], sv[h][c + 1]), sl2x2, nl2[c >> 1]), p0, p1);
        p0 = fast_exp2(p0);
        p1 = fast_exp2(p1);
        p[32 * h + c] = !EDGE || (see >> c & 1u) ? p0 : 0.f;
        p[32 * h + c + 1] = !EDGE || (see >> (c + 1) & 1u) ? p1 : 0.f;
        pk[c >> 1] = pack_bf16(p[32 * h + c], p[32 * h + c + 1]);
      }
    }
    tmem_st16(t_pk + 16 * h, pk);
  }
}

// The (query head, query tile) steps of a key-tile unit, or of a part of them:
// per head of the group the tiles from `top` down to the key tile's own.
struct Steps {
  int left, hq, p, ch, off;      // steps after this one; head, tile, its chunk and number in it
  int first, top, ch_top, off_top;

  __device__ __forceinline__ void begin(const WinTiles& wt, const Window& w, const BwdUnit& u, int G,
                                        const WinPart* parts) {
    first = u.t;
    int ch0, off0;
    wt.split(u.t, ch0, off0);
    const int kmin = wt.pos(ch0, off0), kmax = kmin + wt.rows(off0) - 1;
    top = kmin < w.sinks || kmax >= wt.S - w.window ? wt.nt - 1 : wt.tile_of(kmax + w.window - 1);
    wt.split(top, ch_top, off_top);
    const int nq = top - first + 1;
    int skip = 0;
    left = nq * G - 1;
    if (u.pad) {
      skip = parts[u.pad - 1].skip;
      left = parts[u.pad - 1].steps - 1;
    }
    const int dh = skip / nq;
    hq = u.h * G + dh;
    p = top - (skip - dh * nq);
    wt.split(p, ch, off);
  }
  // advance; false after the last step
  __device__ __forceinline__ bool next(const WinTiles& wt) {
    if (left-- == 0) return false;
    if (p > first) {
      --p;
      if (--off < 0) {
        --ch;
        off = wt.tpc - 1;
      }
    } else {
      ++hq;
      p = top;
      ch = ch_top;
      off = off_top;
    }
    return true;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreadsF, 1) attn_bwd_window_kernel(const __grid_constant__ BwdArgs a) {
  using C = FCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // every offset below assumes a 1024-byte aligned base (no slack is left for
  // aligning by hand); a misaligned base is reported and the CTA does nothing
  if (smem_u32(smem) & 1023u) {
    if (tid == 0) atomicExch(a.err, DEV_SMEM_ALIGN);
    return;
  }
  FBars& bar = *reinterpret_cast<FBars*>(smem + C::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 16);
  volatile StepInfo* info = reinterpret_cast<volatile StepInfo*>(smem + C::OFF_MISC + 32);
  const WinTiles wt = WinTiles::make(a.sh.S, a.sh.cp, a.sh.lb);
  BwdUnit* const us = reinterpret_cast<BwdUnit*>(smem + C::OFF_U);
  const Abort ab{abort_flag, a.err};
  const int G = a.sh.Hq / a.sh.Hkv;

  if (tid == 0) {
    mbar_init(&bar.k_full, 1);
    mbar_init(&bar.k_empty, 1);
    mbar_init(&bar.v_full, 1);
    mbar_init(&bar.v_empty, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 1);
      mbar_init(&bar.q_empty[i], 1);
      mbar_init(&bar.do_full[i], 1);
      mbar_init(&bar.do_empty[i], 1);
    }
    mbar_init(&bar.s_full, 1);
    mbar_init(&bar.p_full, 256);
    mbar_init(&bar.dp_full, 1);
    mbar_init(&bar.dst_full, 256);
    mbar_init(&bar.dss_full, 256);
    mbar_init(&bar.dq_free, 128);
    mbar_init(&bar.staged, 128);
    mbar_init(&bar.staged_ds, 128);
    mbar_init(&bar.ds_free, 1);
    mbar_init(&bar.dv_full, 1);
    mbar_init(&bar.dk_full, 1);
    mbar_init(&bar.done, 1);
    mbar_init(&bar.clc, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.dq_full[i], 1);
      mbar_init(&bar.dq_free2[i], 128);
      mbar_init(&bar.staged2[i], 128);
      mbar_init(&bar.stg_empty[i], 1);
      mbar_init(&bar.unit_full[i], 1);
      mbar_init(&bar.unit_empty[i], kUnitReaders);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  wait_for_previous();
  if (warp == 9) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&a.tq); prefetch_tmap(&a.tk); prefetch_tmap(&a.tv); prefetch_tmap(&a.tdo); prefetch_tmap(&a.tdq);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The unit of run r of this CTA, published by the producer in slot r & 1 (b < 0:
  // there is none).  false if there is none or it did not come.  A warp reads it
  // together, the reducer's thread alone.
  auto unit_of_warp = [&](int r, BwdUnit& u) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(&bar.unit_full[r & 1], (r >> 1) & 1, ab));
    if (!ok) return false;
    u = us[r & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.unit_empty[r & 1]);
    return (bool)__all_sync(0xffffffffu, u.b >= 0);
  };
  // dQ of step j is formed (or the wait failed)
  auto await_dq = [&](int j) { return mbar_wait(&bar.dq_full[j & (C::NDQ - 1)], (j >> (C::NDQ - 1)) & 1, ab); };
  auto unit_of_thread = [&](int r, BwdUnit& u) {
    if (!mbar_wait(&bar.unit_full[r & 1], (r >> 1) & 1, ab)) return false;
    u = us[r & 1];
    mbar_arrive(&bar.unit_empty[r & 1]);
    return u.b >= 0;
  };

  auto dq_readout = [&]() {
    // ------------------------------------------------------------ dQ read-out
    // dQ_j (query rows = TMEM lanes, D fp32 columns): TMEM -> registers -> shared
    // memory for the reducer, in boxes of 32 columns (128-byte swizzle); the
    // columns are released as soon as the last load is done.  At D = 128 the boxes
    // go to the dS tile and the step's dO stage, each staged while the next load
    // is in flight; both are dead once dQ_j is complete: dS_j and dO_j were last
    // read by MMAs that precede it.  The tile goes out unscaled (the final
    // rounding pass applies the softmax scale).
    const int qd = warp & 3;
    const int row = (qd << 5) + lane;  // query row of the tile == TMEM lane
    const uint32_t t_dq = tmem + (uint32_t(qd * 32) << 16) + C::T_DQ;
    auto stage = [&](int gsr, int c, const uint32_t (&o)[32]) {
      unsigned char* bb = C::APART ? smem + C::OFF_STG + (gsr & 1) * C::STG_BYTES + c * (kRows * 128)
                          : c < 2 ? smem + C::OFF_DS + c * (kRows * 128)
                                : smem + C::OFF_DO + (gsr & 1) * C::TILE + (c - 2) * (kRows * 128);
      unsigned char* rp = bb + row * 128;
#pragma unroll
      for (int ch = 0; ch < 8; ++ch)
        *reinterpret_cast<uint4*>(rp + ((ch ^ (row & 7)) << 4)) =
            make_uint4(o[4 * ch + 0], o[4 * ch + 1], o[4 * ch + 2], o[4 * ch + 3]);
    };
    int gs = 0;
    BwdUnit u;
    for (int r = 0; unit_of_warp(r, u); ++r) {
      Steps it;
      it.begin(wt, a.win, u, G, a.parts);
      do {
        await_dq(gs);  // runs on after an abort: the staging is garbage, the waits bounded
        tc_fence_after();
        uint32_t o[2][32];
        if constexpr (C::APART) {
          tmem_ld32(t_dq + (gs & 1) * D, o[0]);
          tmem_ld32(t_dq + (gs & 1) * D + 32, o[1]);
          tmem_ld_wait();
          tc_fence_before();
          mbar_arrive(&bar.dq_free2[gs & 1]);
          if (gs >= 2) mbar_wait(&bar.stg_empty[gs & 1], ((gs >> 1) & 1) ^ 1, ab);  // the tile of two steps ago is added
          stage(gs, 0, o[0]);
          stage(gs, 1, o[1]);
          fence_proxy_async_smem();
          mbar_arrive(&bar.staged2[gs & 1]);
        } else {
          tmem_ld32(t_dq, o[0]);
          tmem_ld32(t_dq + 32, o[1]);
          tmem_ld_wait();
          stage(gs, 0, o[0]);
          tmem_ld32(t_dq + 64, o[0]);
          stage(gs, 1, o[1]);
          tmem_ld32(t_dq + 96, o[1]);
          // the dS tile's chunks are staged: the reducer may add them (and
          // free the tile for the next dS) while the rest is read out
          fence_proxy_async_smem();
          mbar_arrive(&bar.staged_ds);
          tmem_ld_wait();
          tc_fence_before();
          mbar_arrive(&bar.dq_free);
          stage(gs, 2, o[0]);
          stage(gs, 3, o[1]);
          fence_proxy_async_smem();
          mbar_arrive(&bar.staged);
        }
        ++gs;
      } while (it.next(wt));
    }
  };

  // each role's code sits under its own setmaxnreg, so the compiler
  // allocates it against that role's register budget
  if (warp >= 12) {
  regs_to<kRegsWg3>();
  dq_readout();
  } else if (warp >= 8) {
  regs_to<kRegsWg2>();
  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int gs = 0;  // global step index: stage gs & 1, ring phase (gs >> 1) & 1
      int k_loads = 0, v_loads = 0, q_loads = 0, do_loads = 0;
      bool ok = true;
      auto publish = [&](const BwdUnit& x, int r) {
        if (r >= 2 && !(ok = mbar_wait(&bar.unit_empty[r & 1], ((r >> 1) & 1) ^ 1, ab))) return;
        us[r & 1] = x;
        mbar_arrive(&bar.unit_full[r & 1]);
      };
      BwdUnit u = a.units[blockIdx.x];
      publish(u, 0);
      int asked = 0;
      for (int r = 0; ok; ++r) {
        mbar_expect_tx(&bar.clc, 16);
        clc_ask(smem + C::OFF_CLC, &bar.clc);
        ++asked;
        Steps it;
        it.begin(wt, a.win, u, G, a.parts);
        int kch, koff;
        wt.split(u.t, kch, koff);
        const int kmin = wt.pos(kch, koff), kmax = kmin + wt.rows(koff) - 1;
        // everything a load needs is computed before the wait that releases
        // its stage: the dO stage is freed late (it stages dQ), and any work
        // between that release and the load lands on the MMA chain
        const int krow = wt.mem(kch, koff);
        asm volatile("" ::"r"(krow));
        bool more, first = true;
        do {
          const int hq = it.hq, qrow = wt.mem(it.ch, it.off), qlo = wt.pos(it.ch, it.off);
          const int qpos = a.win.all(qlo, qlo + kRows - 1, kmin, kmax) ? qlo : ~qlo;
          const int qt = it.p;
          more = it.next(wt);  // (the step after this one)
          const int st = gs & 1;
          const uint32_t ph = ((gs >> 1) & 1) ^ 1;
          const size_t vo = ((size_t)u.b * a.sh.Hq + hq) * a.Spad + (size_t)qt * kRows;
          unsigned char* vec = smem + C::OFF_VEC + st * C::VEC_BYTES;
          // (an empty asm that reads the values keeps the compiler from sinking
          // their computation below the waits)
          asm volatile("" ::"r"(qrow), "l"(vo), "r"(it.p), "r"(it.hq), "r"((int)more), "r"(qpos));
          if (!(ok = mbar_wait(&bar.q_empty[st], ph, ab))) break;
          info[st].qpos = qpos;
          info[st].last = more ? 0 : 1;
          ++q_loads;
          mbar_expect_tx(&bar.q_full[st], C::TILE + C::VEC_BYTES);  // (release: the info is visible to q_full's waiters)
          for (int bx = 0; bx < D / 64; ++bx)
            tma_load_4d(smem + C::OFF_Q + st * C::TILE + bx * kRows * 128, &a.tq, &bar.q_full[st], bx * 64, hq, qrow,
                        u.b);
          bulk_load(vec, a.lse_l2 + vo, kRows * 4, &bar.q_full[st]);
          bulk_load(vec + kRows * 4, a.delta + vo, kRows * 4, &bar.q_full[st]);
          if (first) {  // (after the first Q, whose stage the last unit left earlier than K)
            if (!(ok = mbar_wait(&bar.k_empty, (r & 1) ^ 1, ab))) break;
            mbar_expect_tx(&bar.k_full, C::TILE);
            ++k_loads;
            for (int bx = 0; bx < D / 64; ++bx)
              tma_load_4d(smem + C::OFF_K + bx * kRows * 128, &a.tk, &bar.k_full, bx * 64, u.h, krow, u.b);
          }
          if (!(ok = mbar_wait(&bar.do_empty[st], ph, ab))) break;
          mbar_expect_tx(&bar.do_full[st], C::TILE);
          ++do_loads;
          for (int bx = 0; bx < D / 64; ++bx)
            tma_load_4d(smem + C::OFF_DO + st * C::TILE + bx * kRows * 128, &a.tdo, &bar.do_full[st], bx * 64, hq, qrow,
                        u.b);
          if (first) {  // (V's space was the last unit's staging)
            first = false;
            if (!(ok = mbar_wait(&bar.v_empty, (r & 1) ^ 1, ab))) break;
            mbar_expect_tx(&bar.v_full, C::TILE);
            ++v_loads;
            for (int bx = 0; bx < D / 64; ++bx)
              tma_load_4d(smem + C::OFF_V + bx * kRows * 128, &a.tv, &bar.v_full, bx * 64, u.h, krow, u.b);
          }
          ++gs;
        } while (more);
        if (!ok) break;
        // with the unit's last step queued the next one is published, and its
        // first tiles go to L2: their loads wait for this unit's end, and would
        // otherwise meet the full HBM latency at every unit boundary
        if (!(ok = mbar_wait(&bar.clc, r & 1, ab))) break;
        const int next = clc_answer(smem + C::OFF_CLC);
        if (next >= 0) u = a.units[next];
        else u.b = -1;
        publish(u, r + 1);
        if (next < 0) break;
        wt.split(u.t, kch, koff);
        it.begin(wt, a.win, u, G, a.parts);
        for (int bx = 0; bx < D / 64; ++bx) {
          tma_prefetch_l2_4d(&a.tk, bx * 64, u.h, wt.mem(kch, koff), u.b);
          tma_prefetch_l2_4d(&a.tv, bx * 64, u.h, wt.mem(kch, koff), u.b);
          tma_prefetch_l2_4d(&a.tdo, bx * 64, it.hq, wt.mem(it.ch, it.off), u.b);
        }
      }
      if (!ok) {
        // let the copies already issued land before the CTA exits (a wait for
        // each barrier's latest phase; none of them waits for long)
        auto drain = [&](uint64_t* b, uint32_t parity) {
          volatile int own = 0;
          mbar_wait(b, parity, Abort{&own, a.err});
        };
        if (asked > 0) drain(&bar.clc, (asked - 1) & 1);
        for (int s = 0; s < 2; ++s) {
          const int nq = (q_loads + 1 - s) >> 1, nd = (do_loads + 1 - s) >> 1;  // loads of stage s
          if (nq > 0) drain(&bar.q_full[s], (nq - 1) & 1);
          if (nd > 0) drain(&bar.do_full[s], (nd - 1) & 1);
        }
        if (k_loads > 0) drain(&bar.k_full, (k_loads - 1) & 1);
        if (v_loads > 0) drain(&bar.v_full, (v_loads - 1) & 1);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    // At D = 64 the whole warp runs this and one lane issues: what it hands over
    // stays in uniform registers.  (In a branch of one thread every product costs
    // several moves to them, each waiting for its turn among the element-wise
    // warps, 100 clocks a product; at D = 128 that is not what it waits for.)
    constexpr bool WARP = C::APART;
    if (WARP || lane == 0) {
      bool lead = true;
      uint32_t tm = tmem;
      if constexpr (WARP) {
        lead = elect_lane();
        tm = __shfl_sync(0xffffffffu, tmem, 0);
      }
      auto wait = [&](uint64_t* b, uint32_t parity) {
        return WARP ? mbar_wait_warp(b, parity, ab) : mbar_wait(b, parity, ab);
      };
      auto last_of = [&](int st) {
        const bool l = info[st].last;
        return WARP ? (bool)__any_sync(0xffffffffu, l) : l;
      };
      constexpr uint32_t IDESC_S = idesc_bf16(128, kRows, 0, 0);  // S^T, dP^T: K-major x K-major
      constexpr uint32_t IDESC_ACC = idesc_bf16(128, D, 0, 1);    // P^T / dS^T (TMEM) x dO / Q (MN-major)
      constexpr uint32_t IDESC_DQ = idesc_bf16(128, D, 1, 1);     // dS (MN-major) x K (MN-major)
      const uint32_t s0 = smem_u32(smem);
      const uint64_t dK_k = sdesc_sw128(s0 + C::OFF_K, 16, 1024);          // K as K-major A
      const uint64_t dV_k = sdesc_sw128(s0 + C::OFF_V, 16, 1024);          // V as K-major A
      const uint64_t dK_mn = sdesc_sw128(s0 + C::OFF_K, kRows * 128, 1024);  // K as MN-major B
      const uint64_t dS_mn = sdesc_sw128(s0 + C::OFF_DS, kRows * 128, 1024); // dS as MN-major A
      auto kstep = [](int kk) { return (uint64_t)((((kk >> 2) * (kRows * 128)) + (kk & 3) * 32) >> 4); };
      auto issue_s = [&](int st) {
        const uint64_t bq = sdesc_sw128(s0 + C::OFF_Q + st * C::TILE, 16, 1024);
        if (lead) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tm + C::T_S, dK_k + kstep(kk), bq + kstep(kk), IDESC_S, kk > 0 ? 1u : 0u);
        mma_commit(&bar.s_full);
        }
      };
      auto issue_dp = [&](int st) {
        const uint64_t bo = sdesc_sw128(s0 + C::OFF_DO + st * C::TILE, 16, 1024);
        if (lead) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tm + C::T_DP, dV_k + kstep(kk), bo + kstep(kk), IDESC_S, kk > 0 ? 1u : 0u);
        mma_commit(&bar.dp_full);
        }
      };
      auto issue_dv = [&](int st, bool acc) {
        const uint64_t bo = sdesc_sw128(s0 + C::OFF_DO + st * C::TILE, kRows * 128, 1024);
        if (lead) {
#pragma unroll
        for (int kk = 0; kk < kRows / 16; ++kk)
          mma_ts(tm + C::T_DV, tm + C::T_S + packed_col<64>(kk * 16), bo + ((kk * 16 * 128) >> 4), IDESC_ACC,
                 (acc || kk > 0) ? 1u : 0u);
        }
      };
      auto issue_dk = [&](int st, bool acc) {
        const uint64_t bq = sdesc_sw128(s0 + C::OFF_Q + st * C::TILE, kRows * 128, 1024);
        if (lead) {
#pragma unroll
        for (int kk = 0; kk < kRows / 16; ++kk)
          mma_ts(tm + C::T_DK, tm + C::T_DP + packed_col<64>(kk * 16), bq + ((kk * 16 * 128) >> 4), IDESC_ACC,
                 (acc || kk > 0) ? 1u : 0u);
        }
      };
      auto issue_dq = [&](int buf) {
        if (lead) {
#pragma unroll
        for (int kk = 0; kk < kRows / 16; ++kk)
          mma_ss(tm + C::T_DQ + buf * D, dS_mn + ((kk * 16 * 128) >> 4), dK_mn + ((kk * 16 * 128) >> 4), IDESC_DQ,
                 kk > 0 ? 1u : 0u);
        mma_commit(&bar.dq_full[buf]);
        }
      };

      int gs = 0;
      bool ok = true;
      BwdUnit u;
      for (int r = 0; ok && (WARP ? unit_of_warp(r, u) : unit_of_thread(r, u)); ++r) {
        if (!(ok = wait(&bar.k_full, r & 1))) break;
        tc_fence_after();
        // prologue: S and dP of the unit's first step
        if (!(ok = wait(&bar.q_full[gs & 1], (gs >> 1) & 1))) break;
        tc_fence_after();
        bool more = !last_of(gs & 1);
        issue_s(gs & 1);
        if (!C::APART && gs > 0 && !(ok = wait(&bar.dq_free, (gs - 1) & 1))) break;  // dQ of the last step read out
        if (!(ok = wait(&bar.v_full, r & 1))) break;
        if (!(ok = wait(&bar.do_full[gs & 1], (gs >> 1) & 1))) break;
        tc_fence_after();
        issue_dp(gs & 1);
        for (int j = 0; ok; ++j, ++gs) {
          const int st = gs & 1;
          const bool this_more = more;
          if (!(ok = wait(&bar.p_full, gs & 1))) break;
          tc_fence_after();
          issue_dv(st, j > 0);
          if (C::APART && lead) mma_commit(&bar.do_empty[st]);  // (dP_j came before)
          if (!this_more) {
            if (lead) mma_commit(&bar.dv_full);
          } else {
            if (!(ok = wait(&bar.q_full[st ^ 1], ((gs + 1) >> 1) & 1))) break;
            tc_fence_after();
            more = !last_of(st ^ 1);
            issue_s(st ^ 1);
          }
          if (!(ok = wait(&bar.dst_full, gs & 1))) break;
          tc_fence_after();
          issue_dk(st, j > 0);
          if (lead) mma_commit(&bar.q_empty[st]);  // Q_j (S_j, dK_j) and its vectors are done
          if (!this_more && lead) mma_commit(&bar.dk_full);
          if constexpr (C::APART) {
            if (this_more) {
              if (!(ok = wait(&bar.do_full[st ^ 1], ((gs + 1) >> 1) & 1))) break;
              tc_fence_after();
              issue_dp(st ^ 1);
            }
            if (!(ok = wait(&bar.dss_full, gs & 1))) break;
            if (gs >= 2 && !(ok = wait(&bar.dq_free2[st], ((gs >> 1) & 1) ^ 1))) break;
            tc_fence_after();
            issue_dq(st);
            if (!this_more) break;
            continue;
          }
          if (!(ok = wait(&bar.dss_full, gs & 1))) break;
          tc_fence_after();
          issue_dq(0);
          if (!this_more) break;
          if (!(ok = wait(&bar.dq_free, gs & 1))) break;
          if (!(ok = wait(&bar.do_full[st ^ 1], ((gs + 1) >> 1) & 1))) break;
          tc_fence_after();
          issue_dp(st ^ 1);
        }
        if (!ok) break;
        ++gs;
        if (lead) mma_commit(&bar.k_empty);  // K (last read by dQ) is done
      }
      if (lead) mma_drain(&bar.done, a.err);
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ dQ reducer
    // adds each staged dQ tile into the fp32 accumulator (rows in the tensors'
    // own order); the boxes in the dS space go first, in their own bulk group,
    // because the next dS waits on them
    if (lane == 0) {
      int gs = 0;
      BwdUnit u;
      for (int r = 0; unit_of_thread(r, u); ++r) {
        Steps it;
        it.begin(wt, a.win, u, G, a.parts);
        do {
          const int hq = it.hq, qrow = wt.mem(it.ch, it.off);
          // (rows past the tile are zero; runs on after an abort: the staging is garbage, the waits bounded)
          if constexpr (C::APART) {
            mbar_wait(&bar.staged2[gs & 1], (gs >> 1) & 1, ab);
#pragma unroll
            for (int box = 0; box < 2; ++box)
              tma_reduce_add_4d(smem + C::OFF_STG + (gs & 1) * C::STG_BYTES + box * (kRows * 128), &a.tdq, box * 32, hq, qrow,
                                u.b);
            bulk_commit_group();
            bulk_wait_read<1>();
            if (gs > 0) mbar_arrive(&bar.stg_empty[(gs - 1) & 1]);  // the tile before is read
          } else {
            mbar_wait(&bar.staged_ds, gs & 1, ab);
#pragma unroll
            for (int box = 0; box < 4; ++box) {
              if (box == 2) mbar_wait(&bar.staged, gs & 1, ab);
              const unsigned char* bb = box < 2 ? smem + C::OFF_DS + box * (kRows * 128)
                                                : smem + C::OFF_DO + (gs & 1) * C::TILE + (box - 2) * (kRows * 128);
              tma_reduce_add_4d(bb, &a.tdq, box * 32, hq, qrow, u.b);
              if (box & 1) bulk_commit_group();
            }
            bulk_wait_read<1>();
            mbar_arrive(&bar.ds_free);  // the dS tile (staging space) may be rewritten
            bulk_wait_read<0>();
            mbar_arrive(&bar.do_empty[gs & 1]);  // the dO stage (staging space) may be reloaded
          }
          ++gs;
        } while (it.next(wt));
      }
      bulk_wait_all();  // every dQ reduce has landed before the CTA retires
    }
  }
  } else {
    regs_to<kRegsEw>();
    // ------------------------------------------------------------ element-wise warps
    // Group g (warps 4g..4g+3) owns query columns [64g, 64g+64) of S^T/dP^T
    // (thread = key row = TMEM lane) and, at the end of a unit, dV/dK columns
    // [gD/2, (g+1)D/2).  A failed wait (abort or timeout) runs on with whatever
    // is in TMEM, so every role walks all of its steps and every wait stays
    // bounded.
    const int g = warp >> 2;
    const int row = ((warp & 3) << 5) + lane;  // TMEM lane
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint64_t sl2x2 = f2pack(a.scale_log2, a.scale_log2);
    int gs = 0;

    BwdUnit u;
    for (int r = 0; unit_of_warp(r, u); ++r) {
      int kch, koff;
      wt.split(u.t, kch, koff);
      const int krows = wt.rows(koff), kmem = wt.mem(kch, koff);
      const bool kvalid = row < krows;
      const int kpos = wt.pos(kch, koff) + row;
      // the last position that sees this row's key (none sees a row past the tile)
      const int qlast = !kvalid ? -1 : (kpos < a.win.sinks || kpos >= wt.S - a.win.window ? wt.S - 1 : kpos + a.win.window - 1);
      bool last;
      do {
        const int st = gs & 1;
        // ---- P into TMEM as bf16 (fp32 copy kept for dS)
        mbar_wait(&bar.s_full, gs & 1, ab);
        mbar_wait(&bar.q_full[st], (gs >> 1) & 1, ab);
        tc_fence_after();
        last = info[st].last != 0;
        const int qpos = info[st].qpos;
        const int q0 = (qpos < 0 ? ~qpos : qpos) + g * 64;  // position of this group's first column
        const float* lse_s = reinterpret_cast<const float*>(smem + C::OFF_VEC + st * C::VEC_BYTES) + g * 64;
        const float* del_s = lse_s + kRows;
        float p[64];
        const uint32_t t_s = tmem + lane_base + C::T_S + g * 64;
        const uint32_t t_pk = tmem + lane_base + C::T_S + packed_col<64>(g * 64);
        if (qpos >= 0 && krows == kRows)
          ew_p<false>(t_s, t_pk, lse_s, sl2x2, p, 0, 0);
        else
          ew_p<true>(t_s, t_pk, lse_s, sl2x2, p, kpos - q0, qlast - q0);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar.p_full);
        // ---- dS = P * (dP - D): bf16 into TMEM (for dK), then shared memory (for dQ)
        mbar_wait(&bar.dp_full, gs & 1, ab);
        tc_fence_after();
        uint32_t dp[2][32], dk[2][16];
        tmem_ld32(tmem + lane_base + C::T_DP + g * 64, dp[0]);
        tmem_ld32(tmem + lane_base + C::T_DP + g * 64 + 32, dp[1]);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t* nd2 = reinterpret_cast<const uint64_t*>(del_s + 32 * h);
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            float d0, d1;
            f2unpack(f2mul(f2pack(p[32 * h + c], p[32 * h + c + 1]), f2add(f2pack_u(dp[h][c], dp[h][c + 1]), nd2[c >> 1])),
                     d0, d1);
            dk[h][c >> 1] = pack_bf16(d0, d1);
          }
          tmem_st16(tmem + lane_base + C::T_DP + packed_col<64>(g * 64 + 32 * h), dk[h]);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar.dst_full);
        // the dS space is free: the last dQ is formed (APART), or its tile has left the space too
        if (gs > 0) C::APART ? await_dq(gs - 1) : mbar_wait(&bar.ds_free, (gs - 1) & 1, ab);
        unsigned char* dsr = smem + C::OFF_DS + g * (kRows * 128) + row * 128;  // this key row of query half g
#pragma unroll
        for (int chunk = 0; chunk < 8; ++chunk)  // 8 query columns per 16-byte chunk
          *reinterpret_cast<uint4*>(dsr + ((chunk ^ (row & 7)) << 4)) =
              make_uint4(dk[chunk >> 2][4 * (chunk & 3)], dk[chunk >> 2][4 * (chunk & 3) + 1],
                         dk[chunk >> 2][4 * (chunk & 3) + 2], dk[chunk >> 2][4 * (chunk & 3) + 3]);
        fence_proxy_async_smem();
        mbar_arrive(&bar.dss_full);
        ++gs;
      } while (!last);
      // dV, then scale*dK, each as soon as its last product is done (dV: while
      // dK's and dQ's still run), through V's space (V was last read by dP) so
      // that warp stores write whole lines: each warp its own 32 rows x D/2
      // columns.  (By all 256 threads together through the dS space, after the
      // unit's last dQ, this took 6,000 clocks of a unit's end; by TMA store,
      // 4,700, behind the dQ reduces in the same queue.)
      unsigned char* const stg = smem + C::OFF_V + warp * (32 * D);
      const int w0 = (warp & 3) * 32, left = krows - w0;  // the warp's first row, rows it has
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const float f = which ? a.scale : 1.f;
        mbar_wait(which ? &bar.dk_full : &bar.dv_full, r & 1, ab);
        tc_fence_after();
        uint32_t o[2][32];
        tmem_ld32(tmem + lane_base + (which ? C::T_DK : C::T_DV) + g * (D / 2), o[0]);
        if (D / 2 > 32) tmem_ld32(tmem + lane_base + (which ? C::T_DK : C::T_DV) + g * (D / 2) + 32, o[1]);
        tmem_ld_wait();
        constexpr int KC = D / 16;  // 16-byte pieces of a row's half (of a quarter in fp32)
        auto at = [&](int rr, int j) { return reinterpret_cast<uint4*>(stg + rr * D + ((j ^ (rr & (KC - 1))) << 4)); };
        if (u.pad) {  // a part: its sums unrounded (rows past the tile are zero), joined afterwards
          float* dst = (which ? a.dk_part : a.dv_part) + ((size_t)(u.pad - 1) * kRows + w0) * D + g * (D / 2);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int j = 0; j < KC; ++j) {
              const uint32_t* x = D == 128 ? &o[q][4 * j] : &o[0][16 * q + 4 * j];
              *at(lane, j) = make_uint4(__float_as_uint(f * __uint_as_float(x[0])), __float_as_uint(f * __uint_as_float(x[1])),
                                        __float_as_uint(f * __uint_as_float(x[2])), __float_as_uint(f * __uint_as_float(x[3])));
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < KC; ++i) {
              const int rr = (lane + 32 * i) / KC, j = lane % KC;
              *reinterpret_cast<uint4*>(dst + rr * D + q * (D / 4) + 4 * j) = *at(rr, j);
            }
            __syncwarp();
          }
          continue;
        }
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          const uint32_t* x = &o[j >> 2][8 * (j & 3)];
          *at(lane, j) = make_uint4(pack_bf16(f * __uint_as_float(x[0]), f * __uint_as_float(x[1])),
                                    pack_bf16(f * __uint_as_float(x[2]), f * __uint_as_float(x[3])),
                                    pack_bf16(f * __uint_as_float(x[4]), f * __uint_as_float(x[5])),
                                    pack_bf16(f * __uint_as_float(x[6]), f * __uint_as_float(x[7])));
        }
        __syncwarp();
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(which ? a.dk : a.dv) +
                             (((size_t)u.b * wt.S + kmem + w0) * a.sh.Hkv + u.h) * D + g * (D / 2);
#pragma unroll
        for (int i = 0; i < KC; ++i) {
          const int rr = (lane + 32 * i) / KC, j = lane % KC;
          if (rr < left) *reinterpret_cast<uint4*>(dst + (size_t)rr * a.sh.Hkv * D + 8 * j) = *at(rr, j);
        }
        __syncwarp();  // (read back: the space may be written again)
      }
      fence_proxy_async_smem();
      if (lane == 0) mbar_arrive(&bar.v_empty);
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// dq (bf16) = scale * the fp32 accumulator, 8 elements a thread at a time (the
// first blocks); dk and dv of the key tiles whose units came in parts: the
// parts' sums, added in order, a float4 of a row a thread (8 blocks per tile).
// (It may start when the products' kernel ends, not before: let in while that
// kernel's units were still being taken over, it cost 3 to 7% of the backward.)
template <int D>
__global__ void __launch_bounds__(256) bwd_window_finish_kernel(const __grid_constant__ BwdArgs a, const WinJoin* joins,
                                                                long long n8, int blocks_dq) {
  wait_for_previous();
  if ((int)blockIdx.x < blocks_dq) {
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n8; i += (long long)blocks_dq * 256) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(a.dq_acc) + 2 * i);
      const float4 y = __ldcs(reinterpret_cast<const float4*>(a.dq_acc) + 2 * i + 1);
      static_cast<uint4*>(a.dq)[i] = make_uint4(pack_bf16(a.scale * x.x, a.scale * x.y), pack_bf16(a.scale * x.z, a.scale * x.w),
                                                pack_bf16(a.scale * y.x, a.scale * y.y), pack_bf16(a.scale * y.z, a.scale * y.w));
    }
    return;
  }
  const int x0 = blockIdx.x - blocks_dq, which = x0 & 1, quarter = (x0 >> 1) & 3;
  const WinJoin jn = joins[x0 >> 3];
  const WinTiles wt = WinTiles::make(a.sh.S, a.sh.cp, a.sh.lb);
  int ch, off;
  wt.split(jn.t, ch, off);
  const int rows = wt.rows(off), mem = wt.mem(ch, off);
  const float* src = (which ? a.dk_part : a.dv_part) + (size_t)jn.part0 * kRows * D;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(which ? a.dk : a.dv);
  for (int x = threadIdx.x + quarter * 256; x < kRows * D / 4; x += 1024) {
    const int row = x / (D / 4), c = x - row * (D / 4);
    if (row >= rows) continue;
    float4 s = reinterpret_cast<const float4*>(src)[x];
    for (int p = 1; p < jn.nparts; ++p) {
      const float4 y = reinterpret_cast<const float4*>(src + (size_t)p * kRows * D)[x];
      s.x += y.x;
      s.y += y.y;
      s.z += y.z;
      s.w += y.w;
    }
    *reinterpret_cast<uint2*>(dst + (((size_t)jn.b * wt.S + mem + row) * a.sh.Hkv + jn.h) * D + 4 * c) =
        make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
  }
}

// Row statistics per tile, [B, Hq, tiles * 128] in tile order: -lse*log2(e) (-inf
// past a tile's rows) and -rowsum(dout*out) (0 there), and the accumulator's rows
// zeroed.  D / 8 lanes a row, 16 bytes of out and dout each.
template <int D>
__global__ void __launch_bounds__(256) bwd_window_prepare_kernel(const __nv_bfloat16* __restrict__ out,
                                                                 const __nv_bfloat16* __restrict__ dout,
                                                                 const float* __restrict__ lse,
                                                                 const __grid_constant__ BwdArgs a) {
  wait_for_previous();
  let_next_start();
  constexpr int LPR = D / 8;
  const WinTiles wt = WinTiles::make(a.sh.S, a.sh.cp, a.sh.lb);
  const int Hq = a.sh.Hq, sub = threadIdx.x % LPR;
  const unsigned gmask = ((1u << LPR) - 1u) << ((threadIdx.x & 31) & ~(LPR - 1));  // this row's lanes
  // a block per (tile, head, batch) and 256 / LPR rows of it at a time
  const int p = blockIdx.x % wt.nt;
  const long long bh = blockIdx.x / wt.nt;
  const int h = (int)(bh % Hq), b = (int)(bh / Hq);
  int ch, off;
  wt.split(p, ch, off);
  const int rows = wt.rows(off), mem = wt.mem(ch, off);
  float* lse_l2 = const_cast<float*>(a.lse_l2) + (bh * wt.nt + p) * kRows;
  float* delta = const_cast<float*>(a.delta) + (bh * wt.nt + p) * kRows;
#pragma unroll 4
  for (int r = threadIdx.x / LPR; r < kRows; r += 256 / LPR) {
    const bool valid = r < rows;
    float acc = 0.f;
    if (valid) {
      const size_t row = ((size_t)b * wt.S + mem + r) * Hq + h;
      const uint4 x = __ldcs(reinterpret_cast<const uint4*>(out + row * D) + sub);
      const uint4 g = __ldcs(reinterpret_cast<const uint4*>(dout + row * D) + sub);
      acc = fmaf(bf16lo(x.x), bf16lo(g.x), fmaf(bf16hi(x.x), bf16hi(g.x), acc));
      acc = fmaf(bf16lo(x.y), bf16lo(g.y), fmaf(bf16hi(x.y), bf16hi(g.y), acc));
      acc = fmaf(bf16lo(x.z), bf16lo(g.z), fmaf(bf16hi(x.z), bf16hi(g.z), acc));
      acc = fmaf(bf16lo(x.w), bf16lo(g.w), fmaf(bf16hi(x.w), bf16hi(g.w), acc));
      float4* z = reinterpret_cast<float4*>(a.dq_acc + row * D);
      z[sub] = make_float4(0.f, 0.f, 0.f, 0.f);
      z[sub + LPR] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) acc += __shfl_xor_sync(gmask, acc, o);
    if (sub == 0) {
      delta[r] = -acc;
      lse_l2[r] = valid ? -lse[bh * wt.S + mem + r] * 1.4426950408889634f : -INFINITY;
    }
  }
}

template <int D>
cudaError_t launch_t(const BwdArgs& a, cudaStream_t st) {
  auto kern = attn_bwd_window_kernel<D>;
  // more than half of an SM's shared memory: one CTA per SM, so the CTA's
  // 512-column TMEM allocation never waits for a neighbour
  constexpr int smem = FCfg<D>::SMEM > 120 * 1024 ? FCfg<D>::SMEM : 120 * 1024;
  // (once per device: driver calls of about a microsecond each)
  static unsigned long long ready = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready >> dev & 1)) {
    // setmaxnreg.inc only succeeds if the launch reserved kRegsLaunchF per thread
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    if (fa.numRegs != kRegsLaunchF) return cudaErrorInvalidConfiguration;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    if (dev < 64) ready |= 1ull << dev;
  }
  return launch_overlapped(kern, dim3(a.n_units), kThreadsF, smem, st, a);
}

}  // namespace

cudaError_t launch_bwd_window_prepare(const void* out, const void* dout, const float* lse, const BwdArgs& a,
                                      cudaStream_t st) {
  const WinTiles wt = WinTiles::make(a.sh.S, a.sh.cp, a.sh.lb);
  const dim3 blocks((unsigned)((long long)a.sh.B * a.sh.Hq * wt.nt));
  const auto* o = static_cast<const __nv_bfloat16*>(out);
  const auto* g = static_cast<const __nv_bfloat16*>(dout);
  return launch_overlapped(a.sh.Dqk == 64 ? bwd_window_prepare_kernel<64> : bwd_window_prepare_kernel<128>, blocks, 256, 0,
                           st, o, g, lse, a);
}

cudaError_t launch_attn_bwd_window(const BwdArgs& a, cudaStream_t st) {
  return a.sh.Dqk == 64 ? launch_t<64>(a, st) : launch_t<128>(a, st);
}

cudaError_t launch_bwd_window_finish(const BwdArgs& a, const WinJoin* joins, int n_joins, int num_sms, cudaStream_t st) {
  const long long n8 = (long long)a.sh.B * a.sh.S * a.sh.Hq * a.sh.Dqk / 8;
  const long long want = (n8 + 255) / 256, most = 16LL * num_sms;
  const int blocks_dq = (int)(want < most ? want : most);
  return launch_overlapped(a.sh.Dqk == 64 ? bwd_window_finish_kernel<64> : bwd_window_finish_kernel<128>,
                           dim3(blocks_dq + 8 * n_joins), 256, 0, st, a, joins, n8, blocks_dq);
}

}  // namespace cpattn
