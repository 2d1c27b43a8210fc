// Grouped-query decode over a sliding window with sinks, on a bf16 or a 4-bit
// KV cache.
//
// One query token per sequence, the one at position L - 1 (L = lens[b]): it
// sees the cache rows [0, min(sinks, L)) and [max(0, L - window), L), which
// are numbered 0 .. n-1 here (the sinks that lie before the window, then the
// window).  Per KV head, with the G = Hq/Hkv query heads of its group as the
// columns of every product:
//   S^T = K q^T            (positions x heads)
//   p = exp2(S^T - m)      running maximum m and sum l per head, fp32
//   O^T = V^T P^T          (channels x heads, fp32 accumulators)
//
// Bound: HBM.  A cached row is used once per KV head, so the floor is the
// visible rows' bytes; the products are m16n8k16 matrix instructions on
// registers (positions or channels as the 16 rows, heads as the 8 columns),
// which need no shared-memory operand tile and no round trip through TMEM: an
// item is 16 or 32 positions, so that a warp works alone on its own ring of
// asynchronous copies and the warps of an SM never wait for one another.
//
// Split: the visible rows of a (b, KV head) are cut into units of 4*CH
// positions, CH for each warp of a CTA; every warp keeps its own (m, l, O),
// and a CTA's warps are joined in shared memory.  Two ways to share the units
// (win_decode_split chooses, with both sides measured):
//  * a cluster of CTAs takes a (b, KV head), its CTAs the units in turn; they
//    join through distributed shared memory, in a fixed order.  No scratch,
//    one launch, nothing to search: least overhead.
//  * every CTA takes an even share of all units of the batch, in order, so
//    that lengths far apart, or few sequences, leave no SM behind; a
//    (b, KV head) that lies in one share is written by it, the others' parts
//    go to the caller's workspace and a second kernel joins them, in order.
// Measured (D = 128): 24 sequences of up to 32768 rows, window 4096, bf16, 8 KV
// heads: 56 us (6.5 TB/s); 8 sequences of 65536 to 131072 rows, 4 bits: 150 us
// (5.9 TB/s); one sequence, window 512: 4.7 us.
//
// 4-bit cache (layout: kv_int4.cu).  A nibble lined up under a mask is an fp16
// subnormal, code * 2^-24 (or * 2^-20 where it is taken one nibble higher), so
// the products run on the codes as they come out of the row, exactly, with no
// conversion; the power of two goes into q (scores) and into the end (output).
// The group's scale and zero enter outside the product:
//   S[t, h]  = sum_g scale[t, g] (codes_g . q_h) + zero[t, g] (sum of q_h over g)
//   O[d, h]  = sum_t (p[t, h] scale[t, g(d)]) code[t, d] + sum_t p[t, h] zero[t, g(d)]
// the scores' scales in fp32 on the accumulators, the output's as one scaled
// copy of P per group; the zeros as one more product each, whose small operand
// is the zeros as they lie in the parameter rows (the sums of q in two fp16
// parts, so that 22 bits of them take part).
//
// P and P scale are fp16, rounded by 2^-11 (against bf16's 2^-8) as long as they
// are no subnormals.  Small values under a row with most of the weight would make
// them such: then their codes lose their weight while their zeros and l keep it,
// and the row stands for its groups' least values.  So P is formed as 2^14 times
// the weight (o, oz and l alike, which cancels at the end), and a group's scales
// are taken over a bound, the least power of two from 2^-14 to 2^14 that no scale
// the warp has met exceeds; where it has to grow the sums so far are rescaled.  A
// subnormal's rounding is then 2^-39 of the bound for P scale, and 2^-25 of it,
// with P's weight, for the scale.
#include <algorithm>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace cpattn {
namespace {

constexpr int kWarpsW = 4;
constexpr int kThreadsW = kWarpsW * 32;
constexpr int kClusterRows = 4096;
// 4-bit cache: log2 of P's factor; pairs of fp16: the least and the most a group's bound may be (2^-14, 2^14), and
// what a pair of powers of two is taken from for their inverses (the exponents mirrored)
constexpr float kLift = 14.f;
constexpr uint32_t kBoundLeast = 0x04000400u, kBoundMost = 0x74007400u, kPow2Inverse = 0x78007800u;
// units of a warp after which the zeros' sums join the codes' (8 sequences of up to 131072 rows, flat scores: error
// 0.0024 -> 0.0017, of which 0.0016 is the result's rounding, 156 -> 161 us; after 4 or 8 units no less)
constexpr int kFold = 16;

// rows a sequence may see at most (the lengths are on the device)
long long win_decode_rows(const WinDecodeArgs& a) {
  return std::min<long long>(a.Smax, (long long)a.window + a.sinks);
}

template <bool INT4, int D>
struct WCfg {
  static constexpr int NG = D / 32;               // groups of a 4-bit row
  static constexpr int CH = INT4 ? 32 : 16;       // positions per step of a warp
  static constexpr int ROW = INT4 ? D / 2 : D * 2;  // bytes of a row (codes or bf16)
  static constexpr int PAR = INT4 ? D / 8 : 0;    // bytes of its parameters
  static constexpr int OFF_KP = CH * ROW;
  static constexpr int OFF_V = OFF_KP + CH * PAR;
  static constexpr int OFF_VP = OFF_V + CH * ROW;
  static constexpr int STAGE = OFF_VP + CH * PAR;
  static constexpr int NS = 2;                    // stages of a warp's ring
  static constexpr int RING = NS * STAGE;
};

template <int NT, int D>
struct WPart {  // a CTA's (or warp's) joined part of up to 8*NT heads
  float o[8 * NT][D + 4];  // (rows four words apart in the banks: a quarter warp's 16-byte stores meet each once)
  float m[8 * NT], l[8 * NT];
};

template <bool INT4, int D, int NT, bool SPLIT>
struct WSmem {
  static constexpr int RING = kWarpsW * WCfg<INT4, D>::RING;
  // a warp's part takes a stage of its ring once the warp has read it, where
  // it fits one (the other then loads ahead), or else the whole ring
  static constexpr bool AHEAD = (int)sizeof(WPart<NT, D>) <= WCfg<INT4, D>::STAGE;
  static_assert((int)sizeof(WPart<NT, D>) <= WCfg<INT4, D>::RING, "a part fits the ring");
  // after the rings: the CTA's joined part (cluster), or the search for its first unit (split)
  static constexpr int SMEM = RING + (SPLIT ? 128 : (int)sizeof(WPart<NT, D>));
  // CTAs per SM the registers are held to
  static constexpr int REGS = NT == 1 ? 4 : 2;
  static constexpr int FIT = 227 * 1024 / (SMEM + 1024);  // and that shared memory has room for
  static constexpr int CTAS = REGS < FIT ? REGS : FIT;
};

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
// the same, or zeros (nothing is read)
template <int BYTES>
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void* src, bool take) {
  const int n = take ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with nothing to add to (no registers to clear)
__device__ __forceinline__ void mma_f16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm2t(uint32_t addr, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {  // (a NaN gives the other operand)
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// both halves of x in [-1, 1]
__device__ __forceinline__ bool at_most_1(uint32_t x) {
  return __hble2(__habs2(*reinterpret_cast<const __half2*>(&x)), __half2half2(__ushort_as_half(0x3c00)));
}
__device__ __forceinline__ float h_lo(uint32_t x) { return __low2float(*reinterpret_cast<const __half2*>(&x)); }
__device__ __forceinline__ float h_hi(uint32_t x) { return __high2float(*reinterpret_cast<const __half2*>(&x)); }
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}

// the four nibble pairs of x, lowest first: fp16 subnormal pairs, the first and
// third worth code * 2^-24, the second and fourth code * 2^-20
__device__ __forceinline__ void nibbles(uint32_t x, uint32_t (&e)[4]) {
  e[0] = x & 0x000f000fu;
  e[1] = x & 0x00f000f0u;
  e[2] = (x >> 8) & 0x000f000fu;
  e[3] = (x >> 8) & 0x00f000f0u;
}

// where 16-byte piece c of row p of a 4-bit tile lies: rows trade places
// within pairs and pieces within the row, so that the score product's loads
// (rows 2m and 2m + 1 by eight lanes) and the value product's (rows 0, 2, 4, 6
// by sixteen lanes, half a row each) meet every bank once
template <int ROW>
__device__ __forceinline__ uint32_t off4(int p, int c) {
  const int s = (p & ~1) | ((p ^ (p >> 1)) & 1);
  return (uint32_t)(s * ROW + ((ROW == 64 ? c ^ (((p >> 2) & 1) << 1) : c) << 4));
}

// rows of a sequence of L positions that its last token sees, and where they lie
struct Visible {
  int n, ns, jump;  // rows; those before the window (sinks); row v >= ns is cache row v + jump
  __device__ __forceinline__ Visible(int L, int window, int sinks) {
    const int w0 = L > window ? L - window : 0;
    ns = sinks < w0 ? sinks : w0;
    n = L - w0 + ns;
    jump = w0 - ns;
  }
};

__device__ __forceinline__ int clamped(int L, int Smax) { return L < 0 ? 0 : (L > Smax ? Smax : L); }

// units of sequence b, for one KV head
__device__ __forceinline__ int units_of(const WinDecodeArgs& a, int b, int per) {
  return (Visible(clamped(a.lens[b], a.Smax), a.window, a.sinks).n + per - 1) / per;
}

template <bool INT4, int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(kThreadsW, WSmem<INT4, D, NT, SPLIT>::REGS)
    gqa_decode_window_kernel(const __grid_constant__ WinDecodeArgs a) {
  using C = WCfg<INT4, D>;
  using M = WSmem<INT4, D, NT, SPLIT>;
  using Part = WPart<NT, D>;
  constexpr int NG = C::NG, CH = C::CH, MT = CH / 16, UNIT = kWarpsW * CH;
  static_assert(C::NS == 2, "two stages");
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;  // row / head and column of the matrix fragments
  const int G = a.Hq / a.Hkv;
  const uint32_t ring = smem_u32(smem) + warp * C::RING;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // inputs written by earlier kernels are visible
  asm volatile("griddepcontrol.launch_dependents;");  // (only now: the joining kernel reads lens before its own wait)

  // ---- this CTA's units -------------------------------------------------------
  // a run of units: (b, g), its first unit, the step to the next and their number
  int b, g, ur, ustep, seg;
  long long left = 0;  // split: units after this run
  if constexpr (!SPLIT) {
    ustep = a.cluster;
    ur = blockIdx.x % ustep;
    const int bg = blockIdx.x / ustep;
    b = bg / a.Hkv;
    g = bg - b * a.Hkv;
    if (g == 0 && ur == 0 && tid == 0 && clamped(a.lens[b], a.Smax) != a.lens[b]) atomicExch(a.err, DEV_LENS_CLAMPED);
  } else {
    ustep = 1;
    long long* const sums = reinterpret_cast<long long*>(smem + M::RING);  // [kWarpsW], then the unit's sequence
    // inclusive scan over the block of 128 sequences' units: the threads' total, and what lies before this thread
    auto block_sum = [&](long long x, long long& before) {
      long long inc = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) sums[warp] = inc;
      __syncthreads();
      long long base = 0, all = 0;
#pragma unroll
      for (int w = 0; w < kWarpsW; ++w) {
        if (w < warp) base += sums[w];
        all += sums[w];
      }
      before = base + inc - x;
      return all;
    };
    long long total = 0, x = 0, before = 0, all = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreadsW) {
      const int bb = b0 + tid;
      x = bb < a.B ? (long long)units_of(a, bb, UNIT) * a.Hkv : 0;
      if (blockIdx.x == 0 && bb < a.B && clamped(a.lens[bb], a.Smax) != a.lens[bb]) atomicExch(a.err, DEV_LENS_CLAMPED);
      if (b0) __syncthreads();
      total += all = block_sum(x, before);
    }
    const long long shares = total < gridDim.x ? total : gridDim.x;  // (none is empty)
    if (blockIdx.x >= shares) return;
    const long long u0 = total * blockIdx.x / shares, u1 = total * (blockIdx.x + 1) / shares;
    // the sequence of unit u0 (of more than 128 sequences, the sums are formed again up to it)
    long long run = 0;
    for (int b0 = 0;; b0 += kThreadsW) {
      if (a.B > kThreadsW) {
        const int bb = b0 + tid;
        x = bb < a.B ? (long long)units_of(a, bb, UNIT) * a.Hkv : 0;
        __syncthreads();
        all = block_sum(x, before);
      }
      if (u0 < run + all) {
        if (u0 >= run + before && u0 < run + before + x) {
          sums[kWarpsW] = b0 + tid;
          sums[kWarpsW + 1] = u0 - run - before;
        }
        break;
      }
      run += all;
    }
    __syncthreads();
    b = (int)sums[kWarpsW];
    const int per = units_of(a, b, UNIT);
    g = (int)(sums[kWarpsW + 1] / per);
    ur = (int)(sums[kWarpsW + 1] - (long long)g * per);
    left = u1 - u0;
  }
  Visible vis(0, 0, 0);
  int nu = 0;       // units of the (b, g)
  size_t row0 = 0;  // its first cache row
  auto enter = [&]() {  // (b, g, ur) set: the rest of the run
    vis = Visible(clamped(a.lens[b], a.Smax), a.window, a.sinks);
    nu = (vis.n + UNIT - 1) / UNIT;
    row0 = ((size_t)b * a.Hkv + g) * a.Smax;
    if constexpr (SPLIT) {
      seg = (int)(nu - ur < left ? nu - ur : left);
      left -= seg;
    } else {
      seg = nu > ur ? (nu - ur + ustep - 1) / ustep : 0;
    }
  };
  enter();

  const unsigned char* kc = static_cast<const unsigned char*>(a.kc);
  const unsigned char* vc = static_cast<const unsigned char*>(a.vc);
  const unsigned char* kp = static_cast<const unsigned char*>(a.kp);
  const unsigned char* vp = static_cast<const unsigned char*>(a.vp);
  constexpr int PC = C::ROW / 16, RI = 32 / PC;  // 16-byte pieces of a row, rows a warp copies at a time
  const int lp = lane / PC, lc = lane % PC;
  const uint32_t loff = INT4 ? off4<C::ROW>(lp, lc) : 0;
  // unit u of the (b, g) into a stage: this warp's CH rows of it
  auto load = [&](int u, int stage) {
    const int n = vis.n, ns = vis.ns, jump = vis.jump;
    const int v0 = (u * kWarpsW + warp) * CH;
    if (v0 < n) {
      const uint32_t st = ring + stage * C::STAGE;
      if (v0 + CH <= n && (v0 >= ns || v0 + CH <= ns)) {
        // CH rows that follow one another in the cache
        const size_t row = row0 + (v0 < ns ? v0 : v0 + jump);
        const unsigned char* gk = kc + row * C::ROW + lane * 16;
        const unsigned char* gv = vc + row * C::ROW + lane * 16;
#pragma unroll
        for (int i = 0; i < CH / RI; ++i) {
          // (rows 8i .. of a 4-bit tile are placed like rows 0 .. 7)
          const int p = i * RI + lp;
          const uint32_t off = INT4 && RI % 8 == 0 ? i * 512 + loff
                               : INT4              ? off4<C::ROW>(p, lc)
                                                   : (uint32_t)(p * C::ROW + ((lc ^ (p & 7)) << 4));
          cp_async<16>(st + off, gk + i * 512);
          cp_async<16>(st + C::OFF_V + off, gv + i * 512);
        }
        if constexpr (INT4) {
          cp_async<C::PAR>(st + C::OFF_KP + lane * C::PAR, kp + (row + lane) * C::PAR);
          cp_async<C::PAR>(st + C::OFF_VP + lane * C::PAR, vp + (row + lane) * C::PAR);
        }
      } else {
        // the sinks' end and the last rows: row by row, zeros past the end
#pragma unroll 1
        for (int i = 0; i < CH / RI; ++i) {
          const int p = i * RI + lp, v = v0 + p;
          const bool in = v < n;
          const size_t row = row0 + (in ? (v < ns ? v : v + jump) : 0);
          const uint32_t off = INT4 ? off4<C::ROW>(p, lc) : (uint32_t)(p * C::ROW + ((lc ^ (p & 7)) << 4));
          cp_async_or_zero<16>(st + off, kc + row * C::ROW + lc * 16, in);
          cp_async_or_zero<16>(st + C::OFF_V + off, vc + row * C::ROW + lc * 16, in);
        }
        if constexpr (INT4) {
          const int v = v0 + lane;
          const bool in = v < n;
          const size_t row = row0 + (in ? (v < ns ? v : v + jump) : 0);
          cp_async_or_zero<C::PAR>(st + C::OFF_KP + lane * C::PAR, kp + row * C::PAR, in);
          cp_async_or_zero<C::PAR>(st + C::OFF_VP + lane * C::PAR, vp + row * C::PAR, in);
        }
      }
    }
  };
  int stage = 0;  // of the next unit
  if (seg > 0) load(ur, stage);
  cp_commit();
  bool opening = true;  // split: the CTA's first run

  while (true) {

  // ---- the group's queries as the B operand of the scores -------------------
  // bf16: plain.  4-bit: fp16, scaled per head by a power of two that takes its
  // largest value to [2^9, 2^10) (so that a sixteenth of it, which meets the
  // nibbles taken one higher, is still exact), and its sums over the groups.
  uint32_t qb[NT][D / 16][2];
  uint32_t qz[NT];                 // 4-bit: the sums over the groups as the B operand of the zeros' product: column k
                                   // < 4 the sum over group k (fp16), column 4 + k what its rounding left
  float sc[NT][2];                 // what takes a score of head 2c, 2c + 1 to the log2 domain
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int h = t * 8 + r;  // this lane's head as the fragment's column
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + ((size_t)b * a.Hq + (size_t)g * G + (h < G ? h : 0)) * D;
    if constexpr (!INT4) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qb[t][kk][0] = h < G ? *reinterpret_cast<const uint32_t*>(q + kk * 16 + 2 * c) : 0u;
        qb[t][kk][1] = h < G ? *reinterpret_cast<const uint32_t*>(q + kk * 16 + 2 * c + 8) : 0u;
      }
      sc[t][0] = sc[t][1] = a.scale_log2;
    } else {
      // channels 32 gg + 8c .. + 7 of every group
      float f[NG][8];
      float mx = 0.f;
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) {
        const uint4 u = h < G ? *reinterpret_cast<const uint4*>(q + gg * 32 + c * 8) : make_uint4(0, 0, 0, 0);
        f[gg][0] = bf16lo(u.x); f[gg][1] = bf16hi(u.x); f[gg][2] = bf16lo(u.y); f[gg][3] = bf16hi(u.y);
        f[gg][4] = bf16lo(u.z); f[gg][5] = bf16hi(u.z); f[gg][6] = bf16lo(u.w); f[gg][7] = bf16hi(u.w);
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(f[gg][i]));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // exponent of the largest value; zero, subnormal and non-finite heads are left as they are
      const int e = (int)(__float_as_uint(mx) >> 23);
      const bool plain = e < 10 || e == 255;
      const float up = plain ? 1.f : __uint_as_float((uint32_t)(127 + 9 + 127 - e) << 23);
      const float down = plain ? 1.f : __uint_as_float((uint32_t)(e - 9) << 23);
      float s8[NG];
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) {
        s8[gg] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[gg][i] *= up;
          s8[gg] += f[gg][i];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          qb[t][2 * gg + j][0] = pack_f16(f[gg][2 * j], f[gg][2 * j + 4]);
          qb[t][2 * gg + j][1] = pack_f16(f[gg][2 * j + 1] * 0.0625f, f[gg][2 * j + 5] * 0.0625f);
        }
        s8[gg] += __shfl_xor_sync(0xffffffffu, s8[gg], 1);
        s8[gg] += __shfl_xor_sync(0xffffffffu, s8[gg], 2);
      }
      // this lane's columns 2c, 2c + 1 (every lane of a head holds all its sums; at D = 64 columns 2, 3, 6, 7 are 0)
      const float z0 = NG == 4 && (c & 1) ? s8[NG - 2] : (c & 1) ? 0.f : s8[0];
      const float z1 = NG == 4 && (c & 1) ? s8[NG - 1] : (c & 1) ? 0.f : s8[1];
      qz[t] = pack_f16(z0, z1);
      if (c >= 2) qz[t] = pack_f16(z0 - h_lo(qz[t]), z1 - h_hi(qz[t]));
      // to the lanes whose accumulator columns are the heads 2c, 2c + 1 (lane 4h holds head h)
#pragma unroll
      for (int j = 0; j < 2; ++j) sc[t][j] = __shfl_sync(0xffffffffu, down, (2 * c + j) * 4) * a.scale_log2;
    }
  }

  // ---- the warp's positions ---------------------------------------------------
  float o[NT][D / 16][4];          // O^T: rows = channels, columns = heads 2c, 2c + 1
  float oz[NT][4];                 // 4-bit: sum of p * zero, row r = group r % NG (D = 128: rows 4 .. 7)
  float m[NT][2], l[NT][2];        // heads 2c, 2c + 1 (log2 domain; l: this lane's rows only)
  uint32_t over[NG / 2];           // 4-bit: 1 over the bounds of the groups' value scales (pairs); o is in their units
#pragma unroll
  for (int i = 0; i < NG / 2; ++i) over[i] = kPow2Inverse - kBoundLeast;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[t][i][j] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) oz[t][j] = 0.f;
    m[t][0] = m[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.f;
  }
  // where this lane's pieces of a 4-bit tile's first rows lie (eight rows on: 8 * ROW bytes on)
  const uint32_t ko = NG == 4 ? off4<C::ROW>(r, c) : off4<C::ROW>(r, c >> 1) + (c & 1) * 8;
  const uint32_t kpo = C::OFF_KP + r * C::PAR;
  const uint32_t vo0 = C::OFF_V + (NG == 4 ? off4<C::ROW>(2 * c, r >> 1) + (r & 1) * 8 : off4<C::ROW>(2 * c, r >> 2) + (r & 3) * 4);
  const uint32_t vo1 =
      C::OFF_V + (NG == 4 ? off4<C::ROW>(2 * c + 1, r >> 1) + (r & 1) * 8 : off4<C::ROW>(2 * c + 1, r >> 2) + (r & 3) * 4);
  const uint32_t vpo = C::OFF_VP + 2 * c * C::PAR;
  // the lanes of accumulator row gg (D = 128: 4 + gg) hold the zeros' share of group gg for the same heads
  auto zeros_of = [&](float x, int gg) { return __shfl_sync(0xffffffffu, x, 4 * (gg + (NG == 4 ? 4 : 0)) + c); };
  for (int i = 0; i < seg; ++i) {
    const int u = ur + i * ustep;
    if (i + 1 < seg) load(u + ustep, stage ^ 1);
    cp_commit();  // (a group per unit, empty at the end of a run, so that all but the newest are the current unit's)
    cp_wait<1>();
    __syncwarp();
    const uint32_t st = ring + stage * C::STAGE;
    const int rows = vis.n - (u * kWarpsW + warp) * CH;  // of this warp's share that exist
    if (rows > 0) {
    // 4-bit: is a value scale of this lane's row (past the end: zeros) beyond its bound?
    const uint32_t va = st + C::OFF_VP + lane * C::PAR;
    bool grow = false;
    if constexpr (INT4) {
      uint2 x = make_uint2(0u, 0u);
      if constexpr (NG == 4) x = lds64(va);
      else x.x = lds32(va);
      grow = !at_most_1(hmul2(x.x, over[0])) || (NG == 4 && !at_most_1(hmul2(x.y, over[NG / 2 - 1])));
    }
    // scores of MT x 16 positions: rows r and r + 8
    float s[NT][MT][4];
    if constexpr (!INT4)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[t][mt][j] = 0.f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if constexpr (!INT4) {
        // lane l gives the address of row l % 16, piece l / 16 of the 16 x 16 block
        const int p = mt * 16 + (lane & 15);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t k4[4];
          ldsm4(st + p * C::ROW + (((2 * kk + (lane >> 4)) ^ (p & 7)) << 4), k4);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_bf16(s[t][mt], k4[0], k4[1], k4[2], k4[3], qb[t][kk][0], qb[t][kk][1]);
        }
      } else {
        uint32_t kw[2][NG];      // codes: rows r, r + 8; this lane's 8 channels of every group
        uint32_t ps[2][NG / 2];  // the rows' scales
        uint32_t z[2];           // their zeros of groups 2c, 2c + 1 (mod NG), the A operand against qz
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t row8 = mt * 2 + hf;
          const uint32_t pa = st + kpo + row8 * (8 * C::PAR);
          if constexpr (NG == 4) {
            const uint4 u = lds128(st + ko + row8 * (8 * C::ROW));
            kw[hf][0] = __byte_perm(u.x, u.z, 0x5410);
            kw[hf][1] = __byte_perm(u.x, u.z, 0x7632);
            kw[hf][2] = __byte_perm(u.y, u.w, 0x5410);
            kw[hf][3] = __byte_perm(u.y, u.w, 0x7632);
            const uint2 v = lds64(pa);
            ps[hf][0] = v.x;
            ps[hf][1] = v.y;
            z[hf] = lds32(pa + 8 + (c & 1) * 4);
          } else {
            const uint2 u = lds64(st + ko + row8 * (8 * C::ROW));
            kw[hf][0] = __byte_perm(u.x, u.y, 0x5410);
            kw[hf][1] = __byte_perm(u.x, u.y, 0x7632);
            const uint2 v = lds64(pa);
            ps[hf][0] = v.x;
            z[hf] = v.y;  // (columns 2, 3, 6, 7 meet zeros of qz)
          }
        }
        float acc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_f16_new(s[t][mt], z[0], z[1], 0u, 0u, qz[t], 0u);
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          uint32_t e0[4], e1[4];
          nibbles(kw[0][gg], e0);
          nibbles(kw[1][gg], e1);
          const float s0 = (gg & 1) ? h_hi(ps[0][gg / 2]) : h_lo(ps[0][gg / 2]);
          const float s1 = (gg & 1) ? h_hi(ps[1][gg / 2]) : h_lo(ps[1][gg / 2]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float x[4];
            mma_f16_new(x, e0[0], e1[0], e0[1], e1[1], qb[t][2 * gg][0], qb[t][2 * gg][1]);
            mma_f16(x, e0[2], e1[2], e0[3], e1[3], qb[t][2 * gg + 1][0], qb[t][2 * gg + 1][1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[t][j] = gg ? fmaf(j < 2 ? s0 : s1, x[j], acc[t][j]) : (j < 2 ? s0 : s1) * x[j];
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[t][mt][j] = fmaf(acc[t][j], 0x1p24f, s[t][mt][j]);
      }
    }
    if (rows < CH) {  // the last rows: none past the end
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (mt * 16 + (j >> 1) * 8 + r >= rows) s[t][mt][j] = -INFINITY;
    }
    // running maximum, probabilities (P^T as the B operand: rows of positions turned into columns)
    uint32_t pb[NT][MT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j & 1] = fmaxf(mx[j & 1], s[t][mt][j]);
      float f[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], off));
        // (4-bit: rounded up, so that no P passes 2^kLift)
        const float mn = fmaxf(m[t][j], INT4 ? __fmul_ru(mx[j], sc[t][j]) : mx[j] * sc[t][j]);
        f[j] = (mn == m[t][j]) ? 1.f : fast_exp2(m[t][j] - mn);
        m[t][j] = mn;
        mx[j] = mn == -INFINITY ? 0.f : (INT4 ? __fadd_ru(mn, -kLift) : mn);
      }
      const bool fold = INT4 && i % kFold == kFold - 1;
      if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f || (INT4 && t == 0 && grow) || fold)) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[t][i][j] *= f[j & 1];
#pragma unroll
        for (int j = 0; j < 4; ++j) oz[t][j] *= f[j & 1];
        l[t][0] *= f[0];
        l[t][1] *= f[1];
        if constexpr (INT4) {
          // (A flat cache's two sums grow with the rows and cancel; the matrix instruction rounds each time by what it
          // adds to.  So now and then the zeros' sums go where the codes' are.)
          if (fold) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
              for (int gg = 0; gg < NG; ++gg) {
                const float z = zeros_of(oz[t][j], gg);
                const float g = ((gg & 1) ? h_hi(over[gg / 2]) : h_lo(over[gg / 2])) * 0x1p-24f;
                o[t][2 * gg][j] = fmaf(z, g, o[t][2 * gg][j]);
                o[t][2 * gg][2 + j] = fmaf(z, g * 16.f, o[t][2 * gg][2 + j]);
                o[t][2 * gg + 1][j] = fmaf(z, g, o[t][2 * gg + 1][j]);
                o[t][2 * gg + 1][2 + j] = fmaf(z, g * 16.f, o[t][2 * gg + 1][2 + j]);
              }
              oz[t][j] = 0.f;
            }
          }
          if (t == 0 && __any_sync(0xffffffffu, grow)) {
            // a scale is past its bound: the bounds raised, what is summed so far (all heads') in units of the new ones
#pragma unroll
            for (int k = 0; k < NG / 2; ++k) {
              const uint32_t was = kPow2Inverse - over[k];
              uint32_t up = hmax2(lds32(va + 4 * k) & 0x7fff7fffu, was);
#pragma unroll
              for (int off = 1; off < 32; off <<= 1) up = hmax2(up, __shfl_xor_sync(0xffffffffu, up, off));
              up = hmin2((up + 0x03ff03ffu) & 0x7c007c00u, kBoundMost);  // to a power of two
              over[k] = kPow2Inverse - up;
              const float g0 = h_lo(was) * h_lo(over[k]), g1 = h_hi(was) * h_hi(over[k]);
#pragma unroll
              for (int tt = 0; tt < NT; ++tt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  o[tt][4 * k][j] *= g0;
                  o[tt][4 * k + 1][j] *= g0;
                  o[tt][4 * k + 2][j] *= g1;
                  o[tt][4 * k + 3][j] *= g1;
                }
            }
          }
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = fast_exp2(fmaf(s[t][mt][j], sc[t][j & 1], -mx[j & 1]));
        l[t][0] += p[0] + p[2];
        l[t][1] += p[1] + p[3];
        pb[t][mt][0] = movmatrix(INT4 ? pack_f16(p[0], p[1]) : pack_bf16(p[0], p[1]));
        pb[t][mt][1] = movmatrix(INT4 ? pack_f16(p[2], p[3]) : pack_bf16(p[2], p[3]));
      }
    }
    // O^T += V^T P^T
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if constexpr (!INT4) {
        // transposed 8 x 8 blocks: lane l gives row l % 8 + 8 * (l / 16) (positions), piece (l / 8) % 2 (channels)
        const int p = mt * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t v4[4];
          ldsm4t(st + C::OFF_V + p * C::ROW + (((2 * i + ((lane >> 3) & 1)) ^ (p & 7)) << 4), v4);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_bf16(o[t][i], v4[0], v4[1], v4[2], v4[3], pb[t][mt][0], pb[t][mt][1]);
        }
      } else {
        // this lane's positions: 2c, 2c + 1 (first pair), 2c + 8, 2c + 9 (second); its
        // channels: 4r .. 4r + 3 of every group
        uint32_t x[2][NG];      // pair, group: nibbles of the pair's two positions
        uint32_t sg[2][NG];     // the pair's scales of the group, over their bound
        uint32_t zz[2];         // the pair's zeros of group r % NG (D = 128: in rows 4 .. 7)
        if constexpr (NG == 4) {
          // the parameter rows (scales, then zeros) of eight positions are an 8 x 8 matrix: transposed, rows 4 .. 7
          // are the groups' zeros as an A operand's rows
          ldsm2t(st + C::OFF_VP + (mt * 16 + (lane & 15)) * C::PAR, zz[0], zz[1]);
        }
#pragma unroll
        for (int pp = 0; pp < 2; ++pp) {
          const uint32_t row8 = mt * 2 + pp;
          const uint32_t va0 = st + vo0 + row8 * (8 * C::ROW), va1 = st + vo1 + row8 * (8 * C::ROW);
          const uint32_t vpa = st + vpo + row8 * (8 * C::PAR);
          if constexpr (NG == 4) {
            const uint2 u0 = lds64(va0), u1 = lds64(va1);
            x[pp][0] = __byte_perm(u0.x, u1.x, 0x5410);
            x[pp][1] = __byte_perm(u0.x, u1.x, 0x7632);
            x[pp][2] = __byte_perm(u0.y, u1.y, 0x5410);
            x[pp][3] = __byte_perm(u0.y, u1.y, 0x7632);
            uint2 a0 = lds64(vpa), a1 = lds64(vpa + C::PAR);
            a0.x = hmul2(a0.x, over[0]);
            a1.x = hmul2(a1.x, over[0]);
            a0.y = hmul2(a0.y, over[NG / 2 - 1]);
            a1.y = hmul2(a1.y, over[NG / 2 - 1]);
            sg[pp][0] = __byte_perm(a0.x, a1.x, 0x5410);
            sg[pp][1] = __byte_perm(a0.x, a1.x, 0x7632);
            sg[pp][2] = __byte_perm(a0.y, a1.y, 0x5410);
            sg[pp][3] = __byte_perm(a0.y, a1.y, 0x7632);
          } else {
            const uint32_t u0 = lds32(va0), u1 = lds32(va1);
            x[pp][0] = __byte_perm(u0, u1, 0x5410);
            x[pp][1] = __byte_perm(u0, u1, 0x7632);
            uint2 a0 = lds64(vpa), a1 = lds64(vpa + C::PAR);
            a0.x = hmul2(a0.x, over[0]);
            a1.x = hmul2(a1.x, over[0]);
            sg[pp][0] = __byte_perm(a0.x, a1.x, 0x5410);
            sg[pp][1] = __byte_perm(a0.x, a1.x, 0x7632);
            zz[pp] = __byte_perm(a0.y, a1.y, (r & 1) ? 0x7632 : 0x5410);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_f16(oz[t], zz[0], 0u, zz[1], 0u, pb[t][mt][0], pb[t][mt][1]);
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          uint32_t e0[4], e1[4];
          nibbles(x[0][gg], e0);
          nibbles(x[1][gg], e1);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint32_t b0 = hmul2(pb[t][mt][0], sg[0][gg]), b1 = hmul2(pb[t][mt][1], sg[1][gg]);
            // rows r: channel 4r + 2j of the group, rows r + 8: channel 4r + 2j + 1
            mma_f16(o[t][2 * gg], e0[0], e0[1], e1[0], e1[1], b0, b1);
            mma_f16(o[t][2 * gg + 1], e0[2], e0[3], e1[2], e1[3], b0, b1);
          }
        }
      }
    }
    }
    __syncwarp();  // every lane has read the stage before it is filled again
    stage ^= 1;
  }

  // ---- join the CTA's warps -----------------------------------------------------
  const int n0 = vis.n;
  const bool whole = SPLIT && ur == 0 && seg == nu;
  __nv_bfloat16* const og = static_cast<__nv_bfloat16*>(a.out) + ((size_t)b * a.Hq + (size_t)g * G) * D;
  // the warp's part goes to the stage it read last; the other loads ahead
  Part& mine = *reinterpret_cast<Part*>(smem + warp * C::RING + (M::AHEAD ? (stage ^ 1) * C::STAGE : 0));
  const bool more = SPLIT && left > 0;
  auto next_run = [&]() {  // the first unit of the next (b, g) that has any
    if (++g == a.Hkv) {
      g = 0;
      do ++b; while (units_of(a, b, UNIT) == 0);  // (more units follow, so there is one)
    }
    ur = 0;
    enter();
    load(0, stage);
  };
  if (M::AHEAD && more) next_run();
  cp_commit();
  {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], off);
        if (r == 0) {
          mine.m[t * 8 + 2 * c + j] = m[t][j];
          mine.l[t * 8 + 2 * c + j] = l[t][j];
        }
      }
      if constexpr (!INT4) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) mine.o[t * 8 + 2 * c + (j & 1)][i * 16 + (j >> 1) * 8 + r] = o[t][i][j];
      } else {
#pragma unroll
        for (int gg = 0; gg < NG; ++gg)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float z = zeros_of(oz[t][j], gg);
            const uint32_t bound = kPow2Inverse - over[gg / 2];
            const float u = (gg & 1) ? h_hi(bound) : h_lo(bound), u0 = u * 0x1p24f, u1 = u * 0x1p20f;
            *reinterpret_cast<float4*>(&mine.o[t * 8 + 2 * c + j][gg * 32 + r * 4]) =
                make_float4(fmaf(o[t][2 * gg][j], u0, z), fmaf(o[t][2 * gg][2 + j], u1, z),
                            fmaf(o[t][2 * gg + 1][j], u0, z), fmaf(o[t][2 * gg + 1][2 + j], u1, z));
          }
      }
    }
  }
  __syncthreads();
  auto part = [&](int w) -> const Part& {
    return *reinterpret_cast<const Part*>(reinterpret_cast<const unsigned char*>(&mine) + (w - warp) * C::RING);
  };
  Part& joined = *reinterpret_cast<Part*>(smem + M::RING);  // cluster
  float* const slot = SPLIT ? a.parts + ((size_t)blockIdx.x * 2 + (opening ? 0 : 1)) * G * (D + 2) : nullptr;
  const int cs = SPLIT ? 1 : a.cluster;
  for (int x = tid; x < G * D; x += kThreadsW) {
    const int h = x / D, d = x - h * D;
    float mj = part(0).m[h];
#pragma unroll
    for (int w = 1; w < kWarpsW; ++w) mj = fmaxf(mj, part(w).m[h]);
    const float ref = mj == -INFINITY ? 0.f : mj;
    float acc = 0.f, ls = 0.f;
#pragma unroll
    for (int w = 0; w < kWarpsW; ++w) {
      const float f = fast_exp2(part(w).m[h] - ref);
      acc = fmaf(part(w).o[h][d], f, acc);
      ls = fmaf(part(w).l[h], f, ls);
    }
    if (SPLIT ? whole : cs == 1) {
      og[x] = __float2bfloat16(n0 ? acc / ls : 0.f);  // a sequence without rows gives zeros
    } else if (SPLIT) {
      slot[x] = acc;
      if (d == 0) {
        slot[G * D + h] = mj;
        slot[G * D + G + h] = ls;
      }
    } else {
      joined.o[h][d] = acc;
      if (d == 0) {
        joined.m[h] = mj;
        joined.l[h] = ls;
      }
    }
  }
  if constexpr (SPLIT) {
    if (!more) return;
    opening = false;
    __syncthreads();  // the parts are read: their space loads again
    if (!M::AHEAD) {
      next_run();
      cp_commit();
    }
    continue;
  }
  if (cs == 1) return;
  // ---- join the cluster's CTAs: each takes a share of the outputs ------------------
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  const uint32_t ja = smem_u32(&joined);
  auto remote = [&](uint32_t addr, int cta) {
    uint32_t ra;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(addr), "r"(cta));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(ra) : "memory");
    return v;
  };
  for (int x = ur * kThreadsW + tid; x < G * D; x += cs * kThreadsW) {
    const int h = x / D, d = x - h * D;
    const uint32_t oo = ja + (uint32_t)offsetof(Part, o) + (h * (D + 4) + d) * 4;
    const uint32_t om = ja + (uint32_t)offsetof(Part, m) + h * 4, ol = ja + (uint32_t)offsetof(Part, l) + h * 4;
    float mj = -INFINITY, acc = 0.f, ls = 0.f;
    for (int k = 0; k < cs; ++k) {
      const float mk = remote(om, k), lk = remote(ol, k), ok = remote(oo, k);
      const float mn = fmaxf(mj, mk), ref = mn == -INFINITY ? 0.f : mn;
      const float fo = fast_exp2(mj - ref), fn = fast_exp2(mk - ref);
      acc = fmaf(ok, fn, acc * fo);
      ls = fmaf(lk, fn, ls * fo);
      mj = mn;
    }
    og[x] = __float2bfloat16(n0 ? acc / ls : 0.f);
  }
  // no CTA leaves while another may still read its part
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  return;
  }
}

// Split: joins the parts of every (b, KV head) that lies in more than one
// CTA's share, in the shares' order, and writes the zeros of sequences without
// rows.  A block per (b, KV head) and query head; JT / D groups of threads take
// the parts in turn.
template <int D, int JT>
__global__ void __launch_bounds__(JT) gqa_decode_join_kernel(const __grid_constant__ WinDecodeArgs a, int unit, int shares) {
  __shared__ long long red[2][JT / 32];
  __shared__ float go[JT / D][D], gm[JT / D], gl[JT / D];
  const int tid = threadIdx.x, G = a.Hq / a.Hkv;
  const int bg = blockIdx.x, h = blockIdx.y, b = bg / a.Hkv, g = bg - b * a.Hkv;
  // (lens was written before the attention kernel passed its own wait, after which this grid may start)
  long long total = 0, before = 0;
  for (int bb = tid; bb < a.B; bb += JT) {
    const long long x = (long long)units_of(a, bb, unit) * a.Hkv;
    total += x;
    if (bb < b) before += x;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if ((tid & 31) == 0) {
    red[0][tid >> 5] = total;
    red[1][tid >> 5] = before;
  }
  __syncthreads();
  total = before = 0;
  for (int w = 0; w < JT / 32; ++w) {
    total += red[0][w];
    before += red[1][w];
  }
  const int nu = units_of(a, b, unit);
  const int grp = tid / D, d = tid - grp * D;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((size_t)b * a.Hq + (size_t)g * G + h) * D + d;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are complete
  asm volatile("griddepcontrol.launch_dependents;");
  if (nu == 0) {
    if (grp == 0) *out = __float2bfloat16(0.f);
    return;
  }
  if (total < shares) shares = (int)total;
  // unit u lies in share ((u + 1) * shares - 1) / total
  const long long p0 = before + (long long)g * nu, p1 = p0 + nu - 1;
  const long long s0 = ((p0 + 1) * shares - 1) / total, s1 = ((p1 + 1) * shares - 1) / total;
  if (s0 == s1) return;  // written by its CTA
  const size_t stride = (size_t)G * (D + 2);
  // the first share's part is its opening run only if the share begins with this (b, g)
  const size_t first = 2 * (size_t)s0 + (total * s0 / shares == p0 ? 0 : 1);
  float m = -INFINITY, l = 0.f, acc = 0.f;
  const int np = (int)(s1 - s0 + 1);
  constexpr int J = JT > 128 ? 8 : 4;  // parts in flight
  for (int i0 = grp; i0 < np; i0 += J * (JT / D)) {
    float po[J], pm[J], pl[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = i0 + j * (JT / D);
      const float* s = a.parts + (i ? 2 * (size_t)(s0 + i) : first) * stride;
      po[j] = i < np ? s[h * D + d] : 0.f;
      pm[j] = i < np ? s[G * D + h] : -INFINITY;
      pl[j] = i < np ? s[G * D + G + h] : 0.f;
    }
    float mn = m;
#pragma unroll
    for (int j = 0; j < J; ++j) mn = fmaxf(mn, pm[j]);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float f = fast_exp2(m - ref);
    acc *= f;
    l *= f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float w = fast_exp2(pm[j] - ref);
      acc = fmaf(po[j], w, acc);
      l = fmaf(pl[j], w, l);
    }
    m = mn;
  }
  if (JT > D) {
    go[grp][d] = acc;
    if (d == 0) {
      gm[grp] = m;
      gl[grp] = l;
    }
    __syncthreads();
    if (grp) return;
    m = gm[0];
    for (int k = 1; k < JT / D; ++k) m = fmaxf(m, gm[k]);
    const float ref = m == -INFINITY ? 0.f : m;
    acc = l = 0.f;
    for (int k = 0; k < JT / D; ++k) {
      const float w = fast_exp2(gm[k] - ref);
      acc = fmaf(go[k][d], w, acc);
      l = fmaf(gl[k], w, l);
    }
  }
  *out = __float2bfloat16(acc / l);
}

template <bool INT4, int D, int NT, bool SPLIT>
cudaError_t launch_t(const WinDecodeArgs& a0, int num_sms, cudaStream_t st) {
  WinDecodeArgs a = a0;
  using M = WSmem<INT4, D, NT, SPLIT>;
  auto kern = gqa_decode_window_kernel<INT4, D, NT, SPLIT>;
  constexpr int smem = M::SMEM, unit = kWarpsW * WCfg<INT4, D>::CH;
  static_assert(smem <= 232448, "shared memory budget");
  // (once per device: a driver call of about a microsecond)
  static unsigned long long ready = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready >> dev & 1)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    if (dev < 64) ready |= 1ull << dev;
  }
  const long long rows = (long long)a.B * a.Hkv, slots = (long long)num_sms * M::CTAS;
  const long long most = ((long long)win_decode_rows(a) + unit - 1) / unit;  // units of a row at most
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // its start overlaps the previous kernel's end
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreadsW);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if constexpr (!SPLIT) {
    // as many CTAs a row as can run at once, as long as each gets a unit
    a.cluster = (int)std::max(1LL, std::min({8LL, slots / rows, most}));
    cfg.gridDim = dim3((unsigned)(rows * a.cluster));
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
  } else {
    const int shares = (int)std::min(slots, rows * most);
    cfg.gridDim = dim3((unsigned)shares);
    if ((e = cudaLaunchKernelEx(&cfg, kern, a)) != cudaSuccess) return e;
    // more threads a block where a row has many parts
    constexpr int J1 = 128, J2 = 512;
    const bool many = shares > 16 * rows;
    cfg.gridDim = dim3((unsigned)rows, (unsigned)(a.Hq / a.Hkv));
    cfg.blockDim = dim3(many ? J2 : J1);
    cfg.dynamicSmemBytes = 0;
    return many ? cudaLaunchKernelEx(&cfg, gqa_decode_join_kernel<D, J2>, a, unit, shares)
                : cudaLaunchKernelEx(&cfg, gqa_decode_join_kernel<D, J1>, a, unit, shares);
  }
}

template <bool INT4, bool SPLIT>
cudaError_t launch_f(const WinDecodeArgs& a, int num_sms, cudaStream_t st) {
  const bool wide = a.Hq / a.Hkv > 8;
  if (a.D == 64) return wide ? launch_t<INT4, 64, 2, SPLIT>(a, num_sms, st) : launch_t<INT4, 64, 1, SPLIT>(a, num_sms, st);
  return wide ? launch_t<INT4, 128, 2, SPLIT>(a, num_sms, st) : launch_t<INT4, 128, 1, SPLIT>(a, num_sms, st);
}

}  // namespace

// Shares of all units cost a search for the first one and a second kernel, 2
// to 5 us; clusters cost what the longest row takes beyond the average one,
// and leave SMs idle where they are few (at most eight CTAs a (b, KV head)).
// So: clusters up to 4096 rows a sequence (4-bit cache, 24 sequences on 8 KV
// heads, 2048 to 4096 rows: clusters 25.4 us, shares 27.5; one sequence of
// 4096: 6.9 against 8.9; of 8000 rows on a bf16 cache: 12.4 against 10.6), and
// beyond where a window shorter than the cache makes the sequences see alike
// and the clusters fill the GPU (24 sequences, window 4096 of 32768, bf16: 56
// against 61 us).  Else shares (4-bit, 7 sequences of 65536 to 131072 rows on
// 8 KV heads: 148 against 213 us; one of 131072: 39 against 99).
bool win_decode_split(const WinDecodeArgs& a, int num_sms) {
  const long long most = win_decode_rows(a);
  if (most <= kClusterRows) return false;
  return most == a.Smax || (long long)a.B * a.Hkv * 8 < 4LL * num_sms;
}

size_t win_decode_bytes(const WinDecodeArgs& a, int num_sms) {
  if (!win_decode_split(a, num_sms)) return 0;
  // two parts a share; at most four shares an SM
  return (size_t)num_sms * 4 * 2 * (a.Hq / a.Hkv) * (a.D + 2) * sizeof(float);
}

cudaError_t launch_gqa_decode_window(const WinDecodeArgs& a, bool int4, int num_sms, cudaStream_t st) {
  if (win_decode_split(a, num_sms)) return int4 ? launch_f<true, true>(a, num_sms, st) : launch_f<false, true>(a, num_sms, st);
  return int4 ? launch_f<true, false>(a, num_sms, st) : launch_f<false, false>(a, num_sms, st);
}

}  // namespace cpattn
