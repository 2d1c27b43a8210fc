// The 4-bit KV cache: rows quantised into it and read back.
//
// A vector of D = 32*NG channels is cut into groups of 32 consecutive
// channels.  Per group (mn, mx its least and largest value, clamped to
// +-57344 so that scale * 15 + zero stays finite in fp16):
//   scale = fp16((mx - mn) / 15),  zero = fp16(mn),
//   code  = clamp(rint((x - zero) / scale), 0, 15)   (0 where scale is 0),
// and the cached value is scale * code + zero.  A group that holds a NaN or an
// infinity gets scale = zero = NaN: what it stands for is NaN, not a number
// that hides it.
//
// A row of codes is D/2 bytes.  Channel 32g + 4r + i (r < 8, i < 4) is nibble
// r*4*NG + 4g + i (low nibble of a byte first): halfword r*NG + g holds the
// four consecutive channels 4r .. 4r+3 of group g.  A row of parameters is NG
// scales, then NG zeros, fp16.  The order serves the decode: a lane of its
// value product takes the halfwords of one r (four channels of every group)
// in one load, a lane of its score product those of two or four, and the pairs
// of nibbles a byte permute lines up always belong to one group.
//
// An element is read and written once (bf16 2 bytes, cache 5/8 byte), which
// makes HBM the floor: reading is bound by it, the append by its instructions.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace cpattn {
namespace {

constexpr int kThreadsKv = 256;
constexpr int kAhead = 2;  // vectors a thread of the append has in flight
constexpr float kInt4Limit = 57344.f;

// n / d for n < 2^31: the quotient is (n * (2^32 + m) / 2^32) >> s with s =
// ceil(log2 d) and m = 2^32 (2^s - d) / d + 1 rounded down, a multiplication and a
// shift (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994)
struct Divider {
  uint32_t m, s;
  explicit Divider(uint32_t d) : s(0) {
    while ((1ull << s) < d) ++s;
    m = (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};

// the tokens of a sequence that take part: count[b] (T without a count array),
// clamped to [0, T] and flagged
__device__ __forceinline__ int kv_count(const KvInt4Args& a, int b) {
  if (!a.count) return a.T;
  const int n = a.count[b];
  if (n < 0 || n > a.T) {
    atomicExch(a.err, DEV_ROWS_SKIPPED);
    return n < 0 ? 0 : a.T;
  }
  return n;
}

// max and min of bf16 pairs that keep a NaN
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// what rounding a - b to d left: d and this are together exactly a - b (Knuth's TwoSum)
__device__ __forceinline__ float rest_of_diff(float a, float b, float d) {
  const float t = __fsub_rn(d, a);
  return __fsub_rn(__fsub_rn(a, __fsub_rn(d, t)), __fadd_rn(b, t));
}
// (v - z) / s to the nearest whole number, ties to the even one, q being the quotient to a few 2^-24: whether to go up
// from k = floor(q) is the sign of v - z - (k + 1/2) s.  Where the difference is not what fp32 makes of it (v far
// smaller than z) its rest decides what looks like a tie: (k + 1/2) s is a multiple of the difference's last place.
__device__ __forceinline__ int nearest_code(float v, float z, float s, float q) {
  const float d = v - z, k = floorf(q);
  float off = fmaf(-(k + 0.5f), s, d);
  if (off == 0.f) off = rest_of_diff(v, z, d);
  const int n = (int)k;
  return n + (off > 0.f || (off == 0.f && (n & 1)) ? 1 : 0);
}
// fp16((hi - lo) / 15), rounded once: the difference and the quotient are rounded to odd (an inexact one gets an odd
// last place, so that it lies on the same side of every fp16 and every midpoint as what it stands for).  This and the
// next, the long way's, are calls: inlined they cost the others registers (4 x 8192 tokens: 46 us instead of 44).
__device__ __noinline__ __half exact_scale(float hi, float lo) {
  uint32_t d = __float_as_uint(hi - lo);
  const float rest = rest_of_diff(hi, lo, hi - lo);
  if (rest < 0.f) d -= 1;
  if (rest != 0.f) d |= 1;
  const float df = __uint_as_float(d), q = __fdiv_rz(df, 15.f);
  const bool inexact = fmaf(-q, 15.f, df) != 0.f;
  return __float2half_rn(__uint_as_float(__float_as_uint(q) | (inexact ? 1u : 0u)));
}
__device__ __noinline__ int clamped_code(float v, float z, float s) {
  return min(max(nearest_code(v, z, s, (v - z) / s), 0), 15);
}
__device__ __forceinline__ float clamp_limit(float x) { return fminf(fmaxf(x, -kInt4Limit), kInt4Limit); }

// Two lanes per group, sixteen channels each (32 bytes, a sector), so that a
// warp reads whole lines: the group's range takes one shuffle, its parameters
// one, and one trade with the neighbouring group's lane turns halfwords of two
// groups into the words a row holds.  Vectors are numbered with the token
// innermost: the rows a warp writes then lie side by side in the cache (D =
// 128: 64 bytes of codes and 16 of parameters each), while it reads whole
// vectors either way.
//
// (x - zero) / scale in units of 2^-16 and half a code on, in one instruction a
// channel: x * (65536 / scale) + c, with c = 1.5 * 2^23 + 32768 - zero * (65536 /
// scale), so that the sum's low bits are the quotient's fixed point: bits 16 ..
// 19 the code rounded to nearest, the 16 bits below how far from a tie.  Two
// channels' codes are lined up in the halves of a register and added into the
// word with its shift, the exponent bits' sum taken off at the end.  c and the
// sum are rounded to half a unit each and 65536 / scale to a few 2^-24, so a
// code is certain three units from a tie.  Closer, the channel is decided
// exactly, by the sign of x - zero - (k + 1/2) scale (a tie goes to the even
// code): bf16 values over an 11-bit scale tie in about one channel of 2000.
// Where a code would leave [0, 15], a value is clamped or not finite, the scale
// is itself close to a rounding border, or zero is above 60 scales (then c
// leaves its binade), the lane goes the long way, with divisions.
//
// Measured on 4 x 8192 tokens of 8 heads (D = 128, 176 MB): 45 us (3.9 TB/s),
// bound by its instructions, 247 a lane and 16 channels, before HBM.  With a
// division each for scale and code it took 122 us, with four lanes a group 75.
template <int NG>
__global__ void __launch_bounds__(kThreadsKv, 4) kv_append_int4_kernel(const __grid_constant__ KvInt4Args a, Divider by_t,
                                                                    Divider by_h) {
  constexpr int D = 32 * NG, VL = 2 * NG;  // lanes of a vector
  const bool is_v = blockIdx.y != 0;
  const uint4* src = static_cast<const uint4*>(is_v ? a.v : a.k);
  unsigned char* codes = static_cast<unsigned char*>(is_v ? a.vcodes : a.kcodes);
  unsigned char* params = static_cast<unsigned char*>(is_v ? a.vparams : a.kparams);
  const uint32_t total = (uint32_t)a.B * a.T * a.Hkv;  // (below 2^31)
  const int l = threadIdx.x % VL, g = l / 2, j = l % 2;
  constexpr uint32_t PER = kThreadsKv / VL;  // vectors of a block at a time
  const uint32_t step = gridDim.x * PER;
  wait_for_previous();
  let_next_start();
  for (uint32_t v0 = blockIdx.x * PER; v0 < total; v0 += step * kAhead) {
    // all of the thread's loads first
    uint4 u[kAhead][2];
    size_t dst[kAhead];
    bool put[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint32_t vec = v0 + k * step + threadIdx.x / VL;
      const bool in = vec < total;
      const uint32_t bh = by_t.div(in ? vec : 0), t = (in ? vec : 0) - bh * (uint32_t)a.T;
      const uint32_t b = by_h.div(bh), h = bh - b * (uint32_t)a.Hkv;
      const long long row = (long long)a.start[b] + t;
      const bool take = in && (int)t < kv_count(a, (int)b);
      put[k] = take && row >= 0 && row < a.Smax;
      if (take && !put[k]) atomicExch(a.err, DEV_ROWS_SKIPPED);
      const uint4* s = src + (size_t)((b * (uint32_t)a.T + t) * (uint32_t)a.Hkv + h) * (D / 8) + 2 * l;
      u[k][0] = put[k] ? __ldcs(s) : make_uint4(0, 0, 0, 0);
      u[k][1] = put[k] ? __ldcs(s + 1) : make_uint4(0, 0, 0, 0);
      dst[k] = (size_t)bh * (size_t)a.Smax + (size_t)row;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint32_t x[8] = {u[k][0].x, u[k][0].y, u[k][0].z, u[k][0].w, u[k][1].x, u[k][1].y, u[k][1].z, u[k][1].w};
      // (greatest, -least) of the lane, then of the group
      uint32_t hi = x[0], lo = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        hi = max2(hi, x[i]);
        lo = min2(lo, x[i]);
      }
      const uint32_t nlo = lo ^ 0x80008000u;
      uint32_t rg = max2(__byte_perm(hi, nlo, 0x5410), __byte_perm(hi, nlo, 0x7632));
      rg = max2(rg, __shfl_xor_sync(0xffffffffu, rg, 1));
      const float mx = bf16lo(rg), mn = -bf16hi(rg);
      // scale: certain where the quotient's neighbours 2^-22 off round to the same
      const float y = (mx - mn) * (1.f / 15.f);
      const uint32_t y2 = pack_f16(y * (1.f - 0x1p-22f), y * (1.f + 0x1p-22f));
      __half hs = __ushort_as_half((unsigned short)y2), hz = __float2half_rn(mn);
      const float s = __half2float(hs), z = __half2float(hz);
      const float inv = s > 0.f ? rcp_approx(s) : 0.f, scale = inv * 65536.f;
      const float c = fmaf(-z, scale, 12582912.f + 32768.f + 3.f);
      uint32_t w[2], near = 0xffffffffu;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        w[q] = 0;
#pragma unroll
        for (int i = 3; i >= 0; --i) {  // channels i and i + 4 of eight
          const uint32_t p0 = x[4 * q + i / 2], p1 = x[4 * q + 2 + i / 2];
          const uint32_t f0 = __float_as_uint(fmaf((i & 1) ? bf16hi(p0) : bf16lo(p0), scale, c));
          const uint32_t f1 = __float_as_uint(fmaf((i & 1) ? bf16hi(p1) : bf16lo(p1), scale, c));
          near = min_u16x2(near, __byte_perm(f0, f1, 0x5410));
          w[q] = (w[q] << 4) + __byte_perm(f0, f1, 0x7632);
        }
        w[q] -= 0x4b404b40u * 0x1111u;  // the four sums' exponent bits
      }
      if ((y2 & 0xffffu) != y2 >> 16 || (mx - z) * inv > 15.49f || (mn - z) * inv < -0.49f || fabsf(z) * inv > 60.f ||
          !(fmaxf(mx, -mn) <= kInt4Limit)) {
        const bool bad = !(mx < INFINITY && mn > -INFINITY);  // a NaN or an infinity
        const float lo2 = clamp_limit(mn);
        hs = bad ? __ushort_as_half(0x7fff) : exact_scale(clamp_limit(mx), lo2);
        hz = bad ? __ushort_as_half(0x7fff) : __float2half_rn(lo2);
        const float s2 = __half2float(hs), z2 = __half2float(hz);
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          uint32_t v = 0;
#pragma unroll
          for (int i = 7; i >= 0; --i) {
            const uint32_t p = q ? x[4 + i / 2] : x[i / 2];
            const float x1 = clamp_limit((i & 1) ? bf16hi(p) : bf16lo(p));
            v = (v << 4) + (uint32_t)(s2 > 0.f ? clamped_code(x1, z2, s2) : 0);
          }
          if (q) w[1] = v;
          else w[0] = v;
        }
      } else if (min(near & 0xffffu, near >> 16) <= 6u) {
        // the pairs that come close to a tie, exactly.  (The other of a pair may lie below zero, which is rounded where
        // the least value is small, by less than half a scale: its code is 0.)
        auto code = [&](float v) { return (uint32_t)nearest_code(v, z, s, (v - z) * inv); };
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t p0 = x[4 * q + i / 2], p1 = x[4 * q + 2 + i / 2];
            const float x0 = (i & 1) ? bf16hi(p0) : bf16lo(p0), x1 = (i & 1) ? bf16hi(p1) : bf16lo(p1);
            if (min(__float_as_uint(fmaf(x0, scale, c)) & 0xffffu, __float_as_uint(fmaf(x1, scale, c)) & 0xffffu) <= 6u)
              w[q] = (w[q] & ~(0x000f000fu << (4 * i))) | (code(x0) | code(x1) << 16) << (4 * i);
          }
      }
      // w[q] holds halfwords r = 4j + 2q, 4j + 2q + 1 of group g.  The even group's lane takes the words of q = 0 of
      // both groups, the odd one's those of q = 1.
      const bool odd = g & 1;
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 2);
      const uint32_t ev = odd ? got : w[0], od = odd ? w[1] : got;  // of the even and of the odd group
      const uint32_t own = (uint32_t)__half_as_ushort(hs) | (uint32_t)__half_as_ushort(hz) << 16;
      const uint32_t oth = __shfl_xor_sync(0xffffffffu, own, 2);
      if (put[k]) {
        const int r = 4 * j + (odd ? 2 : 0);  // words r * NG / 2 + g / 2 and NG / 2 on
        uint32_t* cw = reinterpret_cast<uint32_t*>(codes + dst[k] * (D / 2)) + r * (NG / 2) + g / 2;
        const uint32_t c0 = __byte_perm(ev, od, 0x5410), c1 = __byte_perm(ev, od, 0x7632);
        if (NG == 2) {
          *reinterpret_cast<uint2*>(cw) = make_uint2(c0, c1);
        } else {
          cw[0] = c0;
          cw[NG / 2] = c1;
        }
        if (j == 0)
          reinterpret_cast<uint32_t*>(params + dst[k] * (D / 8))[(odd ? NG / 2 : 0) + g / 2] =
              odd ? __byte_perm(oth, own, 0x7632) : __byte_perm(own, oth, 0x5410);
      }
    }
  }
}

// One lane per 16 bytes of codes: 8 (D = 128) or 16 (D = 64) consecutive
// channels of every group, written as four 16-byte pieces.  Measured on the
// same tokens: 26 us (6.7 TB/s), HBM.
template <int NG>
__global__ void __launch_bounds__(kThreadsKv) kv_read_int4_kernel(const __grid_constant__ KvInt4Args a) {
  constexpr int D = 32 * NG;
  const bool is_v = blockIdx.y != 0;
  uint4* dst = static_cast<uint4*>(const_cast<void*>(is_v ? a.v : a.k));
  const unsigned char* codes = static_cast<const unsigned char*>(is_v ? a.vcodes : a.kcodes);
  const unsigned char* params = static_cast<const unsigned char*>(is_v ? a.vparams : a.kparams);
  const long long total = (long long)a.B * a.T * a.Hkv * NG;
  wait_for_previous();
  let_next_start();
  for (long long x = (long long)blockIdx.x * kThreadsKv + threadIdx.x; x < total; x += (long long)gridDim.x * kThreadsKv) {
    const int c = (int)(x % NG);
    const long long vec = x / NG;
    const int h = (int)(vec % a.Hkv);
    const long long bt = vec / a.Hkv;
    const int t = (int)(bt % a.T), b = (int)(bt / a.T);
    const long long row = (long long)a.start[b] + t;
    const bool take = t < kv_count(a, b);
    const bool load = take && row >= 0 && row < a.Smax;
    if (take && !load) atomicExch(a.err, DEV_ROWS_SKIPPED);
    uint4 u = make_uint4(0, 0, 0, 0);
    uint32_t pr[NG];  // scales, then zeros (pairs)
#pragma unroll
    for (int i = 0; i < NG; ++i) pr[i] = 0;
    if (load) {
      const size_t r = ((size_t)b * a.Hkv + h) * (size_t)a.Smax + (size_t)row;
      u = *reinterpret_cast<const uint4*>(codes + r * (D / 2) + c * 16);
      if (NG == 4) {
        const uint4 p = *reinterpret_cast<const uint4*>(params + r * (D / 8));
        pr[0] = p.x; pr[1] = p.y; pr[NG - 2] = p.z; pr[NG - 1] = p.w;
      } else {
        const uint2 p = *reinterpret_cast<const uint2*>(params + r * (D / 8));
        pr[0] = p.x; pr[1] = p.y;
      }
    }
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float s = __half2float(__ushort_as_half((unsigned short)(pr[g / 2] >> (16 * (g & 1)))));
      const float z = __half2float(__ushort_as_half((unsigned short)(pr[NG / 2 + g / 2] >> (16 * (g & 1)))));
      // this lane's halfwords of group g: r = (8 / NG) * c + j, halfword j * NG + g of the 16 bytes
      uint32_t o[16 / NG];
#pragma unroll
      for (int j = 0; j < 8 / NG; ++j) {
        const int hw = j * NG + g;
        const uint32_t x4 = w[hw / 2] >> (16 * (hw & 1));
#pragma unroll
        for (int i = 0; i < 2; ++i)
          o[2 * j + i] = pack_bf16(fmaf((float)(x4 >> (8 * i) & 15), s, z), fmaf((float)(x4 >> (8 * i + 4) & 15), s, z));
      }
#pragma unroll
      for (int j = 0; j < 4 / NG; ++j)  // 8 channels each
        dst[vec * (D / 8) + g * 4 + c * (4 / NG) + j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
    }
  }
}

// blocks for `lanes` lanes per vector, `ahead` vectors a thread where that leaves two blocks an SM
unsigned kv_blocks(const KvInt4Args& a, int lanes, int ahead, int num_sms) {
  const long long n = ((long long)a.B * a.T * a.Hkv * lanes + kThreadsKv - 1) / kThreadsKv;
  const long long few = 2LL * num_sms;
  return (unsigned)(n <= few ? n : n / ahead > few ? (n + ahead - 1) / ahead : few);
}

}  // namespace

cudaError_t launch_kv_append_int4(const KvInt4Args& a, int num_sms, cudaStream_t st) {
  const Divider by_t(a.T), by_h(a.Hkv);
  const dim3 grid(kv_blocks(a, a.D / 16, kAhead, num_sms), 2);
  return launch_overlapped(a.D == 128 ? kv_append_int4_kernel<4> : kv_append_int4_kernel<2>, grid, kThreadsKv, 0, st, a,
                           by_t, by_h);
}

cudaError_t launch_kv_read_int4(const KvInt4Args& a, int num_sms, cudaStream_t st) {
  const dim3 grid(kv_blocks(a, a.D / 32, 1, num_sms), 2);
  return launch_overlapped(a.D == 128 ? kv_read_int4_kernel<4> : kv_read_int4_kernel<2>, grid, kThreadsKv, 0, st, a);
}

}  // namespace cpattn
