// Key blocks chosen by a cheap score, and the bounds that the score reads.
//
//   bounds   min_e, max_e over the keys of a block, channel by channel (bf16): exact, so the result depends on the keys alone.
//   score    of block c for the queries of a query block (rows i of it, heads h that share the KV head):
//              s(c) = sum_{i,h} sum_e max(q_ihe min_e(c), q_ihe max_e(c)) = sum_e ( Q+_e max_e(c) + Q-_e min_e(c) ),
//            Q+_e = sum_{i,h} max(q_ihe, 0), Q-_e = sum_{i,h} min(q_ihe, 0): an upper bound of <q, k> over the block's keys, summed over
//            the queries. The sums over queries come first, so a block costs one product of 2 d, however many queries there are.
//   choice   the first and last few blocks of the mask's row, and of the others those with the largest score, ties to the lower column.
//
// The choice is that of scores in 64 bits, but hardly any is computed so: this GPU has two FP64 lanes an SM. Q+- are sums of whole numbers
// or of pairs of floats (an error of 2^-44 of their magnitudes, mostly none), the scores 32-bit sums with a bound e on their error. With T the K-th
// largest of these, the true K-th largest lies within e of T, so blocks over T + 2 e are in, blocks under T - 2 e are out, and only where
// those in between do not all fit are they scored again, in pairs of floats (2^-44), or in 64 bits where those would leave their range.
//
// One query a request: choose_kernel alone. Query blocks: pool_kernel (the queries, read once: the bytes of the whole), choose_kernel or, for many
// rows, choose_rows_kernel (scores, search, rows of the table), then the transpose. Times are of one GB300, device time in a captured loop over four inputs.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "fa_launch.h"
#include "fp8.cuh"

namespace fa {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t v) { return *reinterpret_cast<__nv_bfloat162*>(&v); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ uint32_t bits_of(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// ------------------------------------------------------------------------------------------------ bounds of bf16 keys
// A block is at most 128 rows, so every load of a CTA is in flight at once, 16 bytes a lane; two values a comparison. HBM bounds a large call:
// 4 x 4096 keys, 16 heads, d = 128 (67 MB) in 11.6 us, 5.9 TB/s; 64 requests of one new token (512 pages of 64) 3.1 us, a launch.
constexpr uint32_t kBfInf2 = 0x7F807F80u, kBfNegInf2 = 0xFF80FF80u;  // NaN keys propagate: min and max of them are NaN
constexpr int kBoundThreads = 256;

// lo, hi: 8 channels of this thread's rows (lane tid % (D / 8) of a row) -> dst [2][D], by the whole CTA
template <int D>
__device__ __forceinline__ void join_bounds(uint32_t (&lo)[4], uint32_t (&hi)[4], __nv_bfloat16* dst) {
  constexpr int LPR = D / 8, kWarps = kBoundThreads / 32;
  __shared__ uint4 s_box[kWarps][2][LPR];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = bits_of(__hmin2_nan(as_bf2(lo[i]), as_bf2(__shfl_xor_sync(kAll, lo[i], o))));
      hi[i] = bits_of(__hmax2_nan(as_bf2(hi[i]), as_bf2(__shfl_xor_sync(kAll, hi[i], o))));
    }
  if (lane < LPR) {
    s_box[warp][0][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    s_box[warp][1][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
  __syncthreads();
  if (tid < 2 * LPR) {
    const int which = tid / LPR, x = tid % LPR;
    uint32_t v[4] = {s_box[0][which][x].x, s_box[0][which][x].y, s_box[0][which][x].z, s_box[0][which][x].w};
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const uint4 u = s_box[w][which][x];
      const uint32_t t[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = which ? bits_of(__hmax2_nan(as_bf2(v[i]), as_bf2(t[i]))) : bits_of(__hmin2_nan(as_bf2(v[i]), as_bf2(t[i])));
    }
    reinterpret_cast<uint4*>(dst + which * D)[x] = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

template <int D>
__device__ __forceinline__ void block_bounds(const __nv_bfloat16* src, int rows, __nv_bfloat16* dst) {
  constexpr int LPR = D / 8, kRows = kBoundThreads / LPR, kPass = 128 / kRows;
  const int lane = threadIdx.x % LPR, row0 = threadIdx.x / LPR;
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = kBfInf2;
    hi[i] = kBfNegInf2;
  }
  uint4 v[kPass];
#pragma unroll
  for (int k = 0; k < kPass; ++k) {
    const int r = row0 + k * kRows;
    if (r < rows) v[k] = __ldg(reinterpret_cast<const uint4*>(src + (size_t)r * D) + lane);
  }
#pragma unroll
  for (int k = 0; k < kPass; ++k) {
    if (row0 + k * kRows < rows) {
      const uint32_t t[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = bits_of(__hmin2_nan(as_bf2(lo[i]), as_bf2(t[i])));
        hi[i] = bits_of(__hmax2_nan(as_bf2(hi[i]), as_bf2(t[i])));
      }
    }
  }
  join_bounds<D>(lo, hi, dst);
}

// one CTA a block of keys
template <int D>
__global__ void __launch_bounds__(kBoundThreads) key_bounds_kernel(const __grid_constant__ BoundsArgs a) {
  const int c = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
  const int64_t j0 = (int64_t)c * a.page;
  const size_t bh = (size_t)b * a.Hkv + hk;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.k) + (bh * a.kv_len + j0) * D;
  block_bounds<D>(src, (int)min((int64_t)a.page, (int64_t)a.kv_len - j0),
                  static_cast<__nv_bfloat16*>(a.bounds) + (bh * gridDim.x + c) * 2 * D);
}

// The page of a cache that CTA (x, hk, b) works on: the x-th that request b's new tokens reach, and how many of its tokens there are
// after them. False where there is none.
__device__ __forceinline__ bool reached_page(const BoundsArgs& a, int x, int b, int& pid, int& held) {
  const int64_t first = a.q_offset ? (int64_t)__ldg(a.q_offset + b) : 0;
  int n = a.n_new ? __ldg(a.n_new + b) : a.N;
  const bool tell = x == 0 && blockIdx.y == 0 && threadIdx.x == 0;
  if (n < 0 || n > a.N) {
    if (tell) report(a.status, FA_ERR_DEVICE_CHECK);
    n = min(max(n, 0), a.N);
  }
  const int64_t room = (int64_t)a.max_pages * a.page;
  int64_t lo = first, hi = first + n;
  if (n > 0 && (lo < 0 || hi > room)) {  // tokens outside the table are left out
    if (tell) report(a.status, FA_ERR_DEVICE_CHECK);
    lo = max(lo, (int64_t)0);
    hi = min(hi, room);
  }
  if (hi <= lo) return false;
  const int64_t t = lo / a.page + x;
  if (t * a.page >= hi) return false;
  held = (int)min((int64_t)a.page, hi - t * a.page);
  pid = __ldg(a.page_table + (size_t)b * a.max_pages + t);
  if (pid < 0 || pid >= a.n_pages_total) {
    if (threadIdx.x == 0) report(a.status, FA_ERR_DEVICE_CHECK);
    return false;
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(kBoundThreads) kv_bounds_kernel(const __grid_constant__ BoundsArgs a) {
  int pid, held;
  if (!reached_page(a, blockIdx.x, blockIdx.z, pid, held)) return;
  const size_t ph = (size_t)pid * a.Hkv + blockIdx.y;
  block_bounds<D>(static_cast<const __nv_bfloat16*>(a.k) + ph * a.page * D, held, static_cast<__nv_bfloat16*>(a.bounds) + ph * 2 * D);
}

// ------------------------------------------------------------------------------------------------ bounds of e4m3 keys
// A warp takes the 32 tokens of a scale: e4m3 orders as it is (in fp16, exactly), one multiplication by the scale at the end, rounded
// outwards, and outwards again to bf16: with a power-of-two scale nothing is rounded. 8 x up to 2048 new tokens, 8 heads, pages of 128
// (12 MB): 5.3 us, a launch and three loads that wait for one another (n_new, page id, keys).
constexpr int kBound8Threads = 128;

template <int D>
__global__ void __launch_bounds__(kBound8Threads) kv_bounds_fp8_kernel(const __grid_constant__ BoundsArgs a) {
  constexpr int LPR = D / 16, kRows = 32 / LPR, kPass = kScaleTokens / kRows, kWarps = kBound8Threads / 32;
  __shared__ float s_box[kWarps][2][D];
  int pid, held;
  if (!reached_page(a, blockIdx.x, blockIdx.z, pid, held)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, x = lane % LPR;
  const size_t ph = (size_t)pid * a.Hkv + blockIdx.y;
  const int rows = min(held - warp * kScaleTokens, kScaleTokens), used = (held + kScaleTokens - 1) / kScaleTokens;
  if (rows > 0) {
    const uint8_t* src = static_cast<const uint8_t*>(a.k) + (ph * a.page + warp * kScaleTokens) * D;
    const float sc = clamp_scale(__ldg(a.k_scale + ph * (a.page / kScaleTokens) + warp));
    uint4 v[kPass];
#pragma unroll
    for (int k = 0; k < kPass; ++k)
      if (lane / LPR + k * kRows < rows) v[k] = __ldg(reinterpret_cast<const uint4*>(src + (size_t)(lane / LPR + k * kRows) * D) + x);
    uint32_t lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = 0x7C007C00u;  // fp16 infinities
      hi[i] = 0xFC00FC00u;
    }
#pragma unroll
    for (int k = 0; k < kPass; ++k) {
      if (lane / LPR + k * kRows < rows) {
        const uint32_t t[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p, q;
          e4m3x4_to_f16(t[i], p, q);
          lo[2 * i] = bits_of(__hmin2_nan(as_h2(lo[2 * i]), as_h2(p)));
          lo[2 * i + 1] = bits_of(__hmin2_nan(as_h2(lo[2 * i + 1]), as_h2(q)));
          hi[2 * i] = bits_of(__hmax2_nan(as_h2(hi[2 * i]), as_h2(p)));
          hi[2 * i + 1] = bits_of(__hmax2_nan(as_h2(hi[2 * i + 1]), as_h2(q)));
        }
      }
    }
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo[i] = bits_of(__hmin2_nan(as_h2(lo[i]), as_h2(__shfl_xor_sync(kAll, lo[i], o))));
        hi[i] = bits_of(__hmax2_nan(as_h2(hi[i]), as_h2(__shfl_xor_sync(kAll, hi[i], o))));
      }
    if (lane < LPR) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 p = f16x2_to_f32(lo[i]), q = f16x2_to_f32(hi[i]);
        s_box[warp][0][x * 16 + 2 * i] = __fmul_rd(p.x, sc);
        s_box[warp][0][x * 16 + 2 * i + 1] = __fmul_rd(p.y, sc);
        s_box[warp][1][x * 16 + 2 * i] = __fmul_ru(q.x, sc);
        s_box[warp][1][x * 16 + 2 * i + 1] = __fmul_ru(q.y, sc);
      }
    }
  }
  __syncthreads();
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.bounds) + ph * 2 * D;
  for (int e = tid; e < D; e += kBound8Threads) {
    float p = s_box[0][0][e], q = s_box[0][1][e];
    for (int w = 1; w < used; ++w) {  // a NaN on either side stays
      const float u = s_box[w][0][e], t = s_box[w][1][e];
      p = (u < p || u != u) ? u : p;
      q = (t > q || t != t) ? t : q;
    }
    dst[e] = __float2bfloat16_rd(p);
    dst[D + e] = __float2bfloat16_ru(q);
  }
}

// ------------------------------------------------------------------------------------------------ sums over queries
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
constexpr int kThreads = 256, kWarps = kThreads / 32, kPoolThreads = 64;

// s + rest = s + x (+ rest): what the addition rounds off goes to rest
__device__ __forceinline__ void add_exact(float& s, float& rest, float x) {
  const float t = __fadd_rn(s, x), u = __fsub_rn(t, s);
  rest = __fadd_rn(rest, __fadd_rn(__fsub_rn(s, __fsub_rn(t, u)), __fsub_rn(x, u)));
  s = t;
}
// The same, with s the sum rounded once however many terms there were: the scores in 32 bits take s alone, and their bound counts one rounding. (A
// running s is off by half a step for each term, and what rest itself rounds off grows with their number squared.)
__device__ __forceinline__ void add_joined(float& s, float& rest, float x) {
  add_exact(s, rest, x);
  float t = s, off = 0.f;
  add_exact(t, off, rest);
  if (t - t == 0.f) {  // infinities and NaN stay as they are
    s = t;
    rest = off;
  }
}
// Sums of bf16 in whole numbers. For |x| < 2^E, x + C with C = 1.5 * 2^(E + 1) lies in C's binade, so its bits are C's plus x in units of
// 2^(E - 22): an integer sum of the bits is exact, and with max(x, 0) + C = max(x + C, C) the sum of the positive ones takes two
// operations more. What x + C rounds off (of magnitudes under 2^(E - 15)) is summed apart, where there is any, in pairs of floats: E is that of eight channels
// together, and one of them may hold nothing but such rests. At most 256 values a lane.
// Sums in pairs of floats took 7 dependent operations a value: 41 us for 4 x 4096 queries' choice against 37, 118 against 114 for 65536.
struct BitSums {
  uint32_t all[8], pos[8];        // sums of the bits, C's own left in
  float* rest;                    // what was rounded off, of all and of the positive ones, sums and their rests: [2][16], kPoolThreads apart. Seldom touched: in shared memory
  float c, under;                 // C and 2^E
  int n;                          // values so far
  __device__ __forceinline__ float& off(int i, int part) const { return rest[(part * 16 + i) * kPoolThreads]; }  // channel i of all, 8 + i of the positive ones
  __device__ __forceinline__ void add_off(int i, float x) { add_exact(off(i, 0), off(i, 1), x); }
  __device__ __forceinline__ void start(float* mine) {
    rest = mine;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      all[i] = pos[i] = 0u;
      off(i, 0) = off(i, 1) = off(8 + i, 0) = off(8 + i, 1) = 0.f;
    }
    c = under = 0.f;
    n = 0;
  }
  __device__ __forceinline__ float unit() const { return under * 2.384185791015625e-7f; }  // 2^(E - 22)
  // the sums as whole numbers of units, and another E for values up to `top`
  __device__ __forceinline__ void grow(float top) {
    const int ex = min((int)(__float_as_uint(top) >> 23), 251);  // top < 2^(ex - 126)
    const float to = __uint_as_float((uint32_t)(ex + 1) << 23), u = unit();
    const int jump = (int)(__float_as_uint(to) >> 23) - (int)(__float_as_uint(under) >> 23);  // units are 2^jump of the old ones
    const int k = min(31, jump);
    const uint32_t was = __float_as_uint(c) * (uint32_t)n;
    under = to;
    c = 3.f * to;
    const uint32_t now = __float_as_uint(c) * (uint32_t)n;
    if (n == 0) return;  // nothing yet: all and pos are 0
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int a = (int)(all[i] - was), p = (int)(pos[i] - was);
      const int a_up = jump > 31 ? 0 : a >> k, p_up = jump > 31 ? 0 : p >> k;  // past 31 a sum, of either sign, is less than one unit: all of it is rest
      const int a_low = a - (a_up << k), p_low = p - (p_up << k);
      if (jump > 24) {  // of up to 31 bits: a float takes 24
        off(i, 1) += (float)(a_low & 255) * u;
        off(8 + i, 1) += (float)(p_low & 255) * u;
      }
      add_off(i, (float)(jump > 24 ? a_low & ~255 : a_low) * u);
      add_off(8 + i, (float)(jump > 24 ? p_low & ~255 : p_low) * u);
      all[i] = (uint32_t)a_up + now;
      pos[i] = (uint32_t)p_up + now;
    }
  }
  __device__ __forceinline__ void add(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = __fadd_rn((e & 1) ? bf_hi(w[e >> 1]) : bf_lo(w[e >> 1]), c);
      all[e] += __float_as_uint(t);
      pos[e] += __float_as_uint(fmaxf(t, c));
    }
    ++n;
  }
  // Magnitudes from here on, with 8 bits of their own, lose nothing
  __device__ __forceinline__ float kept() const { return 128.f * unit(); }
  // what add(v) rounds off: looked for first, as it is seldom more than one value's, and one after another
  __device__ __forceinline__ void add_rest(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    auto off_by = [&](float y) { return __fsub_rn(y, __fsub_rn(__fadd_rn(y, c), c)); };
    uint32_t some = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) some |= (off_by((e & 1) ? bf_hi(w[e >> 1]) : bf_lo(w[e >> 1])) != 0.f ? 1u : 0u) << e;
#pragma unroll 1
    for (; some; some &= some - 1) {
      const int e = __ffs(some) - 1;
      const uint32_t two = e < 4 ? (e < 2 ? v.x : v.y) : (e < 6 ? v.z : v.w);
      const float y = (e & 1) ? bf_hi(two) : bf_lo(two), d = off_by(y);
      add_off(e, d);
      if (y > 0.f) add_off(8 + e, d);
    }
  }
  // sum + rest, of all and of the positive values
  __device__ __forceinline__ void sums(int i, float& s, float& r, float& sp, float& rp) const {
    const uint32_t own = __float_as_uint(c) * (uint32_t)n;
    const int a = (int)(all[i] - own), p = (int)(pos[i] - own);
    const float u = unit();
    s = (float)a * u;  // of up to 30 bits the upper 24; the others go apart
    r = off(i, 1) + (float)(a - (int)(float)a) * u;
    add_exact(s, r, off(i, 0));
    sp = (float)p * u;
    rp = off(8 + i, 1) + (float)(p - (int)(float)p) * u;
    add_exact(sp, rp, off(8 + i, 0));
  }
};

// The bits of the least magnitude among eight values that is not 0 (2^16: there is none). Volatile: what it shares with other minima is made anew, not
// kept in registers
__device__ __forceinline__ uint32_t least_of(uint4 v) {
  uint32_t m;
  asm volatile(
      "{\n\t.reg .b32 a, b, c, d, e;\n\tmov.b32 e, 0xFFFFFFFF;\n\t"
      "and.b32 a, %1, 0x7FFF7FFF;\n\tand.b32 b, %2, 0x7FFF7FFF;\n\tand.b32 c, %3, 0x7FFF7FFF;\n\tand.b32 d, %4, 0x7FFF7FFF;\n\t"
      "add.u16x2 a, a, e;\n\tadd.u16x2 b, b, e;\n\tadd.u16x2 c, c, e;\n\tadd.u16x2 d, d, e;\n\t"  // less 1: a 0 is the largest
      "min.u16x2 a, a, b;\n\tmin.u16x2 c, c, d;\n\tmin.u16x2 %0, a, c;\n\t}"
      : "=r"(m)
      : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
  return min(m & 0xFFFFu, m >> 16) + 1u;
}

// grid (nq, Hkv * parts, B): Q-, Q+ of one query block over at most 8 of a group's heads, in pairs of floats -> pooled [B, Hkv, nq, parts, 2 (sum,
// rest), 2 D]. Two warps, half of the rows each: long enough a way through memory that the joining at its end costs little. Fourteen CTAs an
// SM: 2048 of them, the two large cases below, are all there at once. HBM and the instructions bound it about alike: 65536 queries of 16 heads
// (268 MB) in 54 us, 5.0 TB/s, 59 % of the issue slots (the whole choice 110 us; with ten CTAs an SM, the rests in registers, 117).
constexpr int kAhead = 8;

// the first of a group's g heads that division `part` takes: part * g passes 32 bits for groups of 46,341 heads and more
__device__ __forceinline__ int first_head(int part, int g, int parts) { return (int)((int64_t)part * g / parts); }

template <int D>
__global__ void __launch_bounds__(kPoolThreads, 14) pool_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int LPR = D / 8, RPL = 32 / LPR;  // lanes a row, rows a load
  __shared__ float s_sum[2][2 * D];
  __shared__ float s_rest[32 * kPoolThreads];
  const int r = blockIdx.x, hk = blockIdx.y / a.parts, part = blockIdx.y % a.parts, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, x = lane % LPR;
  const int g = a.Hq / a.Hkv, h0 = hk * g + first_head(part, g, a.parts), h1 = hk * g + first_head(part + 1, g, a.parts);
  const int i0 = r * a.bq, rows = min(a.bq, a.q_len - i0), half = (rows + 1) / 2;
  const int begin = warp * half + lane / LPR, end = min(rows, warp * half + half);
  const int mine = end > begin ? (end - begin + RPL - 1) / RPL : 0;  // rows of a head that this lane reads
  const int steps = (half + RPL - 1) / RPL;
  BitSums q;
  q.start(s_rest + tid);
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (((size_t)b * a.Hq + h0) * a.q_len + i0 + begin) * D) + x;
  for (int h = h0; h < h1; ++h, src += (size_t)a.q_len * LPR) {
    for (int t = 0; t < steps; t += kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) v[k] = t + k < mine ? __ldg(src + (t + k) * 32) : make_uint4(0, 0, 0, 0);
      uint32_t top = 0u, low = kBfInf2;  // largest and smallest magnitudes, two to a word
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          top = bits_of(__hmax2(as_bf2(top), __habs2(as_bf2(w[j]))));
          low = bits_of(__hmin2(as_bf2(low), __habs2(as_bf2(w[j]))));
        }
      }
      const float most = fmaxf(bf_lo(top), bf_hi(top));
      if (most >= q.under) q.grow(most);
      if (fminf(bf_lo(low), bf_hi(low)) < q.kept()) {
        // Short: which rows hold such a value, and these one after another. Unrolled over the rows, what add_rest does is longer than all of the rest (the whole
        // choice of 65536 queries took 143 us so, 121 with these rows read again, 110 this way). Queries whose magnitudes span 2^60 at random take
        // it for nearly every value: 281 us for 32,768 queries of 16 heads where N(0, 1) takes 66
        uint32_t some = 0u;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          some |= (least_of(v[k]) < __float_as_uint(q.kept()) >> 16 ? 1u : 0u) << k;
        }
#pragma unroll 1
        for (; some; some &= some - 1) {
          const int k = __ffs(some) - 1;
          uint4 r = v[0];
#pragma unroll
          for (int x = 1; x < kAhead; ++x)
            if (k == x) r = v[x];
          q.add_rest(r);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) q.add(v[k]);
    }
  }
  float all[8], all_r[8], pos[8], pos_r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    q.sums(e, all[e], all_r[e], pos[e], pos_r[e]);
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
      const float u = __shfl_xor_sync(kAll, all[e], o), p = __shfl_xor_sync(kAll, pos[e], o);
      all_r[e] += __shfl_xor_sync(kAll, all_r[e], o);
      pos_r[e] += __shfl_xor_sync(kAll, pos_r[e], o);
      add_exact(all[e], all_r[e], u);
      add_exact(pos[e], pos_r[e], p);
    }
  }
  if (warp == 1 && lane < LPR) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s_sum[0][x * 8 + e] = all[e];
      s_sum[1][x * 8 + e] = all_r[e];
      s_sum[0][D + x * 8 + e] = pos[e];
      s_sum[1][D + x * 8 + e] = pos_r[e];
    }
  }
  __syncthreads();
  if (warp == 1 || lane >= LPR) return;
  float* out = a.pooled + ((((size_t)b * a.Hkv + hk) * a.nq + r) * a.parts + part) * 4 * D + x * 8;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    all_r[e] += s_sum[1][x * 8 + e];
    add_exact(all[e], all_r[e], s_sum[0][x * 8 + e]);
    pos_r[e] += s_sum[1][D + x * 8 + e];
    add_exact(pos[e], pos_r[e], s_sum[0][D + x * 8 + e]);
    all_r[e] -= pos_r[e];  // Q- = all - positive
    add_exact(all[e], all_r[e], -pos[e]);
#pragma unroll
    for (int w = 0; w < 2; ++w) {  // the rest below the sum's last bit
      const float s = w ? pos[e] : all[e], rest = w ? pos_r[e] : all_r[e], t = s + rest;
      out[w * D + e] = t;
      out[2 * D + w * D + e] = t - t == 0.f ? rest - (t - s) : 0.f;
    }
  }
}

// ------------------------------------------------------------------------------------------------ scores
// Where the bounds of a (request, KV head)'s blocks lie: block id at base + id * stride
template <int D>
struct Boxes {
  const __nv_bfloat16* base;
  size_t stride;
  const int32_t* table;  // of the request, or NULL: id = column
  int total;
  __device__ __forceinline__ Boxes(const SelectArgs& a, int b, int hk) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.bounds);
    table = a.page_table ? a.page_table + (size_t)b * a.max_pages : nullptr;
    total = a.n_pages_total;
    base = table ? p + (size_t)hk * 2 * D : p + ((size_t)b * a.Hkv + hk) * a.nk * 2 * D;
    stride = table ? (size_t)a.Hkv * 2 * D : 2 * D;
  }
  __device__ __forceinline__ int id(int c) const {  // -1: there is none
    if (!table) return c;
    const int pid = __ldg(table + c);
    return pid < 0 || pid >= total ? -1 : pid;
  }
  __device__ __forceinline__ const __nv_bfloat16* at(int id) const { return base + (size_t)id * stride; }
};

// A warp's part in the scores of one row: the lane's 8 terms of Q-, Q+, and the largest magnitudes of its 8 bounds so far. 16 bytes of a block a
// lane, 8 (d = 64: 16) blocks at a time, whose partial sums meet in a butterfly that halves the blocks a lane still has with every
// step: 8 products in a row, 5 sums.
template <int D>
struct Scorer {
  static constexpr int LPB = D / 4, BPW = 32 / LPB, kStep = 8 * BPW;  // lanes a block, blocks a load, blocks at a time
  float q[8];
  uint32_t most[4];
  // lane t < kStep: the score of the block that its id names (negative: none)
  __device__ __forceinline__ float scores(const Boxes<D>& box, int id) {
    const int lane = threadIdx.x & 31;
    uint4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int w = __shfl_sync(kAll, id, j * BPW + lane / LPB);
      v[j] = w >= 0 ? __ldg(reinterpret_cast<const uint4*>(box.at(w)) + lane % LPB) : make_uint4(0, 0, 0, 0);
    }
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t t[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
      s[j] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[j] = fmaf(q[2 * i], bf_lo(t[i]), s[j]);
        s[j] = fmaf(q[2 * i + 1], bf_hi(t[i]), s[j]);
        most[i] = bits_of(__hmax2(as_bf2(most[i]), __habs2(as_bf2(t[i]))));
      }
    }
    constexpr int O = LPB / 2;
#pragma unroll
    for (int n = 4, o = O; n > 0; n >>= 1, o >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int j = 0; j < n; ++j) {
        const float mine = up ? s[j + n] : s[j], other = up ? s[j] : s[j + n];
        s[j] = mine + __shfl_xor_sync(kAll, other, o);
      }
    }
#pragma unroll
    for (int o = O / 8; o > 0; o >>= 1) s[0] += __shfl_xor_sync(kAll, s[0], o);
    const int slot = (lane / BPW) & 7;
    const int from = (lane % BPW) * LPB + ((slot >> 2) & 1) * O + ((slot >> 1) & 1) * (O / 2) + (slot & 1) * (O / 4);
    return __shfl_sync(kAll, s[0], from);
  }
  // a bound on the magnitudes that any of the scores so far added up
  __device__ __forceinline__ float magnitude() const {
    float err = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      err = fmaf(fabsf(q[2 * i]), bf_lo(most[i]), err);
      err = fmaf(fabsf(q[2 * i + 1]), bf_hi(most[i]), err);
    }
#pragma unroll
    for (int o = LPB / 2; o > 0; o >>= 1) err += __shfl_xor_sync(kAll, err, o);
    if (LPB < 32) {
      const float e = __shfl_xor_sync(kAll, err, LPB & 31);  // the other half's blocks
      err = e > err || e != e ? e : err;
    }
    return err;
  }
};

// ------------------------------------------------------------------------------------------------ the choice
// Order of floats as unsigned numbers, NaN on top, 0 below all of them.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 as 0
  return x != x ? kAll : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k); }
__device__ __forceinline__ uint64_t order_of(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return x != x ? ~0ull : (u >> 63) ? ~u : u | (1ull << 63);
}

// W warps that work on one row of the table (the whole CTA for W > 1)
template <int W>
struct Group {
  int* red;  // [2 W + 1]
  int flip;
  __device__ __forceinline__ static int tid() { return W == 1 ? threadIdx.x & 31 : threadIdx.x; }
  __device__ __forceinline__ static int warp() { return W == 1 ? 0 : threadIdx.x >> 5; }
  __device__ __forceinline__ static void sync() {
    if (W == 1) __syncwarp();
    else __syncthreads();
  }
  __device__ __forceinline__ int sum(int v) {
    v = __reduce_add_sync(kAll, v);
    if (W == 1) return v;
    if ((threadIdx.x & 31) == 0) red[flip * W + warp()] = v;
    __syncthreads();
    int t = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) t += red[flip * W + w];
    flip ^= 1;  // the next sum writes the other half, the one after it behind that one's barrier
    return t;
  }
  // exclusive prefix sums of the set bits of words [0, n) -> pre; returns the total. Begins and ends with a barrier.
  template <class WordFn>
  __device__ __forceinline__ int prefix(WordFn word, int n, uint32_t* pre) {
    sync();
    int run = 0;
    if (warp() == 0) {
      const int lane = threadIdx.x & 31;
      for (int i0 = 0; i0 < n; i0 += 32) {
        const int c = i0 + lane < n ? __popc(word(i0 + lane)) : 0;
        int s = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(kAll, s, o);
          if (lane >= o) s += t;
        }
        if (i0 + lane < n) pre[i0 + lane] = run + s - c;
        run += __shfl_sync(kAll, s, 31);
      }
      if (W > 1 && lane == 0) red[2 * W] = run;
    }
    sync();
    if (W > 1) run = red[2 * W];
    return run;
  }
  __device__ __forceinline__ uint32_t least(uint32_t v) {
    v = __reduce_min_sync(kAll, v);
    if (W == 1) return v;
    if ((threadIdx.x & 31) == 0) red[flip * W + warp()] = (int)v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) v = min(v, (uint32_t)red[flip * W + w]);
    flip ^= 1;
    return v;
  }
  // The want-th largest of the keys that `each` goes over (f(key) for each of this thread's), zeros not counted; want of them are there. A
  // threshold with exactly `want` keys from it on ends the search early, after about log2 of their number steps.
  template <class EachFn>
  __device__ __forceinline__ uint32_t kth(EachFn each, int want) {
    uint32_t lo = kAll, top = kAll;
    each([&](uint32_t k) {
      if (k) lo = min(lo, k);
      top = min(top, ~k);
    });
    lo = least(lo);
    uint32_t hi = ~least(top);
#pragma unroll 1
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2 + 1;
      int m = 0;
      each([&](uint32_t k) { m += k >= mid; });
      m = sum(m);
      if (m == want) {
        uint32_t t = kAll;
        each([&](uint32_t k) {
          if (k >= mid) t = min(t, k);
        });
        return least(t);
      }
      if (m > want) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};

// A row's shared memory, in words
__host__ __device__ constexpr size_t row_words(int nk, int W) { return (size_t)5 * ((nk + 31) / 32) + nk + 2 * W + 3; }
struct RowMem {
  int nk, nw;
  uint32_t *wc, *wp, *wx, *pa, *pb, *key;  // a bit a column: candidates, partial blocks, chosen; prefix sums (two); order of the scores
  int *total, *red;     // partial and full blocks chosen; what Group needs
  __device__ __forceinline__ RowMem(uint32_t* sm, int n) {
    nk = n;
    nw = (n + 31) / 32;
    wc = sm, wp = wc + nw, wx = wp + nw, pa = wx + nw, pb = pa + nw, key = pb + nw;
    total = reinterpret_cast<int*>(key + nk);
    red = total + 2;
  }
};

// Which blocks lie so near the border that 32 bits do not tell: `left` of `z` go in.
struct Border {
  float over, under;
  int left, z;
  __device__ __forceinline__ bool sure(uint32_t k) const { return k != 0u && value_of(k) > over; }
  __device__ __forceinline__ bool near(uint32_t k) const {  // a NaN on either side: near
    const float s = value_of(k);
    return k != 0u && !(s > over) && !(s < under);
  }
};

constexpr int kZone = 32;
struct Zone {  // the blocks near a border, scored exactly
  int n;
  int col[kZone];
  uint64_t key[kZone];
};

// A lane's terms of Q-, Q+ for exact scores, sum and rest
template <int D>
struct ExactQ {
  static constexpr int V = 2 * D / 32;
  float hi[V], lo[V];
};

// Exact score of a block, by a warp: products and sums in pairs of floats (2^-44 of the magnitudes), or where those could overflow or
// underflow (`wide`) in 64 bits.
template <int D>
__device__ __forceinline__ double exact_score(const __nv_bfloat16* box, const ExactQ<D>& q, bool wide) {
  constexpr int V = ExactQ<D>::V;
  const uint32_t* src = reinterpret_cast<const uint32_t*>(box) + (threadIdx.x & 31) * (V / 2);
  uint32_t v[V / 2];
#pragma unroll
  for (int j = 0; j < V / 2; ++j) v[j] = __ldg(src + j);
  if (wide) {
    double s = 0.0;
#pragma unroll
    for (int e = 0; e < V; ++e) s = fma((double)q.hi[e] + (double)q.lo[e], (double)((e & 1) ? bf_hi(v[e / 2]) : bf_lo(v[e / 2])), s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    return s;
  }
  float s = 0.f, rest = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float y = (e & 1) ? bf_hi(v[e / 2]) : bf_lo(v[e / 2]), p = __fmul_rn(q.hi[e], y);
    rest = __fadd_rn(rest, fmaf(q.lo[e], y, fmaf(q.hi[e], y, -p)));
    add_exact(s, rest, p);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float os = __shfl_xor_sync(kAll, s, o), orest = __shfl_xor_sync(kAll, rest, o);
    rest = __fadd_rn(rest, orest);
    add_exact(s, rest, os);
  }
  return (double)s + (double)rest;
}

// Chooses among the scored blocks of a row, by W warps: M.key -> M.wx, with the prefix sums and totals that write_row needs. err bounds the
// magnitudes that a score adds up; exact_q gives the lane's terms of Q-, Q+; zone [nk] is scratch.
template <int W, int D, class QFn>
__device__ void search_row(const SelectArgs& a, uint64_t* zone, const Boxes<D>& box, const RowMem& M, Zone& Z, float err, QFn exact_q) {
  using G = Group<W>;
  G grp{M.red, 0};
  const int lane = threadIdx.x & 31, gw = G::warp(), nk = M.nk, want = a.keep - a.first - a.last;
  const uint32_t below = (1u << lane) - 1u;
  const int n = grp.prefix([&](int i) { return M.wc[i]; }, M.nw, M.pa);
  if (n > a.keep) {
#pragma unroll 1
    for (int i = gw; i < M.nw; i += W) {  // always kept: not among the others
      const int c = i * 32 + lane, place = (int)M.pa[i] + __popc(M.wc[i] & below);
      const bool always = ((M.wc[i] >> lane) & 1u) && (place < a.first || place >= n - a.last);
      const uint32_t w = __ballot_sync(kAll, always);
      if (always) M.key[c] = 0u;
      if (lane == 0) M.wx[i] = w;
    }
    G::sync();
    if (want > 0) {
      // Short loops over the keys in shared memory, four at a time: unrolled over registers the code is several times as long, and a CTA
      // that runs it once waits for its instructions (4 x 4096 queries, rows of 32 blocks: the choice took 40 us so, 36 us this way).
      auto each = [&](auto f) {
#pragma unroll 1
        for (int c = G::tid(); c < nk; c += 128 * W) {
          uint32_t k[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) k[j] = c + j * 32 * W < nk ? M.key[c + j * 32 * W] : 0u;
#pragma unroll
          for (int j = 0; j < 4; ++j) f(k[j]);
        }
      };
      const float t = value_of(grp.kth(each, want));
      // Q rounded (its parts and their sum), a product in 13 steps; the rest is for the rounding of the bound itself
      const float e2 = 2.f * fmaf(17.f * 5.9604644775390625e-8f, err, 1e-42f);
      Border bd{t + e2, t - e2, 0, 0};
      int m = 0, z = 0;
      each([&](uint32_t k) {
        m += bd.sure(k);
        z += bd.near(k);
      });
      bd.left = want - grp.sum(m);
      bd.z = grp.sum(z);
      const bool fits = bd.z == bd.left;
#pragma unroll 1
      for (int i = gw; i < M.nw; i += W) {
        const uint32_t k = i * 32 + lane < nk ? M.key[i * 32 + lane] : 0u, w = __ballot_sync(kAll, bd.sure(k) || (fits && bd.near(k)));
        if (lane == 0) M.wx[i] |= w;
      }
      if (!fits) {  // 32 bits do not tell which of the blocks near the border are in: their scores exactly, a warp each
        const ExactQ<D> xq = exact_q();
        const bool wide = !(err > 8.7e-19f && err < 1e36f);  // 2^-60: what a product rounds off is a normal number still
        const bool few = bd.z <= kZone;
        if (G::tid() == 0) Z.n = 0;
        G::sync();
        for (int i = gw; i < M.nw; i += W) {
          const int c = i * 32 + lane;
          for (uint32_t w = __ballot_sync(kAll, c < nk && bd.near(M.key[c])); w; w &= w - 1) {
            const int cc = i * 32 + __ffs(w) - 1, id = box.id(cc);
            const uint64_t k = order_of(id >= 0 ? exact_score<D>(box.at(id), xq, wide) : -INFINITY);
            if (lane == 0) {
              if (few) {
                const int slot = atomicAdd(&Z.n, 1);  // in any order: their columns are kept with them
                Z.col[slot] = cc;
                Z.key[slot] = k;
              } else {
                zone[cc] = k;
              }
            }
          }
        }
        G::sync();
        if (few) {
          if (gw == 0) {
            const bool mine = lane < bd.z;
            const uint64_t k = mine ? Z.key[lane] : 0;
            const int c = mine ? Z.col[lane] : 0;
            int better = 0;
            for (int j = 0; j < bd.z; ++j) better += Z.key[j] > k || (Z.key[j] == k && Z.col[j] < c);
            if (mine && better < bd.left) atomicOr(&M.wx[c >> 5], 1u << (c & 31));
          }
        } else {
          uint64_t cut = 0;  // the left-th largest of them
          for (uint64_t bit = 1ull << 63; bit; bit >>= 1) {
            int k = 0;
            for (int c = G::tid(); c < nk; c += 32 * W) k += bd.near(M.key[c]) && zone[c] >= (cut | bit);
            if (grp.sum(k) >= bd.left) cut |= bit;
          }
          int k = 0;
          for (int c = G::tid(); c < nk; c += 32 * W) k += bd.near(M.key[c]) && zone[c] > cut;
          const int ties = bd.left - grp.sum(k);  // of those equal to it, the lowest columns
          for (int i = gw; i < M.nw; i += W) {
            const int c = i * 32 + lane;
            const uint32_t w = __ballot_sync(kAll, c < nk && bd.near(M.key[c]) && zone[c] == cut);
            if (lane == 0) M.pb[i] = w;
          }
          grp.prefix([&](int i) { return M.pb[i]; }, M.nw, M.pa);
          for (int i = gw; i < M.nw; i += W) {
            const int c = i * 32 + lane;
            bool in = false;
            if (c < nk && bd.near(M.key[c])) in = zone[c] > cut || (zone[c] == cut && (int)M.pa[i] + __popc(M.pb[i] & below) < ties);
            const uint32_t w = __ballot_sync(kAll, in);
            if (lane == 0) M.wx[i] |= w;
          }
        }
      }
    }
  }
  const int np = grp.prefix([&](int i) { return M.wx[i] & M.wp[i]; }, M.nw, M.pa);
  const int nf = grp.prefix([&](int i) { return M.wx[i] & ~M.wp[i]; }, M.nw, M.pb);
  if (G::tid() == 0) {
    M.total[0] = np;
    M.total[1] = nf;
  }
  G::sync();
}

// The tables of one row from its chosen columns, by W warps
template <int W>
__device__ __forceinline__ void write_row(const SelectArgs& a, size_t row, const RowMem& M) {
  using G = Group<W>;
  const int nk = M.nk, lane = threadIdx.x & 31, np = M.total[0], nf = M.total[1];
  const uint32_t below = (1u << lane) - 1u;
  const MaskOut& T = a.out;
  int32_t *pi = T.kv_idx + row * nk, *fi = T.full_kv_idx + row * nk;
#pragma unroll 1
  for (int i = G::warp(); i < M.nw; i += W) {
    const int c = i * 32 + lane;
    if (c >= nk) continue;
    const uint32_t p = M.wx[i] & M.wp[i], f = M.wx[i] & ~M.wp[i];
    const bool in_p = (p >> lane) & 1u, in_f = (f >> lane) & 1u;
    if (in_p) pi[M.pa[i] + __popc(p & below)] = c;
    if (in_f) fi[M.pb[i] + __popc(f & below)] = c;
    if (c >= np) pi[c] = 0;
    if (c >= nf) fi[c] = 0;
    T.block_class[row * nk + c] = in_p ? FA_BLOCK_PARTIAL : in_f ? FA_BLOCK_FULL : FA_BLOCK_EMPTY;
    if (a.nq == 1) {  // the transpose of one row
      T.q_num[row * nk + c] = in_p;
      T.full_q_num[row * nk + c] = in_f;
      T.q_idx[row * nk + c] = 0;
      T.full_q_idx[row * nk + c] = 0;
    }
  }
  if (G::tid() == 0) {
    T.kv_num[row] = np;
    T.full_kv_num[row] = nf;
  }
}

// Rows of up to kAlone blocks are searched by one warp: the steps are too short for barriers (one request of 600 tokens: 6.0 us, by all eight warps 6.4; 64
// requests, rows of up to 512 blocks: 32.4 us by one warp, 29.4 by eight).
constexpr int kAlone = 128;

// A cluster of `ranks` CTAs a row, grid (nq * ranks, Hkv, B): each scores its share of the blocks into the first one's shared memory, and
// that one chooses. 64 requests of 1k - 32k tokens, 8 KV heads, 32 blocks of up to 512 (76 MB of bounds): 29 us, 9 of them the classes, the
// tables and the launch, 15 the scores (HBM: 11), 5 the search. Two requests of 131,072 tokens, 64 of 2048 blocks: 18 us with eight CTAs a
// row (9, 3.5 and 6 of them; 20 with four CTAs); one of 600 tokens: 6 us.
constexpr int kZoneBlocks = 2048;  // rows of up to so many keep the scores near the border in shared memory, longer ones in the workspace

template <int D>
__global__ void __launch_bounds__(kThreads, 4) choose_kernel(const __grid_constant__ SelectArgs a, int ranks) {
  namespace cg = cooperative_groups;
  using S = Scorer<D>;
  constexpr int V = ExactQ<D>::V, kSteps = 32 / S::kStep;  // steps of the scores a word of columns
  extern __shared__ __align__(8) uint32_t dyn[];
  __shared__ Zone s_zone;
  __shared__ float s_err[8 * kWarps];
  __shared__ float s_q[2][2 * D];  // Q-, Q+: sum and rest
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nk = a.nk;
  const int rank = blockIdx.x % ranks, hk = blockIdx.y, b = blockIdx.z, r = a.nq - 1 - (int)blockIdx.x / ranks;  // causal: long rows first
  const size_t row = ((size_t)b * a.Hkv + hk) * a.nq + r;
  const bool near_by = nk <= kZoneBlocks;
  const RowMem M(dyn + (near_by ? 2 * nk : 0), nk);
  const Boxes<D> box(a, b, hk);
  const uint8_t* cls = a.src_class + ((size_t)(a.src_Bm > 1 ? b : 0) * a.nq + r) * nk;
  const int want = a.keep - a.first - a.last, g = a.Hq / a.Hkv;
  if (ranks > 1) cg::this_cluster().barrier_arrive();  // every CTA of the cluster runs before the first one's memory is written

  // classes and ids of the blocks, 32 columns (a word) at a time, the words in turn to the CTAs: visited blocks are neighbours, and every CTA
  // gets its part of them. A warp's first two words' loads go ahead of the queries'.
  const int i0 = rank + ranks * warp, step = ranks * kWarps;
  int cv[2], ci[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = (i0 + j * step) * 32 + lane;
    cv[j] = c < nk ? cls[c] : 0;
    ci[j] = c < nk ? box.id(c) : -1;
  }
  if (threadIdx.x < 2 * D) {
    float s = 0.f, rest = 0.f;
    if (a.q_len == 1) {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + ((size_t)b * a.Hq + (size_t)hk * g) * D + threadIdx.x % D;
#pragma unroll 4
      for (int h = 0; h < g; ++h) {
        const float x = __bfloat162float(src[(size_t)h * D]);
        add_joined(s, rest, threadIdx.x < D ? min_nan(x, 0.f) : max_nan(x, 0.f));
      }
    } else {
      for (int p = 0; p < a.parts; ++p) {
        const float* src = a.pooled + (row * a.parts + p) * 4 * D + threadIdx.x;
        rest = __fadd_rn(rest, __ldg(src + 2 * D));
        add_joined(s, rest, __ldg(src));
      }
    }
    s_q[0][threadIdx.x] = s;
    s_q[1][threadIdx.x] = rest;
  }
  auto note = [&](int i, int v, int id) {
    const int c = i * 32 + lane;
    const uint32_t some = __ballot_sync(kAll, v != FA_BLOCK_EMPTY), part = __ballot_sync(kAll, v == FA_BLOCK_PARTIAL);
    if (want > 0 && v != FA_BLOCK_EMPTY && id < 0) report(a.status, FA_ERR_DEVICE_CHECK);
    if (c < nk) M.key[c] = v != FA_BLOCK_EMPTY ? (uint32_t)id : (uint32_t)-2;  // until the score takes its place
    if (lane == 0) {
      M.wc[i] = M.wx[i] = some;
      M.wp[i] = part;
    }
  };
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (i0 + j * step < M.nw) note(i0 + j * step, cv[j], ci[j]);
  for (int i = i0 + 2 * step; i < M.nw; i += step) {
    const int c = i * 32 + lane;
    note(i, c < nk ? cls[c] : 0, c < nk ? box.id(c) : -1);
  }
  __syncthreads();

  // the scores, the steps of this CTA's words in turn to the warps
  S sc;
#pragma unroll
  for (int i = 0; i < 8; ++i) sc.q[i] = s_q[0][lane % S::LPB * 8 + i];
#pragma unroll
  for (int i = 0; i < 4; ++i) sc.most[i] = 0u;
  uint32_t* key = M.key;
  if (ranks > 1) {
    cg::this_cluster().barrier_wait();
    key = cg::this_cluster().map_shared_rank(M.key, 0);
    if (rank) {
      uint32_t* words = cg::this_cluster().map_shared_rank(M.wc, 0);
      for (int i = i0; i < M.nw; i += step)
        if (lane < 3) words[lane * M.nw + i] = M.wc[lane * M.nw + i];  // wc, wp, wx follow one another
    }
  }
  for (int t = warp;; t += kWarps) {
    const int c = (rank + ranks * (t / kSteps)) * 32 + t % kSteps * S::kStep + lane;
    if (c - lane >= nk) break;
    const bool mine = lane < S::kStep && c < nk;
    const int id = mine ? (int)M.key[c] : -2;
    float s = -INFINITY;
    if (want > 0 && __any_sync(kAll, id >= 0)) s = sc.scores(box, id);
    if (mine) key[c] = id == -2 ? 0u : order_of(id >= 0 ? s : -INFINITY);
  }
  const float err = sc.magnitude();
  if (lane == 0) (ranks > 1 ? cg::this_cluster().map_shared_rank(s_err, 0) : s_err)[rank * kWarps + warp] = err;
  if (ranks > 1) {
    cg::this_cluster().sync();
    if (rank) return;
  } else {
    __syncthreads();
  }

  auto search = [&](auto warps) {
    float all = 0.f;
    for (int i = 0; i < ranks * kWarps; ++i) all = s_err[i] > all || s_err[i] != s_err[i] ? s_err[i] : all;
    search_row<decltype(warps)::value, D>(a, near_by ? reinterpret_cast<uint64_t*>(dyn) : a.zone + row * nk, box, M, s_zone, all, [&]() {
      ExactQ<D> x;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x.hi[e] = s_q[0][lane * V + e];
        x.lo[e] = s_q[1][lane * V + e];
      }
      return x;
    });
  };
  if (nk <= kAlone) {
    if (warp == 0) search(std::integral_constant<int, 1>{});
    __syncthreads();
  } else {
    search(std::integral_constant<int, kWarps>{});
  }
  write_row<kWarps>(a, row, M);
}

// ------------------------------------------------------------------------------------------------ rows of many query blocks
// Eight neighbouring rows a CTA: a block's bounds are read and unpacked once for all of them (a lane holds 8 of its 2 d terms, and those of Q for
// the eight rows), and the partial sums of the eight meet in a butterfly that halves the rows a lane still has with every step. Then a
// warp a row. A warp for each (row, block) took 2.2 times the instructions. 65536 queries, 4 KV heads, 32 of up to 512 blocks: 47 us, 24 of
// them the scores, 12 the search: the CTAs of long rows, whose warps wait for loads and for one another, two or one to an SM.
constexpr int kRows = kWarps;

__host__ __device__ constexpr size_t rows_pitch(int nk) { return row_words(nk, 1) | 1; }  // odd: the rows' keys of a column lie in different banks

template <int D>
__global__ void __launch_bounds__(kThreads, 2) choose_rows_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int LPB = D / 4, BPW = 32 / LPB, kLoads = 4 / BPW, V = ExactQ<D>::V, O = LPB / 2;
  extern __shared__ uint32_t dyn[];
  __shared__ Zone s_zone[kRows];
  __shared__ float s_err[kWarps][kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nk = a.nk;
  const int hk = blockIdx.x, b = blockIdx.z, top = a.nq - 1 - (int)blockIdx.y * kRows, r = top - warp;  // causal: all heads' long rows first
  const size_t head = ((size_t)b * a.Hkv + hk) * a.nq;
  const Boxes<D> box(a, b, hk);
  const RowMem M(dyn + warp * rows_pitch(nk), nk);
  const uint8_t* cls = a.src_class + ((size_t)(a.src_Bm > 1 ? b : 0) * a.nq + max(r, 0)) * nk;
#pragma unroll 4
  for (int i = 0; i < M.nw; ++i) {
    const int c = i * 32 + lane, v = r >= 0 && c < nk ? cls[c] : 0;
    const uint32_t some = __ballot_sync(kAll, v != FA_BLOCK_EMPTY), part = __ballot_sync(kAll, v == FA_BLOCK_PARTIAL);
    if (c < nk) M.key[c] = 0u;
    if (lane == 0) {
      M.wc[i] = M.wx[i] = some;
      M.wp[i] = part;
    }
  }
  // this lane's terms of Q-, Q+ for the eight rows
  float q[kRows][8];
  const int e0 = lane % LPB * 8;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const float4* src = reinterpret_cast<const float4*>(a.pooled + (head + max(top - k, 0)) * a.parts * 4 * D + e0);
    const float4 u = __ldg(src), v = __ldg(src + 1);
    q[k][0] = u.x, q[k][1] = u.y, q[k][2] = u.z, q[k][3] = u.w, q[k][4] = v.x, q[k][5] = v.y, q[k][6] = v.z, q[k][7] = v.w;
    if (a.parts > 1) {
      float lo[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) lo[e] = 0.f;
      for (int p = 1; p < a.parts; ++p) {
        src += D;
        const float4 u = __ldg(src), v = __ldg(src + 1);
        const float t[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) add_joined(q[k][e], lo[e], t[e]);
      }
    }
  }
  const int slot = ((lane & O) ? 4 : 0) + ((lane & (O / 2)) ? 2 : 0) + ((lane & (O / 4)) ? 1 : 0);  // the row whose sum ends up here
  const bool writer = lane % (LPB / 8) == 0;
  auto meet = [&](float (&s)[kRows]) {
#pragma unroll
    for (int n = 4, o = O; n > 0; n >>= 1, o >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int j = 0; j < n; ++j) {
        const float mine = up ? s[j + n] : s[j], other = up ? s[j] : s[j + n];
        s[j] = mine + __shfl_xor_sync(kAll, other, o);
      }
    }
#pragma unroll
    for (int o = O / 8; o > 0; o >>= 1) s[0] += __shfl_xor_sync(kAll, s[0], o);
    return s[0];
  };
  __syncthreads();
  // the scores: four columns of each 32 a warp, the next ones' loads under the sums
  uint32_t most[4] = {0u, 0u, 0u, 0u};
  int id = -2;
  uint4 v[kLoads];
  auto fetch = [&](int i) {  // the next 32 columns from the i-th on in which any of the rows has one of this warp's four
    for (; i < M.nw; ++i) {
      const uint32_t any = __reduce_or_sync(kAll, lane < kRows ? dyn[lane * rows_pitch(nk) + i] : 0u) >> (warp * 4) & 15u;  // wc of the rows
      if (!any) continue;
      id = -2;
      if (lane < 4 && ((any >> lane) & 1u)) {
        id = box.id(i * 32 + warp * 4 + lane);
        if (id < 0) report(a.status, FA_ERR_DEVICE_CHECK);
      }
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int w = __shfl_sync(kAll, id, j * BPW + lane / LPB);
        v[j] = w >= 0 ? __ldg(reinterpret_cast<const uint4*>(box.at(w)) + lane % LPB) : make_uint4(0, 0, 0, 0);
      }
      break;
    }
    return i;
  };
  if (a.keep > a.first + a.last)
    for (int i = fetch(0); i < M.nw;) {
      const int at = i, c0 = i * 32 + warp * 4, now = id;
      uint4 u[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) u[j] = v[j];
      i = fetch(i + 1);
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const uint32_t t[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
        float s[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) s[k] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = (e & 1) ? bf_hi(t[e >> 1]) : bf_lo(t[e >> 1]);
#pragma unroll
          for (int k = 0; k < kRows; ++k) s[k] = fmaf(q[k][e], y, s[k]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) most[e] = bits_of(__hmax2(as_bf2(most[e]), __habs2(as_bf2(t[e]))));
        const float x = meet(s);
        const int n = j * BPW + lane / LPB, w = __shfl_sync(kAll, now, n);
        uint32_t* row = dyn + slot * rows_pitch(nk);
        if (writer && ((row[at] >> (warp * 4 + n)) & 1u)) row[5 * M.nw + c0 + n] = order_of(w >= 0 ? x : -INFINITY);  // M.key of that row
      }
    }
  {
    float s[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      s[k] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s[k] = fmaf(fabsf(q[k][e]), (e & 1) ? bf_hi(most[e >> 1]) : bf_lo(most[e >> 1]), s[k]);
    }
    float err = meet(s);
    if (LPB < 32) {
      const float e = __shfl_xor_sync(kAll, err, LPB & 31);  // the other half's blocks
      err = e > err || e != e ? e : err;
    }
    if (writer && lane < LPB) s_err[warp][slot] = err;
  }
  __syncthreads();
  if (r < 0) return;
  float err = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) err = s_err[w][warp] > err || s_err[w][warp] != s_err[w][warp] ? s_err[w][warp] : err;
  search_row<1, D>(a, a.zone + (head + r) * nk, box, M, s_zone[warp], err, [&]() {
    ExactQ<D> x;
#pragma unroll
    for (int e = 0; e < V; ++e) x.hi[e] = x.lo[e] = 0.f;
    for (int p = 0; p < a.parts; ++p) {
      const float* src = a.pooled + ((head + r) * a.parts + p) * 4 * D + lane * V;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x.lo[e] = __fadd_rn(x.lo[e], __ldg(src + 2 * D + e));
        add_joined(x.hi[e], x.lo[e], __ldg(src + e));
      }
    }
    return x;
  });
  write_row<1>(a, head + r, M);
}

template <int D>
cudaError_t launch_bounds_d(const BoundsArgs& a, cudaStream_t st) {
  if (!a.page_table) {
    key_bounds_kernel<D><<<dim3((a.kv_len + a.page - 1) / a.page, a.Hkv, a.B), kBoundThreads, 0, st>>>(a);
  } else {
    // N tokens reach so many pages at most, wherever they begin
    const dim3 grid((unsigned)std::min(((int64_t)a.N + 2 * a.page - 2) / a.page, (int64_t)a.max_pages), a.Hkv, a.B);
    if (a.k_scale) kv_bounds_fp8_kernel<D><<<grid, kBound8Threads, 0, st>>>(a);
    else kv_bounds_kernel<D><<<grid, kBoundThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

// Rows of query blocks go eight to a CTA, as long as their keys fit in its shared memory and there are more rows than CTAs with one each would
// run at once (four an SM); fewer or longer ones take a CTA or more each. The whole choice, one row / eight rows a CTA, d = 128 (with rests in single
// floats: the sums take 1 % more now on both sides):
//   256 rows of up to  64 blocks (8192 queries, 4 KV heads)     20.2 / 24.1 us
//   512 rows of up to 256 blocks (32,768 queries, 2 KV heads)   36.6 / 45.2
//  1024 rows of up to 128 blocks (16,384 queries, 8 KV heads)   35.6 / 32.5
//  2048 rows of up to  32 blocks (4 x 4096 queries, 16 heads)   44.5 / 34.7
//  2048 rows of up to 512 blocks (65,536 queries, 4 KV heads)    125 / 109
constexpr int kRowsBlocks = 4096, kAtOnce = 4 * 152;
bool rows_together(int64_t rows, int32_t nq, int32_t nk) { return nq > 1 && nk <= kRowsBlocks && rows > kAtOnce; }

// What a launch's rows need, and what the longest rows that its kernel takes would
size_t choose_smem(int nk) { return (row_words(nk, kWarps) + (nk <= kZoneBlocks ? 2 * nk : 0)) * 4; }
size_t rows_smem(int nk) { return kRows * rows_pitch(nk) * 4; }

// 48 KB without asking, the kernel's own 8 KB at most among them; more always as `most`: the limit is the function's, for all threads' launches, and one
// that another call lowered between here and the launch would refuse it
template <class K>
cudaError_t allow_smem(K kernel, size_t bytes, size_t most) {
  return bytes > 40 * 1024 ? taken(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most)) : cudaSuccess;
}

template <int D>
cudaError_t launch_select_d(const SelectArgs& a, cudaStream_t st) {
  cudaError_t e;
  if (a.q_len > 1) {
    pool_kernel<D><<<dim3(a.nq, a.Hkv * a.parts, a.B), kPoolThreads, 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const int64_t rows = (int64_t)a.B * a.Hkv * a.nq;
  if (rows_together(rows, a.nq, a.nk)) {
    const size_t smem = rows_smem(a.nk);
    if ((e = allow_smem(choose_rows_kernel<D>, smem, rows_smem(kRowsBlocks))) != cudaSuccess) return e;
    choose_rows_kernel<D><<<dim3(a.Hkv, (a.nq + kRows - 1) / kRows, a.B), kThreads, smem, st>>>(a);
    e = cudaGetLastError();
  } else {
    const size_t smem = choose_smem(a.nk);
    const int ranks = select_ranks(rows, a.nk);
    if ((e = allow_smem(choose_kernel<D>, smem, std::max(choose_smem(kSelectMaxBlocks), choose_smem(kZoneBlocks)))) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.nq * ranks, a.Hkv, a.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = taken(cudaLaunchKernelEx(&cfg, choose_kernel<D>, a, ranks));
  }
  if (e != cudaSuccess || a.nq == 1) return e;
  return launch_mask_columns(a.out, st);
}

}  // namespace

// whether the choice needs the workspace for scores near the border
bool select_needs_zone(int64_t rows, int32_t nq, int32_t nk) { return nk > kZoneBlocks || rows_together(rows, nq, nk); }

// CTAs that share the blocks of one row: as many as run at once, each with a step of the scores for every warp. 512 rows of up to 512 blocks: 29 us with
// one CTA each, 37 with two, which take two rounds; 16 rows of 2048 blocks: 18.3 us with eight, 19.7 with four.
int select_ranks(int64_t rows, int32_t nk) {
  int n = 1;
  while (n < 8 && 2 * n * rows <= kAtOnce && nk >= 128 * n) n *= 2;
  return n;
}

cudaError_t launch_bounds(const BoundsArgs& a, cudaStream_t st) {
  return a.d == 64 ? launch_bounds_d<64>(a, st) : launch_bounds_d<128>(a, st);
}

cudaError_t launch_select_blocks(const SelectArgs& a, cudaStream_t st) {
  return a.d == 64 ? launch_select_d<64>(a, st) : launch_select_d<128>(a, st);
}

}  // namespace fa
