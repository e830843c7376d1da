// Key blocks chosen by a cheap score, and the bounds that the score reads.
//
//   bounds   min_e, max_e over the keys of a block, channel by channel (bf16): exact, so the result depends on the keys alone.
//   score    of block c for the queries of a query block (rows i of it, heads h that share the KV head):
//              s(c) = sum_{i,h} sum_e max(q_ihe min_e(c), q_ihe max_e(c)) = sum_e ( Q+_e max_e(c) + Q-_e min_e(c) ),
//            Q+_e = sum_{i,h} max(q_ihe, 0), Q-_e = sum_{i,h} min(q_ihe, 0): an upper bound of <q, k> over the block's keys, summed over
//            the queries. The sums over queries come first, so a block costs one product of 2 d, however many queries there are.
//   choice   the first and last few blocks of the mask's row, and of the others those with the largest score, ties to the lower column.
//
// The choice is that of scores in 64 bits, but hardly any is computed in 64 bits: this GPU has two FP64 lanes an SM. Q+- are summed in
// pairs of floats (an error of 2^-48), the scores in 32 bits with a bound e on their error. With T the K-th largest of these, the true
// K-th largest lies within e of T, so blocks over T + 2 e are in, blocks under T - 2 e are out, and only where those in between do not
// all fit are they scored again in 64 bits.
#include <cooperative_groups.h>

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
// outwards, and outwards again to bf16: with a power-of-two scale nothing is rounded.
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
// hi + lo += x, exactly up to 2^-48 of the result
__device__ __forceinline__ void add_pair(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x), t = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(x, t)));
  hi = s;
}

// Q- [0, D) and Q+ [D, 2 D) of the 8 channels that a thread has
struct Sums {
  float hi[2][8], lo[2][8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) hi[0][i] = hi[1][i] = lo[0][i] = lo[1][i] = 0.f;
  }
  __device__ __forceinline__ void add(uint4 v) {
    const uint32_t t[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = (i & 1) ? bf_hi(t[i >> 1]) : bf_lo(t[i >> 1]);
      add_pair(hi[0][i], lo[0][i], x > 0.f ? 0.f : x);   // NaN goes to Q-, and from there to every score
      add_pair(hi[1][i], lo[1][i], x > 0.f ? x : 0.f);
    }
  }
};

constexpr int kPoolThreads = 256;

// grid (nq, Hkv * parts, B): the sums of one query block over Hq / Hkv / parts heads -> pooled [B, Hkv, nq, parts, 2 (hi, lo), 2 D]
template <int D>
__global__ void __launch_bounds__(kPoolThreads) pool_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int LPR = D / 8, kRows = kPoolThreads / LPR, kWarps = kPoolThreads / 32;
  __shared__ float s_sum[kWarps][2][2 * D];  // hi, lo
  const int r = blockIdx.x, hk = blockIdx.y / a.parts, part = blockIdx.y % a.parts, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, x = tid % LPR;
  const int g = a.Hq / a.Hkv, h0 = hk * g + part * g / a.parts, h1 = hk * g + (part + 1) * g / a.parts;
  const int i0 = r * a.bq, rows = min(a.bq, a.q_len - i0);
  Sums s;
  s.clear();
  for (int h = h0; h < h1; ++h) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (((size_t)b * a.Hq + h) * a.q_len + i0) * D);
#pragma unroll 8
    for (int i = tid / LPR; i < rows; i += kRows) s.add(__ldg(src + (size_t)i * LPR + x));
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float oh = __shfl_xor_sync(kAll, s.hi[w][i], o), ol = __shfl_xor_sync(kAll, s.lo[w][i], o);
        add_pair(s.hi[w][i], s.lo[w][i], oh);
        s.lo[w][i] += ol;
      }
  if (lane < LPR) {
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s_sum[warp][0][w * D + x * 8 + i] = s.hi[w][i];
        s_sum[warp][1][w * D + x * 8 + i] = s.lo[w][i];
      }
  }
  __syncthreads();
  float* out = a.pooled + ((((size_t)b * a.Hkv + hk) * a.nq + r) * a.parts + part) * 4 * D;
  for (int e = tid; e < 2 * D; e += kPoolThreads) {
    float hi = s_sum[0][0][e], lo = s_sum[0][1][e];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      add_pair(hi, lo, s_sum[w][0][e]);
      lo += s_sum[w][1][e];
    }
    out[e] = hi;
    out[2 * D + e] = lo;
  }
}

// ------------------------------------------------------------------------------------------------ scores
// the bounds of block c, or NULL where its page does not exist
template <int D>
__device__ __forceinline__ const __nv_bfloat16* box_of(const SelectArgs& a, int b, int hk, int c) {
  const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(a.bounds);
  if (!a.page_table) return base + (((size_t)b * a.Hkv + hk) * a.nk + c) * 2 * D;
  const int pid = __ldg(a.page_table + (size_t)b * a.max_pages + c);
  return pid < 0 || pid >= a.n_pages_total ? nullptr : base + ((size_t)pid * a.Hkv + hk) * 2 * D;
}

// 32 query blocks x 64 key blocks of one (request, KV head). Sums of products run over 32 of the 2 D terms before they are added up.
constexpr int kTileR = 32, kTileC = 64, kTileK = 32, kTileThreads = 128;

template <int D>
__global__ void __launch_bounds__(kTileThreads) score_tile_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ __align__(16) float s_q[kTileK][kTileR + 4], s_b[kTileK][kTileC + 4];
  __shared__ float s_most[kTileK];
  const int nct = (a.nk + kTileC - 1) / kTileC;
  const int ct = blockIdx.x % nct, c0 = ct * kTileC, r0 = (blockIdx.x / nct) * kTileR, hk = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const size_t row0 = ((size_t)b * a.Hkv + hk) * a.nq + r0;
  const int rn = min(kTileR, a.nq - r0), cn = min(kTileC, a.nk - c0);
  const uint8_t* cls = a.src_class + ((size_t)(a.src_Bm > 1 ? b : 0) * a.nq + r0) * a.nk + c0;
  bool any = false;
  for (int x = tid; x < rn * kTileC; x += kTileThreads) any = any || (x % kTileC < cn && cls[(size_t)(x / kTileC) * a.nk + x % kTileC] != 0);
  if (!__syncthreads_or(any)) {  // no query block here sees any of the key blocks
    if (tid < rn) a.err[(row0 + tid) * nct + ct] = 0.f;
    return;
  }
  const int lc = c0 + tid / 2;
  const __nv_bfloat16* box = lc < a.nk ? box_of<D>(a, b, hk, lc) : nullptr;
  const bool missing = lc < a.nk && !box;
  const int lr = tid / 4, lk = tid % 4 * 8;
  float acc[4][4], err = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  for (int k0 = 0; k0 < 2 * D; k0 += kTileK) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = 0.f;
    if (lr < rn)
      for (int p = 0; p < a.parts; ++p) {
        const float4* src = reinterpret_cast<const float4*>(a.pooled + ((row0 + lr) * a.parts + p) * 4 * D + k0 + lk);
        const float4 u = __ldg(src), v = __ldg(src + 1);
        q[0] += u.x, q[1] += u.y, q[2] += u.z, q[3] += u.w, q[4] += v.x, q[5] += v.y, q[6] += v.z, q[7] += v.w;
      }
    uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (box) {
      const uint4* src = reinterpret_cast<const uint4*>(box + k0 + tid % 2 * 16);
      w[0] = __ldg(src);
      w[1] = __ldg(src + 1);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) s_q[lk + i][lr] = q[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t t = i < 4 ? (&w[0].x)[i & 3] : (&w[1].x)[i & 3];
      s_b[tid % 2 * 16 + 2 * i][tid / 2] = bf_lo(t);
      s_b[tid % 2 * 16 + 2 * i + 1][tid / 2] = bf_hi(t);
    }
    __syncthreads();
    float most = 0.f;  // the largest magnitude of a channel among the tile's blocks
#pragma unroll
    for (int i = 0; i < kTileC / 4; ++i) most = fmaxf(most, fabsf(s_b[tid / 4][tid % 4 + 4 * i]));
    most = fmaxf(most, __shfl_xor_sync(kAll, most, 1));
    most = fmaxf(most, __shfl_xor_sync(kAll, most, 2));
    if (tid % 4 == 0) s_most[tid / 4] = most;
    float part[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) part[i][0] = part[i][1] = part[i][2] = part[i][3] = 0.f;
#pragma unroll 8
    for (int k = 0; k < kTileK; ++k) {
      const float4 u = *reinterpret_cast<const float4*>(&s_q[k][ty * 4]), v = *reinterpret_cast<const float4*>(&s_b[k][tx * 4]);
      const float qq[4] = {u.x, u.y, u.z, u.w}, bb[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[i][j] = fmaf(qq[i], bb[j], part[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += part[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) err = fmaf(fabsf(q[i]), s_most[lk + i], err);
  }
  err += __shfl_xor_sync(kAll, err, 1);
  err += __shfl_xor_sync(kAll, err, 2);
  if (tid % 4 == 0 && lr < rn) a.err[(row0 + lr) * nct + ct] = err;
  __shared__ uint8_t s_missing[kTileC];
  if (tid % 2 == 0) s_missing[tid / 2] = missing;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int rr = ty * 4 + i, cc = tx * 4 + j;
      if (rr < rn && cc < cn) {
        if (s_missing[cc] && cls[(size_t)rr * a.nk + cc]) report(a.status, FA_ERR_DEVICE_CHECK);
        a.scores[(row0 + rr) * a.nk + c0 + cc] = s_missing[cc] ? -INFINITY : acc[i][j];
      }
    }
}

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
};

// shared memory of choose_row, in words
__host__ __device__ constexpr size_t row_words(int nk, int W) { return (size_t)5 * ((nk + 31) / 32) + nk + 2 * W + 2; }

// One row of the mask: query block r of (request b, KV head hk). err bounds the sum of the magnitudes that a score adds up; gamma
// times it bounds the score's error. qd(e): term e of Q-, Q+ in 64 bits.
template <int W, int D, class QFn>
__device__ void choose_row(const SelectArgs& a, int b, int hk, int r, float err, float gamma, uint32_t* sm, QFn qd) {
  using G = Group<W>;
  const int nk = a.nk, nw = (nk + 31) / 32, tid = G::tid(), lane = threadIdx.x & 31, warp = G::warp();
  uint32_t *wc = sm, *wp = wc + nw, *wx = wp + nw, *pa = wx + nw, *pb = pa + nw, *key = pb + nw;
  G grp{reinterpret_cast<int*>(key + nk), 0};
  const uint32_t below = (1u << lane) - 1u;
  const size_t row = ((size_t)b * a.Hkv + hk) * a.nq + r;
  const uint8_t* cls = a.src_class + ((size_t)(a.src_Bm > 1 ? b : 0) * a.nq + r) * nk;
  for (int i = warp; i < nw; i += W) {
    const int c = i * 32 + lane, v = c < nk ? cls[c] : 0;
    const uint32_t some = __ballot_sync(kAll, v != FA_BLOCK_EMPTY), part = __ballot_sync(kAll, v == FA_BLOCK_PARTIAL);
    if (lane == 0) {
      wc[i] = wx[i] = some;
      wp[i] = part;
    }
  }
  const int n = grp.prefix([&](int i) { return wc[i]; }, nw, pa);
  if (n > a.keep) {
    const float* score = a.scores + row * nk;
    const int want = a.keep - a.first - a.last;
    for (int i = warp; i < nw; i += W) {
      const int c = i * 32 + lane, rank = (int)pa[i] + __popc(wc[i] & below);
      const bool seen = (wc[i] >> lane) & 1u, always = seen && (rank < a.first || rank >= n - a.last);
      const uint32_t w = __ballot_sync(kAll, always);
      if (lane == 0) wx[i] = w;
      if (c < nk) key[c] = seen && !always ? order_of(score[c]) : 0u;
    }
    G::sync();
    if (want > 0) {
      uint32_t at = 0;  // the want-th largest
      for (uint32_t bit = 0x80000000u; bit; bit >>= 1) {
        int m = 0;
        for (int c = tid; c < nk; c += 32 * W) m += key[c] >= (at | bit);
        if (grp.sum(m) >= want) at |= bit;
      }
      const float t = value_of(at), e2 = 2.f * fmaf(gamma, err, 1e-42f), over = t + e2, under = t - e2;
      auto sure = [&](uint32_t k) { return k != 0u && value_of(k) > over; };
      auto near = [&](uint32_t k) { const float s = value_of(k); return k != 0u && !(s > over) && !(s < under); };  // NaN: near
      int m = 0, z = 0;
      for (int c = tid; c < nk; c += 32 * W) {
        m += sure(key[c]);
        z += near(key[c]);
      }
      m = grp.sum(m);
      z = grp.sum(z);
      if (z == want - m) {
        for (int i = warp; i < nw; i += W) {
          const int c = i * 32 + lane;
          const uint32_t w = __ballot_sync(kAll, c < nk && (sure(key[c]) || near(key[c])));
          if (lane == 0) wx[i] |= w;
        }
      } else {
        // more candidates than places: their scores in 64 bits, a warp each
        constexpr int V = 2 * D / 32;
        double q[V];
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = qd(lane * V + i);
        uint64_t* zone = a.zone + row * nk;
        for (int i = warp; i < nw; i += W) {
          const int c = i * 32 + lane;
          for (uint32_t w = __ballot_sync(kAll, c < nk && near(key[c])); w; w &= w - 1) {
            const int cc = i * 32 + __ffs(w) - 1;
            const __nv_bfloat16* box = box_of<D>(a, b, hk, cc);
            double s = -INFINITY;
            if (box) {
              s = 0.0;
              const uint32_t* src = reinterpret_cast<const uint32_t*>(box) + lane * (V / 2);
#pragma unroll
              for (int j = 0; j < V / 2; ++j) {
                const uint32_t v = __ldg(src + j);
                s = fma(q[2 * j], (double)bf_lo(v), s);
                s = fma(q[2 * j + 1], (double)bf_hi(v), s);
              }
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
            }
            if (lane == 0) zone[cc] = order_of(s);
          }
        }
        G::sync();
        const int left = want - m;
        uint64_t cut = 0;  // the left-th largest of them
        for (uint64_t bit = 1ull << 63; bit; bit >>= 1) {
          int k = 0;
          for (int c = tid; c < nk; c += 32 * W) k += near(key[c]) && zone[c] >= (cut | bit);
          if (grp.sum(k) >= left) cut |= bit;
        }
        int k = 0;
        for (int c = tid; c < nk; c += 32 * W) k += near(key[c]) && zone[c] > cut;
        const int ties = left - grp.sum(k);  // of those equal to it, the lowest columns
        for (int i = warp; i < nw; i += W) {
          const int c = i * 32 + lane;
          const uint32_t w = __ballot_sync(kAll, c < nk && near(key[c]) && zone[c] == cut);
          if (lane == 0) pb[i] = w;
        }
        grp.prefix([&](int i) { return pb[i]; }, nw, pa);
        for (int i = warp; i < nw; i += W) {
          const int c = i * 32 + lane;
          bool in = false;
          if (c < nk) in = sure(key[c]) || (near(key[c]) && (zone[c] > cut || (zone[c] == cut && (int)pa[i] + __popc(pb[i] & below) < ties)));
          const uint32_t w = __ballot_sync(kAll, in);
          if (lane == 0) wx[i] |= w;
        }
      }
    }
  }
  const int np = grp.prefix([&](int i) { return wx[i] & wp[i]; }, nw, pa);
  const int nf = grp.prefix([&](int i) { return wx[i] & ~wp[i]; }, nw, pb);
  const MaskOut& T = a.out;
  int32_t *pi = T.kv_idx + row * nk, *fi = T.full_kv_idx + row * nk;
  for (int i = warp; i < nw; i += W) {
    const int c = i * 32 + lane;
    if (c >= nk) continue;
    const uint32_t p = wx[i] & wp[i], f = wx[i] & ~wp[i];
    const bool in_p = (p >> lane) & 1u, in_f = (f >> lane) & 1u;
    if (in_p) pi[pa[i] + __popc(p & below)] = c;
    if (in_f) fi[pb[i] + __popc(f & below)] = c;
    T.block_class[row * nk + c] = in_p ? FA_BLOCK_PARTIAL : in_f ? FA_BLOCK_FULL : FA_BLOCK_EMPTY;
    if (a.nq == 1) {  // the transpose of one row
      T.q_num[row * nk + c] = in_p;
      T.full_q_num[row * nk + c] = in_f;
      T.q_idx[row * nk + c] = 0;
      T.full_q_idx[row * nk + c] = 0;
    }
  }
  for (int x = np + tid; x < nk; x += 32 * W) pi[x] = 0;
  for (int x = nf + tid; x < nk; x += 32 * W) fi[x] = 0;
  if (tid == 0) {
    T.kv_num[row] = np;
    T.full_kv_num[row] = nf;
  }
}

constexpr int kRowWarps = 8;
// A score that score_tile_kernel leaves: parts of Q added up (g at most), rounded; 32 products in a row, 8 sums; twice that for the bound's own
__device__ __forceinline__ float tile_gamma(const SelectArgs& a) { return (float)(96 + 2 * a.parts) * 5.9604644775390625e-8f; }

// W = 1: a warp a row, 8 rows a CTA; W = 8: a CTA a row
template <int W, int D>
__global__ void __launch_bounds__(kRowWarps * 32) choose_rows_kernel(const __grid_constant__ SelectArgs a) {
  extern __shared__ uint32_t dyn[];
  const int sub = W == 1 ? threadIdx.x >> 5 : 0, r = blockIdx.x * (kRowWarps / W) + sub, hk = blockIdx.y, b = blockIdx.z;
  if (r >= a.nq) return;
  const size_t row = ((size_t)b * a.Hkv + hk) * a.nq + r;
  const int nct = (a.nk + kTileC - 1) / kTileC;
  float err = 0.f;
  for (int i = threadIdx.x & 31; i < nct; i += 32) {
    const float e = a.err[row * nct + i];
    err = e > err || e != e ? e : err;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float e = __shfl_xor_sync(kAll, err, o);
    err = e > err || e != e ? e : err;
  }
  const float* pooled = a.pooled + row * a.parts * 4 * D;
  choose_row<W, D>(a, b, hk, r, err, tile_gamma(a), dyn + sub * row_words(a.nk, W), [&](int e) {
    double s = 0.0;
    for (int p = 0; p < a.parts; ++p) s += (double)pooled[p * 4 * D + e] + (double)pooled[p * 4 * D + 2 * D + e];
    return s;
  });
}

// ------------------------------------------------------------------------------------------------ one query a request
// A cluster of CTAs a (request, KV head): each sums the heads' queries for itself and scores its share of the blocks, and the first one chooses.
constexpr int kTokenWarps = 8;

template <int D>
__global__ void __launch_bounds__(kTokenWarps * 32) choose_token_kernel(const __grid_constant__ SelectArgs a, int ranks) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t dyn[];
  __shared__ float s_q[2][2 * D];  // hi, lo of Q-, Q+
  constexpr int LPB = 2 * D / 8, BPW = 32 / LPB;  // lanes a block (16 bytes each), blocks a warp has at once
  const int rank = blockIdx.x % ranks, hk = blockIdx.x / ranks, b = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.Hq / a.Hkv, nk = a.nk, nw = (nk + 31) / 32;
  const size_t row = (size_t)b * a.Hkv + hk;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + ((size_t)b * a.Hq + (size_t)hk * g) * D;
  if (tid < 2 * D) {
    const int e = tid % D;
    float hi = 0.f, lo = 0.f;
    for (int h = 0; h < g; ++h) {
      const float x = __bfloat162float(q[(size_t)h * D + e]);
      add_pair(hi, lo, tid < D ? (x > 0.f ? 0.f : x) : (x > 0.f ? x : 0.f));
    }
    s_q[0][tid] = hi;
    s_q[1][tid] = lo;
  }
  __syncthreads();
  const uint8_t* cls = a.src_class + (size_t)(a.src_Bm > 1 ? b : 0) * nk;
  float qf[8], most = 0.f;
  const int x = lane % LPB;
#pragma unroll
  for (int i = 0; i < 8; ++i) qf[i] = s_q[0][x * 8 + i];
  for (int i = rank * kTokenWarps + warp; i < nw; i += ranks * kTokenWarps) {
    const int c = i * 32 + lane;
    const bool seen = c < nk && cls[c] != FA_BLOCK_EMPTY;
    const __nv_bfloat16* mine = seen ? box_of<D>(a, b, hk, c) : nullptr;
    if (seen && !mine) report(a.status, FA_ERR_DEVICE_CHECK);
    float out = -INFINITY;
    const uint32_t w = __ballot_sync(kAll, mine != nullptr);
#pragma unroll 4
    for (int k = 0; k < 32; k += BPW) {
      if (!((w >> k) & ((1u << BPW) - 1u))) continue;
      const int j = k + lane / LPB;
      const uint64_t src = __shfl_sync(kAll, reinterpret_cast<uint64_t>(mine), j);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (src) v = __ldg(reinterpret_cast<const uint4*>(src) + x);
      const uint32_t t[4] = {v.x, v.y, v.z, v.w};
      float s = 0.f, m = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = (e & 1) ? bf_hi(t[e >> 1]) : bf_lo(t[e >> 1]);
        s = fmaf(qf[e], y, s);
        m = fmaf(fabsf(qf[e]), fabsf(y), m);
      }
      most = m > most || m != m ? m : most;
#pragma unroll
      for (int o = LPB / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
      if (BPW == 1) {
        if (lane == k) out = s;
      } else {
        const float s0 = __shfl_sync(kAll, s, 0), s1 = __shfl_sync(kAll, s, 16);
        if (lane == k) out = s0;
        if (lane == k + 1) out = s1;
      }
    }
    if (c < nk) a.scores[row * nk + c] = mine ? out : -INFINITY;
  }
  // a bound on the magnitudes of any block: the lanes' largest parts, added up
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most += __shfl_xor_sync(kAll, most, o);
  if (lane == 0) a.err[row * (8 * kTokenWarps) + rank * kTokenWarps + warp] = most;
  if (ranks > 1) {
    cg::this_cluster().sync();
    if (rank) return;
  } else {
    __syncthreads();
  }
  float err = 0.f;
  for (int i = 0; i < ranks * kTokenWarps; ++i) {
    const float e = __ldcg(a.err + row * (8 * kTokenWarps) + i);
    err = e > err || e != e ? e : err;
  }
  // Q rounded, 8 products in a row, 5 sums; twice that for the bound's own
  choose_row<kTokenWarps, D>(a, b, hk, 0, err, 32.f * 5.9604644775390625e-8f, dyn,
                             [&](int e) { return (double)s_q[0][e] + (double)s_q[1][e]; });
}

template <int D>
cudaError_t launch_bounds_d(const BoundsArgs& a, cudaStream_t st) {
  if (!a.page_table) {
    key_bounds_kernel<D><<<dim3((a.kv_len + a.page - 1) / a.page, a.Hkv, a.B), kBoundThreads, 0, st>>>(a);
  } else {
    const dim3 grid((unsigned)(((int64_t)a.N + 2 * a.page - 2) / a.page), a.Hkv, a.B);
    if (a.k_scale) kv_bounds_fp8_kernel<D><<<grid, kBound8Threads, 0, st>>>(a);
    else kv_bounds_kernel<D><<<grid, kBoundThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

template <class K>
cudaError_t allow_smem(K kernel, size_t bytes) {
  return bytes > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) : cudaSuccess;
}

template <int D>
cudaError_t launch_select_d(const SelectArgs& a, const DevRule& R, cudaStream_t st) {
  cudaError_t e;
  if (a.q_len == 1) {
    const size_t smem = row_words(a.nk, kTokenWarps) * 4;
    const int ranks = select_token_ranks(a.B * (int64_t)a.Hkv, a.nk);
    if ((e = allow_smem(choose_token_kernel<D>, smem)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.Hkv * ranks, a.B);
    cfg.blockDim = dim3(kTokenWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, choose_token_kernel<D>, a, ranks);
  }
  pool_kernel<D><<<dim3(a.nq, a.Hkv * a.parts, a.B), kPoolThreads, 0, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int nct = (a.nk + kTileC - 1) / kTileC, nrt = (a.nq + kTileR - 1) / kTileR;
  score_tile_kernel<D><<<dim3(nct * nrt, a.Hkv, a.B), kTileThreads, 0, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // a warp a row keeps many rows in flight; rows of more than 1024 blocks would take too much shared memory that way
  if (a.nk <= 1024) {
    const size_t smem = kRowWarps * row_words(a.nk, 1) * 4;
    if ((e = allow_smem(choose_rows_kernel<1, D>, smem)) != cudaSuccess) return e;
    choose_rows_kernel<1, D><<<dim3((a.nq + kRowWarps - 1) / kRowWarps, a.Hkv, a.B), kRowWarps * 32, smem, st>>>(a);
  } else {
    const size_t smem = row_words(a.nk, kRowWarps) * 4;
    if ((e = allow_smem(choose_rows_kernel<kRowWarps, D>, smem)) != cudaSuccess) return e;
    choose_rows_kernel<kRowWarps, D><<<dim3(a.nq, a.Hkv, a.B), kRowWarps * 32, smem, st>>>(a);
  }
  if ((e = cudaGetLastError()) != cudaSuccess || a.nq == 1) return e;
  return launch_mask_transpose(R, a.out, st);
}

}  // namespace

// CTAs that share the blocks of one (request, KV head)
int select_token_ranks(int64_t rows, int32_t nk) {
  int n = 1;
  while (n < 8 && rows * n < 2 * 152 && nk >= 128 * n) n *= 2;
  return n;
}

size_t select_err_floats(int32_t q_len, int32_t nk) {
  return q_len == 1 ? 8 * kTokenWarps : (nk + kTileC - 1) / kTileC;
}

cudaError_t launch_bounds(const BoundsArgs& a, cudaStream_t st) {
  return a.d == 64 ? launch_bounds_d<64>(a, st) : launch_bounds_d<128>(a, st);
}

cudaError_t launch_select_blocks(const SelectArgs& a, const DevRule& R, cudaStream_t st) {
  return a.d == 64 ? launch_select_d<64>(a, R, st) : launch_select_d<128>(a, R, st);
}

}  // namespace fa
