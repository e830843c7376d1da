// The attention's inputs: norms of the query and key heads, the rotation by position, and where the rows go.
//
//   r = rsqrt(mean_e x_e^2 + eps),  y = x r w            (no weight: y = x)
//   (z_a, z_b) = (y_a c - y_b s, y_a s + y_b c)          c, s = cos, sin of position * inv_freq[i], pair i = (a, b)
//
// All of it in fp32, one rounding to bf16 (or e4m3) at the end. The angle is taken modulo one turn in 64-bit integers:
// inv_freq / 2 pi is held as a fraction of 2^64 (an integer product, no floating point), a position times it wraps
// around exactly where whole turns do, and the top 32 bits go to sincospif. The error is under 2^-24 turns at any
// position (an fp32 product would be off by position * 2^-24).
//
// Bound: HBM. A row of d values is held by d / 8 lanes, 8 values (16 bytes) a lane: the norm is a few shuffles, and
// the other element of a pair is either in the same lane (neighbouring pairs) or in the same place of one other lane
// (halves: rot is a multiple of 16). cos and sin are computed once a token and shared by all of its heads.
#include "fa_launch.h"
#include "fp8.cuh"

namespace fa {
namespace {

typedef __nv_bfloat16 bf16;

constexpr int kThreads = 256;
constexpr int kTok = 4;          // tokens of a CTA of the row kernels
constexpr int kBatch = 4;        // rows a thread loads before it uses the first

// Fraction of a turn per position, in units of 2^-64 (modulo one turn): inv_freq = m 2^(x-23) times
// floor(2^64 / 2 pi).
__device__ __forceinline__ uint64_t turns_per_position(float inv_freq) {
  const uint32_t u = __float_as_uint(inv_freq);
  int x = (int)((u >> 23) & 255u);
  uint64_t m = u & 0x7FFFFFu;
  if (x > 0) m |= 0x800000u; else x = 1;
  constexpr uint64_t kInv2Pi = 0x28BE60DB9391054Aull;
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  const int sh = 23 - (x - 127);
  uint64_t f;
  if (sh >= 128 || sh <= -64) f = 0;
  else if (sh >= 64) f = hi >> (sh - 64);
  else if (sh > 0) f = (lo >> sh) | (hi << (64 - sh));
  else f = lo << (-sh);
  return (u >> 31) ? 0ull - f : f;
}

__device__ __forceinline__ float2 cos_sin(uint64_t f, int64_t pos) {
  const uint64_t turns = (uint64_t)pos * f;
  float s, c;
  sincospif((float)(int32_t)(turns >> 32) * 4.656612873077393e-10f /* 2^-31: half turns */, &s, &c);
  return make_float2(c, s);
}

// What a lane of a row does for the rotation: element e of the lane's 8 becomes y_e c[e] + p_e s[e], with p_e the
// other element of the pair (s carries the sign).
struct LaneRot {
  int partner;      // lane of the row that holds the other elements (halves)
  int i0;           // first pair index of the lane
  float sign;       // halves: -1 in the first half, +1 in the second; 0: not rotated
  bool inter;
};

template <int D>
__device__ __forceinline__ LaneRot lane_rot(int lane, int rot, int interleaved) {
  LaneRot r;
  const int e0 = lane * 8, half = rot / 2;
  r.inter = interleaved != 0;
  r.partner = lane;
  r.i0 = 0;
  r.sign = 0.f;
  if (e0 < rot) {
    if (r.inter) {
      r.sign = 1.f;
      r.i0 = e0 / 2;
    } else {
      const bool first = e0 < half;
      r.sign = first ? -1.f : 1.f;
      r.i0 = first ? e0 : e0 - half;
      r.partner = first ? lane + half / 8 : lane - half / 8;
    }
  }
  return r;
}

// c[e], s[e] of the lane from a token's table (inverse: the transposed rotation)
template <bool INVERSE>
__device__ __forceinline__ void lane_cos_sin(const float2* table, const LaneRot& r, float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c[e] = 1.f;
    s[e] = 0.f;
  }
  if (r.sign == 0.f) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 t = table[r.inter ? r.i0 + e / 2 : r.i0 + e];
    c[e] = t.x;
    const float g = r.inter ? ((e & 1) ? 1.f : -1.f) : r.sign;
    s[e] = INVERSE ? -g * t.y : g * t.y;
  }
}

// Every lane of the warp calls this (rows that are not there compute on zeros).
template <int LPR>
__device__ __forceinline__ void rotate(float (&y)[8], const LaneRot& r, const float (&c)[8], const float (&s)[8]) {
  float p[8];
  if (r.inter) {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = y[e ^ 1];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = __shfl_sync(0xFFFFFFFFu, y[e], r.partner, LPR);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = fmaf(p[e], s[e], y[e] * c[e]);
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o, LPR);
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o, LPR));
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ void load_w(const float* w, int e0, float (&r)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = w ? __ldg(w + e0 + e) : 1.f;
}

template <int D>
__device__ __forceinline__ void norm_rope(float (&x)[8], bool norm, float eps, const float (&w)[8], bool rope,
                                          const LaneRot& r, const float (&c)[8], const float (&s)[8]) {
  if (norm) {
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) q = fmaf(x[e], x[e], q);
    q = row_sum<D / 8>(q);
    const float rs = rsqrtf(q * (1.f / D) + eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * rs * w[e];
  }
  if (rope) rotate<D / 8>(x, r, c, s);
}

// e4m3 block of one head: rows old tokens keep their place; from scale `was` to scale `now`
template <int D>
__device__ __forceinline__ void rescale_row(uint8_t* row, int e0, float ratio) {
  uint2* p = reinterpret_cast<uint2*>(row + e0);
  const uint2 v = *p;
  uint2 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    e4m3x4_to_f16(i ? v.y : v.x, lo, hi);
    const float2 a = f16x2_to_f32(lo), b = f16x2_to_f32(hi);
    const uint32_t r = pack_e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
    if (i) o.y = r; else o.x = r;
  }
  *p = o;
}

__device__ __forceinline__ uint2 quantise8(const float (&y)[8], float inv) {
  return make_uint2(pack_e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                    pack_e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
}

// ------------------------------------------------------------------------------------------------
// Rows of tokens [first, first + kTok) of the call (token = b * N + n), heads [h0, h1) of the row of heads
// (query heads, then key heads, then value heads, absent ones left out).
// ------------------------------------------------------------------------------------------------
enum { kToHeads = 0, kToPages = 1, kToPagesFp8 = 2 };

__device__ __forceinline__ int new_tokens(const QkvArgs& a, int b) {
  if (!a.n_new) return a.N;
  const int n = __ldg(a.n_new + b);
  if (n < 0 || n > a.N) {
    report(a.status, FA_ERR_DEVICE_CHECK);
    return n < 0 ? 0 : a.N;
  }
  return n;
}

// slot of position pos of request b: page id * page + place, or -1 (reported)
__device__ __forceinline__ int64_t page_slot(const QkvArgs& a, int b, int64_t pos) {
  int64_t at = -1;
  if (pos >= 0 && pos < (int64_t)a.max_pages * a.page) {
    const int c = (int)(pos / a.page);
    const int pid = __ldg(a.page_table + (int64_t)b * a.max_pages + c);
    if (pid >= 0 && pid < a.n_pages_total) at = (int64_t)pid * a.page + (pos - (int64_t)c * a.page);
  }
  if (at < 0) report(a.status, FA_ERR_DEVICE_CHECK);
  return at;
}

template <int D, int DST>
__device__ __forceinline__ void rows_of_tokens(const QkvArgs& a, int64_t first, int h0, int h1, int nq, int nk,
                                               float2 (*s_cs)[D / 2]) {
  constexpr int LPR = D / 8, SLOTS = kThreads / LPR;
  const int tid = threadIdx.x, lane = tid % LPR, slot = tid / LPR, e0 = lane * 8;
  const int64_t tokens = (int64_t)a.B * a.N;
  const bool rope = a.inv_freq != nullptr && h0 < nq + nk;
  const int half = a.rot / 2;
  if (rope) {
    for (int x = tid; x < kTok * half; x += kThreads) {
      const int t = x / half, i = x - t * half;
      const int64_t T = first + t;
      if (T < tokens) {
        const int b = (int)(T / a.N), n = (int)(T - (int64_t)b * a.N);
        s_cs[t][i] = cos_sin(turns_per_position(__ldg(a.inv_freq + i)), (int64_t)n + (a.q_offset ? __ldg(a.q_offset + b) : 0));
      }
    }
    __syncthreads();
  }
  const LaneRot lr = lane_rot<D>(lane, a.inv_freq ? a.rot : 0, a.interleaved);
  float wq[8], wk[8];
  load_w(a.wq, e0, wq);
  load_w(a.wk, e0, wk);
  for (int t = 0; t < kTok; ++t) {
    const int64_t T = first + t;
    if (T >= tokens) break;
    const int b = (int)(T / a.N), n = (int)(T - (int64_t)b * a.N);
    if (DST != kToHeads && n >= new_tokens(a, b)) continue;
    const int64_t pos = (int64_t)n + (a.q_offset ? __ldg(a.q_offset + b) : 0);
    const int64_t at = DST != kToHeads && h1 > nq ? page_slot(a, b, pos) : 0;
    float c[8], s[8];
    if (rope) lane_cos_sin<false>(s_cs[t], lr, c, s);
    // every warp takes the same number of steps: the shuffles want all lanes
    for (int hb = h0; hb < h1; hb += SLOTS * kBatch) {
      uint4 raw[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int h = hb + u * SLOTS + slot;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (h < h1) {
          const bool isq = h < nq, isk = !isq && h < nq + nk;
          const Rows& R = isq ? a.q : isk ? a.k : a.v;
          const int hh = isq ? h : isk ? h - nq : h - nq - nk;
          raw[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const bf16*>(R.p) + b * R.sb + n * R.sn + hh * R.sh + e0));
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (hb + u * SLOTS >= h1) break;  // the same for all threads
        const int h = hb + u * SLOTS + slot;
        const bool live = h < h1, isq = h < nq, isk = !isq && h < nq + nk, isv = !isq && !isk;
        const int hh = isq ? h : isk ? h - nq : h - nq - nk;
        float y[8];
        unpack8(raw[u], y);
        const bool any_qk = __any_sync(0xFFFFFFFFu, live && !isv);
        if (any_qk) {
          float z[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = y[e];
          const bool norm_row = isq ? a.wq != nullptr : a.wk != nullptr;
          if (a.wq || a.wk) {
            float q2 = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) q2 = fmaf(z[e], z[e], q2);
            q2 = row_sum<LPR>(q2);
            if (norm_row) {
              const float rs = rsqrtf(q2 * (1.f / D) + a.eps);
#pragma unroll
              for (int e = 0; e < 8; ++e) z[e] = z[e] * rs * (isq ? wq[e] : wk[e]);
            }
          }
          if (rope) rotate<LPR>(z, lr, c, s);
          if (!isv) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = z[e];
          }
        }
        if (DST == kToPagesFp8) {
          // one new token a request: its 32-token block holds the tokens before it under the scale they have, which
          // one lane reads and writes
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
          m = row_max<LPR>(m);
          const bool mine = live && !isq && at >= 0;
          const int64_t pid = mine ? at / a.page : 0, place = mine ? at - pid * a.page : 0;
          const int before = (int)(place % kScaleTokens);
          float* sc = (isk ? a.k_scale : a.v_scale) + (pid * a.Hkv + hh) * (a.page / kScaleTokens) + place / kScaleTokens;
          float was = 0.f;
          if (mine && before && lane == 0) was = clamp_scale(*sc);
          was = __shfl_sync(0xFFFFFFFFu, was, 0, LPR);
          if (mine) {
            uint8_t* base = static_cast<uint8_t*>(isk ? a.k_pages : a.v_pages) + (pid * a.Hkv + hh) * a.page * D;
            const float now = fmaxf(need_scale(m), was);
            if (before && now != was)
              for (int64_t i = place - before; i < place; ++i) rescale_row<D>(base + i * D, e0, was / now);
            *reinterpret_cast<uint2*>(base + place * D + e0) = quantise8(y, 1.f / now);
            if (lane == 0) *sc = now;
          }
        }
        if (live && (DST != kToPagesFp8 || isq)) {
          bf16* dst;
          if (DST == kToHeads || isq) {
            bf16* o = static_cast<bf16*>(isq ? a.q_out : isk ? a.k_out : a.v_out);
            dst = o + (((int64_t)b * (isq ? a.Hq : a.Hkv) + hh) * a.N + n) * D;
          } else {
            const int64_t pid = at / a.page;
            dst = at < 0 ? nullptr
                         : static_cast<bf16*>(isk ? a.k_pages : a.v_pages) + ((pid * a.Hkv + hh) * a.page + (at - pid * a.page)) * D;
          }
          if (dst) *reinterpret_cast<uint4*>(dst + e0) = isv ? raw[u] : pack8(y);
        }
      }
    }
  }
}

template <int D, int DST>
__global__ void __launch_bounds__(kThreads) qkv_rows_kernel(const __grid_constant__ QkvArgs a, int heads_per_cta) {
  __shared__ float2 s_cs[kTok][D / 2];
  const int nq = a.q.p ? a.Hq : 0, nk = a.k.p ? a.Hkv : 0, nv = a.v.p ? a.Hkv : 0;
  const int h0 = blockIdx.y * heads_per_cta, h1 = min(nq + nk + nv, h0 + heads_per_cta);
  rows_of_tokens<D, DST>(a, (int64_t)blockIdx.x * kTok, h0, h1, nq, nk, s_cs);
}

// ------------------------------------------------------------------------------------------------
// Append to e4m3 pages, several tokens a request. A CTA takes one 32-token block of one request and a group of its
// KV heads: for each head, K and then V, its threads hold the block's new rows, agree on the largest magnitude, and
// write scale and values; rows that the block held before are rescaled where the scale grew. CTAs behind those take
// the query rows.
// ------------------------------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void append_block(const QkvArgs& a, int b, int j, int hk0, int hk1, float2 (*s_cs)[D / 2],
                                             float (*s_max)[kThreads / 32]) {
  constexpr int LPR = D / 8, SLOTS = kThreads / LPR, RPT = kScaleTokens / SLOTS > 0 ? kScaleTokens / SLOTS : 1;
  const int tid = threadIdx.x, lane = tid % LPR, slot = tid / LPR, e0 = lane * 8;
  const int cnt = new_tokens(a, b);
  const int64_t first = a.q_offset ? __ldg(a.q_offset + b) : 0, last = first + cnt;
  const int64_t p0 = ((first >> 5) + j) * kScaleTokens;
  const int64_t lo = max(p0, first), hi = min(p0 + kScaleTokens, last);
  if (lo >= hi) return;
  const int64_t at0 = page_slot(a, b, p0);
  if (at0 < 0) return;
  const int64_t pid = at0 / a.page, place0 = at0 - pid * a.page;
  const bool rope = a.inv_freq != nullptr;
  const int half = a.rot / 2;
  if (rope) {
    for (int x = tid; x < kScaleTokens * half; x += kThreads) {
      const int t = x / half, i = x - t * half;
      s_cs[t][i] = cos_sin(turns_per_position(__ldg(a.inv_freq + i)), p0 + t);
    }
  }
  __syncthreads();
  const LaneRot lr = lane_rot<D>(lane, rope ? a.rot : 0, a.interleaved);
  float wk[8];
  load_w(a.wk, e0, wk);
  float c[RPT][8], s[RPT][8];
  if (rope) {
#pragma unroll
    for (int u = 0; u < RPT; ++u) lane_cos_sin<false>(s_cs[slot + u * SLOTS], lr, c[u], s[u]);
  }
  const int before = (int)(lo - p0);
  const int units = 2 * (hk1 - hk0);  // K and V of each head
  auto load = [&](int x, uint4 (&raw)[RPT]) {
    const Rows& R = (x & 1) ? a.v : a.k;
    const bf16* base = static_cast<const bf16*>(R.p) + b * R.sb + (hk0 + (x >> 1)) * R.sh + e0;
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
      const int64_t pos = p0 + slot + u * SLOTS;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (pos >= lo && pos < hi) raw[u] = __ldg(reinterpret_cast<const uint4*>(base + (pos - first) * R.sn));
    }
  };
  uint4 nxt[RPT];
  load(0, nxt);
  for (int x = 0; x < units; ++x) {
    float y[RPT][8];
#pragma unroll
    for (int u = 0; u < RPT; ++u) unpack8(nxt[u], y[u]);
    if (x + 1 < units) load(x + 1, nxt);
    float m = 0.f;
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
      if (!(x & 1)) norm_rope<D>(y[u], a.wk != nullptr, a.eps, wk, rope, lr, c[u], s[u]);
      const int64_t pos = p0 + slot + u * SLOTS;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = pos >= lo && pos < hi ? fmaxf(m, fabsf(y[u][e])) : m;
    }
    m = row_max<32>(m);
    if ((tid & 31) == 0) s_max[x & 1][tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, s_max[x & 1][w]);
    const int hk = hk0 + (x >> 1);
    float* sc = ((x & 1) ? a.v_scale : a.k_scale) + (pid * a.Hkv + hk) * (a.page / kScaleTokens) + place0 / kScaleTokens;
    uint8_t* base = static_cast<uint8_t*>((x & 1) ? a.v_pages : a.k_pages) + ((pid * a.Hkv + hk) * a.page + place0) * D;
    float now = need_scale(m);
    if (before) {
      const float was = clamp_scale(*sc);
      now = fmaxf(now, was);
      if (now != was)
        for (int i = slot; i < before; i += SLOTS) rescale_row<D>(base + (int64_t)i * D, e0, was / now);
      __syncthreads();  // every thread has read the old scale
    }
    const float inv = 1.f / now;
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
      const int r = slot + u * SLOTS;
      if (p0 + r >= lo && p0 + r < hi) *reinterpret_cast<uint2*>(base + (int64_t)r * D + e0) = quantise8(y[u], inv);
    }
    if (tid == 0) *sc = now;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    append_fp8_kernel(const __grid_constant__ QkvArgs a, int blocks, int heads_per_cta, int groups) {
  __shared__ float2 s_cs[kScaleTokens][D / 2];
  __shared__ float s_max[2][kThreads / 32];
  const int64_t kv_ctas = (int64_t)a.B * blocks * groups;
  if ((int64_t)blockIdx.x < kv_ctas) {
    const int x = blockIdx.x, gi = x % groups, bj = x / groups;
    const int hk0 = gi * heads_per_cta;
    append_block<D>(a, bj / blocks, bj % blocks, hk0, min(a.Hkv, hk0 + heads_per_cta), s_cs, s_max);
  } else {
    rows_of_tokens<D, kToPages>(a, ((int64_t)blockIdx.x - kv_ctas) * kTok, 0, a.Hq, a.Hq, 0, s_cs);
  }
}

// ------------------------------------------------------------------------------------------------
// Backward of the rows: with g = R^T dz (the transposed rotation) and xhat = x r,
//   dw += g xhat,   dx = r (w g - xhat mean(w g xhat))     (no weight: dx = g)
// r is recomputed from x. A CTA walks tokens and keeps its sums of dw in registers (a lane always holds the same 8
// places); they are joined in shared memory, written one row a CTA, and added up by a second kernel in a fixed order:
// no atomics, the same result each time.
// ------------------------------------------------------------------------------------------------
template <int D, bool F32>
__device__ __forceinline__ void store_grad(void* p, int64_t at, const float (&g)[8]) {
  if (F32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    o[0] = make_float4(g[0], g[1], g[2], g[3]);
    o[1] = make_float4(g[4], g[5], g[6], g[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<bf16*>(p) + at) = pack8(g);
  }
}

template <int D, bool F32>
__global__ void __launch_bounds__(kThreads) qkv_bwd_kernel(const __grid_constant__ QkvBwdArgs a) {
  constexpr int LPR = D / 8, SLOTS = kThreads / LPR, U = 2;
  __shared__ float2 s_cs[kTok][D / 2];
  __shared__ float s_dw[SLOTS][D];
  const int tid = threadIdx.x, lane = tid % LPR, slot = tid / LPR, e0 = lane * 8;
  const int nq = a.dq ? a.Hq : 0, nk = a.dk ? a.Hkv : 0, nv = a.dv ? a.Hkv : 0, H = nq + nk + nv;
  const int64_t tokens = (int64_t)a.B * a.N;
  const bool rope = a.inv_freq != nullptr;
  const int half = a.rot / 2;
  const LaneRot lr = lane_rot<D>(lane, rope ? a.rot : 0, a.interleaved);
  float wq[8], wk[8], dwq[8], dwk[8];
  load_w(a.wq, e0, wq);
  load_w(a.wk, e0, wk);
#pragma unroll
  for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;
  for (int64_t first = (int64_t)blockIdx.x * kTok; first < tokens; first += (int64_t)gridDim.x * kTok) {
    if (rope) {
      __syncthreads();  // the table of the last tokens is read
      for (int x = tid; x < kTok * half; x += kThreads) {
        const int t = x / half, i = x - t * half;
        const int64_t T = first + t;
        if (T < tokens) {
          const int b = (int)(T / a.N), n = (int)(T - (int64_t)b * a.N);
          s_cs[t][i] = cos_sin(turns_per_position(__ldg(a.inv_freq + i)), (int64_t)n + (a.q_offset ? __ldg(a.q_offset + b) : 0));
        }
      }
      __syncthreads();
    }
    for (int t = 0; t < kTok; ++t) {
      const int64_t T = first + t;
      if (T >= tokens) break;
      const int b = (int)(T / a.N), n = (int)(T - (int64_t)b * a.N);
      float c[8], s[8];
      if (rope) lane_cos_sin<true>(s_cs[t], lr, c, s);
      for (int hb = 0; hb < H; hb += SLOTS * U) {
        uint4 raw[U];
        float4 g0[U], g1[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = hb + u * SLOTS + slot;
          raw[u] = make_uint4(0, 0, 0, 0);
          g0[u] = g1[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (h < H) {
            const bool isq = h < nq, isk = !isq && h < nq + nk;
            const int hh = isq ? h : isk ? h - nq : h - nq - nk;
            const float* dy = (isq ? a.dq : isk ? a.dk : a.dv) + (((int64_t)b * (isq ? a.Hq : a.Hkv) + hh) * a.N + n) * D + e0;
            g0[u] = __ldg(reinterpret_cast<const float4*>(dy));
            g1[u] = __ldg(reinterpret_cast<const float4*>(dy) + 1);
            const Rows& R = isq ? a.q : a.k;
            if ((isq && a.wq) || (isk && a.wk))
              raw[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const bf16*>(R.p) + b * R.sb + n * R.sn + hh * R.sh + e0));
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (hb + u * SLOTS >= H) break;
          const int h = hb + u * SLOTS + slot;
          const bool live = h < H, isq = h < nq, isk = !isq && h < nq + nk, isv = !isq && !isk;
          const int hh = isq ? h : isk ? h - nq : h - nq - nk;
          float g[8] = {g0[u].x, g0[u].y, g0[u].z, g0[u].w, g1[u].x, g1[u].y, g1[u].z, g1[u].w};
          if (__any_sync(0xFFFFFFFFu, live && !isv)) {
            float z[8], x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = g[e];
            if (rope) rotate<LPR>(z, lr, c, s);
            if (a.wq || a.wk) {
              unpack8(raw[u], x);
              const bool norm_row = isq ? a.wq != nullptr : a.wk != nullptr;
              float q2 = 0.f;
#pragma unroll
              for (int e = 0; e < 8; ++e) q2 = fmaf(x[e], x[e], q2);
              q2 = row_sum<LPR>(q2);
              const float r = rsqrtf(q2 * (1.f / D) + a.eps);
              float dot = 0.f;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                x[e] *= r;
                const float gx = z[e] * x[e], w = isq ? wq[e] : wk[e];
                if (live && norm_row) {
                  if (isq) dwq[e] += gx;
                  if (isk) dwk[e] += gx;
                }
                dot = fmaf(w, gx, dot);
              }
              dot = row_sum<LPR>(dot) * (1.f / D);
              if (norm_row) {
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = r * ((isq ? wq[e] : wk[e]) * z[e] - x[e] * dot);
              }
            }
            if (!isv) {
#pragma unroll
              for (int e = 0; e < 8; ++e) g[e] = z[e];
            }
          }
          if (live) {
            const Rows& R = isq ? a.dq_in : isk ? a.dk_in : a.dv_in;
            store_grad<D, F32>(R.p, b * R.sb + n * R.sn + hh * R.sh + e0, g);
          }
        }
      }
    }
  }
  if (!a.wq && !a.wk) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) s_dw[slot][e0 + e] = which ? dwk[e] : dwq[e];
    __syncthreads();
    if (tid < D) {
      float v = 0.f;
#pragma unroll 4
      for (int i = 0; i < SLOTS; ++i) v += s_dw[i][tid];
      a.partial[((int64_t)blockIdx.x * 2 + which) * D + tid] = v;
    }
  }
}

// Sums of the CTAs' rows: 32 columns of [dwq | dwk] a CTA, 32 rows at a time.
__global__ void __launch_bounds__(1024) dw_reduce_kernel(const float* partial, int ctas, int d, float* dwq, float* dwk) {
  __shared__ float s[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  for (int i = threadIdx.y; i < ctas; i += 32) v += partial[(int64_t)i * 2 * d + col];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = s[threadIdx.x][threadIdx.y];  // lane = row of the sum, warp = column
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (threadIdx.x == 0) {
    const int c = blockIdx.x * 32 + threadIdx.y;
    if (c < d) {
      if (dwq) dwq[c] = v;
    } else if (dwk) {
      dwk[c - d] = v;
    }
  }
}

constexpr int kSms = 152;

// Groups of heads for the row kernels: one CTA a token group where that fills the GPU twice over, else the heads are
// dealt out so that a decode step's few tokens still reach every SM.
int heads_per_cta(int64_t token_ctas, int H, int slots) {
  int groups = 1;
  while (token_ctas * groups < 2 * kSms && (H + groups - 1) / groups > slots) ++groups;
  return (H + groups - 1) / groups;
}

template <int D, int DST>
cudaError_t run_rows(const QkvArgs& a, cudaStream_t st) {
  const int H = (a.q.p ? a.Hq : 0) + (a.k.p ? a.Hkv : 0) + (a.v.p ? a.Hkv : 0);
  const int64_t ctas = ((int64_t)a.B * a.N + kTok - 1) / kTok;
  const int hpc = heads_per_cta(ctas, H, kThreads / (D / 8));
  qkv_rows_kernel<D, DST><<<dim3((unsigned)ctas, (H + hpc - 1) / hpc), kThreads, 0, st>>>(a, hpc);
  return cudaGetLastError();
}

template <int D>
cudaError_t run_append(const QkvArgs& a, cudaStream_t st) {
  if (!a.k_scale) return run_rows<D, kToPages>(a, st);
  if (a.N == 1) return run_rows<D, kToPagesFp8>(a, st);
  const int blocks = (a.N + 2 * kScaleTokens - 2) / kScaleTokens;
  const int hpc = heads_per_cta((int64_t)a.B * blocks, a.Hkv, 1);
  const int groups = (a.Hkv + hpc - 1) / hpc;
  const int64_t ctas = (int64_t)a.B * blocks * groups + (a.q.p ? ((int64_t)a.B * a.N + kTok - 1) / kTok : 0);
  append_fp8_kernel<D><<<(unsigned)ctas, kThreads, 0, st>>>(a, blocks, hpc, groups);
  return cudaGetLastError();
}

template <int D>
cudaError_t run_bwd(const QkvBwdArgs& a, cudaStream_t st) {
  const int ctas = qk_bwd_ctas((int64_t)a.B * a.N);
  if (a.grad_f32)
    qkv_bwd_kernel<D, true><<<ctas, kThreads, 0, st>>>(a);
  else
    qkv_bwd_kernel<D, false><<<ctas, kThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!a.wq && !a.wk)) return e;
  dw_reduce_kernel<<<2 * D / 32, dim3(32, 32), 0, st>>>(a.partial, ctas, D, a.dwq, a.dwk);
  return cudaGetLastError();
}

}  // namespace

int qk_bwd_ctas(int64_t tokens) {
  const int64_t n = (tokens + kTok - 1) / kTok;
  return (int)(n < 4 * kSms ? n : 4 * kSms);
}

cudaError_t launch_qk_norm_rope(const QkvArgs& a, cudaStream_t st) {
  return a.d == 64 ? run_rows<64, kToHeads>(a, st) : run_rows<128, kToHeads>(a, st);
}
cudaError_t launch_kv_append(const QkvArgs& a, cudaStream_t st) {
  return a.d == 64 ? run_append<64>(a, st) : run_append<128>(a, st);
}
cudaError_t launch_qk_norm_rope_backward(const QkvBwdArgs& a, cudaStream_t st) {
  return a.d == 64 ? run_bwd<64>(a, st) : run_bwd<128>(a, st);
}

}  // namespace fa
