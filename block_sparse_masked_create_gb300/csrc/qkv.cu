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
// Bound: HBM, if the instructions are few: with a thread block to a few tokens and the pair's other element fetched by
// shuffles, a step of two rows took 265 instructions and the issue slots were 72 % busy at 37 % of the DRAM rate. So:
//  - a warp takes a token (or, where tokens are few, a share of its heads) and walks its heads, 32 / (d / 8) rows a step:
//    what depends on the token alone is computed once for all of them, the norm's weight is folded into cos and sin;
//  - a lane of a row holds 8 elements as two groups of 4, placed so that both elements of each pair are its own;
//  - arithmetic is on packed pairs of fp32;
//  - loads run ahead through a ring of asynchronous copies in shared memory that only the thread itself reads and
//    writes: many rows in flight without registers to hold them, and no barrier;
//  - the grid is what is resident, and warps walk tokens.
// Measured on one GB300: 4 x 4096 tokens, 16 + 32 heads, d = 128: 66.9 us, 6.0 TB/s of 6.77 measured (first kernel 147; a plain
// copy in the same pattern runs at 5.8); the gradient of 16,384 tokens, 32 + 16 heads: 119.6 us, 6.45 TB/s (first 258); 8 x up
// to 2048 tokens into e4m3 pages: 62.9 us (first 129); one token of 64 requests: 6.3 us (bf16), 7.6 us (e4m3).
#include <algorithm>

#include "fa_launch.h"
#include "fp8.cuh"

namespace fa {
namespace {

typedef __nv_bfloat16 bf16;

constexpr int kSms = 152;

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

// Which elements of a row a lane holds: groups of four at ea and eb. Halves: (ea + k, eb + k) is pair i0 + k; neighbours:
// the 8 elements from ea on are pairs i0 .. i0 + 3. Lanes behind the rotated part hold 8 neighbouring elements.
struct LaneMap {
  int ea, eb, i0;
  bool rot;
};

template <int D, bool INTER>
__device__ __forceinline__ LaneMap lane_map(int lane, int rot) {
  LaneMap m;
  const int half = rot / 2;
  if (!INTER && lane * 4 < half) {
    m.ea = lane * 4;
    m.eb = half + lane * 4;
    m.i0 = lane * 4;
    m.rot = true;
  } else {
    m.ea = INTER ? lane * 8 : rot + (lane - half / 4) * 8;
    m.eb = m.ea + 4;
    m.i0 = lane * 4;
    m.rot = INTER && lane * 8 < rot;
  }
  return m;
}

// A lane's 8 elements as fp32 pairs: a = the first elements of its four pairs, b = the second ones.
struct Eight {
  uint64_t a[2], b[2];
};

__device__ __forceinline__ uint64_t widen(uint32_t w) {
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <bool INTER>
__device__ __forceinline__ Eight unpack(const uint2& va, const uint2& vb) {
  Eight r;
  if (INTER) {
    r.a[0] = f2_pack(__uint_as_float(va.x << 16), __uint_as_float(va.y << 16));
    r.a[1] = f2_pack(__uint_as_float(vb.x << 16), __uint_as_float(vb.y << 16));
    r.b[0] = f2_pack(__uint_as_float(va.x & 0xFFFF0000u), __uint_as_float(va.y & 0xFFFF0000u));
    r.b[1] = f2_pack(__uint_as_float(vb.x & 0xFFFF0000u), __uint_as_float(vb.y & 0xFFFF0000u));
  } else {
    r.a[0] = widen(va.x);
    r.a[1] = widen(va.y);
    r.b[0] = widen(vb.x);
    r.b[1] = widen(vb.y);
  }
  return r;
}

// fp32 values at ea .. ea + 3 and eb .. eb + 3
template <bool INTER>
__device__ __forceinline__ Eight unpack_f32(const float4& va, const float4& vb) {
  Eight r;
  if (INTER) {
    r.a[0] = f2_pack(va.x, va.z);
    r.a[1] = f2_pack(vb.x, vb.z);
    r.b[0] = f2_pack(va.y, va.w);
    r.b[1] = f2_pack(vb.y, vb.w);
  } else {
    r.a[0] = f2_pack(va.x, va.y);
    r.a[1] = f2_pack(va.z, va.w);
    r.b[0] = f2_pack(vb.x, vb.y);
    r.b[1] = f2_pack(vb.z, vb.w);
  }
  return r;
}

// the values in the order of their elements: ea .. ea + 3, eb .. eb + 3
template <bool INTER>
__device__ __forceinline__ void in_order(const Eight& v, float (&y)[8]) {
  float a[4], b[4];
  f2_unpack(v.a[0], a[0], a[1]);
  f2_unpack(v.a[1], a[2], a[3]);
  f2_unpack(v.b[0], b[0], b[1]);
  f2_unpack(v.b[1], b[2], b[3]);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    y[k] = INTER ? ((k & 1) ? b[k >> 1] : a[k >> 1]) : a[k];
    y[4 + k] = INTER ? ((k & 1) ? b[2 + (k >> 1)] : a[2 + (k >> 1)]) : b[k];
  }
}

template <bool INTER>
__device__ __forceinline__ Eight load_weight(const float* w, const LaneMap& m) {
  float4 a = make_float4(1.f, 1.f, 1.f, 1.f), b = a;
  if (w) {
    a = make_float4(__ldg(w + m.ea), __ldg(w + m.ea + 1), __ldg(w + m.ea + 2), __ldg(w + m.ea + 3));
    b = make_float4(__ldg(w + m.eb), __ldg(w + m.eb + 1), __ldg(w + m.eb + 2), __ldg(w + m.eb + 3));
  }
  return unpack_f32<INTER>(a, b);
}

// cos and sin of the lane's four pairs at a position
struct Turn {
  uint64_t c[2], s[2];
};

__device__ __forceinline__ Turn turn_at(const uint64_t (&f)[4], const LaneMap& m, int64_t pos) {
  Turn t;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float2 u = make_float2(1.f, 0.f), v = u;
    if (m.rot) {
      u = cos_sin(f[2 * j], pos);
      v = cos_sin(f[2 * j + 1], pos);
    }
    t.c[j] = f2_pack(u.x, v.x);
    t.s[j] = f2_pack(u.y, v.y);
  }
  return t;
}

__device__ __forceinline__ void lane_frequencies(const float* inv_freq, const LaneMap& m, uint64_t (&f)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = m.rot ? turns_per_position(__ldg(inv_freq + m.i0 + k)) : 0ull;
}

// norm and rotation with the weight folded in: z_a = r (x_a aa + x_b ab), z_b = r (x_a ba + x_b bb)
struct Map2 {
  uint64_t aa[2], ab[2], ba[2], bb[2];
};

__device__ __forceinline__ uint64_t f2_neg(uint64_t v) { return v ^ 0x8000000080000000ull; }

__device__ __forceinline__ Map2 fold(const Turn& t, const Eight& w) {
  Map2 m;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    m.aa[j] = f2_mul(w.a[j], t.c[j]);
    m.ab[j] = f2_neg(f2_mul(w.b[j], t.s[j]));
    m.ba[j] = f2_mul(w.a[j], t.s[j]);
    m.bb[j] = f2_mul(w.b[j], t.c[j]);
  }
  return m;
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

// r of a row; every lane of the warp calls it
template <int D>
__device__ __forceinline__ float row_rsqrt(const Eight& x, float eps) {
  const uint64_t q = f2_fma(x.b[1], x.b[1], f2_fma(x.b[0], x.b[0], f2_fma(x.a[1], x.a[1], f2_mul(x.a[0], x.a[0]))));
  float u, v;
  f2_unpack(q, u, v);
  return rsqrtf(fmaf(row_sum<D / 8>(u + v), 1.f / D, eps));
}

template <int D>
__device__ __forceinline__ Eight norm_rope(const Eight& x, bool norm, float eps, const Map2& m, bool rot) {
  Eight z;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    z.a[j] = f2_mul(x.a[j], m.aa[j]);
    z.b[j] = f2_mul(x.b[j], m.bb[j]);
    if (rot) {  // elsewhere an infinity must not meet its neighbour through a factor of zero
      z.a[j] = f2_fma(x.b[j], m.ab[j], z.a[j]);
      z.b[j] = f2_fma(x.a[j], m.ba[j], z.b[j]);
    }
  }
  if (norm) {
    const float r = row_rsqrt<D>(x, eps);
    const uint64_t rr = f2_pack(r, r);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      z.a[j] = f2_mul(z.a[j], rr);
      z.b[j] = f2_mul(z.b[j], rr);
    }
  }
  return z;
}

template <bool INTER>
__device__ __forceinline__ void store_bf16(bf16* row, const LaneMap& m, const Eight& z) {
  float y[8];
  in_order<INTER>(z, y);
  *reinterpret_cast<uint2*>(row + m.ea) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  *reinterpret_cast<uint2*>(row + m.eb) = make_uint2(pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
}

template <bool INTER>
__device__ __forceinline__ void store_e4m3(uint8_t* row, const LaneMap& m, const Eight& z, float inv) {
  float y[8];
  in_order<INTER>(z, y);
  *reinterpret_cast<uint32_t*>(row + m.ea) = pack_e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
  *reinterpret_cast<uint32_t*>(row + m.eb) = pack_e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
}

__device__ __forceinline__ float largest(const Eight& z) {  // NaN is passed over
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float u, v;
    f2_unpack(z.a[j], u, v);
    m = fmaxf(m, fmaxf(fabsf(u), fabsf(v)));
    f2_unpack(z.b[j], u, v);
    m = fmaxf(m, fmaxf(fabsf(u), fabsf(v)));
  }
  return m;
}

__device__ __forceinline__ void cp_async_8(uint32_t saddr, const void* g) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(saddr), "l"(g) : "memory");
}

// e4m3 block of one head: a row that the block held before goes from one scale to another (ratio of the two)
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

// where position pos of request b lives; pid -1: nowhere (reported)
struct Place {
  int pid, slot;
};
__device__ __forceinline__ Place place_of(const QkvArgs& a, int b, int64_t pos) {
  Place r{-1, 0};
  if (pos >= 0 && pos < (int64_t)a.max_pages * a.page) {  // pos < 2^31 + N: 32 bits without a sign
    const uint32_t c = (uint32_t)pos / (uint32_t)a.page;
    const int pid = __ldg(a.page_table + (int64_t)b * a.max_pages + c);
    if (pid >= 0 && pid < a.n_pages_total) r.pid = pid;
    r.slot = (int)((uint32_t)pos - c * (uint32_t)a.page);
  }
  if (r.pid < 0) report(a.status, FA_ERR_DEVICE_CHECK);
  return r;
}

// ------------------------------------------------------------------------------------------------
// Rows. An item is one token (b, n) and one of `groups` shares of its heads: shares of the query heads, then of the key
// heads, then of the value heads, 32 / (d / 8) heads a step. The warps of the grid deal the items out in turn, so that
// neighbouring warps hold neighbouring tokens, which lie side by side in the head-major tensors.
// ------------------------------------------------------------------------------------------------
struct Shares {
  int groups, q, k;     // heads of a share
};

// Walks the loads: the heads [h, hend) of one kind of one item, then the next kind's or item's. A kind that is left out
// has no heads.
struct Cursor {
  int64_t item;
  int b, n, kind, h, hend;
};

__device__ __forceinline__ bool next_kind(Cursor& c, int64_t items, int64_t step, int N, const Shares& sh, int hq, int hk, int hv,
                                          const int32_t* n_new = nullptr) {
  for (;;) {
    if (++c.kind == 3) {
      c.kind = 0;
      c.item += step;
    }
    if (c.item >= items) return false;
    const int64_t T = sh.groups == 1 ? c.item : c.item / sh.groups;
    const int g = sh.groups == 1 ? 0 : (int)(c.item - T * sh.groups);
    if (c.kind == 0) {
      c.b = (int)((uint32_t)T / (uint32_t)N);  // tokens fit 31 bits
      c.n = (int)((uint32_t)T - (uint32_t)c.b * (uint32_t)N);
      if (n_new && c.n >= __ldg(n_new + c.b)) {  // a token that is not there
        c.kind = 2;
        continue;
      }
    }
    const int per = c.kind == 0 ? sh.q : sh.k;
    c.h = g * per;
    c.hend = min(c.kind == 0 ? hq : c.kind == 1 ? hk : hv, c.h + per);
    if (c.h < c.hend) return true;
  }
}

constexpr int kRing = 8;         // rows in flight a lane (a power of two)
constexpr int kRowThreads = 128;
constexpr int kRowCtas = 5;      // of an SM, by registers; the grid is exactly those: with 8 an SM 75 us where 5 take 67

// One item at a time, with the loads ahead of it.
template <int D, int DST, bool INTER, int THREADS>
struct RowWarp {
  static constexpr int LPR = D / 8, R = 32 / LPR;
  static constexpr int kStep = 2 * THREADS * 8;    // bytes of a ring step: each lane's two groups
  const QkvArgs& a;
  const Shares& sh;
  int lane, row, hq, hk, hv;
  int64_t items, warps;
  LaneMap lm;
  Cursor ld;
  const bf16* src;
  int64_t hop;
  bool more;
  uint32_t ring, in, out;
  Turn turn;
  Place place;
  int b, n;

  __device__ __forceinline__ RowWarp(const QkvArgs& args, const Shares& shares, int64_t warp, int64_t n_warps, uint2* ring_mem)
      : a(args), sh(shares), lane(threadIdx.x % LPR), row((threadIdx.x % 32) / LPR), hq(args.q.p ? args.Hq : 0),
        hk(args.k.p ? args.Hkv : 0), hv(args.v.p ? args.Hkv : 0), items((int64_t)args.B * args.N * shares.groups),
        warps(n_warps), lm(lane_map<D, INTER>(lane, args.inv_freq ? args.rot : 0)), ld{warp, 0, 0, -1, 0, 0}, src(nullptr),
        hop(0), more(true), ring(smem_u32(ring_mem) + threadIdx.x * 8), in(0), out(0), place{-1, 0}, b(0), n(0) {
#pragma unroll 1
    for (int i = 0; i < kRing; ++i) load();
  }

  __device__ __forceinline__ void load() {
    if (more) {
      if (ld.h >= ld.hend) {
        more = next_kind(ld, items, warps, a.N, sh, hq, hk, hv, DST == kToHeads ? nullptr : a.n_new);
        if (more) {
          const Rows& S = ld.kind == 0 ? a.q : ld.kind == 1 ? a.k : a.v;
          src = static_cast<const bf16*>(S.p) + ld.b * S.sb + ld.n * S.sn + (ld.h + row) * S.sh + lm.ea;
          hop = R * S.sh;
        }
      }
      if (more) {
        if (ld.h + row < ld.hend) {
          cp_async_8(ring + in, src);
          cp_async_8(ring + in + THREADS * 8, src + (lm.eb - lm.ea));
        }
        src += hop;
        ld.h += R;
      }
    }
    in = (in + kStep) & (kRing * kStep - 1);
    cp_async_commit();
  }

  // KIND 0: query rows, 1: key rows, 2: value rows
  template <int KIND>
  __device__ __forceinline__ void heads_of(int g) {
    const int per = KIND == 0 ? sh.q : sh.k, H = KIND == 0 ? hq : KIND == 1 ? hk : hv;
    int h = g * per + row;
    const int hend = min(H, g * per + per);
    int left = (hend - g * per + R - 1) / R;
    if (left <= 0) return;
    constexpr bool kToCache = DST != kToHeads && KIND != 0;
    const float* w = KIND == 0 ? a.wq : KIND == 1 ? a.wk : nullptr;
    Map2 m;
    if (KIND != 2) m = fold(turn, load_weight<INTER>(w, lm));
    bf16* dst = nullptr;
    int64_t step = 0;
    if (!kToCache) {
      step = (int64_t)R * a.N * D;
      dst = static_cast<bf16*>(KIND == 0 ? a.q_out : KIND == 1 ? a.k_out : a.v_out) +
            (((int64_t)b * (KIND == 0 ? a.Hq : a.Hkv) + h) * a.N + n) * D + lm.ea;
    } else if (DST == kToPages && place.pid >= 0) {
      step = (int64_t)R * a.page * D;
      dst = static_cast<bf16*>(KIND == 1 ? a.k_pages : a.v_pages) +
            (((int64_t)place.pid * a.Hkv + h) * a.page + place.slot) * D + lm.ea;
    }
    const bool writes = dst != nullptr;
    for (; left > 0; --left) {
      cp_async_wait<kRing - 1>();
      const bool live = h < hend;
      uint2 va = make_uint2(0, 0), vb = va;
      if (live) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(va.x), "=r"(va.y) : "r"(ring + out) : "memory");
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(vb.x), "=r"(vb.y) : "r"(ring + out + THREADS * 8) : "memory");
      }
      out = (out + kStep) & (kRing * kStep - 1);
      load();
      if (KIND == 2 && DST != kToPagesFp8) {  // as it is
        if (live && writes) {
          *reinterpret_cast<uint2*>(dst) = va;
          *reinterpret_cast<uint2*>(dst + (lm.eb - lm.ea)) = vb;
        }
      } else {
        Eight z = unpack<INTER>(va, vb);
        if (KIND != 2) z = norm_rope<D>(z, w != nullptr, a.eps, m, lm.rot);
        if (kToCache && DST == kToPagesFp8) {
          quantise(z, KIND == 1 ? a.k_pages : a.v_pages, KIND == 1 ? a.k_scale : a.v_scale, h, live);
        } else if (live && writes) {
          float y[8];
          in_order<INTER>(z, y);
          *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
          *reinterpret_cast<uint2*>(dst + (lm.eb - lm.ea)) = make_uint2(pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
        }
      }
      dst += step;
      h += R;
    }
  }

  // One new token a request: its 32-token block holds the tokens before it under the scale they have, which one lane
  // reads and writes. The whole warp calls it.
  __device__ __forceinline__ void quantise(const Eight& z, void* pages, float* scales, int h, bool live) {
    const float need = need_scale(row_max<LPR>(largest(z)));
    const bool mine = live && place.pid >= 0;
    const int before = place.slot % kScaleTokens;
    const int64_t head = (int64_t)place.pid * a.Hkv + h;
    float* sc = scales + head * (a.page / kScaleTokens) + place.slot / kScaleTokens;
    float was = 0.f;
    if (mine && before && lane == 0) was = clamp_scale(*sc);
    was = __shfl_sync(0xFFFFFFFFu, was, 0, LPR);
    if (mine) {
      uint8_t* base = static_cast<uint8_t*>(pages) + head * a.page * D;
      const float now = fmaxf(need, was);
      if (before && now != was)
        for (int r = place.slot - before; r < place.slot; ++r) rescale_row<D>(base + r * D, lane * 8, was / now);
      store_e4m3<INTER>(base + place.slot * D, lm, z, 1.f / now);
      if (lane == 0) *sc = now;
    }
  }

  __device__ __forceinline__ void run(int64_t warp) {
    uint64_t f[4] = {0, 0, 0, 0};
    if (a.inv_freq) lane_frequencies(a.inv_freq, lm, f);
    for (int64_t item = warp; item < items; item += warps) {
      const int64_t T = sh.groups == 1 ? item : item / sh.groups;
      const int g = sh.groups == 1 ? 0 : (int)(item - T * sh.groups);
      b = (int)((uint32_t)T / (uint32_t)a.N);
      n = (int)((uint32_t)T - (uint32_t)b * (uint32_t)a.N);
      if (DST != kToHeads && n >= new_tokens(a, b)) continue;  // no loads are under way for it either
      const int64_t pos = (int64_t)n + (a.q_offset ? __ldg(a.q_offset + b) : 0);
      turn = turn_at(f, lm, pos);
      if (DST != kToHeads && hk && sh.k) place = place_of(a, b, pos);
      heads_of<0>(g);
      heads_of<1>(g);
      heads_of<2>(g);
    }
    cp_async_wait<0>();
  }
};

template <int D, int DST, bool INTER>
__global__ void __launch_bounds__(kRowThreads, kRowCtas) qkv_rows_kernel(const __grid_constant__ QkvArgs a, const __grid_constant__ Shares sh) {
  __shared__ __align__(16) uint2 ring[kRing * 2 * kRowThreads];
  const int64_t warp = (int64_t)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
  RowWarp<D, DST, INTER, kRowThreads> w(a, sh, warp, (int64_t)gridDim.x * (kRowThreads / 32), ring);
  w.run(warp);
}

// ------------------------------------------------------------------------------------------------
// Append to e4m3 pages, several tokens a request. A CTA takes one 32-token block of one request and a share of its
// KV heads: for each head its threads hold the block's new K and V rows, agree on the two largest magnitudes (one
// barrier), and write scales and values; rows that the block held before are rescaled where the scale grew. Other CTAs
// take the query rows.
// ------------------------------------------------------------------------------------------------
constexpr int kBlockThreads = 256;

// A head's rows of one block: the lane's values to e4m3 under the block's scale.
template <int D, bool INTER, int RPT, int SLOTS>
__device__ __forceinline__ void write_block(uint8_t* base, float* sc, float big, float was, int before, int slot,
                                            const LaneMap& lm, const Eight (&z)[RPT], const bool (&in)[RPT], int lane) {
  const float now = fmaxf(need_scale(big), was), inv = 1.f / now;
  if (now != was)  // was = 0 where the block has no tokens yet: nothing to rescale
    for (int i = slot; i < before; i += SLOTS) rescale_row<D>(base + i * D, lane * 8, was / now);
#pragma unroll
  for (int u = 0; u < RPT; ++u)
    if (in[u]) store_e4m3<INTER>(base + (slot + u * SLOTS) * D, lm, z[u], inv);
  if (threadIdx.x == 0) *sc = now;
}

template <int D, bool INTER>
__device__ __forceinline__ void append_block(const QkvArgs& a, int b, int j, int hk0, int hk1, uint2* ring_mem,
                                             uint32_t (*s_max)[2][kBlockThreads / 32]) {
  constexpr int LPR = D / 8, SLOTS = kBlockThreads / LPR, RPT = kScaleTokens / SLOTS, kWarps = kBlockThreads / 32;
  constexpr int kAhead = kRing / (2 * RPT), kStep = 2 * kBlockThreads * 8;
  const int tid = threadIdx.x, lane = tid % LPR, slot = tid / LPR;
  const int64_t first = a.q_offset ? __ldg(a.q_offset + b) : 0;
  const int cnt = new_tokens(a, b);
  const int64_t p0 = ((first >> 5) + j) * kScaleTokens;
  const int64_t lo = max(p0, first), hi = min(p0 + kScaleTokens, first + cnt);
  if (lo >= hi) return;
  const LaneMap lm = lane_map<D, INTER>(lane, a.inv_freq ? a.rot : 0);
  bool in[RPT];
  const bf16 *kp[RPT], *vp[RPT];
#pragma unroll
  for (int u = 0; u < RPT; ++u) {
    const int64_t pos = p0 + slot + u * SLOTS;
    in[u] = pos >= lo && pos < hi;
    const int64_t n = in[u] ? pos - first : 0;
    kp[u] = static_cast<const bf16*>(a.k.p) + b * a.k.sb + hk0 * a.k.sh + n * a.k.sn + lm.ea;
    vp[u] = static_cast<const bf16*>(a.v.p) + b * a.v.sb + hk0 * a.v.sh + n * a.v.sn + lm.ea;
  }
  const uint32_t ring = smem_u32(ring_mem) + tid * 8;
  const int far = lm.eb - lm.ea, heads = hk1 - hk0;
  uint32_t at_in = 0, at_out = 0;
  int loaded = 0;
  auto load = [&]() {  // K and V rows of the next head
    if (loaded < heads) {
#pragma unroll
      for (int u = 0; u < RPT; ++u) {
        if (in[u]) {
          const uint32_t to = ring + at_in + u * kStep;
          cp_async_8(to, kp[u]);
          cp_async_8(to + kBlockThreads * 8, kp[u] + far);
          cp_async_8(to + RPT * kStep, vp[u]);
          cp_async_8(to + RPT * kStep + kBlockThreads * 8, vp[u] + far);
        }
        kp[u] += a.k.sh;
        vp[u] += a.v.sh;
      }
      ++loaded;
    }
    at_in = (at_in + 2 * RPT * kStep) & (kRing * kStep - 1);
    cp_async_commit();
  };
#pragma unroll
  for (int x = 0; x < kAhead; ++x) load();
  const Place place = place_of(a, b, p0);
  Map2 m[RPT];
  {
    uint64_t f[4] = {0, 0, 0, 0};
    if (a.inv_freq) lane_frequencies(a.inv_freq, lm, f);
    const Eight w = load_weight<INTER>(a.wk, lm);
#pragma unroll
    for (int u = 0; u < RPT; ++u) m[u] = fold(turn_at(f, lm, p0 + slot + u * SLOTS), w);
  }
  const int before = (int)(lo - p0), spp = a.page / kScaleTokens;
  const int64_t head0 = (int64_t)place.pid * a.Hkv + hk0;
  float* ks = a.k_scale + head0 * spp + place.slot / kScaleTokens;
  float* vs = a.v_scale + head0 * spp + place.slot / kScaleTokens;
  const int64_t at0 = (head0 * a.page + place.slot) * D;
  uint8_t *kd = static_cast<uint8_t*>(a.k_pages) + at0, *vd = static_cast<uint8_t*>(a.v_pages) + at0;
  for (int x = 0; x < (place.pid < 0 ? 0 : heads); ++x) {
    cp_async_wait<kAhead - 1>();
    float k_was = 0.f, v_was = 0.f;
    if (before) {
      k_was = clamp_scale(*ks);
      v_was = clamp_scale(*vs);
    }
    Eight zk[RPT], zv[RPT];
    float k_big = 0.f, v_big = 0.f;
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
      uint2 ka = make_uint2(0, 0), kb = ka, va = ka, vb = ka;
      if (in[u]) {
        const uint32_t from = ring + at_out + u * kStep;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(ka.x), "=r"(ka.y) : "r"(from) : "memory");
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(kb.x), "=r"(kb.y) : "r"(from + kBlockThreads * 8) : "memory");
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(va.x), "=r"(va.y) : "r"(from + RPT * kStep) : "memory");
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                     : "=r"(vb.x), "=r"(vb.y)
                     : "r"(from + RPT * kStep + kBlockThreads * 8)
                     : "memory");
      }
      zk[u] = norm_rope<D>(unpack<INTER>(ka, kb), a.wk != nullptr, a.eps, m[u], lm.rot);
      zv[u] = unpack<INTER>(va, vb);
      if (in[u]) {  // rows of zeros may be NaN without an eps
        k_big = fmaxf(k_big, largest(zk[u]));
        v_big = fmaxf(v_big, largest(zv[u]));
      }
    }
    at_out = (at_out + 2 * RPT * kStep) & (kRing * kStep - 1);
    load();
    // magnitudes order as their bits do
    const uint32_t kw = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(k_big));
    const uint32_t vw = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v_big));
    if ((tid & 31) == 0) {
      s_max[x & 1][0][tid >> 5] = kw;
      s_max[x & 1][1][tid >> 5] = vw;
    }
    __syncthreads();  // the old scales are read, too
    uint32_t km = 0, vm = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      km = max(km, s_max[x & 1][0][w]);
      vm = max(vm, s_max[x & 1][1][w]);
    }
    write_block<D, INTER, RPT, SLOTS>(kd, ks, __uint_as_float(km), k_was, before, slot, lm, zk, in, lane);
    write_block<D, INTER, RPT, SLOTS>(vd, vs, __uint_as_float(vm), v_was, before, slot, lm, zv, in, lane);
    ks += spp;
    vs += spp;
    kd += (int64_t)a.page * D;
    vd += (int64_t)a.page * D;
  }
  cp_async_wait<0>();
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kBlockThreads, 3)
    append_fp8_kernel(const __grid_constant__ QkvArgs a, int blocks, int heads_per_cta, int groups) {
  __shared__ __align__(16) uint2 ring[kRing * 2 * kBlockThreads];
  __shared__ __align__(16) uint32_t s_max[2][2][kBlockThreads / 32];
  // the two kinds of CTAs take turns: the blocks are bound by their instructions, the query rows by HBM
  const int kv_ctas = a.B * blocks * groups, q_ctas = (int)gridDim.x - kv_ctas, both = min(kv_ctas, q_ctas);
  const int x = (int)blockIdx.x;
  const bool turn = x < 2 * both;
  if (turn ? (x & 1) == 0 : kv_ctas > q_ctas) {
    const int i = turn ? x >> 1 : x - both, gi = i % groups, bj = i / groups;
    const int hk0 = gi * heads_per_cta;
    append_block<D, INTER>(a, bj / blocks, bj % blocks, hk0, min(a.Hkv, hk0 + heads_per_cta), ring, s_max);
  } else {
    constexpr int kWarps = kBlockThreads / 32;
    const int64_t warp = (int64_t)(turn ? x >> 1 : x - both) * kWarps + threadIdx.x / 32;
    const Shares all{1, a.Hq, 0};  // the query rows alone
    RowWarp<D, kToPages, INTER, kBlockThreads> w(a, all, warp, (int64_t)q_ctas * kWarps, ring);
    w.run(warp);
  }
}

// ------------------------------------------------------------------------------------------------
// Backward of the rows: with g = R^T dz (the transposed rotation) and xhat = x r,
//   dw += g xhat,   dx = r (w g - xhat mean(w g xhat))     (no weight: dx = g)
// r is recomputed from x. A warp walks items as in the forward and keeps its sums of dw in registers (a lane always
// holds the same 8 places); they are joined in shared memory, written one row a CTA, and added up by a second kernel in
// a fixed order: no atomics, the same result each time.
// ------------------------------------------------------------------------------------------------
constexpr int kBwdThreads = 256;
constexpr int kBwdCtas = 2;                                 // of an SM, the grid is exactly those
constexpr int kBwdRing = 4;
constexpr int kBwdStep = kBwdThreads * 48;                  // a row's 48 bytes a lane: 32 of dz, 16 of x
constexpr int kBwdRingBytes = kBwdRing * kBwdStep;

template <bool F32, bool INTER>
__device__ __forceinline__ void store_grad(void* p, int64_t at, const LaneMap& m, const Eight& g) {
  if (F32) {
    float y[8];
    in_order<INTER>(g, y);
    float* o = static_cast<float*>(p) + at;
    *reinterpret_cast<float4*>(o + m.ea) = make_float4(y[0], y[1], y[2], y[3]);
    *reinterpret_cast<float4*>(o + m.eb) = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    store_bf16<INTER>(static_cast<bf16*>(p) + at, m, g);
  }
}

template <int D, bool F32, bool INTER>
struct BwdWarp {
  static constexpr int LPR = D / 8, R = 32 / LPR;
  const QkvBwdArgs& a;
  const Shares& sh;
  int lane, row, hq, hk, hv;
  int64_t items, warps;
  LaneMap lm;
  Cursor ld;
  const float* dy;
  const bf16* src;
  int64_t dy_hop, hop;
  bool more;
  uint32_t ring, in, out;
  Turn turn;
  Eight dwq, dwk;
  int b, n;

  __device__ __forceinline__ BwdWarp(const QkvBwdArgs& args, const Shares& shares, int64_t warp, int64_t n_warps, void* ring_mem)
      : a(args), sh(shares), lane(threadIdx.x % LPR), row((threadIdx.x % 32) / LPR), hq(args.dq ? args.Hq : 0),
        hk(args.dk ? args.Hkv : 0), hv(args.dv ? args.Hkv : 0), items((int64_t)args.B * args.N * shares.groups),
        warps(n_warps), lm(lane_map<D, INTER>(lane, args.inv_freq ? args.rot : 0)), ld{warp, 0, 0, -1, 0, 0}, dy(nullptr),
        src(nullptr), dy_hop((int64_t)R * args.N * D), hop(0), more(true), ring(smem_u32(ring_mem) + threadIdx.x * 16), in(0),
        out(0), b(0), n(0) {
#pragma unroll
    for (int j = 0; j < 2; ++j) dwq.a[j] = dwq.b[j] = dwk.a[j] = dwk.b[j] = 0ull;
#pragma unroll 1
    for (int i = 0; i < kBwdRing; ++i) load();
  }

  __device__ __forceinline__ void load() {
    if (more) {
      if (ld.h >= ld.hend) {
        more = next_kind(ld, items, warps, a.N, sh, hq, hk, hv);
        if (more) {
          const int H = ld.kind == 0 ? a.Hq : a.Hkv;
          dy = (ld.kind == 0 ? a.dq : ld.kind == 1 ? a.dk : a.dv) + (((int64_t)ld.b * H + ld.h + row) * a.N + ld.n) * D + lm.ea;
          const Rows& S = ld.kind == 0 ? a.q : a.k;
          const bool with_x = ld.kind == 0 ? a.wq != nullptr : ld.kind == 1 && a.wk != nullptr;
          src = with_x ? static_cast<const bf16*>(S.p) + ld.b * S.sb + ld.n * S.sn + (ld.h + row) * S.sh + lm.ea : nullptr;
          hop = with_x ? R * S.sh : 0;
        }
      }
      if (more) {
        if (ld.h + row < ld.hend) {
          cp_async_16(ring + in, dy, true);
          cp_async_16(ring + in + kBwdThreads * 16, dy + (lm.eb - lm.ea), true);
          if (src) {
            cp_async_8(ring + in + kBwdThreads * 32, src);
            cp_async_8(ring + in + kBwdThreads * 32 + 8, src + (lm.eb - lm.ea));
          }
        }
        dy += dy_hop;
        src += hop;
        ld.h += R;
      }
    }
    in = in + kBwdStep == kBwdRingBytes ? 0 : in + kBwdStep;
    cp_async_commit();
  }

  // KIND 0: query rows, 1: key rows, 2: value rows; NORM: with a weight
  template <int KIND, bool NORM>
  __device__ __forceinline__ void heads_of(int g) {
    const int per = KIND == 0 ? sh.q : sh.k, H = KIND == 0 ? hq : KIND == 1 ? hk : hv;
    int h = g * per + row;
    const int hend = min(H, g * per + per);
    int left = (hend - g * per + R - 1) / R;
    if (left <= 0) return;
    Eight w;
    if (NORM) w = load_weight<INTER>(KIND == 0 ? a.wq : a.wk, lm);
    const Rows& S = KIND == 0 ? a.dq_in : KIND == 1 ? a.dk_in : a.dv_in;
    int64_t to = b * S.sb + n * S.sn + h * S.sh;
    const int64_t step = R * S.sh;
    Eight& dw = KIND == 0 ? dwq : dwk;
    for (; left > 0; --left) {
      cp_async_wait<kBwdRing - 1>();
      const bool live = h < hend;
      float4 ga = make_float4(0.f, 0.f, 0.f, 0.f), gb = ga;
      uint4 xr = make_uint4(0, 0, 0, 0);
      if (live) {
        const uint32_t at = ring + out;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(ga.x), "=f"(ga.y), "=f"(ga.z), "=f"(ga.w) : "r"(at) : "memory");
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(gb.x), "=f"(gb.y), "=f"(gb.z), "=f"(gb.w)
                     : "r"(at + kBwdThreads * 16)
                     : "memory");
        if (NORM)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(xr.x), "=r"(xr.y), "=r"(xr.z), "=r"(xr.w)
                       : "r"(at + kBwdThreads * 32)
                       : "memory");
      }
      out = out + kBwdStep == kBwdRingBytes ? 0 : out + kBwdStep;
      load();
      Eight g8 = unpack_f32<INTER>(ga, gb);
      if (KIND != 2) {
        if (lm.rot) {
          const Eight d = g8;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            g8.a[j] = f2_fma(d.a[j], turn.c[j], f2_mul(d.b[j], turn.s[j]));
            g8.b[j] = f2_fma(d.b[j], turn.c[j], f2_neg(f2_mul(d.a[j], turn.s[j])));
          }
        }
        if (NORM) {
          const Eight x = unpack<INTER>(make_uint2(xr.x, xr.y), make_uint2(xr.z, xr.w));
          const float r = row_rsqrt<D>(x, a.eps);
          const uint64_t rr = f2_pack(r, r);
          Eight gx, wg;
          uint64_t acc = 0ull;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            gx.a[j] = f2_mul(g8.a[j], x.a[j]);
            gx.b[j] = f2_mul(g8.b[j], x.b[j]);
            acc = f2_fma(w.a[j], gx.a[j], acc);
            acc = f2_fma(w.b[j], gx.b[j], acc);
            wg.a[j] = f2_mul(w.a[j], g8.a[j]);
            wg.b[j] = f2_mul(w.b[j], g8.b[j]);
          }
          if (live) {  // a row that is not there may have r = inf
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              dw.a[j] = f2_fma(gx.a[j], rr, dw.a[j]);
              dw.b[j] = f2_fma(gx.b[j], rr, dw.b[j]);
            }
          }
          float u, v;
          f2_unpack(acc, u, v);
          const float dot = row_sum<LPR>(u + v) * r;              // sum of w g xhat
          const float k = -dot * (1.f / D) * r * r;
          const uint64_t kk = f2_pack(k, k);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            g8.a[j] = f2_fma(wg.a[j], rr, f2_mul(x.a[j], kk));
            g8.b[j] = f2_fma(wg.b[j], rr, f2_mul(x.b[j], kk));
          }
        }
      }
      if (live) store_grad<F32, INTER>(S.p, to, lm, g8);
      to += step;
      h += R;
    }
  }

  __device__ __forceinline__ void run(int64_t warp) {
    uint64_t f[4] = {0, 0, 0, 0};
    if (a.inv_freq) lane_frequencies(a.inv_freq, lm, f);
    for (int64_t item = warp; item < items; item += warps) {
      const int64_t T = sh.groups == 1 ? item : item / sh.groups;
      const int g = sh.groups == 1 ? 0 : (int)(item - T * sh.groups);
      b = (int)((uint32_t)T / (uint32_t)a.N);
      n = (int)((uint32_t)T - (uint32_t)b * (uint32_t)a.N);
      turn = turn_at(f, lm, (int64_t)n + (a.q_offset ? __ldg(a.q_offset + b) : 0));
      if (a.wq) heads_of<0, true>(g); else heads_of<0, false>(g);
      if (a.wk) heads_of<1, true>(g); else heads_of<1, false>(g);
      heads_of<2, false>(g);
    }
    cp_async_wait<0>();
  }
};

template <int D, bool F32, bool INTER>
__global__ void __launch_bounds__(kBwdThreads, kBwdCtas) qkv_bwd_kernel(const __grid_constant__ QkvBwdArgs a,
                                                                        const __grid_constant__ Shares sh) {
  constexpr int LPR = D / 8, SLOTS = kBwdThreads / LPR;
  extern __shared__ uint4 ring[];
  const int tid = threadIdx.x;
  const int64_t warp = (int64_t)blockIdx.x * (kBwdThreads / 32) + tid / 32;
  BwdWarp<D, F32, INTER> w(a, sh, warp, (int64_t)gridDim.x * (kBwdThreads / 32), ring);
  w.run(warp);
  if (!a.wq && !a.wk) return;
  float (*s_dw)[D] = reinterpret_cast<float (*)[D]>(ring);  // the rings are read: [SLOTS][D]
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
    float y[8];
    in_order<INTER>(which ? w.dwk : w.dwq, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s_dw[tid / LPR][w.lm.ea + e] = y[e];
      s_dw[tid / LPR][w.lm.eb + e] = y[4 + e];
    }
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

// Shares of the heads: a token's heads stay together where that gives every warp that fits the GPU an item, else they
// are dealt out so that a decode step's few tokens still reach every SM.
Shares shares(int64_t tokens, int64_t warps, int Hq, int Hkv, int rows_a_step) {
  int groups = 1;
  const int most = (std::max(Hq, Hkv) + rows_a_step - 1) / rows_a_step;
  while (groups < most && tokens * groups < warps) groups *= 2;
  return Shares{groups, (Hq + groups - 1) / groups, (Hkv + groups - 1) / groups};
}

template <int D, int DST>
cudaError_t run_rows(const QkvArgs& a, cudaStream_t st) {
  constexpr int kWarps = kRowThreads / 32;
  const int64_t tokens = (int64_t)a.B * a.N;
  const Shares sh = shares(tokens, kSms * kRowCtas * kWarps, a.Hq, a.Hkv, 32 / (D / 8));
  const int64_t ctas = std::min<int64_t>((tokens * sh.groups + kWarps - 1) / kWarps, kSms * kRowCtas);
  auto kern = a.interleaved ? qkv_rows_kernel<D, DST, true> : qkv_rows_kernel<D, DST, false>;
  kern<<<(unsigned)ctas, kRowThreads, 0, st>>>(a, sh);
  return cudaGetLastError();
}

template <int D>
cudaError_t run_append(const QkvArgs& a, cudaStream_t st) {
  if (!a.k_scale) return run_rows<D, kToPages>(a, st);
  if (a.N == 1) return run_rows<D, kToPagesFp8>(a, st);
  const int blocks = (a.N + 2 * kScaleTokens - 2) / kScaleTokens;
  int groups = 1;
  while (groups < a.Hkv && (int64_t)a.B * blocks * groups < 2 * kSms) ++groups;
  const int hpc = (a.Hkv + groups - 1) / groups;
  groups = (a.Hkv + hpc - 1) / hpc;
  const int64_t q_items = a.q.p ? (int64_t)a.B * a.N : 0, per = kBlockThreads / 32;
  const int64_t ctas = (int64_t)a.B * blocks * groups + std::min<int64_t>((q_items + per - 1) / per, kSms * 16);
  if (ctas > 0x3FFFFFFF) return cudaErrorInvalidConfiguration;
  auto kern = a.interleaved ? append_fp8_kernel<D, true> : append_fp8_kernel<D, false>;
  kern<<<(unsigned)ctas, kBlockThreads, 0, st>>>(a, blocks, hpc, groups);
  return cudaGetLastError();
}

template <int D>
cudaError_t run_bwd(const QkvBwdArgs& a, cudaStream_t st) {
  const int64_t tokens = (int64_t)a.B * a.N;
  const int ctas = qk_bwd_ctas(tokens);
  const Shares sh = shares(tokens, (int64_t)ctas * (kBwdThreads / 32), a.Hq, a.Hkv, 32 / (D / 8));
  auto kern = a.grad_f32 ? (a.interleaved ? qkv_bwd_kernel<D, true, true> : qkv_bwd_kernel<D, true, false>)
                         : (a.interleaved ? qkv_bwd_kernel<D, false, true> : qkv_bwd_kernel<D, false, false>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBwdRingBytes);
  if (e != cudaSuccess) return e;
  kern<<<ctas, kBwdThreads, kBwdRingBytes, st>>>(a, sh);
  e = cudaGetLastError();
  if (e != cudaSuccess || (!a.wq && !a.wk)) return e;
  dw_reduce_kernel<<<2 * D / 32, dim3(32, 32), 0, st>>>(a.partial, ctas, D, a.dwq, a.dwk);
  return cudaGetLastError();
}

}  // namespace

// CTAs of the backward's persistent grid, two an SM; fewer where there are not four tokens' worth of work for each
int qk_bwd_ctas(int64_t tokens) {
  const int64_t n = (tokens + 3) / 4;
  return (int)(n < kBwdCtas * kSms ? n : kBwdCtas * kSms);
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
