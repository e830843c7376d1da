// Paged split-KV decode over an 8-bit cache: e4m3 pages with an fp32 scale for each 32 tokens and KV head.
//
//   s_j = scale * ks[j/32] * <q, k8_j>,   O = sum_j p_j vs[j/32] v8_j / sum_j p_j
//
// Bound: HBM, one byte a cached value. The shape is that of the bf16 decode: a CTA takes a span of pages of one
// (request, KV head) for all its query heads, each of its 4 warps streams 32-token sub-tiles through its own ring of
// TMA copies, and a second kernel joins the spans. At half the bytes the on-chip work weighs twice as much, so:
//  - the bytes become fp16 in registers, straight from ldmatrix: e4m3 is exact in fp16, and so are bf16 queries once
//    each row is divided by a power of two. The order of k inside an MMA is free as long as both operands agree, so a
//    32-bit register of four neighbouring bytes feeds one MMA step as it is; V comes through a transposing ldmatrix of
//    16-bit pairs, one byte permute splits even and odd columns, and a lane ends up with four neighbouring columns of O.
//  - P is fp16 (2^-12 relative, against 2^-9 for bf16), unscaled: O is held in units of the current V scale and changes
//    units only where the scale does. P's own unit lies 2^7 or more under the largest P of the warp's keys (1024 at most) and
//    moves only past a factor of 2^8, so that a P below 2^-21 of that largest is off by at most 2^-32 of it.
//  - what a sub-tile needs besides its bytes (page, scales, mask bits) is looked up by one lane for each sub-tile of the
//    warp at the start, all at once, and handed round by shuffles.
//  - groups of at most 8 query heads (HALF) leave rows 8 .. 15 of the MMA tile out of the softmax.
// Measured on one GB300: 64 requests of 1k - 32k tokens, 32 / 8 heads, d = 128: 338 us, 6.55 TB/s of 6.77 measured (with all
// 16 rows 377); two requests of 131,072 tokens 92 us, 5.5 TB/s; 64 requests of 16,000 tokens, 8 / 8 heads, d = 64: 174 us.
#include <type_traits>

#include "fa_launch.h"
#include "fp8.cuh"

namespace fa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4;
// P in fp16, in units of 2^m: m is set 2^7 under a sub-tile's largest and kept until one lies past 2^15 of it
constexpr float kUnitBelow = 7.f, kMost = 15.f;
constexpr int kSub = kScaleTokens;   // tokens per sub-tile: one K scale and one V scale

template <int D>
struct Cfg {
  static constexpr int kStages = 3;
  static constexpr int kCtas = fp8_decode_ctas(D);       // resident an SM
  static constexpr int kTile = kSub * D;                 // bytes of a K or V sub-tile
  static constexpr int kStage = 2 * kTile;
  static constexpr int kWarpBytes = kStages * kStage;
  static constexpr int kSmem = kWarps * kWarpBytes + 1024;
};

// byte offset of 16-byte chunk c of row `row` in a TMA-written [32][D] byte tile (128-byte swizzle for D = 128,
// 64-byte for D = 64)
template <int D>
__device__ __forceinline__ uint32_t tile_at(int row, int c) {
  return D == 128 ? (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)) : (uint32_t)(row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
}

template <int D, bool HALF>
__global__ void __launch_bounds__(kWarps * 32, Cfg<D>::kCtas)
    decode_fp8_kernel(const __grid_constant__ DecFp8Args A, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV) {
  using C = Cfg<D>;
  constexpr int kStages = C::kStages;
  const DecArgs& a = A.d;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t bars[kWarps][kStages];
  __shared__ int32_t s_abort;
  __shared__ float sM[kWarps][16], sL[kWarps][16];

  const int s = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, t4 = lane & 3;
  const int g = a.Hq / a.Hkv, PAGE = a.page;
  const DevMask& M = a.mask;
  const int bm = M.Bm > 1 ? b : 0;
  const size_t mrow = (size_t)bm * M.Hm * M.nq;  // Hm == 1, nq == 1
  const int n_full = __ldg(M.full_kv_num + mrow), n_vis = n_full + __ldg(M.kv_num + mrow);
  const int e0 = s * a.pages_per_split;
  const size_t hq0 = (size_t)b * a.Hq + (size_t)hk * g;
  if (e0 >= n_vis) {  // nothing here: the join never reads it, and a request without any key is written by span 0
    if (s == 0) {
      for (int x = tid; x < g * D; x += kWarps * 32) {
        if (a.out_f32) reinterpret_cast<float*>(a.out)[hq0 * D + x] = 0.f;
        else reinterpret_cast<__nv_bfloat16*>(a.out)[hq0 * D + x] = __float2bfloat16_rn(0.f);
      }
      if (tid < g) a.lse[hq0 + tid] = -INFINITY;
    }
    return;
  }
  const int e1 = min(n_vis, e0 + a.pages_per_split);
  const int spp = PAGE / kSub;
  const int n_sub = (e1 - e0) * spp;

  if (tid == 0) {
    s_abort = 0;
    for (int w = 0; w < kWarps; ++w)
      for (int st = 0; st < kStages; ++st) mbar_init(&bars[w][st], 1);
    fence_mbar_init();
    if (a.counters) {
      const int nf = max(0, min(e1, n_full) - e0), np = (e1 - e0) - nf;
      unsigned long long* ct = reinterpret_cast<unsigned long long*>(a.counters);
      atomicAdd(ct + 0, 1ull);
      atomicAdd(ct + 1, (unsigned long long)nf);
      atomicAdd(ct + 2, (unsigned long long)np);
      atomicAdd(ct + 3, (unsigned long long)(2 * (e1 - e0)));
    }
  }
  if (tid == 32) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  __syncthreads();
  WaitCtl wc{a.timeout_ns, a.status, &s_abort};

  // sub-tiles of this warp: u = warp, warp + 4, ...; at most 32 of them (a span is at most 4096 tokens). Lane i looks
  // up number i: first position, row of its bytes in the pages (-1: nothing to read), scales, and visible tokens.
  const int my_count = warp < n_sub ? (n_sub - warp + kWarps - 1) / kWarps : 0;
  const int64_t ig = a.rule.q_offset ? (int64_t)__ldg(a.rule.q_offset + (M.Bm > 1 ? b : 0)) : 0;
  const int doc_i = a.rule.any_doc ? doc_at(a.rule, bm, ig) : -1;
  int l_j0 = 0, l_row = -1;
  uint32_t l_bits = 0;
  float l_ks = 1.f, l_vs = 1.f;
  if (lane < my_count) {
    const int u = warp + lane * kWarps, e = e0 + u / spp, t0 = (u % spp) * kSub;
    const int c = e < n_full ? __ldg(M.full_kv_idx + mrow * M.nk + e) : __ldg(M.kv_idx + mrow * M.nk + e - n_full);
    const int pid = __ldg(a.page_table + (size_t)b * a.max_pages + c);
    l_j0 = c * PAGE + t0;
    if (pid < 0 || pid >= a.n_pages_total) {
      report(a.status, FA_ERR_DEVICE_CHECK);
    } else {
      const int64_t at = ((int64_t)pid * a.Hkv + hk) * spp + t0 / kSub;
      l_ks = clamp_scale(__ldg(A.k_scale + at));
      l_vs = clamp_scale(__ldg(A.v_scale + at));
      l_bits = 0xFFFFFFFFu;
      if (e >= n_full) {
        const int w = (int)min((int64_t)kSub, (int64_t)M.kv_len - l_j0);
        l_bits = rule_row_bits(a.rule, ig, l_j0, w, doc_i, [&](int dd) {
          return doc_bits<1>(w, dd, [&](int cc) { return doc_at(a.rule, bm, (int64_t)l_j0 + cc); });
        }).w[0];
      }
      if (l_bits) l_row = (pid * a.Hkv + hk) * PAGE + t0;
    }
  }
  __syncwarp();

  uint8_t* my = smem + warp * C::kWarpBytes;
  auto issue = [&](int k) {  // the whole warp; lane 0 copies
    const int row = __shfl_sync(0xFFFFFFFFu, l_row, k);
    if (lane == 0) {
      uint64_t* bar = &bars[warp][k % kStages];
      if (row < 0) {
        mbar_arrive(bar);
      } else {
        uint8_t* st = my + (k % kStages) * C::kStage;
        mbar_arrive_expect_tx(bar, C::kStage);
        tma_load_2d(st, &tmK, 0, row, bar);
        tma_load_2d(st + C::kTile, &tmV, 0, row, bar);
      }
    }
  };
  for (int k = 0; k < min(kStages, my_count); ++k) issue(k);

  // Q fragments in fp16, each row divided by the power of two under its largest magnitude. Step c of the product
  // covers columns 16 c .. 16 c + 15; lane t4 holds columns 16 c + 4 t4 .. + 3 as k slots {2 t4, 2 t4 + 1} and {+ 8, + 9}.
  const int ra = lane >> 2, rb = ra + 8;
  const __nv_bfloat16* Qb = reinterpret_cast<const __nv_bfloat16*>(a.q) + hq0 * D;
  uint32_t qf[D / 16][4];
  float sr_a = 0.f, sr_b = 0.f;  // scale * log2(e) * the row's power of two
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (HALF && half) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c) qf[c][1] = qf[c][3] = 0u;
      break;
    }
    const int row = half ? rb : ra;
    uint2 v[D / 16];
    float m = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      v[c] = row < g ? __ldg(reinterpret_cast<const uint2*>(Qb + (size_t)row * D + c * 16 + t4 * 4)) : make_uint2(0, 0);
      m = fmaxf(m, fmaxf(fabsf(__uint_as_float(v[c].x << 16)), fabsf(__uint_as_float(v[c].x & 0xFFFF0000u))));
      m = fmaxf(m, fmaxf(fabsf(__uint_as_float(v[c].y << 16)), fabsf(__uint_as_float(v[c].y & 0xFFFF0000u))));
    }
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const uint32_t ex = (__float_as_uint(m) >> 23) & 255u;
    const int e = (ex == 0u || ex == 255u) ? 0 : min(max((int)ex - 127, -126), 126);
    const float up = __uint_as_float((uint32_t)(127 + e) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
    if (half) sr_b = a.scale * kLog2e * up; else sr_a = a.scale * kLog2e * up;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      qf[c][half] = pack_f16x2(__uint_as_float(v[c].x << 16) * down, __uint_as_float(v[c].x & 0xFFFF0000u) * down);
      qf[c][2 + half] = pack_f16x2(__uint_as_float(v[c].y << 16) * down, __uint_as_float(v[c].y & 0xFFFF0000u) * down);
    }
  }
  const bool has_score = a.score.alibi || a.score.rel || a.score.softcap > 0.f;
  const float slope_a = (a.score.alibi && ra < g) ? __ldg(a.score.alibi + hk * g + ra) : 0.f;
  const float slope_b = (a.score.alibi && rb < g) ? __ldg(a.score.alibi + hk * g + rb) : 0.f;

  float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f, vref = 1.f;
  float o[D / 16][2][4];  // [16 columns][even, odd][row a: columns 4 t4, 4 t4 + 2 (+ 1 odd); row b]
#pragma unroll
  for (int c = 0; c < D / 16; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) o[c][h][0] = o[c][h][1] = o[c][h][2] = o[c][h][3] = 0.f;

  bool ok = true;
  int k_fail = my_count;
  for (int k = 0; k < my_count; ++k) {
    const int stg = k % kStages;
    ok = mbar_wait(&bars[warp][stg], (uint32_t)((k / kStages) & 1), wc);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (!ok) {
      k_fail = k;
      break;
    }
    const uint32_t bits = __shfl_sync(0xFFFFFFFFu, l_bits, k);
    const float ks = __shfl_sync(0xFFFFFFFFu, l_ks, k), vs = __shfl_sync(0xFFFFFFFFu, l_vs, k);
    const int j0 = __shfl_sync(0xFFFFFFFFu, l_j0, k);
    if (bits) {
      const uint32_t kb = smem_u32(my + stg * C::kStage), vb = kb + C::kTile;
      float sc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        uint32_t r[4];  // token groups 8 i .. 8 i + 7
        ldsm_x4(kb + tile_at<D>(lane, c), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t b0, b1;
          e4m3x4_to_f16(r[i], b0, b1);
          mma_f16_16816(sc[i], qf[c], b0, b1);
        }
      }
      float mx_a = -INFINITY, mx_b = -INFINITY;
      const float sl_a = sr_a * ks, sl_b = sr_b * ks;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int e = 0; e < (HALF ? 2 : 4); ++e) {
          const int col = i * 8 + t4 * 2 + (e & 1);
          const bool up = e >= 2;
          float x = sc[i][e] * (up ? sl_b : sl_a);
          if (has_score) {
            x *= kLn2;
            const int64_t dist = ig - ((int64_t)j0 + col);
            if (a.score.alibi) x -= (up ? slope_b : slope_a) * (float)dist;
            if (a.score.rel && (up ? rb : ra) < g) {
              const int64_t hi = 2 * (int64_t)a.score.kv_len - 2;
              int64_t ix = dist + a.score.kv_len - 1;
              ix = ix < 0 ? 0 : (ix > hi ? hi : ix);
              x += __ldg(a.score.rel + (size_t)(hk * g + (up ? rb : ra)) * (size_t)(hi + 1) + ix);
            }
            if (a.score.softcap > 0.f) x = softcap_exact(x, a.score.softcap, a.score.inv_softcap);
            x *= kLog2e;
          }
          if (!((bits >> col) & 1u)) x = -INFINITY;
          sc[i][e] = x;
          if (up) mx_b = fmaxf(mx_b, x); else mx_a = fmaxf(mx_a, x);
        }
      }
      mx_a = fmaxf(mx_a, __shfl_xor_sync(0xFFFFFFFFu, mx_a, 1));
      mx_a = fmaxf(mx_a, __shfl_xor_sync(0xFFFFFFFFu, mx_a, 2));
      if (!HALF) {
        mx_b = fmaxf(mx_b, __shfl_xor_sync(0xFFFFFFFFu, mx_b, 1));
        mx_b = fmaxf(mx_b, __shfl_xor_sync(0xFFFFFFFFu, mx_b, 2));
      }
      const float mn_a = mx_a > m_a + kMost ? mx_a - kUnitBelow : m_a, mn_b = mx_b > m_b + kMost ? mx_b - kUnitBelow : m_b;
      const float ref_a = mn_a == -INFINITY ? 0.f : mn_a, ref_b = mn_b == -INFINITY ? 0.f : mn_b;
      if (__any_sync(0xFFFFFFFFu, mn_a != m_a || mn_b != m_b || vs != vref)) {
        const float al_a = ex2_approx(m_a - ref_a), al_b = HALF ? 0.f : ex2_approx(m_b - ref_b), w = vref / vs;
        l_a *= al_a;
        if (!HALF) l_b *= al_b;
        const float f_a = al_a * w, f_b = al_b * w;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            o[c][h][0] *= f_a;
            o[c][h][1] *= f_a;
            if (!HALF) {
              o[c][h][2] *= f_b;
              o[c][h][3] *= f_b;
            }
          }
        m_a = mn_a;
        m_b = mn_b;
        vref = vs;
      }
      uint32_t pf[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p0 = ex2_approx(sc[i][0] - ref_a), p1 = ex2_approx(sc[i][1] - ref_a);
        l_a += p0 + p1;
        pf[i >> 1][(i & 1) * 2 + 0] = pack_f16x2(p0, p1);
        pf[i >> 1][(i & 1) * 2 + 1] = 0u;
        if (!HALF) {
          const float p2 = ex2_approx(sc[i][2] - ref_b), p3 = ex2_approx(sc[i][3] - ref_b);
          l_b += p2 + p3;
          pf[i >> 1][(i & 1) * 2 + 1] = pack_f16x2(p2, p3);
        }
      }
      auto pv = [&](auto kind) {
        constexpr bool masked = decltype(kind)::value;
        uint32_t keep[4];
        if (masked) {
          // bytes of tokens that are not visible become zero: a masked slot may hold anything, NaN too
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t two = bits >> (i * 8 + t4 * 2);
            keep[i] = ((two & 1u) ? 0x00FF00FFu : 0u) | ((two & 2u) ? 0xFF00FF00u : 0u);
          }
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t r[4], ev[4], od[4];
          ldsm_x4_t(vb + tile_at<D>(lane, c), r[0], r[1], r[2], r[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t x = __byte_perm(r[i], 0, 0x3120);  // {t0 d0, t1 d0, t0 d1, t1 d1}
            if (masked) x &= keep[i];
            e4m3x4_to_f16(x, ev[i], od[i]);
          }
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            mma_f16_16816(o[c][0], pf[kk], ev[2 * kk], ev[2 * kk + 1]);
            mma_f16_16816(o[c][1], pf[kk], od[2 * kk], od[2 * kk + 1]);
          }
        }
      };
      if (bits == 0xFFFFFFFFu) pv(std::false_type{}); else pv(std::true_type{});
    }
    __syncwarp();
    if (k + kStages < my_count) {
      if (lane == 0) fence_proxy_async_smem();
      issue(k + kStages);
    }
  }
  if (!ok) {
    // drain this warp's copies still in flight before the CTA and its shared memory go away
    if (lane == 0) {
      for (int k = k_fail; k < min(my_count, k_fail + kStages); ++k)
        mbar_wait_drain(&bars[warp][k % kStages], (uint32_t)((k / kStages) & 1), a.timeout_ns);
    }
    __syncwarp();
  }
  __syncthreads();
  if (s_abort) return;

  // ---- join the 4 warps' states (the rings are free: every copy has landed)
  l_a += __shfl_xor_sync(0xFFFFFFFFu, l_a, 1);
  l_a += __shfl_xor_sync(0xFFFFFFFFu, l_a, 2);
  if (!HALF) {
    l_b += __shfl_xor_sync(0xFFFFFFFFu, l_b, 1);
    l_b += __shfl_xor_sync(0xFFFFFFFFu, l_b, 2);
  }
  float* sO = reinterpret_cast<float*>(smem);  // [4][16][D]
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    const int col = c * 16 + t4 * 4;
    *reinterpret_cast<float4*>(sO + (warp * 16 + ra) * D + col) =
        make_float4(o[c][0][0] * vref, o[c][1][0] * vref, o[c][0][1] * vref, o[c][1][1] * vref);
    if (!HALF)
      *reinterpret_cast<float4*>(sO + (warp * 16 + rb) * D + col) =
          make_float4(o[c][0][2] * vref, o[c][1][2] * vref, o[c][0][3] * vref, o[c][1][3] * vref);
  }
  if (t4 == 0) {
    sM[warp][ra] = m_a;
    sL[warp][ra] = l_a;
    if (!HALF) {
      sM[warp][rb] = m_b;
      sL[warp][rb] = l_b;
    }
  }
  __syncthreads();
  const bool only = n_vis <= a.pages_per_split;  // the request's one span: the result itself
  for (int x = tid; x < g * D; x += kWarps * 32) {
    const int row = x / D, col = x % D;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sM[w][row]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float u = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float wt = ex2_approx(sM[w][row] - ref);
      u += wt * sO[(w * 16 + row) * D + col];
      l += wt * sL[w][row];
    }
    if (only) {
      const float r = mm == -INFINITY ? 0.f : u / l;
      if (a.out_f32) reinterpret_cast<float*>(a.out)[(hq0 + row) * D + col] = r;
      else reinterpret_cast<__nv_bfloat16*>(a.out)[(hq0 + row) * D + col] = __float2bfloat16_rn(r);
      if (col == 0) a.lse[hq0 + row] = mm == -INFINITY ? -INFINITY : (mm + log2f(l)) * kLn2;
    } else {
      const size_t slot = (hq0 + row) * (size_t)a.n_splits + s;
      a.ws_u[slot * D + col] = u;
      if (col == 0) {
        a.ws_m[slot] = mm;
        a.ws_l[slot] = l;
      }
    }
  }
}

// Joins the spans of one query head: m = max m_s, l = sum 2^(m_s - m) l_s, O = sum 2^(m_s - m) u_s / l. Requests of
// one span are done already. Four groups of threads take every fourth span.
constexpr int kJoin = 4;

template <int D>
__global__ void __launch_bounds__(kJoin * D) decode_fp8_join_kernel(const __grid_constant__ DecArgs a) {
  __shared__ float s_u[kJoin][D], s_red[kJoin * D / 32], s_l[kJoin];
  const int hq = blockIdx.x, b = blockIdx.y, col = threadIdx.x % D, part = threadIdx.x / D;
  const DevMask& M = a.mask;
  const size_t mrow = (size_t)(M.Bm > 1 ? b : 0) * M.Hm * M.nq;
  const int n_vis = __ldg(M.full_kv_num + mrow) + __ldg(M.kv_num + mrow);
  if (n_vis <= a.pages_per_split) return;
  const int ns = (n_vis + a.pages_per_split - 1) / a.pages_per_split;
  const size_t base = ((size_t)b * a.Hq + hq) * (size_t)a.n_splits, obase = ((size_t)b * a.Hq + hq) * D;
  float mm = -INFINITY;
  for (int s = threadIdx.x; s < ns; s += kJoin * D) mm = fmaxf(mm, a.ws_m[base + s]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o));
  if (threadIdx.x % 32 == 0) s_red[threadIdx.x / 32] = mm;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoin * D / 32; ++w) mm = fmaxf(mm, s_red[w]);
  const float ref = mm == -INFINITY ? 0.f : mm;
  float l = 0.f, u = 0.f;
#pragma unroll 8
  for (int s = part; s < ns; s += kJoin) {
    const float wt = ex2_approx(a.ws_m[base + s] - ref);
    l += wt * a.ws_l[base + s];
    u += wt * a.ws_u[(base + s) * D + col];
  }
  s_u[part][col] = u;
  if (col == 0) s_l[part] = l;
  __syncthreads();
  if (part) return;
  l = 0.f;
  u = 0.f;
#pragma unroll
  for (int p = 0; p < kJoin; ++p) {
    l += s_l[p];
    u += s_u[p][col];
  }
  const float r = mm == -INFINITY ? 0.f : u / l;
  if (a.out_f32) reinterpret_cast<float*>(a.out)[obase + col] = r;
  else reinterpret_cast<__nv_bfloat16*>(a.out)[obase + col] = __float2bfloat16_rn(r);
  if (col == 0) a.lse[(size_t)b * a.Hq + hq] = mm == -INFINITY ? -INFINITY : (mm + log2f(l)) * kLn2;
}

template <int D>
int launch_d(const DecFp8Args& A, cudaStream_t st) {
  using C = Cfg<D>;
  const DecArgs& a = A.d;
  CUtensorMap tk, tv;
  const uint64_t dims[2] = {(uint64_t)D, (uint64_t)a.n_pages_total * a.Hkv * a.page};
  const uint64_t strides[1] = {(uint64_t)D};
  const uint32_t box[2] = {D, kSub};
  if (encode_tmap_u8(&tk, a.k_pages, 2, dims, strides, box) != 0) return FA_ERR_CUDA;
  if (encode_tmap_u8(&tv, a.v_pages, 2, dims, strides, box) != 0) return FA_ERR_CUDA;
  auto kern = a.Hq / a.Hkv <= 8 ? decode_fp8_kernel<D, true> : decode_fp8_kernel<D, false>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
    return FA_ERR_CUDA;
  kern<<<dim3(a.n_splits, a.Hkv, a.Bz), kWarps * 32, C::kSmem, st>>>(A, tk, tv);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  if (a.n_splits > 1) {
    decode_fp8_join_kernel<D><<<dim3(a.Hq, a.Bz), kJoin * D, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // namespace

int launch_decode_fp8(const DecFp8Args& a, cudaStream_t st) {
  return a.d.d == 64 ? launch_d<64>(a, st) : launch_d<128>(a, st);
}

}  // namespace fa
