// Masked attention forward over an 8-bit paged cache on 5th-generation tensor cores: queries bf16, keys and values e4m3
// with a scale for each 32 tokens and KV head, 128 x 128 blocks, head dim 64 or 128.
//
//   s_ij = scale * ks[j/32] * <q_i, k8_j> (+ score rule, mask),   O_i = sum_j p_ij vs[j/32] v8_j / sum_j p_ij
//
// The tiles, the order of blocks and the roles are those of the bf16 forward (fwd_tc5.cu); what differs is that K and V
// arrive as bytes and all products run in fp16:
//   warps 0 .. 7    softmax, a thread a query row. Before the loop each thread turns its row of Q into fp16, divided by a
//                   power of two (exact but for what is 2^-24 of the row's largest). A score column is multiplied by its
//                   block's K scale, P carries its block's V scale (a factor in the exponent, four a row and block, from
//                   registers); the row sum is taken without it. The unit that a row's O and sum are held in is a power of
//                   two by the largest P times V scale that the row sees: scales of what it does not see play no part.
//   warp 8          TMA producer: the pages of each key block of the union, as bytes, into a ring of staging tiles.
//   warp 9          MMA issuer, as in the bf16 forward.
//   warps 12 .. 15  converters: a staging tile's bytes to fp16 (exact, no scale) in the swizzled layout that the products
//                   read, a row a thread; rows that no query may see, and pages that are not there, become zero.
// Few queries a request (heads of a KV head times positions at most 128): the heads share a tile, so that each page is read
// and converted once for all of them, and the two tiles of a CTA are two chunks of the keys.
// Bytes to fp16 is one conversion for two values: 128 a thread and tile, about a fifth of the issue slots that a block's
// softmax leaves. The whole saves writing and reading the expanded cache, 3 + 2 bytes a value.
// Bound: the tensor pipe and the softmax, as the bf16 forward, and the instruction cache, which the roles share (its stalls fell
// when the converters' loop was rolled: 142 -> 134 us). Measured on one GB300: 256 queries after 130,816 tokens, 8 heads, d =
// 128: 132 us with the merge of the cut rows, 1040 TFLOP/s (expanding first: 263); long rows take 1.2 times the bf16 forward.
// Registers: 512 threads launch with 128 each; the softmax warps go up to 192 and the others down to 64, together the
// same 65,536 (with 168 and 88 the softmax spilled).
#include <cfloat>
#include <cstring>

#include "fp8.cuh"
#include "fwd_tiles.cuh"

namespace fa {
namespace {

constexpr int kLoadWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kConvWarp = 12;
constexpr int kThreads = 16 * 32;
constexpr int kSoftmaxRegs = 192, kOtherRegs = 64;
static_assert(256 * kSoftmaxRegs + 256 * kOtherRegs <= 512 * 128, "registers of the launch");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The row's unit, 2^ref: P times its V scale lies in fp16, whose smallest step is 2^-24 and largest value just under 2^16. A new unit
// is set 2^7 under a block's largest, and kept while a block's largest stays within 2^-1 .. 2^15 of it, so that a key 2^-13 of its
// block's largest keeps all its bits and one 2^-23 of it is not lost. (A unit that only rises leaves the many small keys of a long row
// that one key outweighs to the subnormals: 20,000 keys at e^-17 of one with V = 0 were off by 44 %.) Units are not lowered
// beyond 2^-24 of the row's largest so far: what is lost there is 2^-49 of it a key, 2^-29 over a million keys, and ALiBi's scores, which
// fall without end, take three passes over O and not one every 2^8. The rows of a warp change units together, as a pass serves all:
// 512 queries of 2 requests over 8192 keys, 32 / 8 heads, ALiBi: 142 us (154 row by row and down to 2^-40; no ALiBi: 131).
constexpr float kUnitBelow = 7.f, kMost = 15.f, kLeast = -1.f, kUnitSpan = 24.f;

enum ScoreKind { SK_NONE = 0, SK_ALIBI = 1, SK_SOFTCAP = 2, SK_GENERIC = 3 };

template <int D>
struct Cfg {
  static constexpr int kQBytes = 128 * D * 2;      // one Q tile (also the O staging tile)
  static constexpr int kSlotBytes = 128 * D * 2;   // one K or V tile in fp16
  static constexpr int kRawBytes = 128 * D;        // the same in bytes
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRaw = D == 128 ? 4 : 8;    // staging tiles
  static constexpr int kOffRing = 2 * kQBytes;
  static constexpr int kOffRaw = kOffRing + kStages * kSlotBytes;
  static constexpr int kOffBar = kOffRaw + kRaw * kRawBytes;
  static constexpr int kBars = 11 + 2 * kStages + 2 * kRaw;
  static constexpr int kSmem = kOffBar + 512;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kBars * 8 + 8 + 4 * kStages + 8 * kRaw <= 512, "barrier region");
  static constexpr uint32_t kTmemCols = 512;
  // tensor memory as in the bf16 forward: S_t at 256 t (P_t over its first 64 columns), O_t at 256 t + 128
  __device__ static constexpr uint32_t col_s(int t) { return (uint32_t)t * 256u; }
  __device__ static constexpr uint32_t col_o(int t) { return (uint32_t)t * 256u + 128u; }
};

struct Params {
  FwdFp8Args f;
  int ahead, pair_rows, desc, group;  // as in the bf16 forward
};

// fp16 A and B, fp32 accumulation (type fields 0)
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// byte offset of 16-byte chunk c of row `row` in a TMA-written [128][D] byte tile (128-byte swizzle for D = 128, 64-byte
// for D = 64)
template <int D>
__device__ __forceinline__ uint32_t raw_at(int row, int c) {
  return D == 128 ? (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)) : (uint32_t)(row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
}

// 2^n of a whole n; 0 below 2^-126
__device__ __forceinline__ float pow2_whole(float n) {
  return __uint_as_float((uint32_t)(int)(fminf(fmaxf(n, -127.f), 127.f) + 127.f) << 23);
}

// PACK: P.f.pack > 1. As a run-time choice the turns cost the other calls 6 % (the producer's registers and instructions).
template <int D, int SK, bool PACK>
__global__ void __launch_bounds__(kThreads, 1)
    fwd_fp8_kernel(const __grid_constant__ Params P, const __grid_constant__ CUtensorMap tmQ,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ CUtensorMap tmO) {
  using C = Cfg<D>;
  constexpr int NST = C::kStages, NRAW = C::kRaw;
  const FwdArgs& a = P.f.a;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* const bar_q = bars;                      // [2] Q tile landed
  uint64_t* const bar_qc = bars + 2;                 // [2] Q tile is fp16 (each softmax warp arrives)
  uint64_t* const bar_s = bars + 4;                  // [2] S = Q K^T complete
  uint64_t* const bar_p = bars + 6;                  // [2] P stored in tensor memory (each softmax warp arrives)
  uint64_t* const bar_o = bars + 8;                  // [2] O += P V complete
  uint64_t* const bar_full = bars + 10;              // [NST] fp16 tile written (each converter warp arrives)
  uint64_t* const bar_empty = bar_full + NST;        // [NST] fp16 tile consumed
  uint64_t* const bar_raw = bar_empty + NST;         // [NRAW] staging tile landed
  uint64_t* const bar_rawfree = bar_raw + NRAW;      // [NRAW] staging tile read (each converter warp arrives)
  uint64_t& bar_drain = *(bar_rawfree + NRAW);
  uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(bars + C::kBars);
  int32_t& s_abort = *(reinterpret_cast<int32_t*>(bars + C::kBars) + 1);
  // per fp16 slot of a K tile: which tiles visit its element (bits 0, 1), whether it is the union's last (bit 2)
  volatile int32_t* const s_uflag = reinterpret_cast<volatile int32_t*>(bars + C::kBars + 1);
  // per staging tile: the key block, and those flags with, from bit 8 on, which of its pages are there
  volatile int32_t* const s_raw = s_uflag + NST;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem) & 1023u) {  // uniform across the CTA, before any barrier or allocation
    if (tid == 0) report(a.status, FA_ERR_DEVICE_CHECK);
    return;
  }
  const DevMask& M = a.mask;
  const bool desc = P.desc != 0;
  int b, h0, h1, r0, r1;
  work_item(a, P.pair_rows, P.group, blockIdx.x, b, h0, h1, r0, r1);
  const Tile T0 = make_tile(a, b, h0, r0);
  const Tile T1 = make_tile(a, b, h1, r1);
  const bool any = T0.n + T1.n > 0;
  const KeyRange keys = key_range(a.rule, M.Bm, b, P.f.rule_q_len, a.kv_len);
  const int begin = keys.begin, end = keys.end;
  const int page = P.f.page, page_log = 31 - __clz(page);

  uint8_t* sQ0 = smem;
  uint8_t* sQ1 = smem + C::kQBytes;
  uint8_t* sRing = smem + C::kOffRing;
  uint8_t* sRaw = smem + C::kOffRaw;

  // ring loads (producer warp); the first one starts before the CTA-wide barrier below
  int issued = 0, l_pid = -1;
  uint32_t there = 0;
  const int boxes = 128 / page;
  auto load = [&](bool is_v, int c, int fl, const WaitCtl& wc) -> bool {
    const int s = issued % NRAW, j = c * 128 + lane * page;
    const bool need = lane < boxes && j < end && j + page > begin;
    if (!is_v) {  // the block's pages, one a lane (V takes the same); the look-up is under way while the warp waits
      l_pid = -1;
      if (need) asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(l_pid) : "l"(a.page_table + (size_t)b * a.max_pages + (j >> page_log)));
    }
    if (issued >= NRAW &&
        !__all_sync(0xFFFFFFFFu, mbar_wait(&bar_rawfree[s], (uint32_t)(((issued / NRAW) - 1) & 1), wc)))
      return false;
    if (!is_v) {
      const bool in = l_pid >= 0 && l_pid < a.n_pages_total;
      if (need && !in) report(a.status, FA_ERR_DEVICE_CHECK);
      there = __ballot_sync(0xFFFFFFFFu, in);
    }
    if (lane == 0) {
      s_raw[2 * s] = c;
      s_raw[2 * s + 1] = fl | (int)(there << 8);
      const uint32_t bytes = (uint32_t)__popc(there) * (uint32_t)(page * D);
      if (bytes) mbar_arrive_expect_tx(&bar_raw[s], bytes); else mbar_arrive(&bar_raw[s]);
    }
    for (int k = 0; k < boxes; ++k) {
      const int pid = __shfl_sync(0xFFFFFFFFu, l_pid, k);
      if (lane == 0 && ((there >> k) & 1u))
        tma_load_2d(sRaw + s * C::kRawBytes + k * page * D, is_v ? &tmV : &tmK, 0, (pid * a.Hkv + T0.hk) * page, &bar_raw[s]);
    }
    __syncwarp();
    ++issued;
    return true;
  };
  // the next element: its column, and which tiles visit it (bits 0, 1) and whether it is the last (bit 2)
  Union uw;
  auto take_next = [&](int& flags) -> int {
    bool i0, i1;
    int c;
    if (!PACK) {
      c = uw.take(T0, T1, desc, i0, i1);
    } else {  // the two tiles are chunks of one row: in turns, so that one's softmax runs under the other's products
      const int k0 = uw.w0.next_key(), k1 = uw.w1.next_key();
      i0 = k1 == INT_MAX || (k0 != INT_MAX && uw.w0.f + uw.w0.p <= uw.w1.f + uw.w1.p);
      i1 = !i0;
      c = key_col(i0 ? k0 : k1, desc);
      if (i0) uw.w0.advance(T0, desc); else uw.w1.advance(T1, desc);
    }
    flags = (int)i0 | ((int)i1 << 1) | (uw.done() ? 4 : 0);
    return c;
  };
  int c_first = -1;  // producer: column of the first element
  if (warp == kLoadWarp) {
    if (lane == 0) {
      s_abort = 0;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        mbar_init(&bar_q[t], 1);
        mbar_init(&bar_qc[t], 4);
        mbar_init(&bar_s[t], 1);
        mbar_init(&bar_p[t], 4);
        mbar_init(&bar_o[t], 1);
      }
      for (int s = 0; s < NST; ++s) {
        mbar_init(&bar_full[s], 4);
        mbar_init(&bar_empty[s], 1);
      }
      for (int s = 0; s < NRAW; ++s) {
        mbar_init(&bar_raw[s], 1);
        mbar_init(&bar_rawfree[s], 4);
      }
      mbar_init(&bar_drain, 1);
      fence_mbar_init();
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmO);
    }
    __syncwarp();
    const uint64_t qpol = l2_evict_first_policy();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const Tile& T = t ? T1 : T0;
      if (T.n > 0) {
        mbar_arrive_expect_tx_elect(&bar_q[t], C::kQBytes);
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          tma_load_3d_elect_hint((t ? sQ1 : sQ0) + x * 16384, &tmQ, x * 64, T.rq * 128, b * a.Hq + T.h, &bar_q[t], qpol);
      }
    }
    if (any) {  // K of the first element: there is room, so nothing is waited for
      uw.init(T0, T1, desc);
      int fl;
      c_first = take_next(fl);
      load(false, c_first, fl, WaitCtl{a.timeout_ns, a.status, &s_abort});
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&s_tmem, C::kTmemCols);
    tmem_relinquish();
  }
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  const uint32_t tmem = s_tmem;
  WaitCtl wc{a.timeout_ns, a.status, &s_abort};
  // the four warps of each warpgroup take the same branch
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
    // =============================== TMA producer ===============================
    // the Q tiles of the CTA that will take this SM after the next wave go to L2 now
    if (P.ahead > 0 && blockIdx.x + P.ahead < gridDim.x && lane == 0) {
      int bn, hn0, hn1, rn0, rn1;
      work_item(a, P.pair_rows, P.group, blockIdx.x + P.ahead, bn, hn0, hn1, rn0, rn1);
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const Tile Tn = make_tile(a, bn, tt ? hn1 : hn0, tt ? rn1 : rn0);
        if (Tn.n == 0) continue;
#pragma unroll
        for (int x = 0; x < D / 64; ++x) tma_prefetch_l2_3d(&tmQ, x * 64, Tn.rq * 128, bn * a.Hq + Tn.h);
      }
    }
    __syncwarp();
    // K(u0), then V(u_k) K(u_k+1) for each element u_k of the union: the order in which the products take them.
    bool ok = true;
    int c = c_first;
    while (c >= 0 && ok) {
      ok = load(true, c, 0, wc);
      if (!ok || uw.done()) break;
      int fl;
      c = take_next(fl);
      ok = load(false, c, fl, wc);
    }
    if (!ok || *wc.abort) {
      // drain: the last copies may still be landing in shared memory
      for (int i = max(0, issued - NRAW); i < issued; ++i)
        mbar_wait_drain(&bar_raw[i % NRAW], (uint32_t)((i / NRAW) & 1), a.timeout_ns);
      if (T0.n > 0) mbar_wait_drain(&bar_q[0], 0, a.timeout_ns);
      if (T1.n > 0) mbar_wait_drain(&bar_q[1], 0, a.timeout_ns);
    }
  } else if (warp >= kConvWarp) {
    // =============================== converters ===============================
    const int row = tid - kConvWarp * 32;
    const uint32_t seen = (uint32_t)max(end - begin, 0);
    bool last = false;
    for (int i = 0; any; ++i) {
      const int sr = i % NRAW, s = i % NST;
      const bool is_v = i & 1;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bar_raw[sr], (uint32_t)((i / NRAW) & 1), wc))) break;
      const int c = s_raw[2 * sr], fl = s_raw[2 * sr + 1];
      const bool zero = (uint32_t)(c * 128 + row - begin) >= seen || !((fl >> (8 + (row >> page_log))) & 1);
      const uint32_t src = smem_u32(sRaw + sr * C::kRawBytes);
      uint8_t* const dst = sRing + s * C::kSlotBytes;
      if (i >= NST && !__all_sync(0xFFFFFFFFu, mbar_wait(&bar_empty[s], (uint32_t)(((i / NST) - 1) & 1), wc))) break;
#pragma unroll 2
      for (int k = 0; k < D / 16; ++k) {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(src + raw_at<D>(row, k))
                     : "memory");
        if (zero) v = make_uint4(0, 0, 0, 0);
        uint4 lo, hi;
        e4m3x4_to_f16(v.x, lo.x, lo.y);
        e4m3x4_to_f16(v.y, lo.z, lo.w);
        e4m3x4_to_f16(v.z, hi.x, hi.y);
        e4m3x4_to_f16(v.w, hi.z, hi.w);
        *reinterpret_cast<uint4*>(dst + tile_off(row, 2 * k)) = lo;
        *reinterpret_cast<uint4*>(dst + tile_off(row, 2 * k + 1)) = hi;
      }
      if (row == 0 && !is_v) s_uflag[s] = fl & 7;
      fence_proxy_async_smem();  // the products read the tile, and a copy refills the staging tile, by the async proxy
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar_full[s]);
        mbar_arrive(&bar_rawfree[sr]);
      }
      if (!is_v) last = fl & 4;
      else if (last) break;
    }
  } else if (warp == kMmaWarp) {
    // =============================== MMA issuer ===============================
    // The order of the bf16 forward: at union step k, for tile 0 then tile 1 (each on its own elements), O_t +=
    // P_t(u_k-1) V(u_k-1) once P_t is ready, then S_t = Q_t K(u_k)^T; a slot is released after its last reader.
    constexpr uint32_t idesc_qk = idesc_f16_f32(128, 128, false);
    constexpr uint32_t idesc_pv = idesc_f16_f32(128, D, true);
    const uint64_t qdesc0 = sdesc_sw128(smem_u32(sQ0), 16, 1024), qdesc1 = sdesc_sw128(smem_u32(sQ1), 16, 1024);
    const uint64_t kdesc = sdesc_sw128(smem_u32(sRing), 16, 1024);
    const uint64_t vdesc = sdesc_sw128(smem_u32(sRing), 128 * 128, 1024);
    int consumed = 0;
    bool ok = true;
    if (T0.n > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_qc[0], 0, wc));
    if (ok && T1.n > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_qc[1], 0, wc));
    tc5_fence_after();
    auto take = [&]() -> int {
      const int s = consumed % NST;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bar_full[s], (uint32_t)((consumed / NST) & 1), wc))) return -1;
      tc5_fence_after();
      ++consumed;
      return s;
    };
    struct Step {
      bool live, in0, in1;
      int sk, sv;  // slots of the element's K and V
    };
    Step cur{false, false, false, -1, -1}, prev = cur;
    bool more = any;
    int np[2] = {0, 0};  // P blocks consumed so far per tile
    while (ok) {
      cur.live = more;
      if (!cur.live && !prev.live) break;
      if (prev.live && (prev.sv = take()) < 0) { ok = false; break; }
      if (cur.live) {
        if ((cur.sk = take()) < 0) { ok = false; break; }
        const int fl = s_uflag[cur.sk];
        cur.in0 = fl & 1;
        cur.in1 = (fl >> 1) & 1;
        more = !(fl & 4);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const bool use_v = prev.live && (t ? prev.in1 : prev.in0);
        const bool use_k = cur.live && (t ? cur.in1 : cur.in0);
        if (use_v) {
          if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_p[t], (uint32_t)(np[t] & 1), wc)))) break;
          tc5_fence_after();
          mma_pv_product(tmem + C::col_o(t), tmem + C::col_s(t), vdesc + (uint64_t)(prev.sv * (C::kSlotBytes >> 4)), idesc_pv,
                         np[t] > 0 ? 1u : 0u);
          tc5_commit_elect(&bar_o[t]);
          ++np[t];
          if (t == 1 || !prev.in1) tc5_commit_elect(&bar_empty[prev.sv]);
        }
        if (use_k) {
          mma_qk_product<D / 16>(tmem + C::col_s(t), t ? qdesc1 : qdesc0, kdesc + (uint64_t)(cur.sk * (C::kSlotBytes >> 4)),
                                 idesc_qk);
          tc5_commit_elect(&bar_s[t]);
          if (t == 1 || !cur.in1) tc5_commit_elect(&bar_empty[cur.sk]);
        }
      }
      prev = cur;
    }
    tc5_commit_elect(&bar_drain);
    mbar_wait_drain(&bar_drain, 0, a.timeout_ns);
  }
  } else {
    // =============================== softmax warpgroups ===============================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const Tile TT = t ? T1 : T0;
    uint8_t* const sQt = t ? sQ1 : sQ0;
    const int q_row = TT.rq * 128 + row;  // row of the tile's head
    const int o_row = TT.r * 128 + row;   // output row (the same unless rows are split)
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + C::col_s(t);
    const uint32_t tO = tmem + lane_base + C::col_o(t);
    float* Lg = a.lse + ((size_t)b * a.Hq + TT.h) * a.out_q_len;
    const bool issuer = (warp & 3) == 0 && lane == 0;
    if (TT.valid && TT.n == 0) {
      const int row_bytes = D * (a.out_f32 ? 4 : 2);
      uint8_t* Ob = reinterpret_cast<uint8_t*>(a.out) + (((size_t)b * a.Hq + TT.h) * a.out_q_len) * row_bytes;
      if (q_row < a.q_len) {
        if (a.split_ncm <= 1)
          for (int c16 = 0; c16 < row_bytes / 16; ++c16)
            *reinterpret_cast<uint4*>(Ob + (size_t)o_row * row_bytes + c16 * 16) = make_uint4(0, 0, 0, 0);
        Lg[o_row] = -INFINITY;
      }
    } else if (TT.valid) {
      const int64_t off_b = a.rule.q_offset ? (int64_t)__ldg(a.rule.q_offset + (M.Bm > 1 ? b : 0)) : 0;
      // the row's query head and position (a packed tile holds the heads of a KV head one after the other)
      const int sub_head = PACK ? min(q_row / P.f.rule_q_len, P.f.pack - 1) : 0;
      const int head = PACK ? TT.h * P.f.pack + sub_head : TT.h;
      const int64_t ig = (int64_t)(PACK ? q_row - sub_head * P.f.rule_q_len : q_row) + off_b;
      const int bm = M.Bm > 1 ? b : 0;
      bool ok = true;
      // ---- the row of Q to fp16, divided by the power of two under its largest magnitude
      float up = 1.f;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_q[t], 0u, wc));
      if (ok) {
        uint32_t big = 0;  // magnitudes order as their bits do
#pragma unroll
        for (int c16 = 0; c16 < D / 8; ++c16) {
          const uint4 v = *reinterpret_cast<const uint4*>(sQt + tile_off(row, c16));
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) big = max(big, max((u[i] << 16) & 0x7FFF0000u, u[i] & 0x7FFF0000u));
        }
        const uint32_t ex = big >> 23;
        const int e = (ex == 0u || ex == 255u) ? 0 : min(max((int)ex - 127, -126), 126);
        up = __uint_as_float((uint32_t)(127 + e) << 23);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int c16 = 0; c16 < D / 8; ++c16) {
          uint4* const at = reinterpret_cast<uint4*>(sQt + tile_off(row, c16));
          const uint4 v = *at;
          auto half2 = [&](uint32_t u) {
            return pack_f16x2(__uint_as_float(u << 16) * down, __uint_as_float(u & 0xFFFF0000u) * down);
          };
          *at = make_uint4(half2(v.x), half2(v.y), half2(v.z), half2(v.w));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_qc[t]);
      }
      const float qs = a.scale * up;                    // times a K scale: the factor of a score column
      const float slope2 = (SK == SK_ALIBI || SK == SK_GENERIC) && a.score.alibi ? __ldg(a.score.alibi + head) * kLog2e : 0.f;
      const float cap2 = SK == SK_SOFTCAP ? a.score.softcap * kLog2e : 1.f;
      float ref = -INFINITY, largest = -INFINITY, le = 0.f;  // O and the row sum are held in units of 2^ref
      // scales of a block, looked up one block ahead: lane q holds the K scale of its tokens 32 q .. (q < 4), lane 4 + q
      // the V scale. (A second walk two blocks ahead, so that no step of list -> page table -> scale is waited for, was 10 %
      // slower: the instructions weigh more than the waits, which lie under the products.)
      const int sub = lane & 3;
      const float* const scales = (lane & 4) ? P.f.v_scale : P.f.k_scale;
      auto fetch = [&](int c) -> float {
        const int j = c * 128 + sub * 32;
        if (j >= end) return kScaleMin;  // no row sees it
        const int pid = __ldg(a.page_table + (size_t)b * a.max_pages + (j >> page_log));
        if (pid < 0 || pid >= a.n_pages_total) return kScaleMin;
        return clamp_scale(__ldg(scales + ((int64_t)pid * a.Hkv + TT.hk) * (page / 32) + (j & (page - 1)) / 32));
      };
      Walk wk;  // this tile's blocks, in the order the MMA warp issues them
      wk.init(TT, desc);
      float sc_next = fetch(key_col(wk.next_key(), desc));
      for (int j = 0; j < TT.n; ++j) {
        const bool partial = wk.next_partial();
        const int c = key_col(wk.next_key(), desc);
        wk.advance(TT, desc);
        const float sc = sc_next;
        if (j + 1 < TT.n) sc_next = fetch(key_col(wk.next_key(), desc));
        const int64_t j0 = (int64_t)c * 128;
        Bits128 bits = {{0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu}};
        if (partial) {
          const int w = (int)max((int64_t)0, min((int64_t)128, (int64_t)a.kv_len - j0));
          bits = {{0u, 0u, 0u, 0u}};
          if (q_row < a.q_len && w > 0) {
            const int doc_i = a.rule.any_doc ? doc_at(a.rule, bm, ig) : -1;
            const bool runs = a.rule.any_doc && ig >= 0 && ig < a.rule.doc_len && doc_runs_usable(a.rule, bm);
            int64_t run_lo = 0, run_hi = 0;
            if (runs) doc_run_of(a.rule, bm, ig, run_lo, run_hi);
            bits = rule_row_bits(a.rule, ig, j0, w, doc_i, [&](int dq) {
              if (runs) return range_bits(clamp_rel(run_lo - j0, w), clamp_rel(run_hi - j0, w));
              return doc_bits<4>(w, dq, [&](int cc) { return doc_at(a.rule, bm, j0 + cc); });
            });
          }
        }
        // log2 and inverse of the lane's scale: the whole part exact, the rest good to 2^-22 (the row sum undoes the factor)
        const uint32_t sb = __float_as_uint(sc);
        float l_inv, l_log;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(l_inv) : "f"(sc));
        asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(l_log) : "f"(__uint_as_float((sb & 0x7FFFFFu) | 0x3F800000u)));
        l_log += (float)((int)(sb >> 23) - 127);
        if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_s[t], (uint32_t)(j & 1), wc));
        if (!ok) continue;
        tc5_fence_after();
        float x[128];
#pragma unroll
        for (int k = 0; k < 4; ++k) tc5_ld32(tS + 32 * k, *reinterpret_cast<uint32_t(*)[32]>(&x[32 * k]));
        tc5_wait_ld();
        // ---- score rule (log2 domain, SK_NONE: the factor is left to the exponent's FMA)
        float mult[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mult[k] = qs * __shfl_sync(0xFFFFFFFFu, sc, k);
        if (SK == SK_NONE) {
#pragma unroll
          for (int k = 0; k < 4; ++k)  // never 0: a masked column is -inf. (Under it every visible score rounds to 0 all the same.)
            mult[k] = fmaxf(mult[k] * kLog2e, FLT_MIN);
        } else if (SK == SK_ALIBI) {
          // the bias is linear in the column: four chains step by 8 columns (see the bf16 forward)
          const float base = -slope2 * (float)(ig - j0);
          const uint64_t step = f2_pack(8.f * slope2, 8.f * slope2);
          uint64_t bch[4];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            bch[r] = f2_pack(fmaf(slope2, (float)(2 * r), base), fmaf(slope2, (float)(2 * r + 1), base));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t s2 = f2_pack(mult[k] * kLog2e, mult[k] * kLog2e);
#pragma unroll
            for (int i = 32 * k; i < 32 * k + 32; i += 2) {
              const int r = (i >> 1) & 3;
              f2_unpack(f2_fma(f2_pack(x[i], x[i + 1]), s2, bch[r]), x[i], x[i + 1]);
              bch[r] = f2_add(bch[r], step);
            }
          }
        } else if (SK == SK_SOFTCAP) {
          // tanh |u| = (1 - e) / (1 + e), e = 2^(-2 log2(e) |u|), two columns at a time: 1 - e is exact where it is small, so
          // the error is e's, 2^-23.5 of the cap (tanh.approx: 8e-6, which a cap of 50 would turn into 4e-4 of a score).
          // log2(e) c is left to the exponent's FMA. 4 x 1024 queries over 4096 keys, 32 / 8 heads: 431 us; 2^-22 with 1 -
          // 2 / (1 + e^2u) takes 391, the series of tanh_exact where scores are small 442, no cap 253.
          const uint64_t one2 = f2_pack(1.f, 1.f), neg2 = f2_pack(-1.f, -1.f);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float in = mult[k] * a.score.inv_softcap * (2.f * kLog2e);
            const uint64_t in2 = f2_pack(in, in);
#pragma unroll
            for (int i = 32 * k; i < 32 * k + 32; i += 2) {
              float y0, y1, s0, s1, r0, r1;
              f2_unpack(f2_mul(f2_pack(x[i], x[i + 1]), in2), y0, y1);
              const uint64_t e = f2_pack(ex2_approx(-fabsf(y0)), ex2_approx(-fabsf(y1)));
              f2_unpack(f2_add(e, one2), s0, s1);
              asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(s0));
              asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(s1));
              f2_unpack(f2_mul(f2_fma(e, neg2, one2), f2_pack(r0, r1)), r0, r1);
              x[i] = copysignf(r0, y0);
              x[i + 1] = copysignf(r1, y1);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            for (int i = 32 * k; i < 32 * k + 32; ++i) {
              float v = x[i] * mult[k];
              const int64_t dist = ig - (j0 + i);
              if (a.score.alibi) v -= (slope2 * kLn2) * (float)dist;
              if (a.score.rel) {
                int64_t ix = dist + a.score.kv_len - 1;
                ix = ix < 0 ? 0 : (ix > 2 * (int64_t)a.score.kv_len - 2 ? 2 * (int64_t)a.score.kv_len - 2 : ix);
                v += __ldg(a.score.rel + (size_t)head * (2 * (size_t)a.score.kv_len - 1) + ix);
              }
              if (a.score.softcap > 0.f) v = softcap_exact(v, a.score.softcap, a.score.inv_softcap);
              x[i] = v * kLog2e;
            }
          }
        }
        if (SK != SK_NONE) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mult[k] = cap2;
        }
        // ---- mask after the score rule, partial blocks only
        if (partial) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t wd = bits.w[k];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[k * 32 + i] = ((wd >> i) & 1u) ? x[k * 32 + i] : -INFINITY;
          }
        }
        // ---- the row's largest p * vs in the block, a chain for each factor. What a row does not see has no part in it
        float lg[4], top;
        {
          float mx[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            lg[k] = __shfl_sync(0xFFFFFFFFu, l_log, 4 + k);
            mx[k] = fmaxf(x[32 * k], x[32 * k + 1]);
#pragma unroll
            for (int i = 2; i < 32; i += 2) mx[k] = fmax3(mx[k], x[32 * k + i], x[32 * k + i + 1]);
            mx[k] = fmaf(mx[k], mult[k], lg[k]);
          }
          top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
        }
        float alpha = 1.f;
        bool rescale = false;
        largest = fmaxf(largest, top);
        const bool leaves = top > ref + kMost || (top < ref + kLeast && top > -INFINITY);
        if (__any_sync(0xFFFFFFFFu, leaves) && top > -INFINITY) {
          const float to = floorf(fmaxf(top - kUnitBelow, largest - kUnitSpan));  // whole: units change by powers of two
          rescale = ref != -INFINITY && to != ref;
          if (rescale) alpha = pow2_whole(ref - to);
          ref = to;
        }
        const float rf = ref == -INFINITY ? 0.f : ref;
        // ---- P vs = 2^(mult x + log2 vs - ref) in fp16, and the row sum of P in the same unit
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float add = lg[k] - rf, inv_k = __shfl_sync(0xFFFFFFFFu, l_inv, 4 + k);
          const uint64_t mul2 = f2_pack(mult[k], mult[k]), add2 = f2_pack(add, add);
          uint64_t se[2] = {0, 0};
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int at = 32 * k + 16 * ch + 2 * i;
              float y0, y1;
              f2_unpack(f2_fma(f2_pack(x[at], x[at + 1]), mul2, add2), y0, y1);
              const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
              pk[i] = pack_f16x2(p0, p1);
              se[i & 1] = f2_add(se[i & 1], f2_pack(p0, p1));
            }
            tc5_st8(tS + 16 * k + 8 * ch, pk);
          }
          float e0, e1;
          f2_unpack(f2_add(se[0], se[1]), e0, e1);
          sum = fmaf(e0 + e1, inv_k, sum);
        }
        le = le * alpha + sum;
        // ---- O is stable here: S_t completed, and O_t's previous update was issued before it
        if (j > 0 && __any_sync(0xFFFFFFFFu, rescale)) {
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            tc5_ld32(tO + c0, o);
            tc5_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tc5_st32(tO + c0, o);
          }
        }
        tc5_wait_st();
        tc5_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_p[t]);
      }
      // ---- epilogue: wait for the tile's last O update, normalise and store through the Q buffer
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_o[t], (uint32_t)((TT.n - 1) & 1), wc));
      tc5_fence_after();
      const bool empty = ref == -INFINITY;
      const float inv = empty ? 0.f : 1.f / le;
      if (ok && q_row < a.q_len) Lg[o_row] = empty ? -INFINITY : (ref + log2f(le)) * kLn2;
      constexpr int QB = D / 64;  // bf16 boxes, and fp32 boxes of a round, that the Q buffer holds
      const int rounds = a.out_f32 ? (D / 32) / QB : 1;
      for (int rd = 0; rd < rounds; ++rd) {
        if (rd > 0) {
          if (issuer) bulk_wait_group_read0();  // the previous round's boxes have left shared memory
          named_bar_sync(1 + t, 128);
        }
        if (ok) {
#pragma unroll
          for (int col = 0; col < D; col += 32) {
            const int kb = col / 32;
            if (a.out_f32 && kb / QB != rd) continue;
            uint32_t o[32];
            tc5_ld32(tO + col, o);
            tc5_wait_ld();
            if (!a.out_f32) {
#pragma unroll
              for (int q4 = 0; q4 < 4; ++q4) {
                uint4 v;
                v.x = pack_bf16x2(__uint_as_float(o[8 * q4 + 0]) * inv, __uint_as_float(o[8 * q4 + 1]) * inv);
                v.y = pack_bf16x2(__uint_as_float(o[8 * q4 + 2]) * inv, __uint_as_float(o[8 * q4 + 3]) * inv);
                v.z = pack_bf16x2(__uint_as_float(o[8 * q4 + 4]) * inv, __uint_as_float(o[8 * q4 + 5]) * inv);
                v.w = pack_bf16x2(__uint_as_float(o[8 * q4 + 6]) * inv, __uint_as_float(o[8 * q4 + 7]) * inv);
                *reinterpret_cast<uint4*>(sQt + tile_off(row, col / 8 + q4)) = v;
              }
            } else {
              uint8_t* const stg = sQt + (kb % QB) * 16384;
#pragma unroll
              for (int q4 = 0; q4 < 8; ++q4) {
                const float4 v = make_float4(__uint_as_float(o[4 * q4 + 0]) * inv, __uint_as_float(o[4 * q4 + 1]) * inv,
                                             __uint_as_float(o[4 * q4 + 2]) * inv, __uint_as_float(o[4 * q4 + 3]) * inv);
                *reinterpret_cast<float4*>(stg + row * 128 + ((q4 ^ (row & 7)) << 4)) = v;
              }
            }
          }
        }
        // every thread of the tile reaches these barriers (ok or not); the store runs only if no role gave up
        fence_proxy_async_smem();
        named_bar_sync(1 + t, 128);
        if (!*wc.abort && issuer) {
          const uint64_t pol = l2_evict_first_policy();
#pragma unroll
          for (int x = 0; x < QB; ++x)
            tma_store_3d_hint(&tmO, sQt + x * 16384, a.out_f32 ? (rd * QB + x) * 32 : x * 64, TT.r * 128, b * a.Hq + TT.h, pol);
          bulk_commit_group();
        }
      }
      if (issuer) bulk_wait_group_read0();
    }
  }
  tc5_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc5_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, int SK>
int launch_k(const FwdFp8Args& f, cudaStream_t st) {
  using C = Cfg<D>;
  const FwdArgs& a = f.a;
  CUtensorMap tq, tk, tv, to;
  const uint64_t dq[3] = {(uint64_t)D, (uint64_t)a.q_len, (uint64_t)a.B * a.Hq};
  const uint64_t sq[2] = {(uint64_t)D * 2, (uint64_t)a.q_len * D * 2};
  const uint32_t box[3] = {64, 128, 1};
  const uint64_t dk[2] = {(uint64_t)D, (uint64_t)a.n_pages_total * a.Hkv * f.page};
  const uint64_t sk[1] = {(uint64_t)D};
  const uint32_t boxk[2] = {D, (uint32_t)f.page};
  if (encode_tmap_bf16(&tq, a.q, 3, dq, sq, box) || encode_tmap_u8(&tk, a.k, 2, dk, sk, boxk) ||
      encode_tmap_u8(&tv, a.v, 2, dk, sk, boxk))
    return FA_ERR_CUDA;
  const uint64_t dout[3] = {(uint64_t)D, (uint64_t)a.out_q_len, (uint64_t)a.B * a.Hq};
  const int el = a.out_f32 ? 4 : 2;
  const uint64_t so[2] = {(uint64_t)D * el, (uint64_t)a.out_q_len * D * el};
  const uint32_t boxo[3] = {32, 128, 1};
  if (a.out_f32 ? encode_tmap_f32(&to, a.out, 3, dout, so, boxo) : encode_tmap_bf16(&to, a.out, 3, dout, so, box))
    return FA_ERR_CUDA;
  Params p;
  std::memset(&p, 0, sizeof(p));
  p.f = f;
  p.ahead = 152;
  p.pair_rows = (a.Hq / a.Hkv) % 2 != 0;
  p.desc = a.score.alibi != nullptr;
  p.group = p.pair_rows && (a.mask.nq + 1) / 2 >= 128 ? 4 : 8;
  const int n_items = p.pair_rows ? a.B * a.Hq * ((a.mask.nq + 1) / 2) : a.B * ((a.Hq + 1) / 2) * a.mask.nq;
  auto kern = f.pack > 1 ? fwd_fp8_kernel<D, SK, true> : fwd_fp8_kernel<D, SK, false>;
  cudaFuncAttributes at;  // the register split counts on what the launch allocates
  if (cudaFuncGetAttributes(&at, kern) != cudaSuccess || at.numRegs * kThreads < 256 * (kSoftmaxRegs + kOtherRegs))
    return FA_ERR_CUDA;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
    return FA_ERR_CUDA;
  kern<<<n_items, kThreads, C::kSmem, st>>>(p, tq, tk, tv, to);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D>
int launch_sk(const FwdFp8Args& f, cudaStream_t st) {
  const DevScore& s = f.a.score;
  const bool al = s.alibi != nullptr, rel = s.rel != nullptr, cap = s.softcap > 0.f;
  if (!al && !rel && !cap) return launch_k<D, SK_NONE>(f, st);
  if (al && !rel && !cap) return launch_k<D, SK_ALIBI>(f, st);
  if (!al && !rel && cap) return launch_k<D, SK_SOFTCAP>(f, st);
  return launch_k<D, SK_GENERIC>(f, st);
}

}  // namespace

int launch_fwd_fp8(const FwdFp8Args& f, cudaStream_t st) {
  return f.a.d == 128 ? launch_sk<128>(f, st) : launch_sk<64>(f, st);
}

}  // namespace fa
