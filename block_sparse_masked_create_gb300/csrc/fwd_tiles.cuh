// Query tiles and block lists of the tcgen05 forwards (bf16 K / V: fwd_tc5.cu, e4m3 pages: fwd_fp8.cu): which two tiles a
// CTA takes, the order in which it visits their key blocks, and the issue of a whole product.
#pragma once

#include <climits>

#include "fa_launch.h"

namespace fa {
namespace {

// byte offset of 16-byte chunk c16 of row `row` in a [128][D] tile stored as D/64 sub-tiles [128][64]
// with the 128-byte swizzle (TMA SWIZZLE_128B layout; also the UMMA K-major SW128 layout)
__device__ __forceinline__ uint32_t tile_off(int row, int c16) {
  return (uint32_t)((c16 >> 3) * 16384 + row * 128 + (((c16 & 7) ^ (row & 7)) << 4));
}

// One 128-row query tile: query head h (KV head hk), BlockMask row r, and the query block rq it reads
// (rq = r, or with split rows the block of entry r). O and LSE go to rows r * 128 .. of the output.
struct Tile {
  int valid;     // a tile exists (Hq or the number of query blocks may be odd)
  int h, hk, r, rq;
  int n_full, n_part, n;
  const int32_t* full_idx;
  const int32_t* part_idx;
};

__device__ __forceinline__ Tile make_tile(const FwdArgs& a, int b, int h, int r) {
  const DevMask& M = a.mask;
  Tile T;
  T.valid = h < a.Hq && r >= 0;
  T.h = T.valid ? h : 0;
  T.r = T.valid ? r : 0;
  T.rq = a.split_ncm > 1 ? T.r / a.split_ncm : T.r;
  T.hk = T.h / (a.Hq / a.Hkv);
  const int bm = M.Bm > 1 ? b : 0, hm = M.Hm > 1 ? T.h : 0;
  const size_t mrow = ((size_t)bm * M.Hm + hm) * M.nq + T.r;
  T.n_full = T.valid ? __ldg(M.full_kv_num + mrow) : 0;
  T.n_part = T.valid ? __ldg(M.kv_num + mrow) : 0;
  T.n = T.n_full + T.n_part;
  T.full_idx = M.full_kv_idx + mrow * M.nk;
  T.part_idx = M.kv_idx + mrow * M.nk;
  return T;
}

// A tile's visited blocks in column order, its full and partial lists (each ascending) merged. Ordering
// keys are the column (ascending walk) or minus the column (descending walk); an exhausted list has key
// INT_MAX. Every role of the CTA walks the same lists the same way.
struct Walk {
  int f, p, kf, kp;
  // The load is issued where the walk advances and read one element later; as a volatile asm statement
  // it keeps its place in the program (a read-only __ldg may be sunk to its first use, which would put a
  // cache round trip on the issuing warp's critical path at every element).
  static __device__ __forceinline__ int key(const int32_t* idx, int n, int i, bool desc) {
    const int k = i < n ? (desc ? n - 1 - i : i) : 0;
    int v;
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(idx + k));
    return i >= n ? INT_MAX : (desc ? -v : v);
  }
  __device__ __forceinline__ void init(const Tile& T, bool desc) {
    f = p = 0;
    kf = key(T.full_idx, T.n_full, 0, desc);
    kp = key(T.part_idx, T.n_part, 0, desc);
  }
  __device__ __forceinline__ int next_key() const { return min(kf, kp); }
  __device__ __forceinline__ bool next_partial() const { return kp < kf; }
  __device__ __forceinline__ void advance(const Tile& T, bool desc) {
    if (kp < kf) {
      ++p;
      kp = key(T.part_idx, T.n_part, p, desc);
    } else {
      ++f;
      kf = key(T.full_idx, T.n_full, f, desc);
    }
  }
};
__device__ __forceinline__ int key_col(int key, bool desc) { return desc ? -key : key; }

// The same walk with the loaded column ids kept as loaded: the ordering keys are derived where they are
// compared, so the load that advance() issues is first waited for at the next element rather than at once
// (the producer walks the union between its loads; a cache round trip per element would delay them).
struct LazyWalk {
  int f, p, nf, np, vf, vp, dsc;
  static __device__ __forceinline__ int load(const int32_t* idx, int n, int i, bool desc) {
    const int k = i < n ? (desc ? n - 1 - i : i) : 0;
    int v;
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(idx + k));
    return v;
  }
  __device__ __forceinline__ void init(const Tile& T, bool desc) {
    f = p = 0;
    nf = T.n_full;
    np = T.n_part;
    dsc = desc;
    vf = load(T.full_idx, nf, 0, desc);
    vp = load(T.part_idx, np, 0, desc);
  }
  __device__ __forceinline__ int kf() const { return f < nf ? (dsc ? -vf : vf) : INT_MAX; }
  __device__ __forceinline__ int kp() const { return p < np ? (dsc ? -vp : vp) : INT_MAX; }
  __device__ __forceinline__ int next_key() const { return min(kf(), kp()); }
  __device__ __forceinline__ bool next_partial() const { return kp() < kf(); }
  __device__ __forceinline__ void advance(const Tile& T, bool desc) {
    if (kp() < kf()) {
      ++p;
      vp = load(T.part_idx, np, p, desc);
    } else {
      ++f;
      vf = load(T.full_idx, nf, f, desc);
    }
  }
};

// The union of the two tiles' block sequences (both tiles read the same K / V: one batch row, one KV
// head), in the same order; each element says which tiles visit it. The producer walks it, loads K and V of
// each element once and passes the element's flags to the MMA warp with its K slot; the MMA warp issues each
// tile's products on its own elements.
struct Union {
  LazyWalk w0, w1;
  __device__ __forceinline__ void init(const Tile& T0, const Tile& T1, bool desc) {
    w0.init(T0, desc);
    w1.init(T1, desc);
  }
  __device__ __forceinline__ bool done() const { return min(w0.next_key(), w1.next_key()) == INT_MAX; }
  // column of the next element, which tiles visit it (and whether it is partial for them); then step past it
  __device__ __forceinline__ int take(const Tile& T0, const Tile& T1, bool desc, bool& in0, bool& in1,
                                      bool* part0 = nullptr, bool* part1 = nullptr) {
    const int k = min(w0.next_key(), w1.next_key());
    in0 = w0.next_key() == k;
    in1 = w1.next_key() == k;
    if (part0) *part0 = w0.next_partial();
    if (part1) *part1 = w1.next_partial();
    if (in0) w0.advance(T0, desc);
    if (in1) w1.advance(T1, desc);
    return key_col(k, desc);
  }
};

// Work item p -> batch b and the two tiles' (head, query block). Units of work, (batch, head pair) for
// sibling heads or (batch, head) for row pairs, are taken in groups of `group`; within a group the
// query blocks follow the mask's row order (longest rows first, so the short ones fill the tail; for
// causal masks the last block first) with the group's units side by side, so the CTAs resident at any
// time share the K / V of a few heads in L2. Row pairs are consecutive entries of the row order (for
// causal and sliding-window masks two adjacent query blocks), whose block lists mostly coincide.
__device__ __forceinline__ void work_item(const FwdArgs& a, int pair_rows, int group, int p, int& b, int& h0,
                                          int& h1, int& r0, int& r1) {
  const int HP = pair_rows ? a.Hq : (a.Hq + 1) / 2;         // units per batch row
  const int nq = a.mask.nq;
  const int RPU = pair_rows ? (nq + 1) / 2 : nq;             // items per unit
  const int NP = a.B * HP;
  const int GS = NP < group ? NP : group;
  const int g = p / (GS * RPU), g0 = g * GS, gs = min(GS, NP - g0);
  const int rem = p - g * GS * RPU;
  const int unit = g0 + rem % gs;
  const int k = rem / gs;                                    // rank of the item within its unit
  const int hu = unit % HP;
  b = unit / HP;
  const DevMask& M = a.mask;
  const int hm_head = pair_rows ? hu : 2 * hu;
  const int32_t* ro = M.row_order ? M.row_order + ((size_t)(M.Bm > 1 ? b : 0) * M.Hm + (M.Hm > 1 ? hm_head : 0)) * nq
                                  : nullptr;
  auto row = [&](int i) { return ro ? __ldg(ro + i) : nq - 1 - i; };
  if (pair_rows) {
    h0 = h1 = hu;
    r0 = row(2 * k);
    r1 = 2 * k + 1 < nq ? row(2 * k + 1) : -1;
  } else {
    h0 = 2 * hu;
    h1 = 2 * hu + 1;
    r0 = r1 = row(k);
  }
}

// A whole product is issued from one asm statement: one elect.sync picks the issuing lane for all its
// K-steps (an elect and a separate statement per K-step cost the single MMA warp more issue time than the
// tensor core spends on the step). Operand offsets per K-step ks, in 16-byte descriptor units:
//  S = Q K^T (K-major, 128-byte swizzle, [128][64] sub-tiles of 16 KiB): (ks / 4) * 1024 + (ks % 4) * 2 on
//  both operands; the first step overwrites S, the others accumulate.
//  O += P V: P (bf16 pairs) at tensor-memory column 8 ks, V rows 16 ks .. 16 ks + 15 at 128 ks; the first
//  step accumulates only if `acc`.
#define FA_MMA_HEAD                                                                                       \
  "{\n\t.reg .pred P, Q, T;\n\t.reg .b64 da, db;\n\t.reg .b32 ta;\n\telect.sync _|P, 0xffffffff;\n\t" \
  "setp.ne.b32 Q, %4, 0;\n\tsetp.eq.b32 T, %4, %4;\n\t"
#define FA_QK_FIRST "@P tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, Q;\n\t"
#define FA_QK_STEP(OFF) \
  "add.s64 da, %1, " #OFF ";\n\tadd.s64 db, %2, " #OFF ";\n\t@P tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, T;\n\t"
#define FA_PV_FIRST "@P tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, Q;\n\t"
#define FA_PV_STEP(COL, OFF)                                                                               \
  "add.s32 ta, %1, " #COL ";\n\tadd.s64 db, %2, " #OFF ";\n\t@P tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, " \
  "%3, T;\n\t"

template <int NK>  // D / 16 K-steps
__device__ __forceinline__ void mma_qk_product(uint32_t d_tmem, uint64_t qdesc, uint64_t kdesc, uint32_t idesc) {
  static_assert(NK == 4 || NK == 8, "d = 64 or 128");
  if constexpr (NK == 8) {
    asm volatile(FA_MMA_HEAD FA_QK_FIRST FA_QK_STEP(2) FA_QK_STEP(4) FA_QK_STEP(6) FA_QK_STEP(1024) FA_QK_STEP(1026)
                     FA_QK_STEP(1028) FA_QK_STEP(1030) "}" ::"r"(d_tmem),
                 "l"(qdesc), "l"(kdesc), "r"(idesc), "r"(0u)
                 : "memory");
  } else {
    asm volatile(FA_MMA_HEAD FA_QK_FIRST FA_QK_STEP(2) FA_QK_STEP(4) FA_QK_STEP(6) "}" ::"r"(d_tmem), "l"(qdesc),
                 "l"(kdesc), "r"(idesc), "r"(0u)
                 : "memory");
  }
}
__device__ __forceinline__ void mma_pv_product(uint32_t d_tmem, uint32_t p_tmem, uint64_t vdesc, uint32_t idesc,
                                               uint32_t acc) {
  asm volatile(FA_MMA_HEAD FA_PV_FIRST FA_PV_STEP(8, 128) FA_PV_STEP(16, 256) FA_PV_STEP(24, 384) FA_PV_STEP(32, 512)
                   FA_PV_STEP(40, 640) FA_PV_STEP(48, 768) FA_PV_STEP(56, 896) "}" ::"r"(d_tmem),
               "r"(p_tmem), "l"(vdesc), "r"(idesc), "r"(acc)
               : "memory");
}
#undef FA_MMA_HEAD
#undef FA_QK_FIRST
#undef FA_QK_STEP
#undef FA_PV_FIRST
#undef FA_PV_STEP

}  // namespace
}  // namespace fa
