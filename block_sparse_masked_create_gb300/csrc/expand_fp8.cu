// e4m3 pages -> bf16 K and V in token order, for the key blocks that a BlockMask lists: the first step of the
// forward over an 8-bit paged cache. The tcgen05 forward then reads bf16 tiles as it always does.
//
// Bound: HBM, 1 byte read and 2 written a value (and read again by the forward, mostly from L2 for short contexts): about
// 25 us of 182 for 4 x 1024 queries over 4096 keys, 32 / 8 heads. It is taken where more than 16 query tiles share a key
// block, or the blocks are smaller than 128; few tiles go through the kernel that reads the pages, single tokens through the
// decode.
//
// Positions that no query row may see (past the last key of a causal or prefix term, before the first of a window) become
// zero, so what a page holds there does not matter.
#include "fa_launch.h"
#include "fp8.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

// CTA: one 32-token block of one (batch row, KV head), K and V
template <int D>
__global__ void __launch_bounds__(kThreads) expand_kernel(const __grid_constant__ ExpandArgs a) {
  constexpr int LPR = D / 16;                       // lanes a row: 16 bytes in, 32 bytes out
  constexpr int kRows = kThreads / 2 / LPR;         // rows a pass, K by the first half of the threads, V by the second
  const int hk = blockIdx.y, b = blockIdx.z;
  const int64_t j0 = (int64_t)blockIdx.x * kScaleTokens;
  const DevMask& M = a.mask;
  const int c = (int)(j0 / M.bk);
  bool listed = false;
  const int per = M.Hm > 1 ? M.Hm / a.Hkv : 0;      // rows of the mask for this KV head (Hm = 1: the one row of all heads)
  for (int h = 0; h < max(per, 1); ++h) {
    const size_t col = ((size_t)(M.Bm > 1 ? b : 0) * M.Hm + hk * per + h) * M.nk + c;
    listed = listed || __ldg(M.q_num + col) + __ldg(M.full_q_num + col) > 0;
  }
  if (!listed) return;  // the forward reads nothing of it
  const int pid = __ldg(a.page_table + (size_t)b * a.max_pages + j0 / a.page);
  const KeyRange keys = key_range(a.rule, M.Bm, b, a.q_len, a.kv_len);
  // the block's rows that some query row sees
  const int lo = (int)max((int64_t)0, keys.begin - j0), rows = (int)min((int64_t)kScaleTokens, keys.end - j0) - lo;
  const bool seen = rows > 0;
  const bool have = pid >= 0 && pid < a.n_pages_total && seen;
  if (!have && seen) report(a.status, FA_ERR_DEVICE_CHECK);
  const int which = threadIdx.x / (kThreads / 2), tid = threadIdx.x % (kThreads / 2);
  const int lane = tid % LPR;
  float sc = 1.f;
  const uint8_t* src = nullptr;
  if (have) {
    const int64_t ph = (int64_t)pid * a.Hkv + hk, place = j0 % a.page;
    sc = clamp_scale(__ldg((which ? a.v_scale : a.k_scale) + ph * (a.page / kScaleTokens) + place / kScaleTokens));
    src = static_cast<const uint8_t*>(which ? a.v_pages : a.k_pages) + (ph * a.page + place) * D + lane * 16;
  }
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(which ? a.v_out : a.k_out) +
                       (((size_t)b * a.Hkv + hk) * a.kv_len + j0) * D + lane * 16;
#pragma unroll
  for (int r = tid / LPR; r < kScaleTokens; r += kRows) {
    if (j0 + r >= a.kv_len) break;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (have && (uint32_t)(r - lo) < (uint32_t)rows) v = __ldg(reinterpret_cast<const uint4*>(src + (size_t)r * D));
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo, hi;
      e4m3x4_to_f16(in[i], lo, hi);
      const float2 x = f16x2_to_f32(lo), y = f16x2_to_f32(hi);
      out[2 * i] = pack_bf16x2(x.x * sc, x.y * sc);      // exact where the scale is a power of two
      out[2 * i + 1] = pack_bf16x2(y.x * sc, y.y * sc);
    }
    uint4* o = reinterpret_cast<uint4*>(dst + (size_t)r * D);
    o[0] = make_uint4(out[0], out[1], out[2], out[3]);
    o[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

}  // namespace

cudaError_t launch_expand_fp8(const ExpandArgs& a, cudaStream_t st) {
  const dim3 grid((a.kv_len + kScaleTokens - 1) / kScaleTokens, a.Hkv, a.B);
  if (a.d == 64)
    expand_kernel<64><<<grid, kThreads, 0, st>>>(a);
  else
    expand_kernel<128><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
