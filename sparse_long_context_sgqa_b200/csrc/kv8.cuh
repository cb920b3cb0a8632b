// The 8-bit K/V cache: E4M3 codes with one scale for the eight tokens of a
// block in one group's K or V.
//
//   kv8      [S, blocks, G, 2 (K, V), 8, 192] codes: a (block, group)'s K and V
//            are one contiguous run, the unit the attention kernels gather
//   kv_scale [S, blocks, G, 2] FP32
//
// The scale is the smallest power of two that brings the block's largest
// magnitude to at most 448, the largest E4M3 value.  E4M3 is a floating
// format, so a scale between two powers of two would not make its codes more
// exact, while x / scale and scale * code are exact with a power of two:
// the only rounding of the cache is the code's own (half a step, 2^-4).
#pragma once
#include "attn_mma.cuh"

namespace sgqa {

constexpr int kQ8Tok = 8;                        // tokens per block
constexpr int kQ8Half = kQ8Tok * kD;             // codes of a block's K (or V) in one group
constexpr int kQ8Blk = 2 * kQ8Half;              // codes of a (block, group)
constexpr int kQ8MinExp = -100;                  // smallest scale 2^-100: a block of zeros, or of values below 448 * 2^-100
constexpr int kAppendWarps = 8;

// ---------------------------------------------------------------------------
// Append: quantise the K/V rows of positions [pos0, pos0 + n).  One warp takes
// the eight rows of one (sequence, block, K or V, group): lane 4 r + c holds
// the 16-element pieces c, c + 4, c + 8 of row r, so a row's four lanes read
// 128 contiguous bytes and write 64.  A block that was begun by an earlier
// call takes its older rows from `tail` (the rows themselves, in BF16) and is
// quantised again from them: the codes do not depend on how the tokens were
// cut into calls.  Rows that do not exist yet get code 0.  The warp of the
// call's first block also leaves the rows of the incomplete last block in
// `tail`; each lane has read its own pieces of the old rows by then.
// A block that holds an infinity or NaN gets scale NaN and codes 0: whoever
// attends it reads NaN, nobody else is touched.
// Bound: HBM, 2 bytes read and 1 written per element.  Measured, in a CUDA graph:
// 8192 tokens 8.0 us (4.7 TB/s; 5.8 us at the copy rate), 3 x 1001 tokens 4.0 us,
// 16 sequences x 1 token 2.7 us (launch); the call from Python takes 8 to 11 us of
// host time in all three.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kAppendWarps * 32)
kv_append_q8_kernel(const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                    __nv_bfloat16* __restrict__ tail, uint8_t* __restrict__ kv8, float* __restrict__ kv_scale,
                    int64_t pos0, int64_t n, int G, int64_t blocks, int64_t nb, int64_t units) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int g = static_cast<int>(unit % G);
  const int x = static_cast<int>((unit / G) & 1);  // 0: K, 1: V
  const int64_t j = (unit / (2 * G)) % nb;         // block of the call
  const int64_t seq = unit / (2 * G * nb);
  const int row = lane >> 2, c = lane & 3;
  const int64_t first = pos0 / kQ8Tok, end = pos0 + n;
  const int64_t tok = (first + j) * kQ8Tok + row;
  const __nv_bfloat16* src = x ? v : k;
  // rows of tail: [S, 2, 8, G, D]
  uint4* trow = reinterpret_cast<uint4*>(tail + (((seq * 2 + x) * kQ8Tok + row) * G + g) * static_cast<int64_t>(kD));
  uint4 w[3][2];
  {
    const uint4* p = nullptr;
    if (tok < pos0) p = trow;
    else if (tok < end) p = reinterpret_cast<const uint4*>(src + ((seq * n + tok - pos0) * G + g) * kD);
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[i][h] = p != nullptr ? p[2 * (c + 4 * i) + h] : make_uint4(0u, 0u, 0u, 0u);
  }
  uint32_t top = 0;  // two running maxima of the magnitudes' bits
#pragma unroll
  for (int i = 0; i < 3; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a[4] = {w[i][h].x, w[i][h].y, w[i][h].z, w[i][h].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) top = __vmaxu2(top, a[e] & 0x7FFF7FFFu);
    }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
  const uint32_t amax = max(top & 0xFFFFu, top >> 16);  // BF16 bits
  const bool finite = amax < 0x7F80u;
  // smallest e with amax <= 1.75 * 2^8 * 2^e
  const int e = max(static_cast<int>(amax >> 7) - 127 - 8 + ((amax & 0x7Fu) > 0x60u ? 1 : 0), kQ8MinExp);
  const float inv = finite ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 0.f;
  const int64_t bg = (seq * blocks + first + j) * G + g;
  uint8_t* dst = kv8 + bg * kQ8Blk + x * kQ8Half + row * kD;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    uint32_t o[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a[4] = {w[i][h].x, w[i][h].y, w[i][h].z, w[i][h].w};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float2 f0 = make_float2(__uint_as_float(a[2 * q] << 16) * inv, __uint_as_float(a[2 * q] & 0xFFFF0000u) * inv);
        const float2 f1 = make_float2(__uint_as_float(a[2 * q + 1] << 16) * inv,
                                      __uint_as_float(a[2 * q + 1] & 0xFFFF0000u) * inv);
        o[2 * h + q] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(f0, __NV_SATFINITE, __NV_E4M3)) |
                       (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(f1, __NV_SATFINITE, __NV_E4M3)) << 16);
      }
    }
    if (!finite) o[0] = o[1] = o[2] = o[3] = 0u;
    *reinterpret_cast<uint4*>(dst + 16 * (c + 4 * i)) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (lane == 0) kv_scale[bg * 2 + x] = finite ? __uint_as_float(static_cast<uint32_t>(127 + e) << 23) : __uint_as_float(0x7FC00000u);
  if (j == 0 && end % kQ8Tok != 0) {
    const int64_t tt = (end / kQ8Tok) * kQ8Tok + row;
    if (tt >= pos0 && tt < end) {
      const uint4* p = reinterpret_cast<const uint4*>(src + ((seq * n + tt - pos0) * G + g) * kD);
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) trow[2 * (c + 4 * i) + h] = p[2 * (c + 4 * i) + h];
    }
  }
}

// One unit of an accumulated attention weight (integer sums: the order of the
// additions cannot change them).
constexpr float kAccUnits = 4294967296.f;  // 2^32
__device__ __forceinline__ void acc_add(int64_t* acc, float w) {
  if (w == w)  // NaN weights (a block with NaN was attended) are not counted
    atomicAdd(reinterpret_cast<unsigned long long*>(acc), static_cast<unsigned long long>(__float2ll_rn(w * kAccUnits)));
}

}  // namespace sgqa
