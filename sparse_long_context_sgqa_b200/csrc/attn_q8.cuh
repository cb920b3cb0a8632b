// Sparse attention over the 8-bit K/V cache (layout: kv8.cuh) on the tcgen05
// tensor cores.  The scores take the E4M3 codes of K as they lie; few queries take
// those of V so too, many queries widen V.
//
// A query is not rounded to 8 bits: it is split into two E4M3 values, x = hi +
// lo / 16 with hi = E4M3(x), lo = E4M3(16 (x - hi)), which carry a BF16 value (8
// significant bits) exactly down to 2^-13.8 of the row's largest; below, a value
// is off by at most 2^-21.8 of that (many queries: see there).  Softmax
// weights need more range than E4M3 has: where one token takes most of a row (a
// sink), the result lies in weights 2^-14 of the largest and below.  Few queries
// split them into three E5M2 values (2^-9 of a weight, in FP16's range), many
// queries take FP16 weights and V widened to FP16.  The parts of a value are MMA
// columns (or MMA steps) side by side, so K or V is read once for all.  With one
// scale per (block, group), a block's K scale multiplies its scores and its V
// scale its weights.
//
// Softmax reference.  The weights that enter the MMA are 2^(s - ref) vs: the
// reference follows the scores plus the exponent of the V scale, so that blocks
// of small values keep their bits where they carry the result.  The sum of the
// weights, FP32, uses the same reference without the V scale.
#pragma once
#include <cooperative_groups.h>

#include "kv8.cuh"
#include "tc.cuh"

namespace sgqa {

// Byte offset of byte c (0..63) of row r in tiles of 64-byte rows (512-byte atoms).
__device__ __forceinline__ uint32_t sw64_offset(uint32_t r, uint32_t c) {
  const uint32_t a = r * 64u + c;
  return a ^ (((a >> 7) & 3u) << 4);
}

// Exponent e of the smallest power of two with amax / 2^e <= 448 (amax > 0
// finite or zero; at least kQ8MinExp).
__device__ __forceinline__ int e4m3_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  return max(static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0), kQ8MinExp);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {  // a in the low byte
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t v) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v & 0xFFFFu), __NV_E4M3);
  return __half22float2(__half2(h));
}
// Two weights as three E5M2 values each, x = c0 + c1 / 8 + c2 / 64: every value
// takes three significant bits, the next one what is left.  In FP16 (11 bits,
// exact differences; an E5M2 code is the upper byte of an FP16 number).
__device__ __forceinline__ void split_e5m2(float a, float b, uint32_t (&c)[3]) {
  __half2 r = __floats2half2_rn(a, b);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    c[i] = static_cast<uint32_t>(__nv_cvt_halfraw2_to_fp8x2(r, __NV_SATFINITE, __NV_E5M2));
    if (i < 2) {
      const uint32_t v = __byte_perm(c[i], 0u, 0x1404);  // bytes 0, 1 into the upper halves' high bytes
      r = __hmul2(__hsub2(r, *reinterpret_cast<const __half2*>(&v)), __float2half2_rn(8.f));
    }
  }
}
// hi and 16 x lo codes of two values (low 16 bits each).
__device__ __forceinline__ void split_e4m3(float a, float b, uint32_t& hi, uint32_t& lo, float lo_scale) {
  hi = e4m3x2(a, b);
  const float2 h = e4m3x2_value(hi);
  lo = e4m3x2((a - h.x) * lo_scale, (b - h.y) * lo_scale);
}

// ---------------------------------------------------------------------------
// Few queries (decode): an HBM-bound gather.  One CTA takes a range of one
// (query, group)'s blocks (split-K), 16 blocks = 128 tokens at a time, and
// computes transposed, so that the 16 heads are the narrow MMA side:
//   S^T [128 tokens x 32] = K [128 x 192] Q^T     6 MMAs (M128 N32 K32): columns
//                           16 heads' hi | 16 heads' lo; K as gathered (K-major)
//   softmax               one thread per token and half of the heads
//   O^T [192 dims x 48] += V^T [192 x 128] P^T    2 x 4 MMAs (M128 N48 K32): V as
//                           gathered (MN-major), dims 0-127 and 64-191 (the rows
//                           computed twice are not read); P through shared memory,
//                           columns 16 heads' first, second and third E5M2 values
// A token's scores never cross threads for a maximum: the reference moves only
// when some weight exceeds 2^14 (one barrier-or per tile tells), and only then
// are a head's maxima reduced over the tile and O rescaled in TMEM.
// K and V are gathered by a warp each (16 lanes, one 1.5 KB box per block) into
// rings of their own: a K stage is free again after its MMA, a V stage only
// after the softmax of its tile.  The splits of a row form one cluster and
// combine through distributed shared memory.
// Measured, in a CUDA graph: 16 contexts of 262144 tokens, 512 blocks each, 28.0 us
// (the bytes at the copy rate: 15.5 us), 16 x 32768 with gate and weights 32.0 us,
// one query at position 1024 8.8 us.  Of the last little is bytes: lists, scales,
// gather, two products and combine follow one another.
// ---------------------------------------------------------------------------
constexpr int kQdTile = 16;       // blocks per tile
constexpr int kQdStages = 2;      // of K and of V
constexpr int kQdMeta = 8;        // tiles whose scales and masks are held
constexpr int kQdThreads = 384;   // K and V producers, QK and PV issuers, 8 softmax warps
constexpr int kQdS = 4;           // score buffers: the QK issuer runs ahead, so that K stages are free early
constexpr int kQdCols = 256;      // TMEM: S 4 x 32, O 2 x 64 (48 used)
constexpr int kQdMaxSplit = 8;    // splits of a row = one (portable) cluster
constexpr int kQdStage = kQdTile * kQ8Half;  // bytes of a stage

struct __align__(512) QdSmem {
  uint8_t k[kQdStages][kQdTile][3][8][64];    // [block][chunk of 64 dims][8 rows][64 B], 64-byte swizzle
  uint8_t v[kQdStages][kQdTile][3][8][64];
  uint8_t q[3][32][64];                       // [chunk][16 hi, 16 lo][64 B], 64-byte swizzle
  uint8_t p[kQdTile * kQ8Tok][64];            // [token][16 first, 16 second, 16 third values, unused], 64-byte swizzle
  float2 scale[kQdMeta][kQdTile];             // a tile's blocks: K scale, V scale
  int32_t mask[kQdMeta][kQdTile];             // attended tokens (bits 0-7), floor(log2(V scale)) above them
  float wmax[4][kHg];                         // a reference change: maxima of the four lane quadrants
  float qscale[kHg];
  uint64_t k_full[kQdStages], k_empty[kQdStages], v_full[kQdStages], v_empty[kQdStages], meta_full[kQdMeta];
  uint64_t s_full[kQdS], s_free[kQdS], p_full, pv_done, q_full, o_final, drain[2];
  uint32_t tmem;
  int abort;
};

constexpr int kQdOStride = kD + 2;
// The combine's view of the K ring, once the last MMA is done.
struct QdOut {
  float m[kHg];                    // this split's reference
  float f[kQdMaxSplit][kHg], lr[kQdMaxSplit][kHg];  // every split's, then its factor
  float fin[kHg], wfac[kHg];       // normalisation (and gate); weight normalisation
  float mu[kHg];                   // the splits' common reference
  float wl[4][kHg];                // and its sums by lane quadrant
  float o[kHg][kQdOStride];
};
static_assert(sizeof(QdOut) <= kQdStages * kQdStage, "the combine fits the K ring");

// Workspace of the weights: per (row, block of the row) 16 heads' sums, then per
// (row, tile) the references they refer to.
struct QdWeights {
  int64_t* acc;   // nullptr: not wanted
  float* sums;    // [rows, k + 1, 16]
  float* refs;    // [rows, tiles, 16]
  int tiles;      // per row (nsplit x tiles of a split)
};

template <bool WEIGHTS>
__global__ void __launch_bounds__(kQdThreads, 2)
attn_q8_decode_kernel(const __grid_constant__ CUtensorMap kvmap, const __nv_bfloat16* __restrict__ q,
                      const float* __restrict__ kv_scale, const int32_t* __restrict__ sel,
                      const int32_t* __restrict__ sel_count, const __nv_bfloat16* __restrict__ gate,
                      __nv_bfloat16* __restrict__ out, QdWeights wts, int64_t nq, int G, int k, int64_t q_pos0,
                      int64_t blocks, int nsplit, float scale_log2) {
  extern __shared__ uint8_t smem_raw[];
  QdSmem& sm = *reinterpret_cast<QdSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 511) & ~static_cast<uintptr_t>(511));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % nsplit;
  const int64_t row = blockIdx.x / nsplit;  // (seq * nq + i) * G + g
  const int g = static_cast<int>(row % G);
  const int64_t i = (row / G) % nq;
  const int64_t seq = row / (G * nq);
  const int64_t t = q_pos0 + i, hist = t / kQ8Tok;
  const int32_t* ids = sel + row * k;
  // Positions [0, kh) are the list's (kh: the longest it can be; positions from
  // the count on are empty), position kh is the current block.  The split does
  // not wait for the count.
  const int kh = static_cast<int>(min(static_cast<int64_t>(k), hist));
  const int per = (kh + nsplit) / nsplit;
  const int b0 = min(kh + 1, split * per), b1 = min(kh + 1, b0 + per);
  const int n_tiles = (b1 - b0 + kQdTile - 1) / kQdTile;
  volatile int* abort = &sm.abort;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  // block at position b: -1 none, -2 an id that breaks the contract
  auto block_at = [&](int b, int cnt, int id, int prev) -> int32_t {
    if (b >= b1) return -1;
    if (b == kh) return static_cast<int32_t>(hist);
    if (b >= cnt) return -1;
    return id < 0 || id >= hist || id <= prev ? -2 : id;
  };
  int issued = 0;  // producers: tiles whose copies this warp issued
  const bool is_k = warp == 0;
  // ids and their predecessors are fetched two tiles ahead, scales one
  int id2 = -1, prev2 = -1, cnt = 0;
  int32_t blk = -1;
  float2 sc = make_float2(0.f, 1.f);
  auto fetch = [&](int j, int& id, int& prev) {
    const int b = b0 + j * kQdTile + lane;
    id = prev = -1;
    if (lane < kQdTile && b < min(b1, kh)) {
      id = __ldg(ids + b);
      if (b > 0) prev = __ldg(ids + b - 1);
    }
  };
  auto resolve = [&](int j, int id, int prev) -> int32_t {
    const int32_t r = block_at(lane < kQdTile ? b0 + j * kQdTile + lane : b1, cnt, id, prev);
    if (r == -2 && is_k) report(kDevBounds);
    return r;
  };
  auto scales = [&](int32_t x) -> float2 {
    return is_k && x >= 0 ? __ldg(reinterpret_cast<const float2*>(kv_scale) + (seq * blocks + x) * G + g)
                          : make_float2(0.f, 1.f);
  };
  auto copy = [&](int s) {  // this lane's block into stage s; no block: a box outside the cache, filled with zeros
    const uint32_t full = bar(is_k ? sm.k_full[s] : sm.v_full[s]);
    tc::mbar_expect_tx(full, kQ8Half);
    tc::tma_load_5d(smem_u32(is_k ? &sm.k[s][lane][0][0][0] : &sm.v[s][lane][0][0][0]), &kvmap, 0, is_k ? 0 : kQ8Tok, 0,
                    blk >= 0 ? g : 0, blk >= 0 ? static_cast<int32_t>(seq * blocks + blk) : -1, full);
  };
  if (warp == 0 || warp == 11) {
    // Each producer sets up its own barriers and sends its first tile off before
    // the CTA-wide set-up is through.
    int id1, prev1;
    fetch(0, id1, prev1);
    fetch(1, id2, prev2);
    cnt = min(max(__ldg(sel_count + row), 0), k);
    if (lane == 0) {
      tc::prefetch_tmap(&kvmap);
      for (int s = 0; s < kQdStages; ++s) {
        tc::mbar_init(bar(is_k ? sm.k_full[s] : sm.v_full[s]), kQdTile);
        tc::mbar_init(bar(is_k ? sm.k_empty[s] : sm.v_empty[s]), 1);
      }
      if (is_k)
        for (int s = 0; s < kQdMeta; ++s) tc::mbar_init(bar(sm.meta_full[s]), kQdTile);
      tc::mbar_fence_init();
    }
    __syncwarp();
    blk = resolve(0, id1, prev1);
    sc = scales(blk);
    if (n_tiles > 0) {
      if (lane < kQdTile) copy(0);
      issued = 1;
    }
    __syncwarp();
  } else if (warp == 1) {
    tc::tmem_alloc(smem_u32(&sm.tmem), kQdCols);
  } else if (warp == 10) {
    if (lane == 0) {
      sm.abort = 0;
      for (int b = 0; b < kQdS; ++b) {
        tc::mbar_init(bar(sm.s_full[b]), 1);
        tc::mbar_init(bar(sm.s_free[b]), 256);
      }
      for (int b = 0; b < 2; ++b) tc::mbar_init(bar(sm.drain[b]), 1);
      tc::mbar_init(bar(sm.p_full), 256);
      tc::mbar_init(bar(sm.pv_done), 1);
      tc::mbar_init(bar(sm.q_full), 256);
      tc::mbar_init(bar(sm.o_final), 1);
      tc::mbar_fence_init();
    }
    __syncwarp();
  }
  // the softmax warps' queries: a warp packs two heads, a lane dims 2 lane and
  // 2 lane + 1 of every chunk
  uint32_t qw[2][3];
  const int qh = 2 * (warp - 2);
  if (warp >= 2 && warp <= 9) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
      for (int c = 0; c < 3; ++c) qw[hh][c] = __ldg(reinterpret_cast<const uint32_t*>(q + (row * kHg + qh + hh) * kD) + 32 * c + lane);
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tS = sm.tmem, tO = sm.tmem + 32 * kQdS;

  // per-head state of the softmax threads
  float ref[8], l[8];
#pragma unroll
  for (int h = 0; h < 8; ++h) { ref[h] = -INFINITY; l[h] = 0.f; }

  if (warp == 0 || warp == 11) {
    // ---------------------------------------------------------------- producers
    for (int j = 0; j < n_tiles; ++j) {
      const int s = j % kQdStages;
      if (j >= kQdStages && !tc::warp_wait(bar(is_k ? sm.k_empty[s] : sm.v_empty[s]), ((j / kQdStages) - 1) & 1, abort)) break;
      if (lane < kQdTile) {
        if (j > 0) copy(s);
        if (is_k) {
          const int32_t m = blk < 0 ? 0 : blk == hist ? (2 << (t % kQ8Tok)) - 1 : 0xFF;
          const int32_t e = blk < 0 || !isfinite(sc.y) ? 0 : static_cast<int32_t>(__float_as_uint(sc.y) >> 23) - 127;
          sm.scale[j % kQdMeta][lane] = make_float2(sc.x, blk < 0 ? 0.f : sc.y);
          sm.mask[j % kQdMeta][lane] = e * 256 + m;
          tc::mbar_arrive(bar(sm.meta_full[j % kQdMeta]));
        }
      }
      __syncwarp();
      issued = j + 1;
      blk = resolve(j + 1, id2, prev2);
      sc = scales(blk);
      fetch(j + 2, id2, prev2);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- S^T = K Q^T
    const uint32_t id_qk = tc::idesc_e4m3(128, 32, false, false);
    const uint64_t dk0 = tc::sdesc(smem_u32(&sm.k[0][0][0][0][0]), 16, kQ8Half, tc::kSw64);
    const uint64_t dq0 = tc::sdesc(smem_u32(&sm.q[0][0][0]), 16, 512, tc::kSw64);
    bool ok = tc::warp_wait(bar(sm.q_full), 0, abort);
    for (int j = 0; ok && j < n_tiles; ++j) {
      const int s = j % kQdStages, b = j % kQdS;
      ok = tc::warp_wait(bar(sm.k_full[s]), (j / kQdStages) & 1, abort);
      if (ok && j >= kQdS) ok = tc::warp_wait(bar(sm.s_free[b]), ((j / kQdS) - 1) & 1, abort);
      if (!ok) break;
      tc::fence_after();
      if (tc::elect_one()) {
        const uint64_t dk = dk0 + (kQdStage / 16) * s;
#pragma unroll
        for (int kk = 0; kk < 6; ++kk)  // K: +512 B per 64 dims; Q: +2 KB; both +32 B per 32 dims
          tc::mma_f8(tS + 32 * b, dk + (kk >> 1) * 32 + (kk & 1) * 2, dq0 + (kk >> 1) * 128 + (kk & 1) * 2, id_qk,
                     kk > 0 ? 1u : 0u);
        tc::mma_commit(bar(sm.s_full[b]));
        tc::mma_commit(bar(sm.k_empty[s]));
      }
      __syncwarp();
    }
  } else if (warp == 10) {
    // ---------------------------------------------------------------- O^T += V^T P^T
    const uint32_t id_pv = tc::idesc_e4m3_e5m2(128, 48, true, true);
    // V: 64-dim chunks 512 B apart, 8-token groups one block apart; P: 8-token groups 512 B apart
    const uint64_t dv0 = tc::sdesc(smem_u32(&sm.v[0][0][0][0][0]), 512, kQ8Half, tc::kSw64);
    const uint64_t dp = tc::sdesc(smem_u32(&sm.p[0][0]), 512, 512, tc::kSw64);
    bool ok = true;
    for (int j = 0; ok && j < n_tiles; ++j) {
      const int s = j % kQdStages;
      ok = tc::warp_wait(bar(sm.v_full[s]), (j / kQdStages) & 1, abort) && tc::warp_wait(bar(sm.p_full), j & 1, abort);
      if (!ok) break;
      tc::fence_after();
      if (tc::elect_one()) {
        const uint64_t dv = dv0 + (kQdStage / 16) * s;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {  // 32 tokens: V +4 blocks, P +2 KB
          const uint32_t acc = (j > 0 || kk > 0) ? 1u : 0u;
          tc::mma_f8(tO, dv + kk * (4 * kQ8Half / 16), dp + kk * 128, id_pv, acc);
          tc::mma_f8(tO + 64, dv + 32 + kk * (4 * kQ8Half / 16), dp + kk * 128, id_pv, acc);
        }
        tc::mma_commit(bar(sm.v_empty[s]));
        tc::mma_commit(bar(sm.pv_done));
        if (j + 1 == n_tiles) tc::mma_commit(bar(sm.o_final));
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- softmax
    // Warps 2-5 take heads 0-7, warps 6-9 heads 8-15; the four warps of a half
    // (one per TMEM lane quadrant) agree on its references by a barrier of their own.
    const int sw = warp - 2, quad = warp & 3, half = sw >> 2, h0 = 8 * half, hbar = 1 + half;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const int tok = quad * 32 + lane;  // token of the tile = TMEM lane
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int h = qh + hh;
      float x[3][2], mx = 0.f;
      bool fin = true;
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const uint32_t w = qw[hh][c];
        x[c][0] = __uint_as_float(w << 16);
        x[c][1] = __uint_as_float(w & 0xFFFF0000u);
        fin = fin && isfinite(x[c][0]) && isfinite(x[c][1]);
        mx = fmaxf(mx, fmaxf(fabsf(x[c][0]), fabsf(x[c][1])));
      }
      mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
      fin = __all_sync(0xffffffffu, fin);
      const int e = fin ? e4m3_exp(mx) : 0;
      const float inv = pow2f(-e);
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        uint32_t hi, lo;
        split_e4m3(x[c][0] * inv, x[c][1] * inv, hi, lo, 16.f);
        *reinterpret_cast<uint16_t*>(&sm.q[c][0][0] + sw64_offset(h, 2 * lane)) = static_cast<uint16_t>(hi);
        *reinterpret_cast<uint16_t*>(&sm.q[c][0][0] + sw64_offset(16 + h, 2 * lane)) = static_cast<uint16_t>(lo);
      }
      // a query with an infinity or NaN: every score NaN
      if (lane == 0) sm.qscale[h] = fin ? pow2f(e) * scale_log2 : __uint_as_float(0x7FC00000u);
    }
    tc::fence_proxy_async_smem();
    tc::mbar_arrive(bar(sm.q_full));
    asm volatile("bar.sync %0, 128;" ::"r"(hbar) : "memory");
    float rc[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) rc[h] = sm.qscale[h0 + h];
    bool ok = true;
    for (int j = 0; j < n_tiles; ++j) {
      const int sb = j % kQdS;
      ok = ok && tc::mbar_wait(bar(sm.meta_full[j % kQdMeta]), (j / kQdMeta) & 1, abort);
      const float2 sc = sm.scale[j % kQdMeta][tok >> 3];
      const int32_t msk = sm.mask[j % kQdMeta][tok >> 3];
      const bool use = (msk >> (tok & 7)) & 1;
      const float lvs = static_cast<float>(msk >> 8);
      ok = ok && tc::mbar_wait(bar(sm.s_full[sb]), (j / kQdS) & 1, abort);
      tc::fence_after();
      uint32_t sh[8], sl[8];
      tc::tmem_ld8(tS + 32 * sb + lane_off + h0, sh);
      tc::tmem_ld8(tS + 32 * sb + lane_off + 16 + h0, sl);
      tc::tmem_ld_wait();
      tc::fence_before();
      tc::mbar_arrive(bar(sm.s_free[sb]));
      float x[8];
      bool grow = false;
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const float v = fmaf(__uint_as_float(sl[h]), 0.0625f, __uint_as_float(sh[h])) * (sc.x * rc[h]);
        x[h] = use ? v : -INFINITY;
        grow = grow || x[h] + lvs > ref[h] + 14.f;
      }
      // does any weight of the tile exceed 2^14?  (2^15 with a V scale between two
      // powers of two: still in FP16's range)
      int any;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n selp.s32 %0, 1, 0, q;\n}"
          : "=r"(any)
          : "r"(static_cast<int>(grow)), "r"(hbar)
          : "memory");
      if (any) {
        // new references: the largest score (plus log2 of its V scale) - 4, so that
        // they stay until the scores grow by 2^10
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const int v = __float_as_int(fmaxf(x[h] + lvs, -INFINITY));
          const int mx = __reduce_max_sync(0xffffffffu, v ^ ((v >> 31) & 0x7FFFFFFF));
          if (lane == 0) sm.wmax[quad][h0 + h] = __int_as_float(mx ^ ((mx >> 31) & 0x7FFFFFFF));
        }
        asm volatile("bar.sync %0, 128;" ::"r"(hbar) : "memory");
        float al[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const float mx = fmaxf(fmaxf(sm.wmax[0][h0 + h], sm.wmax[1][h0 + h]), fmaxf(sm.wmax[2][h0 + h], sm.wmax[3][h0 + h]));
          const float nr = mx > ref[h] + 14.f ? mx - 4.f : ref[h];
          al[h] = nr == ref[h] ? 1.f : exp2f(ref[h] - nr);
          ref[h] = nr;
          l[h] *= al[h];
        }
        if (j > 0) {  // O holds P(j-1) V(j-1) by then
          ok = ok && tc::mbar_wait(bar(sm.pv_done), (j - 1) & 1, abort);
          tc::fence_after();
#pragma unroll 1
          for (int part = 0; part < 6; ++part) {  // dims 0-127, 64-191; the three values' columns
            uint32_t o[8];
            const uint32_t at = tO + 64 * (part / 3) + 16 * (part % 3) + h0 + lane_off;
            tc::tmem_ld8(at, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int h = 0; h < 8; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * al[h]);
            tc::tmem_st8(at, o);
          }
          tc::tmem_st_wait();
        }
      }
      uint32_t p3[3][2];  // the three values of 8 heads
#pragma unroll
      for (int h = 0; h < 8; h += 2) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[h + e] = fast_exp2(x[h + e] - (ref[h + e] == -INFINITY ? 0.f : ref[h + e]));
          l[h + e] += x[h + e];
        }
        uint32_t c[3];
        split_e5m2(x[h] * sc.y, x[h + 1] * sc.y, c);
#pragma unroll
        for (int i = 0; i < 3; ++i) p3[i][h >> 2] = (h & 2) ? p3[i][h >> 2] | (c[i] << 16) : c[i];
      }
      // P is free once O += P(j-1) V(j-1) has read it
      if (j >= 1) ok = ok && tc::mbar_wait(bar(sm.pv_done), (j - 1) & 1, abort);
#pragma unroll
      for (int i = 0; i < 3; ++i)
        *reinterpret_cast<uint2*>(&sm.p[0][0] + sw64_offset(tok, 16 * i + h0)) = make_uint2(p3[i][0], p3[i][1]);
      tc::fence_proxy_async_smem();
      tc::fence_before();
      tc::mbar_arrive(bar(sm.p_full));
      if (WEIGHTS) {
        // sums over the block's eight tokens (lanes): every exchange halves the
        // heads a lane holds; lane r of a block ends with head r
        float y[4], z[2];
        const bool h4 = lane & 4, h2 = lane & 2, h1 = lane & 1;
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = (h4 ? x[4 + c] : x[c]) + __shfl_xor_sync(0xffffffffu, h4 ? x[c] : x[4 + c], 4);
#pragma unroll
        for (int c = 0; c < 2; ++c) z[c] = (h2 ? y[2 + c] : y[c]) + __shfl_xor_sync(0xffffffffu, h2 ? y[c] : y[2 + c], 2);
        const float w = (h1 ? z[1] : z[0]) + __shfl_xor_sync(0xffffffffu, h1 ? z[0] : z[1], 1);
        const int blk = b0 + j * kQdTile + (tok >> 3);
        if (blk < b1) wts.sums[(row * (k + 1) + blk) * kHg + h0 + (lane & 7)] = w;
        if (tok == 0) {
          float* r = wts.refs + (row * wts.tiles + split * (wts.tiles / nsplit) + j) * kHg + h0;
#pragma unroll
          for (int h = 0; h < 8; ++h) r[h] = ref[h];
        }
      }
    }
    // the threads' sums, while the last product runs (the wait below covers it)
#pragma unroll
    for (int h = 0; h < 8; ++h) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
    }
    if (n_tiles > 0) ok = ok && tc::mbar_wait(bar(sm.o_final), 0, abort);
  }
  // Every role has left its loop, so the abort flag is final; on the failure
  // path the copies and MMAs in flight land before their memory is reused.
  __syncthreads();
  if (sm.abort) {
    if (warp == 0 || warp == 11) {
      for (int j = max(issued - kQdStages, 0); j < issued; ++j)
        tc::mbar_drain(bar(warp == 0 ? sm.k_full[j % kQdStages] : sm.v_full[j % kQdStages]), (j / kQdStages) & 1);
    } else if (warp == 1 || warp == 10) {
      uint64_t& d = sm.drain[warp == 1 ? 0 : 1];
      if (tc::elect_one()) tc::mma_commit(bar(d));
      __syncwarp();
      tc::mbar_drain(bar(d), 0);
    }
    __syncthreads();
  }
  QdOut& po = *reinterpret_cast<QdOut*>(&sm.k[0][0][0][0][0]);
  if (warp >= 2 && warp <= 9) {
    const int quad = warp & 3, h0 = 8 * ((warp - 2) >> 2);
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    if (n_tiles > 0) {
      tc::fence_after();
      const int d = quad * 32 + lane;
      const int parts = quad >= 2 ? 2 : 1;  // dims 0-127; of 64-191 the upper half
      for (int part = 0; part < parts; ++part) {
        uint32_t c0[8], c1[8], c2[8];
        tc::tmem_ld8(tO + 64 * part + h0 + lane_off, c0);
        tc::tmem_ld8(tO + 64 * part + 16 + h0 + lane_off, c1);
        tc::tmem_ld8(tO + 64 * part + 32 + h0 + lane_off, c2);
        tc::tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < 8; ++h)
          po.o[h0 + h][64 * part + d] = fmaf(fmaf(__uint_as_float(c2[h]), 0.125f, __uint_as_float(c1[h])), 0.125f, __uint_as_float(c0[h]));
      }
    } else {
      for (int x = threadIdx.x - 64; x < kHg * kQdOStride; x += 256) (&po.o[0][0])[x] = 0.f;
    }
    if (lane == 0) {
      // a split that gave up has no sums: NaN makes the whole row NaN and keeps its
      // weights out of acc, which outlives the call
      const bool gave_up = sm.abort != 0;
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        po.wl[quad][h0 + h] = gave_up ? __uint_as_float(0x7FC00000u) : l[h];
        if (quad == 0) po.m[h0 + h] = ref[h];
      }
    }
    tc::fence_before();
  }
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  if (warp == 1) {
    tc::fence_after();
    tc::tmem_dealloc(sm.tmem, kQdCols);
  }
  // This split finalises pairs [split * n, split * n + n) of the row's 16 x 96
  // pairs of outputs.  Every remote read of a step is issued before the first
  // is used: one trip through the cluster for the references, one for O.
  const int n = (kHg * kD / 2 + nsplit - 1) / nsplit;
  const int i1 = min(kHg * kD / 2, split * n + n);
  float2 part[kQdMaxSplit];
  auto read_parts = [&](int x) {
    const int h = x / (kD / 2), d = 2 * (x - h * (kD / 2));
#pragma unroll
    for (int r = 0; r < kQdMaxSplit; ++r)
      if (r < nsplit) part[r] = *reinterpret_cast<const float2*>(cluster.map_shared_rank(&po.o[h][d], r));
  };
  if (static_cast<int>(threadIdx.x) < nsplit * kHg) {
    const int r = threadIdx.x / kHg, h = threadIdx.x % kHg;
    const QdOut* other = cluster.map_shared_rank(&po, r);
    const float m = other->m[h], w0 = other->wl[0][h], w1 = other->wl[1][h], w2 = other->wl[2][h], w3 = other->wl[3][h];
    po.f[r][h] = m;
    po.lr[r][h] = (w0 + w1) + (w2 + w3);
  }
  const int x0 = split * n + threadIdx.x;
  if (x0 < i1) read_parts(x0);
  __syncthreads();
  if (threadIdx.x < kHg) {
    const int h = threadIdx.x;
    float mm = -INFINITY;
    for (int r = 0; r < nsplit; ++r) mm = fmaxf(mm, po.f[r][h]);
    const float mu = mm == -INFINITY ? 0.f : mm;
    float ls = 0.f;
    for (int r = 0; r < nsplit; ++r) {
      const float a = exp2f(po.f[r][h] - mu);
      po.f[r][h] = a;
      ls += po.lr[r][h] == 0.f ? 0.f : a * po.lr[r][h];
    }
    po.fin[h] = gate_factor(gate, row * kHg + h) / ls;
    po.wfac[h] = 1.f / ls;  // a weight sum with reference r counts 2^(r - mu) / ls
    po.mu[h] = mu;
  }
  __syncthreads();
  for (int x = x0; x < i1; x += kQdThreads) {
    if (x != x0) read_parts(x);
    const int h = x / (kD / 2);
    float2 a = make_float2(0.f, 0.f);
#pragma unroll
    for (int r = 0; r < kQdMaxSplit; ++r)
      if (r < nsplit) {
        a.x = fmaf(po.f[r][h], part[r].x, a.x);
        a.y = fmaf(po.f[r][h], part[r].y, a.y);
      }
    reinterpret_cast<uint32_t*>(out)[row * (kHg * kD / 2) + x] = pack_bf16x2(a.x * po.fin[h], a.y * po.fin[h]);
  }
  if (WEIGHTS) {
    const int n_cnt = min(max(sel_count[row], 0), k);
    for (int x = threadIdx.x; x < b1 - b0; x += kQdThreads) {
      const int b = b0 + x;
      const int32_t blk = block_at(b, n_cnt, b < kh ? ids[b] : 0, b > 0 && b < kh ? ids[b - 1] : -1);
      if (blk < 0) continue;
      const float* ws = wts.sums + (row * (k + 1) + b) * kHg;
      const float* rs = wts.refs + (row * wts.tiles + split * (wts.tiles / nsplit) + x / kQdTile) * kHg;
      float w = 0.f;
#pragma unroll
      for (int h = 0; h < kHg; ++h) {
        const float v = ws[h];
        const float u = v == 0.f ? 0.f : v * exp2f((rs[h] == -INFINITY ? 0.f : rs[h]) - po.mu[h]) * po.wfac[h];
        w += u == u ? u : 0.f;  // NaN: not counted
      }
      acc_add(wts.acc + seq * blocks + blk, w);
    }
  }
  cluster.sync();  // no split leaves while others still read its shared memory
}

// ---------------------------------------------------------------------------
// Many queries (prefill).  The unit and the union of its queries' blocks are
// those of attn_tc_kernel (attn_tc.cuh): 8 adjacent queries x 16 heads = the 128 MMA rows, 64-token tiles of the union, then a
// tile with the current blocks.  What differs is the operands:
//   S = Q K^T   2 x 6 MMAs (E4M3, M128 N64 K32): Q's hi and lo halves from TMEM,
//               K's codes as gathered.  Twice the passes at twice the BF16 rate.
//   O += P V    4 MMAs (FP16, M128 N192 K16): P from TMEM, V's codes widened to
//               FP16 (exact) in shared memory by a warpgroup of its own.  P needs the
//               range of 16 bits: where one token takes most of a row (a sink), the
//               result lies in weights 2^-14 of the largest and below, which two
//               E4M3 halves in one accumulator lose.
// lo is not multiplied by 16 here (both halves add into one accumulator): a query
// value is exact down to 2^-9.8 of the row's largest, smaller ones are off by at
// most 2^-17.8 of it (half a step of the smallest E4M3 values, 2^-10, where the
// largest is just above 224).
// A block's K scale and the row's query scale multiply its scores; its V scale
// enters the exponent (2^(s + log2 vs - ref)) and leaves the block's sum again.
//
// WEIGHTS: the second sweep of a call that accumulates weights.  With every
// row's log-sum known, S alone is computed again, and each block's weights are
// summed over the unit's 128 rows, eight blocks of a tile at a time.
// Measured, in a CUDA graph with the plan of the unions: 2048 queries at 8192, 512
// blocks each, 553-564 us; 2 x 1001 queries with gate and weights 532 us.  Bound by
// the softmax warps' issue and latency: the tensor pipe is active 43% of the time.
// Sixteen softmax warps (575 us) and a maximum taken ahead of the exponentials (580
// us) were slower than this form in the same run (558 us).
// ---------------------------------------------------------------------------
constexpr int kQpStages = 8;      // K ring depth, 12 KB each
constexpr int kQpVStages = 4;     // V ring depth (codes)
constexpr int kQpThreads = 512;   // producers and issuers, V widening, 2 x softmax: a warpgroup each
constexpr int kQpTile = 8;        // blocks per tile
constexpr int kQpMeta = 4;        // batches (of 4 tiles) whose scales are held
// Registers: 512 x 128 at launch = 256 x 80 (the first two warpgroups) + 256 x 176 (softmax).
constexpr int kQpRegsFew = 80, kQpRegsMany = 176;

struct __align__(1024) QpSmem {
  uint8_t v16[2][kQpTile][3][1024];          // widened V: [block][chunk][8 rows x 128 B], 128-byte swizzle
  uint8_t k[kQpStages][kQpTile][3][8][64];   // [block][chunk][8 rows][64 B], 64-byte swizzle
  uint8_t v[kQpVStages][kQpTile][3][8][64];
  float4 meta[kQpMeta][32];                 // per block: K scale, log2(V scale), 1 / V scale (NaN scales as 0, 0, 1)
  float4 meta_cur[8];                       // of the current blocks (two are used)
  uint32_t meta_nan[kQpMeta + 1];           // batch (last: the current blocks): bit i: block i's K or V scale is NaN
  uint32_t meta_nan_k[kQpMeta + 1];         // its K scale is
  int32_t ids[kQpMeta][32];                 // WEIGHTS: the blocks
  uint64_t q_full;
  uint64_t k_full[kQpStages], k_empty[kQpStages], v_full[kQpVStages], v_empty[kQpVStages], meta_full[kQpMeta];
  uint64_t w_full[2], w_empty[2];           // widened V
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t o_final, drain, drain_pv;
  float mchain[128];                        // the rows' reference after the latest tile
  float lsum[2][128];                       // partial row sums of the two warps of a pair
  float gfac[128];
  uint32_t tmem;
  int abort;
};

template <bool WEIGHTS, bool SKIP_PAIRS>
__global__ void __launch_bounds__(kQpThreads, 1)
attn_q8_prefill_kernel(const __grid_constant__ CUtensorMap kvmap, const __nv_bfloat16* __restrict__ q,
                       const float* __restrict__ kv_scale, const int32_t* __restrict__ plan_ids,
                       const uint8_t* __restrict__ plan_mask, const int32_t* __restrict__ plan_count,
                       const __nv_bfloat16* __restrict__ gate, __nv_bfloat16* __restrict__ out, float* __restrict__ lse,
                       int64_t* __restrict__ acc, int64_t nq, int G, int k, int64_t q_pos0, int64_t blocks,
                       float scale_log2) {
  extern __shared__ uint8_t smem_raw[];
  QpSmem& sm = *reinterpret_cast<QpSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // group-major order: CTAs resident together read one group's K/V (L2 reuse)
  const int64_t nqb = (nq + 7) / 8;
  const int64_t per_group = static_cast<int64_t>(gridDim.x) / G;
  const int g = static_cast<int>(blockIdx.x / per_group);
  const int64_t sq = blockIdx.x % per_group;  // seq * nqb + qb
  const int64_t qb = sq % nqb;
  const int64_t seq = sq / nqb;
  const int64_t unit = sq * G + g;
  const int U = plan_count[unit];
  const int32_t* uid = plan_ids + unit * (8 * static_cast<int64_t>(k));
  const uint8_t* umask = plan_mask + unit * (8 * static_cast<int64_t>(k));
  const int n_union_tiles = (U + kQpTile - 1) / kQpTile;
  const int n_tiles = n_union_tiles + 1;
  const int64_t t_first = q_pos0 + qb * 8;
  const int64_t t_last = q_pos0 + min(nq, qb * 8 + 8) - 1;
  const int64_t cb = t_first / 8;  // the first query's current block
  const int64_t c0 = 8 * cb;
  volatile int* abort = &sm.abort;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  if (threadIdx.x == 0) {
    sm.abort = 0;
    tc::mbar_init(bar(sm.q_full), 256);
    for (int s = 0; s < kQpStages; ++s) {
      tc::mbar_init(bar(sm.k_full[s]), 1);
      tc::mbar_init(bar(sm.k_empty[s]), 1);
    }
    for (int s = 0; s < kQpVStages; ++s) {
      tc::mbar_init(bar(sm.v_full[s]), 1);
      tc::mbar_init(bar(sm.v_empty[s]), 128);
    }
    for (int b = 0; b < kQpMeta; ++b) tc::mbar_init(bar(sm.meta_full[b]), 32);
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(bar(sm.s_full[b]), 1);
      tc::mbar_init(bar(sm.s_free[b]), 128);
      tc::mbar_init(bar(sm.p_full[b]), 128);
      tc::mbar_init(bar(sm.pv_done[b]), 1);
      tc::mbar_init(bar(sm.w_full[b]), 128);
      tc::mbar_init(bar(sm.w_empty[b]), 1);
    }
    tc::mbar_init(bar(sm.o_final), 1);
    tc::mbar_init(bar(sm.drain), 1);
    tc::mbar_init(bar(sm.drain_pv), 1);
    tc::mbar_fence_init();
  }
  if (warp == 1) tc::tmem_alloc(smem_u32(&sm.tmem), 512);
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sm.tmem;
  const uint32_t tO = tmem;                              // columns [0, 192)
  const uint32_t tS0 = tmem + 192;                       // S buffers of 64 columns
  const uint32_t tP0 = tmem + 320;                       // P buffers [320, 352), [352, 384), two FP16 per column
  const uint32_t tQ = tmem + 384;                        // Q: hi [384, 432), lo [432, 480)
  int issued = 0;

  if (warp < 4) {
    tc::regs_dec<kQpRegsFew>();
    if (warp == 0 || warp == 2) {
      // ---------------------------------------------------------------- producers
      const bool is_k = warp == 0;
      if (tc::elect_one()) tc::prefetch_tmap(&kvmap);
      __syncwarp();
      // Union blocks one per lane in batches of four tiles, fetched a whole batch
      // ahead; lane 8 t + e holds block e of tile 4 b + t (-1: a zero-filled box).
      auto load_batch = [&](int bt) -> int32_t {
        const int idx = 32 * bt + lane;
        return idx < U ? uid[idx] : -1;
      };
      auto scales = [&](int64_t blk) -> float2 {
        return blk < 0 ? make_float2(0.f, 1.f)
                       : __ldg(reinterpret_cast<const float2*>(kv_scale) + (seq * blocks + blk) * G + g);
      };
      auto publish = [&](float4* dst, int slot, float2 x) {  // by the whole warp
        const bool nk = !(x.x == x.x), nv = !(x.y == x.y);
        if (dst != nullptr) *dst = make_float4(nk ? 0.f : x.x, nv ? 0.f : log2f(x.y), nv ? 1.f : 1.f / x.y, 0.f);
        const uint32_t bk = __ballot_sync(0xffffffffu, nk), bv = __ballot_sync(0xffffffffu, nv);
        if (lane == 0) {
          sm.meta_nan[slot] = bk | bv;
          sm.meta_nan_k[slot] = bk;
        }
        __syncwarp();
      };
      if (!WEIGHTS || is_k) {
        int32_t ids_cur = load_batch(0), ids_next = n_union_tiles > 4 ? load_batch(1) : -1;
        float2 sc_next = make_float2(0.f, 1.f);
        if (is_k) {
          publish(lane < 8 ? &sm.meta_cur[lane] : nullptr, kQpMeta,
                  scales(lane == 0 || (lane == 1 && c0 + 8 <= t_last) ? cb + lane : -1));
          publish(&sm.meta[0][lane], 0, scales(ids_cur));
          sm.ids[0][lane] = ids_cur;
          tc::mbar_arrive(bar(sm.meta_full[0]));
          sc_next = scales(ids_next);
        }
        for (int j = 0; j < n_tiles; ++j) {
          const int nst = is_k ? kQpStages : kQpVStages;
          const int s = j % nst;
          if (j > 0 && (j & 3) == 0) {
            const int bt = j / 4;
            ids_cur = ids_next;
            if (is_k && j < n_union_tiles) {
              // Batch bt - 4 was read: this stage's last QK (tile j - 8) waited for the
              // score buffer of tile j - 10, which the softmax frees after its scales.
              if (j >= kQpStages && !tc::warp_wait(bar(sm.k_empty[s]), ((j / kQpStages) - 1) & 1, abort)) break;
              publish(&sm.meta[bt % kQpMeta][lane], bt % kQpMeta, sc_next);
              sm.ids[bt % kQpMeta][lane] = ids_cur;
              tc::mbar_arrive(bar(sm.meta_full[bt % kQpMeta]));
            }
            ids_next = 4 * (bt + 1) < n_union_tiles ? load_batch(bt + 1) : -1;
            if (is_k) sc_next = scales(ids_next);
          }
          int32_t blk[kQpTile];
#pragma unroll
          for (int e = 0; e < kQpTile; ++e) {
            const int32_t id = __shfl_sync(0xffffffffu, ids_cur, 8 * (j & 3) + e);
            if (j < n_union_tiles) blk[e] = id;
            else blk[e] = (e == 0 || (e == 1 && c0 + 8 <= t_last)) ? static_cast<int32_t>(cb) + e : -1;
          }
          if (j >= nst && !tc::warp_wait(bar(is_k ? sm.k_empty[s] : sm.v_empty[s]), ((j / nst) - 1) & 1, abort)) break;
          if (tc::elect_one()) {
            const uint32_t full = bar(is_k ? sm.k_full[s] : sm.v_full[s]);
            tc::mbar_expect_tx(full, kQpTile * kQ8Half);
            const uint32_t dst = smem_u32(is_k ? &sm.k[s][0][0][0][0] : &sm.v[s][0][0][0][0]);
#pragma unroll
            for (int e = 0; e < kQpTile; ++e)
              tc::tma_load_5d(dst + e * kQ8Half, &kvmap, 0, is_k ? 0 : kQ8Tok, 0, blk[e] >= 0 ? g : 0,
                              blk[e] >= 0 ? static_cast<int32_t>(seq * blocks + blk[e]) : -1, full);
          }
          __syncwarp();
          issued = j + 1;
        }
      }
    } else if (warp == 1 || warp == 3) {
      // ---------------------------------------------------------------- MMA issuers
      const uint32_t id_qk = tc::idesc_e4m3(128, 64, false, false);
      const uint32_t id_pv = tc::idesc_f16(128, 192, true);
      const uint64_t dk0 = tc::sdesc(smem_u32(&sm.k[0][0][0][0][0]), 16, kQ8Half, tc::kSw64);
      const uint64_t dv0 = tc::sdesc_sw128(smem_u32(&sm.v16[0][0][0][0]), 1024, 2 * kQ8Half);
      constexpr uint32_t kStage = kQpTile * kQ8Half / 16;
      bool ok = true;
      if (warp == 1) {
        ok = tc::warp_wait(bar(sm.q_full), 0, abort);
        for (int j = 0; ok && j < n_tiles; ++j) {
          const int s = j % kQpStages, b = j % 2;
          ok = tc::warp_wait(bar(sm.k_full[s]), (j / kQpStages) & 1, abort);
          if (ok && j >= 2) ok = tc::warp_wait(bar(sm.s_free[b]), ((j / 2) - 1) & 1, abort);
          if (!ok) break;
          tc::fence_after();
          if (tc::elect_one()) {
            const uint64_t dk = dk0 + kStage * s;
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int kk = 0; kk < 6; ++kk)  // Q: 8 columns per 32 dims; K: +512 B per 64 dims, +32 B per 32
                tc::mma_f8_tmem_a(tS0 + 64 * b, tQ + 48 * half + 8 * kk,
                                  dk + (kk >> 1) * 32 + (kk & 1) * 2, id_qk, (kk > 0 || half > 0) ? 1u : 0u);
            tc::mma_commit(bar(sm.k_empty[s]));
            tc::mma_commit(bar(sm.s_full[b]));
          }
          __syncwarp();
        }
      } else if (!WEIGHTS) {
        for (int j = 0; ok && j < n_tiles; ++j) {
          const int b = j % 2;
          ok = tc::warp_wait(bar(sm.w_full[b]), (j / 2) & 1, abort) && tc::warp_wait(bar(sm.p_full[b]), (j / 2) & 1, abort);
          if (!ok) break;
          tc::fence_after();
          if (tc::elect_one()) {
            const uint64_t dv = dv0 + 2 * kStage * b;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 16 tokens: V +2 blocks, P +8 columns
              tc::mma_f16_tmem_a(tO, tP0 + 32 * b + 8 * kk, dv + (4 * kQ8Half / 16) * kk, id_pv, (j > 0 || kk > 0) ? 1u : 0u);
            tc::mma_commit(bar(sm.w_empty[b]));
            tc::mma_commit(bar(sm.pv_done[b]));
          }
          __syncwarp();
        }
        if (ok) {
          if (tc::elect_one()) tc::mma_commit(bar(sm.o_final));
          __syncwarp();
        }
      }
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- V codes -> FP16
    tc::regs_dec<kQpRegsFew>();
    // A warp takes six of a tile's 24 (block, chunk) pieces, a lane one 16-byte
    // piece of a row in each: 512 contiguous bytes in, two conflict-free 16-byte
    // stores per lane out.
    if (!WEIGHTS) {
      const uint32_t r = lane >> 2, c = lane & 3;
      const uint32_t src_off = sw64_offset(r, 16 * c);
      const uint32_t dst0 = r * 128 + (((2 * c) ^ r) << 4), dst1 = r * 128 + (((2 * c + 1) ^ r) << 4);
      bool ok = true;
      for (int j = 0; ok && j < n_tiles; ++j) {
        const int s = j % kQpVStages, b = j % 2;
        ok = tc::warp_wait(bar(sm.v_full[s]), (j / kQpVStages) & 1, abort);
        if (ok && j >= 2) ok = tc::warp_wait(bar(sm.w_empty[b]), ((j / 2) - 1) & 1, abort);
        if (!ok) break;
        const uint8_t* src = &sm.v[s][0][0][0][0] + src_off;
        uint8_t* dst = &sm.v16[b][0][0][0];
        uint4 x[6];
#pragma unroll
        for (int i = 0; i < 6; ++i) x[i] = *reinterpret_cast<const uint4*>(src + (6 * (warp - 4) + i) * 512);
#pragma unroll
        for (int i = 0; i < 6; ++i) {
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t o[8];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const __half2 lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[y] & 0xFFFFu), __NV_E4M3);
            const __half2 hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[y] >> 16), __NV_E4M3);
            o[2 * y] = *reinterpret_cast<const uint32_t*>(&lo);
            o[2 * y + 1] = *reinterpret_cast<const uint32_t*>(&hi);
          }
          uint8_t* d = dst + (6 * (warp - 4) + i) * 1024;
          *reinterpret_cast<uint4*>(d + dst0) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(d + dst1) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        tc::fence_proxy_async_smem();
        tc::mbar_arrive(bar(sm.v_empty[s]));
        tc::mbar_arrive(bar(sm.w_full[b]));
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax + epilogue
    tc::regs_inc<kQpRegsMany>();
    // Two warps per TMEM lane quadrant take alternate tiles (`half`: which), so that
    // one's exponentials run beside the other's loads and stores.  The rows'
    // reference goes from tile to tile through shared memory (bar.arrive, bar.sync);
    // where a tile's weights show that it has to move, they are computed once more.
    // A failed wait clears `ok` but keeps every barrier step in place.
    const int quad = warp & 3, half = (warp - 8) >> 2;
    const int pair_bar = 1 + quad;
    const int pub_mine = 5 + 2 * quad + half, pub_other = 5 + 2 * quad + (half ^ 1);
    const int m = quad * 32 + lane;  // TMEM lane = row = (query slot, head)
    const int qs = m >> 4;
    const int64_t qi = qb * 8 + qs;
    const bool qvalid = qi < nq;
    const int64_t t = q_pos0 + (qvalid ? qi : qb * 8);
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const int64_t orow_idx = ((seq * nq + (qvalid ? qi : 0)) * G + g) * kHg + (m & 15);
    if (!WEIGHTS && half == 0) sm.gfac[m] = gate_factor(gate, orow_idx);
    // Q row m, dims [96 half, 96 half + 96): the row's scale, then codes into TMEM
    float rc;
    {
      const uint4* src = reinterpret_cast<const uint4*>(q + orow_idx * kD + 96 * half);
      uint32_t w[48];
#pragma unroll
      for (int c = 0; c < 12; ++c) {
        const uint4 x = qvalid ? src[c] : make_uint4(0u, 0u, 0u, 0u);
        w[4 * c] = x.x;
        w[4 * c + 1] = x.y;
        w[4 * c + 2] = x.z;
        w[4 * c + 3] = x.w;
      }
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < 48; ++c) top = __vmaxu2(top, w[c] & 0x7FFF7FFFu);
      top = max(top & 0xFFFFu, top >> 16);  // BF16 bits of the largest magnitude
      sm.lsum[half][m] = __uint_as_float(top << 16);
      asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
      const uint32_t t2 = max(__float_as_uint(sm.lsum[0][m]), __float_as_uint(sm.lsum[1][m]));
      const bool fin = t2 < 0x7F800000u;
      const int e = fin ? e4m3_exp(__uint_as_float(t2)) : 0;
      const float inv = pow2f(-e);
      rc = fin ? pow2f(e) * scale_log2 : __uint_as_float(0x7FC00000u);  // infinity or NaN: every score NaN
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        uint32_t h8[8], l8[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const uint32_t a = w[16 * c + 2 * x], b = w[16 * c + 2 * x + 1];
          uint32_t ha, la, hb, lb;
          split_e4m3(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xFFFF0000u) * inv, ha, la, 1.f);
          split_e4m3(__uint_as_float(b << 16) * inv, __uint_as_float(b & 0xFFFF0000u) * inv, hb, lb, 1.f);
          h8[x] = ha | (hb << 16);
          l8[x] = la | (lb << 16);
        }
        tc::tmem_st8(tQ + lane_off + 24 * half + 8 * c, h8);
        tc::tmem_st8(tQ + 48 + lane_off + 24 * half + 8 * c, l8);
      }
      tc::tmem_st_wait();
      tc::fence_before();
      tc::mbar_arrive(bar(sm.q_full));
      asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");  // lsum is reused at the end
    }
    float ref = -INFINITY;           // the row's reference, as this warp knows it
    float m_l = -INFINITY, l = 0.f;  // this warp's part of the row's sum, relative to 2^m_l
    uint32_t nan_v = 0, nan_k = 0;   // the row attends a block whose V (or K), its K, holds an infinity or NaN
    const float row_lse = WEIGHTS ? (qvalid ? lse[orow_idx] : INFINITY) : 0.f;
    bool ok = tc::mbar_wait(bar(sm.meta_full[0]), 0, abort);  // (the current blocks' scales come with it)
    uint2 mb_next = make_uint2(0u, 0u);  // mask bytes of this warp's next tile
    if (half < n_union_tiles) mb_next = *reinterpret_cast<const uint2*>(umask + 8 * half);
    for (int j = half; j < n_tiles; j += 2) {
      const int b = half;
      const bool last = j >= n_union_tiles;  // the current-block tile
      const int slot = last ? kQpMeta : (j / 4) % kQpMeta, at = last ? 0 : 8 * (j & 3);
      const uint32_t tS = tS0 + 64 * b + lane_off, tP = tP0 + 32 * b + lane_off;
      // bit 8 e of word h: the row's query attends block 4 h + e (the plan's bytes
      // behind the union are zeros)
      const uint32_t use[2] = {last ? 1u << (8 * (t / 8 - cb)) : (mb_next.x >> qs) & 0x01010101u,
                               last ? 0u : (mb_next.y >> qs) & 0x01010101u};
      if (j + 2 < n_union_tiles) mb_next = *reinterpret_cast<const uint2*>(umask + 8 * (j + 2));
      if (!last && (j & 3) < 2) ok = ok && tc::mbar_wait(bar(sm.meta_full[slot]), (j / (4 * kQpMeta)) & 1, abort);
      const float4* meta = last ? sm.meta_cur : &sm.meta[slot][at];
      if (const uint32_t nan = (sm.meta_nan[slot] >> at) & 0xFFu) {  // rare
        const uint32_t nk = sm.meta_nan_k[slot] >> at;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          nan_v |= (use[e >> 2] >> (8 * (e & 3))) & (nan >> e) & 1u;
          nan_k |= (use[e >> 2] >> (8 * (e & 3))) & (nk >> e) & 1u;
        }
      }
      ok = ok && tc::mbar_wait(bar(sm.s_full[b]), (j / 2) & 1, abort);
      tc::fence_after();
      uint32_t sr[64];
      tc::tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
      tc::tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
      tc::tmem_ld_wait();
      float rct = rc;  // this tile's row scale
      if (last) {
        // Tokens of the row's current block behind t get score -inf.  Where the row's
        // and the block's scale underflow together (a head of zeros at keys of
        // zeros), -inf times their product would be NaN: the scores are 0 then, and
        // stay apart from the masked ones under a row scale of 1.
        const int end = static_cast<int>(t - c0);
        const bool flat = meta[use[0] >> 8 ? 1 : 0].x * rc == 0.f;
        if (flat) rct = 1.f;
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if ((use[0] >> (8 * (x >> 3))) & 1u) sr[x] = x > end ? __float_as_uint(-INFINITY) : flat ? 0u : sr[x];
      }
      if constexpr (WEIGHTS) {
        tc::fence_before();
        tc::mbar_arrive(bar(sm.s_free[b]));
        // weights of the row, summed by block, then over the warp's 32 rows: lane
        // 8 i + e ends with block e
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float cf = meta[e].x * rct;
          const uint64_t c2 = pack_f32x2(cf, cf), o2 = pack_f32x2(-row_lse, -row_lse);
          uint64_t p[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint64_t v = fma_f32x2(pack_f32x2(__uint_as_float(sr[8 * e + 2 * x]), __uint_as_float(sr[8 * e + 2 * x + 1])), c2, o2);
            p[x] = pack_f32x2(fast_exp2(f32x2_lo(v)), fast_exp2(f32x2_hi(v)));
          }
          const uint64_t sum = add_f32x2(add_f32x2(p[0], p[1]), add_f32x2(p[2], p[3]));
          w[e] = f32x2_lo(sum) + f32x2_hi(sum);
          if (!((use[e >> 2] >> (8 * (e & 3))) & 1u) || !(w[e] == w[e])) w[e] = 0.f;
        }
        float y[4], z[2];
        const bool h4 = lane & 4, h2 = lane & 2, h1 = lane & 1;
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = (h4 ? w[4 + c] : w[c]) + __shfl_xor_sync(0xffffffffu, h4 ? w[c] : w[4 + c], 4);
#pragma unroll
        for (int c = 0; c < 2; ++c) z[c] = (h2 ? y[2 + c] : y[c]) + __shfl_xor_sync(0xffffffffu, h2 ? y[c] : y[2 + c], 2);
        float v = (h1 ? z[1] : z[0]) + __shfl_xor_sync(0xffffffffu, h1 ? z[0] : z[1], 1);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        // After a wait that gave up, anywhere in the unit, scores may be overwritten
        // early and block numbers never written: nothing more is added.
        if (ok && !*abort && lane < 8 && v > 0.f) {
          const int64_t id = last ? cb + lane : sm.ids[slot][at + lane];
          if (id >= 0 && id < blocks) acc_add(acc + seq * blocks + id, v);
        }
      } else {
        tc::fence_before();
        tc::mbar_arrive(bar(sm.s_free[b]));
        // P buffer b is free once O += P(j-2) V(j-2) has read it
        if (j >= 2) ok = ok && tc::mbar_wait(bar(sm.pv_done[b]), ((j / 2) - 1) & 1, abort);
        tc::fence_after();
        // The reference after tile j-1, from the other warp.  Waiting for it here
        // lets the two warps' exponentials take turns (one sub-partition's).
        if (j > 0) {
          asm volatile("bar.sync %0, 64;" ::"r"(pub_other) : "memory");
          ref = sm.mchain[m];
        }
        float ls;
        for (int pass = 0; pass < 2; ++pass) {
          const float neg = ref == -INFINITY ? 0.f : -ref;
          float top = 0.f;  // largest sum of a block's weights
          ls = 0.f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[16];
            const uint32_t wuse = SKIP_PAIRS ? __reduce_or_sync(0xffffffffu, use[h]) : 0x01010101u;
#pragma unroll
            for (int e2 = 0; e2 < 4; e2 += 2) {
              if (!SKIP_PAIRS || ((wuse >> (8 * e2)) & 0x0101u)) {
#pragma unroll
                for (int e = e2; e < e2 + 2; ++e) {
                  // P = 2^(s + log2 vs - ref); a block the row does not attend has offset -inf
                  const float4 mt = meta[4 * h + e];
                  const float cf = mt.x * rct, off = (use[h] >> (8 * e)) & 1u ? mt.y + neg : -INFINITY;
                  const uint64_t c2 = pack_f32x2(cf, cf), o2 = pack_f32x2(off, off);
                  uint64_t pe[4];
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    const int at2 = 32 * h + 8 * e + 2 * x;
                    const uint64_t v = fma_f32x2(pack_f32x2(__uint_as_float(sr[at2]), __uint_as_float(sr[at2 + 1])), c2, o2);
                    const float p0 = fast_exp2(f32x2_lo(v)), p1 = fast_exp2(f32x2_hi(v));
                    pe[x] = pack_f32x2(p0, p1);
                    pk[4 * e + x] = pack_f16x2(p0, p1);
                  }
                  const uint64_t sum = add_f32x2(add_f32x2(pe[0], pe[1]), add_f32x2(pe[2], pe[3]));
                  const float bs = f32x2_lo(sum) + f32x2_hi(sum);
                  top = fmaxf(top, bs);
                  ls = fmaf(bs, mt.z, ls);
                }
              } else {
#pragma unroll
                for (int x = 4 * e2; x < 4 * e2 + 8; ++x) pk[x] = 0u;
              }
            }
            tc::tmem_st16(tP + 16 * h, pk);
          }
          if (pass == 1) break;
          // these weights stand unless a block's sum leaves FP16's range (one of its
          // weights is above 2^12 then), or the row has no reference yet
          const bool high = top > 60000.f || (ref == -INFINITY && (use[0] | use[1]) != 0u);
          if (!__any_sync(0xffffffffu, high)) break;
          tc::tmem_st_wait();  // the second pass stores to the same columns: stores keep no order of their own
          float mx = -INFINITY;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 mt = meta[e];
            float v = __uint_as_float(sr[8 * e]);
#pragma unroll
            for (int x = 1; x < 8; ++x) v = fmaxf(v, __uint_as_float(sr[8 * e + x]));
            mx = fmaxf(mx, (use[e >> 2] >> (8 * (e & 3))) & 1u ? fmaf(v, mt.x * rct, mt.y) : -INFINITY);
          }
          // A new reference lies 4 below the largest weight: FP16 then holds weights
          // down to 2^-18 of it in full and resolves 2^-28 of it, and the reference
          // stays until the scores grow by 2^8 at least.
          const bool need = mx > ref + 12.f;
          const float old = ref;
          if (need) ref = mx - 4.f;
          if (j > 0 && __any_sync(0xffffffffu, need)) {
            const float alpha = need ? exp2f(old - ref) : 1.f;
            // O must hold P(j-1) V(j-1) before it is rescaled.  (This warp knows the
            // product of tile j-2 done, so tile j-3's too: the phase is tile j-1's.)
            ok = ok && tc::mbar_wait(bar(sm.pv_done[b ^ 1]), ((j - 1) / 2) & 1, abort);
            tc::fence_after();
#pragma unroll 1
            for (int h = 0; h < 6; ++h) {
              uint32_t o[32];
              tc::tmem_ld32(tO + lane_off + 32 * h, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
              tc::tmem_st32(tO + lane_off + 32 * h, o);
            }
          }
        }
        sm.mchain[m] = ref;
        if (j + 1 < n_tiles) asm volatile("bar.arrive %0, 64;" ::"r"(pub_mine) : "memory");
        if (m_l != ref) {
          l = m_l == -INFINITY ? l : l * exp2f(m_l - ref);  // (at -inf: 0, or NaN)
          m_l = ref;
        }
        l += ls;
        tc::tmem_st_wait();
        tc::fence_before();
        tc::mbar_arrive(bar(sm.p_full[b]));
      }
    }
    if (!WEIGHTS) {
      ok = ok && tc::mbar_wait(bar(sm.o_final), 0, abort);
      if (nan_v) sm.gfac[m] = __uint_as_float(0x7FC00000u);
      // both loops are done: the final reference is in mchain; combine the two partial sums
      asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
      ref = sm.mchain[m];
      sm.lsum[half][m] = nan_k ? __uint_as_float(0x7FC00000u) : m_l == -INFINITY ? l : l * exp2f(m_l - ref);
      asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
      const float ltot = sm.lsum[0][m] + sm.lsum[1][m];
      if (ok) {
        tc::fence_after();
        const float inv = sm.gfac[m] / ltot;  // softmax normalisation and output gate
        if (lse != nullptr && half == 0 && qvalid) lse[orow_idx] = (ref == -INFINITY ? 0.f : ref) + log2f(ltot);
        __nv_bfloat16* orow = out + orow_idx * kD;
#pragma unroll 1
        for (int h = 3 * half; h < 3 * half + 3; ++h) {
          uint32_t o[32];
          tc::tmem_ld32(tO + lane_off + 32 * h, o);
          tc::tmem_ld_wait();
          if (qvalid) {
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4) {
              uint4 w;
              w.x = pack_bf16x2(__uint_as_float(o[8 * v4 + 0]) * inv, __uint_as_float(o[8 * v4 + 1]) * inv);
              w.y = pack_bf16x2(__uint_as_float(o[8 * v4 + 2]) * inv, __uint_as_float(o[8 * v4 + 3]) * inv);
              w.z = pack_bf16x2(__uint_as_float(o[8 * v4 + 4]) * inv, __uint_as_float(o[8 * v4 + 5]) * inv);
              w.w = pack_bf16x2(__uint_as_float(o[8 * v4 + 6]) * inv, __uint_as_float(o[8 * v4 + 7]) * inv);
              *reinterpret_cast<uint4*>(orow + 32 * h + 8 * v4) = w;
            }
          }
        }
      }
    }
  }
  // The abort flag is final here; after a failed wait the copies and MMAs in
  // flight land before shared memory and TMEM are released.
  __syncthreads();
  if (sm.abort) {
    if (warp == 0 || warp == 2) {
      const int nst = warp == 0 ? kQpStages : kQpVStages;
      for (int j = issued > nst ? issued - nst : 0; j < issued; ++j)
        tc::mbar_drain(bar(warp == 0 ? sm.k_full[j % nst] : sm.v_full[j % nst]), (j / nst) & 1);
    } else if (warp == 1 || warp == 3) {
      uint64_t& d = warp == 1 ? sm.drain : sm.drain_pv;
      if (tc::elect_one()) tc::mma_commit(bar(d));
      __syncwarp();
      tc::mbar_drain(bar(d), 0);
    } else if (!WEIGHTS && lse != nullptr && warp >= 12) {
      // no log-sums: the weights' sweep, which may well succeed, adds nothing for these rows
      const int m = threadIdx.x - 384;
      const int64_t qi = qb * 8 + (m >> 4);
      if (qi < nq) lse[((seq * nq + qi) * G + g) * kHg + (m & 15)] = __uint_as_float(0x7FC00000u);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

}  // namespace sgqa
