// Eviction of cache blocks by accumulated attention weight.
//
// Of a sequence's n complete blocks (slots 0 .. n-1) the `keep` with the
// largest weight stay; blocks among the first or the most recent ones of the
// sequence are protected; equal weights keep the smaller original number.
// Attention over past blocks does not depend on their order, so the cache is
// not shifted together: the i-th freed slot below `keep` takes the i-th kept
// block found behind it.  At most min(keep, n - keep) blocks move instead of
// nearly all of them.
#pragma once
#include "common.cuh"

namespace sgqa {

constexpr int kMaxArrays = 8;
struct EvictArrays {
  uint8_t* base[kMaxArrays];
  int64_t bytes[kMaxArrays];  // per block
  int shift[kMaxArrays];      // log2 of the copied word (1 .. 16 bytes)
  int tail_only[kMaxArrays];
  int count;
};

constexpr int kEvictThreads = 1024;

struct EvictWs {
  int64_t cap;       // slots per sequence in the lists
  int2* moves;       // [S, cap] (to, from)
  int64_t* moved_acc;  // [S, cap + 1]: acc of each move's block; the incomplete block's at the end
  int32_t* moved_pos;  // [S, cap]
  int32_t* count;    // [S]
};

__device__ __forceinline__ int32_t evict_pos(const int32_t* pos, int64_t slot, int64_t known, int64_t evicted) {
  return slot < known ? pos[slot] : static_cast<int32_t>(slot + evicted);
}

// Larger key = kept first; protected blocks above every weight.
__device__ __forceinline__ uint64_t evict_key(int64_t acc, int32_t pos, int64_t first, int64_t recent_from) {
  if (pos < first || pos >= recent_from) return ~0ull;
  const uint64_t k = static_cast<uint64_t>(acc) ^ 0x8000000000000000ull;
  return k == ~0ull ? k - 1 : k;
}

// Block-wide exclusive scan of two counts (packed); returns this thread's
// prefix and the totals.
__device__ __forceinline__ uint2 evict_scan(uint2 v, uint2* warp_tot, uint2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint2 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) { x.x += a; x.y += b; }
  }
  __syncthreads();
  if (lane == 31) warp_tot[warp] = x;
  __syncthreads();
  uint2 before = make_uint2(0, 0), all = make_uint2(0, 0);
  for (int w = 0; w < kEvictThreads / 32; ++w) {
    if (w < warp) { before.x += warp_tot[w].x; before.y += warp_tot[w].y; }
    all.x += warp_tot[w].x;
    all.y += warp_tot[w].y;
  }
  total = all;
  return make_uint2(before.x + x.x - v.x, before.y + x.y - v.y);
}

// One CTA per sequence: radix select of the smallest kept key (8 bits at a
// time), then of the largest kept original number among the blocks that tie
// there; the lists of freed slots and moved blocks; the weights and numbers of
// the kept blocks in their new slots.
__global__ void __launch_bounds__(kEvictThreads)
evict_select_kernel(const int64_t* acc, const int32_t* pos, int64_t known, int64_t evicted, int64_t n, int part,
                    int64_t keep, int64_t first, int64_t recent, int64_t slots, EvictWs ws, int64_t* acc_out,
                    int32_t* pos_out) {
  __shared__ uint32_t hist[256];
  __shared__ uint2 warp_tot[kEvictThreads / 32];
  __shared__ uint64_t s_key;
  __shared__ int64_t s_need;
  const int64_t seq = blockIdx.x;
  const int tid = threadIdx.x;
  const int64_t* a = acc + seq * slots;
  const int32_t* p = pos + seq * slots;  // read below `known` only
  const int64_t recent_from = n + evicted - recent;
  uint64_t key = 0;      // digits of the boundary key found so far
  int64_t need = keep;   // blocks still to take among those that match them
  for (int sh = 56; sh >= 0; sh -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int64_t s = tid; s < n; s += kEvictThreads) {
      const uint64_t x = evict_key(a[s], evict_pos(p, s, known, evicted), first, recent_from);
      if (sh == 56 || (x >> (sh + 8)) == (key >> (sh + 8))) atomicAdd(&hist[(x >> sh) & 255], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      int64_t left = need;
      int d = 255;
      for (; d > 0 && hist[d] < left; --d) left -= hist[d];
      s_key = key | (static_cast<uint64_t>(d) << sh);
      s_need = left;
    }
    __syncthreads();
    key = s_key;
    need = s_need;
    __syncthreads();
  }
  // among the blocks with that key: the `need` smallest numbers
  uint32_t pkey = 0;
  int64_t pneed = need;
  for (int sh = 24; sh >= 0; sh -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int64_t s = tid; s < n; s += kEvictThreads) {
      const int32_t ps = evict_pos(p, s, known, evicted);
      if (evict_key(a[s], ps, first, recent_from) == key) {
        const uint32_t x = static_cast<uint32_t>(ps);
        if (sh == 24 || (x >> (sh + 8)) == (pkey >> (sh + 8))) atomicAdd(&hist[(x >> sh) & 255], 1u);
      }
    }
    __syncthreads();
    if (tid == 0) {
      int64_t left = pneed;
      int d = 0;
      for (; d < 255 && hist[d] < left; ++d) left -= hist[d];
      s_key = pkey | (static_cast<uint32_t>(d) << sh);
      s_need = left;
    }
    __syncthreads();
    pkey = static_cast<uint32_t>(s_key);
    pneed = s_need;
    __syncthreads();
  }
  int2* moves = ws.moves + seq * ws.cap;
  int64_t* macc = ws.moved_acc + seq * (ws.cap + 1);
  int32_t* mpos = ws.moved_pos + seq * ws.cap;
  auto kept = [&](int64_t s) {
    const int32_t ps = evict_pos(p, s, known, evicted);
    const uint64_t x = evict_key(a[s], ps, first, recent_from);
    return keep > 0 && (x > key || (x == key && static_cast<uint32_t>(ps) <= pkey));
  };
  uint32_t holes = 0, late = 0;
  for (int64_t s0 = 0; s0 < n; s0 += kEvictThreads) {
    const int64_t s = s0 + tid;
    const bool in = s < n;
    const bool kp = in && kept(s);
    const bool hole = in && !kp && s < keep, mv = kp && s >= keep;
    uint2 tot;
    const uint2 at = evict_scan(make_uint2(hole, mv), warp_tot, tot);
    if (hole) moves[holes + at.x].x = static_cast<int32_t>(s);
    if (mv) {
      moves[late + at.y].y = static_cast<int32_t>(s);
      macc[late + at.y] = a[s];
      mpos[late + at.y] = evict_pos(p, s, known, evicted);
    }
    holes += tot.x;
    late += tot.y;
  }
  if (tid == 0) {
    if (holes != late) report(kDevBounds);  // original numbers that occur twice
    ws.count[seq] = static_cast<int32_t>(min(holes, late));
    if (part) macc[ws.cap] = a[n];
  }
  __syncthreads();
  // new weights and numbers: kept blocks that stay, then the moved ones; no
  // weight behind them
  uint32_t h0 = 0;
  for (int64_t s0 = 0; s0 < slots; s0 += kEvictThreads) {
    const int64_t s = s0 + tid;
    const bool hole = s < min(n, keep) && !kept(s);
    uint2 tot;
    const uint2 at = evict_scan(make_uint2(hole, 0), warp_tot, tot);
    int64_t v = 0;
    int32_t ps = -1;
    if (s < keep) {
      const uint32_t r = h0 + at.x;
      if (hole) {
        if (r < late) { v = macc[r]; ps = mpos[r]; }
      } else {
        v = a[s];
        ps = evict_pos(p, s, known, evicted);
      }
    } else if (s == keep && part) {
      v = macc[ws.cap];
    }
    __syncthreads();  // every read of these slots before the writes (acc_out may be acc)
    if (s < slots) {
      acc_out[seq * slots + s] = v;
      if (s < keep) pos_out[seq * slots + s] = ps;
    }
    h0 += tot.x;
  }
}

// Moves the blocks' bytes.  A CTA takes the moves of one sequence in turn; a
// thread copies the same pieces of a block in every step, so that where the
// incomplete block's new slot held a block that moves, one thread reads each
// piece before it writes it.
__global__ void __launch_bounds__(256)
evict_move_kernel(EvictArrays ar, EvictWs ws, int64_t n, int part, int64_t keep, int64_t slots) {
  const int64_t seq = blockIdx.y;
  const int count = ws.count[seq];
  const int2* moves = ws.moves + seq * ws.cap;
  auto copy = [&](int64_t to, int64_t from, bool tail) {
    for (int x = 0; x < ar.count; ++x) {
      if (ar.tail_only[x] && !tail) continue;
      uint8_t* dst = ar.base[x] + (seq * slots + to) * ar.bytes[x];
      const uint8_t* src = ar.base[x] + (seq * slots + from) * ar.bytes[x];
      const int64_t words = ar.bytes[x] >> ar.shift[x];
      for (int64_t i = threadIdx.x; i < words; i += blockDim.x) {
        switch (ar.shift[x]) {
          case 4: reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(src)[i]; break;
          case 3: reinterpret_cast<uint2*>(dst)[i] = reinterpret_cast<const uint2*>(src)[i]; break;
          case 2: reinterpret_cast<uint32_t*>(dst)[i] = reinterpret_cast<const uint32_t*>(src)[i]; break;
          case 1: reinterpret_cast<uint16_t*>(dst)[i] = reinterpret_cast<const uint16_t*>(src)[i]; break;
          default: dst[i] = src[i];
        }
      }
    }
  };
  bool tail_done = false;
  for (int m = blockIdx.x; m < count; m += gridDim.x) {
    copy(moves[m].x, moves[m].y, false);
    if (part && moves[m].y == keep) {
      copy(keep, n, true);
      tail_done = true;
    }
  }
  // the first block behind `keep` moves first, if it moves at all: move 0
  if (blockIdx.x == 0 && part && keep < n && !tail_done) copy(keep, n, true);
}

}  // namespace sgqa
