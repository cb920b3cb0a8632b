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
#include <cooperative_groups.h>

#include "common.cuh"

namespace sgqa {

constexpr int kMaxArrays = 8;
struct EvictArrays {
  uint8_t* base[kMaxArrays];
  int64_t bytes[kMaxArrays];  // per block
  int shift[kMaxArrays];      // log2 of the copied word (16, 4 or 1 bytes)
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

// Exclusive scan of two counts per warp over the block's 32 warps: `v` of lane 0
// counts; every lane gets its warp's prefix, and the totals.
__device__ __forceinline__ uint2 evict_warp_scan(uint2 v, uint2* warp_tot, uint2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) warp_tot[warp] = v;
  __syncthreads();
  const uint2 own = warp_tot[lane];  // every warp scans the 32 totals itself
  uint2 x = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) { x.x += a; x.y += b; }
  }
  total = make_uint2(__shfl_sync(0xffffffffu, x.x, 31), __shfl_sync(0xffffffffu, x.y, 31));
  return make_uint2(__shfl_sync(0xffffffffu, x.x - own.x, warp), __shfl_sync(0xffffffffu, x.y - own.y, warp));
}

// The same per thread.
__device__ __forceinline__ uint2 evict_scan(uint2 v, uint2* warp_tot, uint2& total) {
  const int lane = threadIdx.x & 31;
  uint2 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) { x.x += a; x.y += b; }
  }
  const uint2 sum = make_uint2(__shfl_sync(0xffffffffu, x.x, 31), __shfl_sync(0xffffffffu, x.y, 31));
  const uint2 before = evict_warp_scan(sum, warp_tot, total);
  return make_uint2(before.x + x.x - v.x, before.y + x.y - v.y);
}

// Sequences of more blocks than a cluster holds (evict_select_kernel below):
// one CTA per sequence re-reads the weights for every step.  Radix select of the
// smallest kept key (8 bits at a time), then of the largest kept original number
// among the blocks that tie there; the lists of freed slots and moved blocks;
// the weights and numbers of the kept blocks in their new slots.
__global__ void __launch_bounds__(kEvictThreads)
evict_select_long_kernel(const int64_t* acc, const int32_t* pos, int64_t known, int64_t evicted, int64_t n, int part,
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

// ---------------------------------------------------------------------------
// One cluster per sequence, every CTA a contiguous range of slots whose weights
// and numbers it keeps in shared memory (12 bytes each, 16384 slots at most).
// The `keep`-th block of the order (weight down, number up) is found by
// histograms of 2048 bins that the cluster adds up through distributed shared
// memory: first on a logarithmic scale (32 bins per power of two, so that
// weights that fall off over decades spread), then linear in the bin where the
// boundary lies.  Once at most 512 blocks are left there, they are ranked by
// counting; usually after two histograms.  Blocks with equal weights that reach
// the last step are told apart by further histograms of their numbers.
// Bound: latency (barriers and dependent passes), not bytes.
// Measured: 456 of 520 blocks kept 9.4 us, 16 x 4096 -> 2800 11.7 us, 2 x 65536 ->
// 49152 28.6 us.
// ---------------------------------------------------------------------------
constexpr int kEvBins = 2048;
constexpr int kEvSlots = 16384;      // per CTA
constexpr int kEvMaxCluster = 8;     // portable
constexpr int kEvRank = 512;

struct EvictSmem {
  uint32_t hist[2][kEvBins];         // two, so that the next pass can clear while others still read
  uint64_t ckey[kEvRank];            // the last candidates (rank 0's copy is used)
  uint32_t cpos[kEvRank];
  uint2 warp_tot[kEvictThreads / 32];
  uint32_t ccount;
  uint2 sums;                        // freed slots and moved blocks of this CTA
  uint32_t bin, above, inside;       // boundary bin, blocks in the bins above it and in it
  uint64_t tkey;                     // the last kept block
  uint32_t tpos;
  int64_t acc[kEvSlots];
  int32_t pos[kEvSlots];
};

// Bin of a key on the logarithmic scale: 0 negative weights, 1 none, 2047 protected.
__device__ __forceinline__ uint32_t evict_log_bin(uint64_t key) {
  if (key == ~0ull) return kEvBins - 1;
  if (!(key >> 63)) return 0;
  const uint64_t a = key ^ 0x8000000000000000ull;
  if (a == 0) return 1;
  const int m = 63 - __clzll(static_cast<long long>(a));
  const uint32_t frac = static_cast<uint32_t>(m >= 5 ? a >> (m - 5) : a << (5 - m)) & 31u;
  return 2 + 32 * m + frac;
}
// Smallest and largest key of a bin.
__device__ __forceinline__ void evict_log_range(uint32_t bin, uint64_t& lo, uint64_t& hi) {
  constexpr uint64_t kZero = 0x8000000000000000ull;
  if (bin == kEvBins - 1) {
    lo = hi = ~0ull;
  } else if (bin == 0) {
    lo = 0;
    hi = kZero - 1;
  } else if (bin == 1) {
    lo = hi = kZero;
  } else {
    const int m = static_cast<int>(bin - 2) / 32;
    const uint64_t f = 32 + (bin - 2) % 32;
    lo = kZero + (m >= 5 ? f << (m - 5) : f >> (5 - m));
    hi = m >= 5 ? lo + (1ull << (m - 5)) - 1 : lo;
  }
}

__global__ void __launch_bounds__(kEvictThreads, 1)
evict_select_kernel(const int64_t* acc, const int32_t* pos, int64_t known, int64_t evicted, int64_t n, int part,
                    int64_t keep, int64_t first, int64_t recent, int64_t slots, EvictWs ws, int64_t* acc_out,
                    int32_t* pos_out) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint8_t raw[];
  EvictSmem& sm = *reinterpret_cast<EvictSmem*>(raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int ncta = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int64_t seq = blockIdx.x / ncta;
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t recent_from = n + evicted - recent;
  const int64_t per = (n + ncta - 1) / ncta, s0 = rank * per;
  const int cnt = static_cast<int>(max(static_cast<int64_t>(0), min(n, s0 + per) - s0));
  const int64_t* a = acc + seq * slots;
  const int32_t* p = pos + seq * slots;  // read below `known` only
  // for the lists: a contiguous range per warp, at most 16 rounds of 32 slots
  const int its = static_cast<int>((per + kEvictThreads - 1) / kEvictThreads);
  const int w0 = (tid >> 5) * 32 * its + lane;
  const int64_t tail_acc = part ? a[n] : 0;
  for (int i = tid; i < cnt; i += 4 * kEvictThreads) {  // four loads of each in flight
    int64_t va[4];
    int32_t vp[4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (i + x * kEvictThreads < cnt) {
        va[x] = a[s0 + i + x * kEvictThreads];
        vp[x] = evict_pos(p, s0 + i + x * kEvictThreads, known, evicted);
      }
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (i + x * kEvictThreads < cnt) {
        sm.acc[i + x * kEvictThreads] = va[x];
        sm.pos[i + x * kEvictThreads] = vp[x];
      }
  }
  for (int i = tid; i < 2 * kEvBins; i += kEvictThreads) (&sm.hist[0][0])[i] = 0;
  if (tid == 0) sm.ccount = 0;
  __syncthreads();
  auto key_at = [&](int i) { return evict_key(sm.acc[i], sm.pos[i], first, recent_from); };
  // Adds the cluster's histograms and finds, from the highest bin down, the one
  // with the need-th block; every CTA computes the same.
  auto boundary = [&](int h, uint32_t need) {
    cluster.sync();
    uint32_t c[2] = {0, 0};  // bins 2047 - 2 tid, 2046 - 2 tid
#pragma unroll
    for (int r = 0; r < kEvMaxCluster; ++r)
      if (r < ncta) {
        const uint2 v = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&sm.hist[h][kEvBins - 2 - 2 * tid], r));
        c[0] += v.y;
        c[1] += v.x;
      }
    uint2 tot;
    const uint32_t before = evict_scan(make_uint2(c[0] + c[1], 0), sm.warp_tot, tot).x;
    if (before < need && before + c[0] >= need) {
      sm.bin = kEvBins - 1 - 2 * tid;
      sm.above = before;
      sm.inside = c[0];
    } else if (before + c[0] < need && before + c[0] + c[1] >= need) {
      sm.bin = kEvBins - 2 - 2 * tid;
      sm.above = before + c[0];
      sm.inside = c[1];
    }
    __syncthreads();
    return sm.inside;
  };
  auto count = [&](int h, uint32_t bin, bool in) {
    // warps whose blocks all fall in one bin (no weight, protected) add once
    const uint32_t live = __ballot_sync(0xffffffffu, in);
    if (live == 0u) return;
    const uint32_t lead = __shfl_sync(0xffffffffu, bin, __ffs(live) - 1);
    if (__all_sync(0xffffffffu, !in || bin == lead)) {
      if (lane == __ffs(live) - 1) atomicAdd(&sm.hist[h][bin], static_cast<uint32_t>(__popc(live)));
    } else if (in) {
      atomicAdd(&sm.hist[h][bin], 1u);
    }
  };
  uint64_t tkey = ~0ull;
  uint32_t tpos = 0;
  if (keep > 0) {
    const int rounds = (cnt + kEvictThreads - 1) / kEvictThreads;
    uint32_t need = static_cast<uint32_t>(keep);
    for (int r = 0; r < rounds; ++r) {
      const int i = r * kEvictThreads + tid;
      count(0, i < cnt ? evict_log_bin(key_at(i)) : 0u, i < cnt);
    }
    uint32_t left = boundary(0, need);
    need -= sm.above;
    uint64_t lo, hi;            // the boundary's range of keys, then (by_pos) of numbers, smaller ones first
    uint32_t plo = 0, phi = 0xFFFFFFFFu;
    evict_log_range(sm.bin, lo, hi);
    bool by_pos = lo == hi;
    int h = 1;
    while (left > kEvRank && !(by_pos && plo == phi)) {
      int sh = 0;
      const uint64_t width = by_pos ? static_cast<uint64_t>(phi - plo) : hi - lo;
      while ((width >> sh) >= kEvBins) ++sh;
      for (int r = 0; r < rounds; ++r) {
        const int i = r * kEvictThreads + tid;
        bool in = i < cnt;
        uint32_t bin = 0;
        if (in) {
          const uint64_t k = key_at(i);
          const uint32_t ps = static_cast<uint32_t>(sm.pos[i]);
          in = k >= lo && k <= hi && (!by_pos || (ps >= plo && ps <= phi));
          bin = by_pos ? kEvBins - 1 - ((ps - plo) >> sh) : static_cast<uint32_t>((k - lo) >> sh);
        }
        count(h, bin, in);
      }
      left = boundary(h, need);
      need -= sm.above;
      const uint32_t bin = sm.bin;
      if (by_pos) {
        plo += (kEvBins - 1 - bin) << sh;
        phi = static_cast<uint32_t>(min(static_cast<unsigned long long>(phi), plo + ((1ull << sh) - 1)));
      } else {
        lo += static_cast<uint64_t>(bin) << sh;
        hi = min(static_cast<unsigned long long>(hi), lo + ((1ull << sh) - 1));
        by_pos = lo == hi;
      }
      // the histogram before this one has been read by everybody: clear it for the next
      h ^= 1;
      for (int i = tid; i < kEvBins; i += kEvictThreads) sm.hist[h][i] = 0;
      __syncthreads();
    }
    if (left > kEvRank) {
      // more blocks than that with one weight and one number: the call's contract is broken
      tkey = lo;
      tpos = phi;
    } else {
      // rank the last candidates by counting, in CTA 0
      EvictSmem* lead = cluster.map_shared_rank(&sm, 0);
      for (int i = tid; i < cnt; i += kEvictThreads) {
        const uint64_t k = key_at(i);
        const uint32_t ps = static_cast<uint32_t>(sm.pos[i]);
        if (k >= lo && k <= hi && (!by_pos || (ps >= plo && ps <= phi))) {
          const uint32_t at = atomicAdd(&lead->ccount, 1u);
          if (at < kEvRank) {
            lead->ckey[at] = k;
            lead->cpos[at] = ps;
          }
        }
      }
      cluster.sync();
      if (rank == 0) {
        const uint32_t c = min(sm.ccount, static_cast<uint32_t>(kEvRank));
        for (uint32_t x = tid >> 5; x < c; x += kEvictThreads / 32) {  // a warp counts who stands before x
          const uint64_t k = sm.ckey[x];
          const uint32_t ps = sm.cpos[x];
          uint32_t better = 0;
          for (uint32_t i = lane; i < c; i += 32) {
            const uint64_t ki = sm.ckey[i];
            const uint32_t pi = sm.cpos[i];
            better += (ki > k || (ki == k && (pi < ps || (pi == ps && i < x)))) ? 1u : 0u;
          }
          better = __reduce_add_sync(0xffffffffu, better);
          if (lane == 0 && better == need - 1) {
            sm.tkey = k;
            sm.tpos = ps;
          }
        }
      }
      cluster.sync();
      tkey = lead->tkey;
      tpos = lead->tpos;
    }
  }
  auto kept = [&](int i) {
    const uint64_t k = key_at(i);
    return keep > 0 && (k > tkey || (k == tkey && static_cast<uint32_t>(sm.pos[i]) <= tpos));
  };
  // freed slots below `keep`, kept blocks behind it: ranks over the whole sequence
  uint2 mine = make_uint2(0, 0), tot;
  uint32_t keeps = 0;  // bit t: round t's slot is kept
  for (int t = 0; t < its; ++t) {
    const int i = w0 + 32 * t;
    const bool in = i < cnt, k = in && kept(i), below = in && s0 + i < keep;
    keeps |= (k ? 1u : 0u) << t;
    mine.x += __popc(__ballot_sync(0xffffffffu, below && !k));
    mine.y += __popc(__ballot_sync(0xffffffffu, k && !below));
  }
  uint2 at = evict_warp_scan(mine, sm.warp_tot, tot);  // of this warp
  if (tid == 0) sm.sums = tot;
  cluster.sync();
  uint2 all = make_uint2(0, 0);
#pragma unroll
  for (int r = 0; r < kEvMaxCluster; ++r)
    if (r < ncta) {
      const uint2 v = cluster.map_shared_rank(&sm, r)->sums;
      if (r < rank) {
        at.x += v.x;
        at.y += v.y;
      }
      all.x += v.x;
      all.y += v.y;
    }
  int2* moves = ws.moves + seq * ws.cap;
  int64_t* macc = ws.moved_acc + seq * (ws.cap + 1);
  int32_t* mpos = ws.moved_pos + seq * ws.cap;
  const uint32_t lt = (1u << lane) - 1u;
  uint2 r = at;
  for (int t = 0; t < its; ++t) {
    const int i = w0 + 32 * t;
    const bool in = i < cnt, k = (keeps >> t) & 1u, below = in && s0 + i < keep;
    const uint32_t free_slots = __ballot_sync(0xffffffffu, below && !k), late = __ballot_sync(0xffffffffu, k && !below);
    if (below && !k) moves[r.x + __popc(free_slots & lt)].x = static_cast<int32_t>(s0 + i);
    if (k && !below) {
      const uint32_t to = r.y + __popc(late & lt);
      moves[to].y = static_cast<int32_t>(s0 + i);
      macc[to] = sm.acc[i];
      mpos[to] = sm.pos[i];
    }
    r.x += __popc(free_slots);
    r.y += __popc(late);
  }
  if (tid == 0 && rank == 0) {
    if (all.x != all.y) report(kDevBounds);  // original numbers that occur twice
    ws.count[seq] = static_cast<int32_t>(min(all.x, all.y));
  }
  __threadfence();
  cluster.sync();  // the lists are complete, and every weight has been read
  // new weights and numbers: kept blocks that stay, then the moved ones; no weight behind them
  int64_t* ao = acc_out + seq * slots;
  int32_t* po = pos_out + seq * slots;
  uint32_t hole = at.x;
#pragma unroll 4
  for (int t = 0; t < its; ++t) {
    const int i = w0 + 32 * t;
    const bool k = (keeps >> t) & 1u, below = i < cnt && s0 + i < keep;
    const uint32_t free_slots = __ballot_sync(0xffffffffu, below && !k);
    if (below) {
      const uint32_t h = hole + __popc(free_slots & lt);
      ao[s0 + i] = k ? sm.acc[i] : h < all.y ? macc[h] : 0;
      po[s0 + i] = k ? sm.pos[i] : h < all.y ? mpos[h] : -1;
    }
    hole += __popc(free_slots);
  }
  for (int64_t s = keep + static_cast<int64_t>(rank) * kEvictThreads + tid; s < slots; s += static_cast<int64_t>(ncta) * kEvictThreads)
    ao[s] = s == keep && part ? tail_acc : 0;
  cluster.sync();  // no CTA leaves while others may read its shared memory
}

// ---------------------------------------------------------------------------
// Moves the blocks' bytes, 256 words (4 KB of 16-byte words) per warp and step,
// eight loads per lane in flight: a piece of one move's block, or, for arrays of
// at most 128 words per block, as many whole blocks of consecutive moves as fit.
// Where the incomplete block's new slot held a block that moves (it is the
// first move then), the lane that copies a word of that move copies the same word
// of the incomplete block after it.
// Bound: HBM, every moved byte read and written once.
// ---------------------------------------------------------------------------
constexpr int kMovePiece = 256;
constexpr int kMoveWarps = 8;

// Warp steps that `count` moves of an array with that many words per block take.
__host__ __device__ inline int64_t move_steps(int64_t words, int64_t count) {
  if (words > kMovePiece / 2) return count * ((words + kMovePiece - 1) / kMovePiece);
  const int64_t group = kMovePiece / words;
  return (count + group - 1) / group;
}

// One step of large blocks: words [w0, w0 + 256) of a block.
template <typename T>
__device__ __forceinline__ void move_large(T* dst, const T* src, int w0, int words, int lane) {
  src += w0 + lane;
  dst += w0 + lane;
  if (w0 + kMovePiece <= words) {
    T v[kMovePiece / 32];
#pragma unroll
    for (int i = 0; i < kMovePiece / 32; ++i) v[i] = src[32 * i];
#pragma unroll
    for (int i = 0; i < kMovePiece / 32; ++i) dst[32 * i] = v[i];
  } else {
#pragma unroll 1
    for (int w = w0 + lane; w < words; w += 32, src += 32, dst += 32) *dst = *src;
  }
}

// One step of small blocks: the blocks of moves [m0, m0 + 256 / words).
template <typename T>
__device__ __forceinline__ void move_small(T* base, int words, int64_t m0, const int2* moves, int64_t count, int lane) {
  const int group = static_cast<int>(min(static_cast<int64_t>(kMovePiece / words), count - m0));
#pragma unroll 4
  for (int x = lane; x < group * words; x += 32) {
    const int g = x / words, w = x - g * words;
    const int2 mv = moves[m0 + g];
    base[static_cast<int64_t>(mv.x) * words + w] = base[static_cast<int64_t>(mv.y) * words + w];
  }
}

template <typename T>
__device__ __forceinline__ void move_step(T* base, int words, int64_t step, const int2* moves, int64_t count, bool chained,
                                          int64_t to0, int64_t from0, int lane) {
  if (words > kMovePiece / 2) {
    const int per = (words + kMovePiece - 1) / kMovePiece;
    const int64_t m = step / per;
    const int w0 = static_cast<int>(step - m * per) * kMovePiece;
    const int2 mv = moves[m];
    move_large(base + static_cast<int64_t>(mv.x) * words, base + static_cast<int64_t>(mv.y) * words, w0, words, lane);
    if (chained && m == 0) move_large(base + to0 * words, base + from0 * words, w0, words, lane);
  } else {
    const int64_t m0 = step * (kMovePiece / words);
    move_small(base, words, m0, moves, count, lane);
    if (chained && m0 == 0) {  // word w of move 0 was lane w % 32's
      for (int w = lane; w < words; w += 32) base[to0 * words + w] = base[from0 * words + w];
    }
  }
}

// Moves of the kept blocks into the freed slots, array by array.
// Bound: HBM.  Measured with the selection, in a CUDA graph: 16 x 4096 -> 2800 blocks
// 76.9 us and 2 x 65536 -> 49152 132.7 us (bytes at the copy rate: 53.7, 93.1 us).
__global__ void __launch_bounds__(kMoveWarps * 32, 4)
evict_move_kernel(const __grid_constant__ EvictArrays ar, int arrays, int tail_arrays, EvictWs ws, int64_t n, int part, int64_t keep, int64_t slots) {
  const int64_t seq = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int count = ws.count[seq];
  const int2* moves = ws.moves + seq * ws.cap;
  const bool tail = part && keep < n;                       // the incomplete block moves to slot `keep`
  const bool chained = tail && count > 0 && moves[0].y == keep;
  const int2 tail_move = make_int2(static_cast<int32_t>(keep), static_cast<int32_t>(n));
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kMoveWarps;
  int64_t it = static_cast<int64_t>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5);
  // steps in order: the moves of every array, then the incomplete block's
  // (unless the lanes of move 0 take it along)
  for (int x = 0; x < arrays + (tail ? arrays + tail_arrays : 0); ++x) {
    const bool t = x >= arrays;
    const int y = t ? x - arrays : x;
    if (t && chained && y < arrays) continue;
    const int words = static_cast<int>(ar.bytes[y] >> ar.shift[y]);
    const int64_t cnt = t ? 1 : count;
    const int64_t steps = move_steps(words, cnt);
    const int2* mv = t ? &tail_move : moves;
    const bool ch = !t && chained;
    uint8_t* base = ar.base[y] + seq * slots * ar.bytes[y];
    for (; it < steps; it += warps) {
      switch (ar.shift[y]) {
        case 4: move_step(reinterpret_cast<uint4*>(base), words, it, mv, cnt, ch, keep, n, lane); break;
        case 2: move_step(reinterpret_cast<uint32_t*>(base), words, it, mv, cnt, ch, keep, n, lane); break;
        default: move_step(base, words, it, mv, cnt, ch, keep, n, lane);
      }
    }
    it -= steps;
  }
}

}  // namespace sgqa
