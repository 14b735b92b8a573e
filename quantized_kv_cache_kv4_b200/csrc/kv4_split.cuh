// A batch of T work items (runs of pages, in sequence order) split into equal contiguous shares,
// one per worker (a warp, or a CTA): no work list, no counter and no launch of its own. Every CTA
// scans the sequences' item counts itself (a few KB of lengths from L2), so that a share starts
// with a search over the block's scan and a walk over one thread's run of sequences.
#pragma once

#include <stdint.h>

namespace kv4 {

constexpr int kSplitThreads = 128;  // threads of a CTA that scan (its first 4 warps)

// The share of worker w and the owner of item t, for T items over up to W workers with at
// least `least` items each: the first `more` workers take per + 1 items, the others per.
struct Shares {
  long long per, more;
  __device__ __forceinline__ Shares(long long T, int W, int least) {
    const long long w = max(1LL, min(static_cast<long long>(W), T / least));
    per = T / w;
    more = T - per * w;
  }
  __device__ __forceinline__ long long begin(long long w) const { return w * per + min(w, more); }
  __device__ __forceinline__ int owner(long long t) const {
    const long long cut = more * (per + 1);
    return static_cast<int>(t < cut ? t / (per + 1) : more + (t - cut) / max(1LL, per));
  }
};

struct SplitSmem {
  long long scan[kSplitThreads + 1];
  long long wsum[kSplitThreads / 32];
};

// The share [begin, end) of a worker, and the sequence its first item is in (whose first item is
// seq_first). An empty share has begin >= end.
struct Share {
  long long begin, end, seq_first;
  int b;
};

// The share of worker `me` of W from the block's scan (after take_share; no barrier).
// items(b, check): items of sequence b (>= 0).
template <class Items>
__device__ __forceinline__ Share find_share(int B, int me, int W, int least, const SplitSmem &sm,
                                            Items items) {
  const int run = (B + kSplitThreads - 1) / kSplitThreads;
  const long long T = sm.scan[kSplitThreads];
  const Shares sh(T, W, least);
  Share s{sh.begin(me), min(sh.begin(me + 1), T), 0, 0};
  if (s.begin >= s.end) return s;
  int lo = 0, hi = kSplitThreads - 1;  // the last run that starts at or before the share
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sm.scan[mid] <= s.begin) lo = mid; else hi = mid - 1;
  }
  s.b = lo * run;
  s.seq_first = sm.scan[lo];
  for (;;) {
    const long long n = items(s.b, false);
    if (s.begin < s.seq_first + n) break;
    s.seq_first += n;
    ++s.b;
  }
  return s;
}

// The block's scan, and the share of worker `me` (a warp's lanes pass the same). All threads of the
// block call it; items are asked for with check set once per sequence and block.
template <class Items>
__device__ __forceinline__ Share take_share(int B, int me, int W, int least, SplitSmem &sm, Items items) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int run = (B + kSplitThreads - 1) / kSplitThreads;
  long long mine = 0;
  const bool scans = threadIdx.x < kSplitThreads;
  for (int i = 0; scans && i < run; ++i) {
    const int b = threadIdx.x * run + i;
    if (b < B) mine += items(b, true);
  }
  long long incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (scans && lane == 31) sm.wsum[warp] = incl;
  __syncthreads();
  if (scans) {
    long long base = 0;
    for (int i = 0; i < warp; ++i) base += sm.wsum[i];
    sm.scan[threadIdx.x + 1] = base + incl;
  }
  if (threadIdx.x == 0) sm.scan[0] = 0;
  __syncthreads();
  return find_share(B, me, W, least, sm, items);
}

}  // namespace kv4
