// Attention over the 8-bit block-scaled cache for many query rows of a sequence: prefill
// chunks and the verification of drafted tokens, on the tcgen05 tensor cores.
//
// Rows. Row r of a (sequence, kv head) is position i = r / G of its last n positions and query
// head g = r % G, so a tile of 128 rows shares every K and V block it reads. Key tiles are 128
// positions (8 pages).
//
// A CTA runs two pipelines of 128 rows each:
//   softmax warps (4 + 4)  one thread per row: the row's logits from TMEM, the running maximum
//                          and sum, the weights back to TMEM over the logits;
//   MMA warp               one thread issues S = Q K^T (both operands in shared memory) and
//                          O += P V (P in TMEM); accumulators S and O in TMEM, 4 x 128 columns;
//   loading warp           page ids, scales, and the pages' codes into shared memory by bulk copies;
//   convert warps (4)      write the codes as fp16 (exact for both formats) into the 128-byte-
//                          swizzled tiles the MMAs read;
//   scheduling warp        the CTA's runs of key tiles.
// The pipelines hold rows 0-127 and 128-255 of one unit and read the same key tiles, which are
// converted once (two stages).
//
// Scales. A key block's scale multiplies its 16 logits, a value block's scale its 16 weights:
// P = p 2^7 vs / 2^vref with vref the exponent of the largest value scale so far, so P is at
// most 2^15 (p up to 2^8: the maximum a row subtracts is moved only when it is outgrown by
// that factor, which spares most rescales of O). fp16 keeps 11 significant bits of P down to
// 2^-14, and 2^-25 below: about 2^-31 of the largest weight times the largest value scale.
//
// Split. The key tiles of all units, in order, are dealt to the workers in equal contiguous
// shares; units that two or more workers share leave partial records (first and last unit of
// a worker) for the merge.
//
// What bounds it. 2 chunks of 3900-4096 positions over 7000-8192 (743 GFLOP): 875 us a call among
// others in INT8 (850 TFLOP/s), 2 to 3 % less in e4m3. Of the ~5000 cycles of a key tile the products
// take 2050 (both pipelines'), a pipeline's softmax 2900 (of which the exponentials 1100-2100, as the
// other's fall together with them), and a pipeline's softmax waits for its own products. One MMA warp
// that takes the pipelines in turn keeps them out of phase (two warps, one per pipeline: 999 us). The
// roles' instructions contend: the loops are short in code where they can be (the convert loop
// unrolled by 8 instead of 1 costs a fifth of the kernel, exponentials by polynomial on the FMA pipe 6
// to 20 %, half rows per thread with 16 softmax warps 2 %).
#include <algorithm>

#include "kv4_block8.cuh"

namespace kv4 {

constexpr int kTile = 128;               // rows of a pipeline, positions of a key tile
constexpr int kUnitRows = 2 * kTile;     // query rows of a unit: both pipelines'
constexpr int kTilePages = kTile / kPage;
constexpr int kOperandBytes = kTile * kHeadDim * 2;  // one fp16 operand tile: 32 KB
constexpr int kTileThreads = 512;        // 8 softmax and 4 convert warps, one each for MMA, scheduling, loading
// registers per thread of the three kinds: 256 x 192 + 128 x 64 + 128 x 64 = 512 x 128, what
// the block is launched with
constexpr int kSoftmaxRegs = 192, kConvertRegs = 64, kMmaRegs = 64;
constexpr int kRawBytes = kTilePages * kInt8CodeBytes;  // a key tile's K or V codes: 16 KB
constexpr int kTileSmem = 6 * kOperandBytes + 2 * kRawBytes + 1024;  // Q, K, V x 2, codes (+ alignment)
constexpr int kTileCtas = 148;           // one per SM (shared memory)
constexpr int kTileMinShare = 1;         // key tiles of a worker: ~2.5 us of work, a record's join is less
constexpr float kLazy = 8.0f;            // log2 of how far a row may outgrow its maximum
constexpr float kPShift = 7.0f;          // P is at most 2^(kLazy + kPShift)
constexpr uint32_t kTileWait = 1u << 18;  // attempts of one bounded wait

// ---------------------------------------------------------------------------
// tcgen05
// ---------------------------------------------------------------------------
// Instruction descriptor of kind::f16, fp16 x fp16 -> fp32, M = N = 128: D format f32 at bit 4,
// B transposed (MN-major) at bit 16, N / 8 at bit 17, M / 16 at bit 24.
constexpr uint32_t kIdescQK = (1u << 4) | ((kTile / 8) << 17) | ((kTile / 16) << 24);
constexpr uint32_t kIdescPV = kIdescQK | (1u << 16);

// Shared-memory operand descriptor, 128-byte swizzle: address / 16, leading offset / 16 at bit
// 16, stride offset / 16 at bit 32, version 1 at bit 46, swizzle mode 2 at bit 61. Operand
// tiles are [2 halves of 64 dims][128 rows][128 bytes]: groups of 8 rows are 1024 bytes apart
// (stride offset), the halves 16384 bytes (leading offset, read for the MN-major V).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(16384 >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// 1 in one lane of the warp, the same one each time.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// Issued by the lane whose `one` is set; the whole warp calls it.
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(one)
      : "memory");
}
// The barrier gets one arrival when every MMA this thread has issued so far is done.
__device__ __forceinline__ void mma_commit(uint32_t one, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)), "r"(one)
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 32 columns of this warp's 32 TMEM lanes, one lane per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::
          "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(addr));
}

template <int N>
struct Setmax {
  static __device__ __forceinline__ void inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
  static __device__ __forceinline__ void dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
};

// ---------------------------------------------------------------------------
// units and segments
// ---------------------------------------------------------------------------
struct SeqTiles : SeqRows {
  int units, per_head;  // units of a kv head, and their key tiles together
  int gqa;
  __device__ __forceinline__ int unit_tiles(int u) const {  // at least 1: an empty unit writes zeros
    const int last = min(n - 1, ((u + 1) * kUnitRows - 1) / gqa);  // its last position
    return max(0, L - n + last) / kTile + 1;
  }
};

__device__ __forceinline__ SeqTiles tiles_of_seq(const CacheView &c, const Queries &qs, int b,
                                                       int32_t *err) {
  SeqTiles s;
  static_cast<SeqRows &>(s) = rows_of(c, qs, b, err);
  s.gqa = c.gqa;
  s.units = static_cast<int>((static_cast<long long>(s.n) * c.gqa + kUnitRows - 1) / kUnitRows);
  s.per_head = 0;
  for (int u = 0; u < s.units; ++u) s.per_head += s.unit_tiles(u);
  return s;
}

// A worker's next run of key tiles of one unit.
struct Segments {
  const CacheView &c;
  const Queries &qs;
  Share share;
  long long at;
  int b;
  long long seq_first;
  SeqTiles sq;
  // the segment: unit u of kv head h, its key tiles [k0, k1) of nt
  int h, u, k0, k1, nt;
  bool first;  // the worker's first

  __device__ __forceinline__ Segments(const CacheView &cc, const Queries &q, const Share &s)
      : c(cc), qs(q), share(s), at(s.begin), b(s.b), seq_first(s.seq_first) {
    if (share.begin < share.end) sq = tiles_of_seq(c, qs, b, nullptr);
  }
  __device__ __forceinline__ bool next() {
    if (at >= share.end) return false;
    while (at >= seq_first + static_cast<long long>(c.num_kv_heads) * sq.per_head) {
      seq_first += static_cast<long long>(c.num_kv_heads) * sq.per_head;
      sq = tiles_of_seq(c, qs, ++b, nullptr);
    }
    const long long in_seq = at - seq_first;
    h = static_cast<int>(in_seq / sq.per_head);
    int rest = static_cast<int>(in_seq - static_cast<long long>(h) * sq.per_head);
    u = 0;
    while (rest >= (nt = sq.unit_tiles(u))) {
      rest -= nt;
      ++u;
    }
    k0 = rest;
    k1 = static_cast<int>(min(static_cast<long long>(nt), k0 + (share.end - at)));
    first = at == share.begin;
    at += k1 - k0;
    return true;
  }
};

// What a key tile's blocks are scaled by; a ring of four, so that a slot is written again only after
// the softmax threads have left it.
struct alignas(16) TileScales {
  float ks[kTilePages];  // negative: the page is left out
  float cv[kTilePages];  // vs 2^(kPShift - vref)
  float vref;            // exponent with every value scale of the segment so far at most 2^vref
  float moved;           // vref before this tile, less vref (0: it has not moved)
  int left;              // positions of the tile within the length (negative: no more tiles)
  int pages;             // bit p: page p of the tile was copied
  int any_bad;
};

// A segment as the scheduling warp hands it to the others (b < 0: no more).
struct Seg {
  int b, h, u, k0, k1, nt, first;
  int L, n, row0;  // the sequence's length, queries and first query row
};
constexpr int kSegRing = 4;

struct TileBars {
  uint64_t seg_full[kSegRing], seg_empty[kSegRing];
  uint64_t q_full[2], s_full[2], p_full[2];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t raw_full[2], raw_empty[2];  // the codes of K, of V
  uint64_t idle;                       // the last of the products is done
};

// The logits of positions that a row does not see, -inf: all but the tile's first `left`, and
// those of pages that are left out.
__device__ __forceinline__ void mask_logits(uint32_t (&s)[4][32], const TileScales &sl, int left) {
#pragma unroll
  for (int x = 0; x < kTilePages; ++x) {
    const int n = sl.ks[x] < 0.f ? 0 : left - 16 * x;
#pragma unroll
    for (int y = 0; y < 16; ++y) {
      uint32_t &v = s[x >> 1][16 * (x & 1) + y];
      v = y < n ? v : 0xff800000u;
    }
  }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int F>
__global__ void __launch_bounds__(kTileThreads, 1) block8_tile_kernel(CacheView c, Queries qs, Outputs out,
                                                                     float *__restrict__ partials,
                                                                     Crossing *__restrict__ notes,
                                                                     Waits waits, int32_t *err) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ SplitSmem split;
  __shared__ TileBars bars;
  __shared__ TileScales scales[4];
  __shared__ Seg segs[kSegRing];
  __shared__ uint32_t tmem_base_s;
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int H = c.num_kv_heads, G = c.gqa;
  // pipeline of a softmax warp: warps 0-3 and 4-7; convert warps 8-11, the MMA warp 12, the scheduling
  // warp 14 and the loading warp 15 serve both
  const int pipe = (warp >> 2) & 1;

  if (threadIdx.x == 0) {
    for (int k = 0; k < kSegRing; ++k) {
      mbar_init(&bars.seg_full[k], 1);
      mbar_init(&bars.seg_empty[k], 10);  // warps that read it
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 4);
      mbar_init(&bars.s_full[i], 2);  // the MMAs' completion, and the issuing thread itself
      mbar_init(&bars.p_full[i], 4);
      mbar_init(&bars.k_full[i], 4);
      mbar_init(&bars.v_full[i], 4);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_empty[i], 1);
      mbar_init(&bars.raw_full[i], 1);
      mbar_init(&bars.raw_empty[i], 4);
    }
    mbar_init(&bars.idle, 1);
    fence_barrier_init();
  }
  if (warp == 12) {  // all 512 columns: S and O of both pipelines
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base_s))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  const int me = blockIdx.x, workers = gridDim.x;
  auto items = [&](int i, bool check) {
    return static_cast<long long>(H) *
           tiles_of_seq(c, qs, i, check && blockIdx.x == 0 ? err : nullptr).per_head;
  };
  const Share share = take_share(c.num_seqs, me, workers, kTileMinShare, split, items);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  const uint32_t tm_s = tmem + 256 * pipe, tm_o = tm_s + 128;
  uint8_t *q_tile = smem + pipe * kOperandBytes;
  uint8_t *k_tiles = smem + 2 * kOperandBytes, *v_tiles = smem + 4 * kOperandBytes;
  uint8_t *raw = smem + 6 * kOperandBytes;  // K's codes, then V's
  auto stage_of = [](int k) { return k & 1; };  // of the worker's k-th tile
  auto phase_of = [](int k) { return (k >> 1) & 1; };
  auto slot_of = [&](int k) -> TileScales & { return scales[k & 3]; };
  auto wait = [&](uint64_t *bar, int parity) {
    if (mbar_wait_bounded(bar, parity, waits.limit)) return true;
    set_err(err, KV4_DEVERR_TIMEOUT);
    return false;
  };
  int kt = 0;      // tiles of the worker so far
  int seg_no = 0;  // segments read from the ring so far
  bool ok = true;  // no wait has given up
  auto read_seg = [&](int no, Seg &s) {  // all lanes of a warp; false: no more
    const int at = no & (kSegRing - 1);
    ok = __all_sync(0xffffffffu, wait(&bars.seg_full[at], (no / kSegRing) & 1));
    if (!ok) return false;
    s = segs[at];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.seg_empty[at]);
    return s.b >= 0;
  };

  // (a warpgroup's warps execute one setmaxnreg together, before they part)
  if (warp >= 12) {
    Setmax<kMmaRegs>::dec();
    if (warp == 15) {
      // ------------------------------- load -------------------------------
      // Page ids a tile ahead of their scales, and those a tile ahead of the copies.
      struct Meta {
        int kt;         // the worker's tile number, -1: no tile
        int k, L;       // the key tile, the length
        int h, pid;     // kv head; page (lane % 8) of the tile (-2: behind the length)
        uint16_t ks, vs;  // and its scales
        bool first;     // the segment's first tile
      };
      Seg sg;
      int at = 0, end = 0, n_tiles = 0;
      bool more = true;
      float vref = 0.f;
      auto ask_page = [&]() {  // the next tile and its page ids
        Meta m{-1, 0, 0, 0, -2, 0, 0, false};
        if (at == end) {
          more = more && read_seg(seg_no++, sg);
          if (!more) return m;
          at = sg.k0;
          end = sg.k1;
        }
        m.kt = n_tiles++;
        m.first = at == sg.k0;
        m.k = at++;
        m.L = sg.L;
        m.h = sg.h;
        const int page = m.k * kTilePages + (lane & 7);
        if (page < (m.L + kPage - 1) / kPage)
          m.pid = __ldg(c.page_table + static_cast<size_t>(sg.b) * c.max_pages + page);
        return m;
      };
      auto ask_scales = [&](Meta &m) {  // of its pages, and whether the ids are any
        if (m.kt < 0 || m.k * kTilePages + (lane & 7) >= (m.L + kPage - 1) / kPage) return;
        if (m.pid < 0 || m.pid >= c.num_pages) {
          set_err(err, KV4_DEVERR_PAGE_ID);
          m.pid = -1;
        } else {
          m.ks = __ldg(c.k_params + static_cast<size_t>(m.pid) * H + m.h);
          m.vs = __ldg(c.v_params + static_cast<size_t>(m.pid) * H + m.h);
        }
      };
      Meta cur = ask_page();
      ask_scales(cur);
      Meta nxt = ask_page();
      int k = 0;
      for (; ok; ++k) {
        ok = __all_sync(0xffffffffu, wait(&bars.raw_empty[0], (k & 1) ^ 1));
        if (!ok) break;
        TileScales &sl = slot_of(k);
        if (cur.kt < 0) {  // no more tiles
          if (lane == 0) {
            sl.left = -1;
            mbar_arrive(&bars.raw_full[0]);
          }
          break;
        }
        const float ks = cur.pid == -1 ? -1.f : __half2float(__ushort_as_half(cur.ks));
        const float vs = __half2float(__ushort_as_half(cur.vs));
        float top = vs;
#pragma unroll
        for (int off = 1; off < kTilePages; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const unsigned there = __ballot_sync(0xffffffffu, cur.pid >= 0) & 0xffu;
        const unsigned bad = __ballot_sync(0xffffffffu, cur.pid == -1);
        int e = -24;
        if (top > 0.f) frexpf(top, &e);  // top < 2^e
        const float before = cur.first ? static_cast<float>(e) : vref;
        vref = fmaxf(before, static_cast<float>(e));
        if (lane < kTilePages) {
          sl.ks[lane] = ks;
          sl.cv[lane] = vs * fast_exp2(kPShift - vref);
        }
        if (lane == 0) {
          sl.vref = vref;
          sl.moved = before - vref;
          sl.left = min(kTile, max(0, cur.L - cur.k * kTile));
          sl.pages = static_cast<int>(there);
          sl.any_bad = bad != 0u;
        }
        __syncwarp();
        const size_t off = (static_cast<size_t>(max(cur.pid, 0)) * H + cur.h) * kInt8CodeBytes;
        const uint32_t bytes = __popc(there) * kInt8CodeBytes;
        fence_proxy_async_smem();
        const bool asks = k > 0 || me != waits.withheld;  // (the testing hook)
        if (lane == 0 && asks) mbar_arrive_expect_tx(&bars.raw_full[0], bytes);
        __syncwarp();
        if (lane < kTilePages && cur.pid >= 0 && asks)
          bulk_g2s(raw + lane * kInt8CodeBytes, c.k_codes + off, kInt8CodeBytes, &bars.raw_full[0]);
        ok = __all_sync(0xffffffffu, wait(&bars.raw_empty[1], (k & 1) ^ 1));
        if (!ok) {  // (this tile's K, the last one's V)
          wait(&bars.raw_full[0], k & 1);
          if (k > 0) wait(&bars.raw_full[1], (k & 1) ^ 1);
          k = 0;
          break;
        }
        fence_proxy_async_smem();
        if (lane == 0) mbar_arrive_expect_tx(&bars.raw_full[1], bytes);
        __syncwarp();
        if (lane < kTilePages && cur.pid >= 0)
          bulk_g2s(raw + kRawBytes + lane * kInt8CodeBytes, c.v_codes + off, kInt8CodeBytes, &bars.raw_full[1]);
        cur = nxt;
        ask_scales(cur);
        nxt = ask_page();
      }
      // However the loop ended (by a wait for the next segment that gave up, too), the last copies land
      // before the block ends: the convert warps may have given up on them. (Before the end's mark,
      // which is a phase of K's barrier, K's last copy has been converted.)
      if (k > 0 && !ok) wait(&bars.raw_full[0], (k & 1) ^ 1);
      if (k > 0) wait(&bars.raw_full[1], (k & 1) ^ 1);
    } else if (warp == 14) {
      // ------------------------------- schedule -------------------------------
      if (lane == 0) {
        Segments sg(c, qs, share);
        notes[me].rows = 0;
        for (int no = 0;; ++no) {
          const bool more = sg.next();
          if (no == 0 && more)
            notes[me] = crossing(Shares(split.scan[kSplitThreads], workers, kTileMinShare), me, share.begin - sg.k0,
                                 sg.nt, sg.k0, sg.sq.row0, sg.h, sg.u * kUnitRows,
                                 min(kUnitRows, sg.sq.n * G - sg.u * kUnitRows));
          const int at = no & (kSegRing - 1);
          if (!wait(&bars.seg_empty[at], ((no / kSegRing) & 1) ^ 1)) break;
          segs[at] = more ? Seg{sg.b, sg.h, sg.u, sg.k0, sg.k1, sg.nt, sg.first, sg.sq.L, sg.sq.n, sg.sq.row0}
                                : Seg{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0};
          mbar_arrive(&bars.seg_full[at]);
          if (!more) break;
        }
      }
    } else if (warp == 12) {
      // ------------------------------- MMA -------------------------------
      // One warp for both pipelines, in turn: a step's products of one are issued together (mixed with
      // the other's, both would end at the time of the later one), so that they run under the other's
      // softmax. The warp goes through this together and one lane issues: descriptors and barrier
      // addresses are then the warp's (uniform registers), not to be moved there for each instruction.
      int seg = 0, pp0 = 0, pp1 = 0, q1 = 0;  // segments; phases of the p_full and of the second q_full
      const uint32_t one = elect_one();
      const uint64_t qd0 = smem_desc(smem_u32(smem));
      const uint64_t kd0 = smem_desc(smem_u32(k_tiles)), vd0 = smem_desc(smem_u32(v_tiles));
      auto all = [&](uint64_t *bar, int parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
      // S (or the last O) is there; the thread's own arrival hands on what it has seen of the convert
      // warps' writes (the tile's scales)
      auto done = [&](int p) {
        mma_commit(one, &bars.s_full[p]);
        if (one) mbar_arrive(&bars.s_full[p]);
      };
      auto qk = [&](int p, int k) {  // (K is there)
        const uint64_t qd = qd0 + static_cast<uint64_t>((p * kOperandBytes) >> 4);
        const uint64_t kd = kd0 + static_cast<uint64_t>((stage_of(k) * kOperandBytes) >> 4);
#pragma unroll
        for (int x = 0; x < 8; ++x) {  // 16 dims: 32 bytes of a row; the halves 16 KB apart
          const uint64_t off = static_cast<uint64_t>(((x >> 2) * 16384 + (x & 3) * 32) >> 4);
          mma_ss(one, tmem + 256 * p, qd + off, kd + off, kIdescQK, x > 0);
        }
      };
      auto pv = [&](int p, int k, bool acc) {
        const uint64_t vd = vd0 + static_cast<uint64_t>((stage_of(k) * kOperandBytes) >> 4);
#pragma unroll
        for (int x = 0; x < 8; ++x)  // 16 positions: 16 rows of 128 bytes, 8 columns of P
          mma_ts(one, tmem + 256 * p + 128, tmem + 256 * p + 8 * x, vd + static_cast<uint64_t>((x * 2048) >> 4),
                 kIdescPV, acc || x > 0);
      };
      Seg sg;
      while (ok && read_seg(seg_no++, sg)) {
        const int n = __reduce_max_sync(0xffffffffu, sg.k1 - sg.k0);  // (uniform, and known to be)
        const bool two = __all_sync(0xffffffffu, sg.u * kUnitRows + kTile < sg.n * G);  // second pipeline has rows
        ok = all(&bars.k_full[stage_of(kt)], phase_of(kt)) && all(&bars.q_full[0], seg & 1);
        ++seg;
        if (!ok) break;
        tc_fence_after();
        qk(0, kt);
        done(0);
        if (two) {
          ok = all(&bars.q_full[1], q1 & 1);
          ++q1;
          if (!ok) break;
          tc_fence_after();
          qk(1, kt);
          done(1);
        }
        mma_commit(one, &bars.k_empty[stage_of(kt)]);
        for (int j = 0; ok && j < n; ++j) {
          const int st = stage_of(kt + j), next = stage_of(kt + j + 1);
          const bool more = j + 1 < n;
          // all that the products need but the weights is waited for ahead of them
          ok = all(&bars.v_full[st], phase_of(kt + j));
          if (more) ok = ok && all(&bars.k_full[next], phase_of(kt + j + 1));
          ok = ok && all(&bars.p_full[0], pp0 & 1);
          ++pp0;
          if (!ok) break;
          tc_fence_after();
          pv(0, kt + j, j > 0);
          if (more) qk(0, kt + j + 1);
          done(0);
          if (two) {
            ok = all(&bars.p_full[1], pp1 & 1);
            ++pp1;
            if (!ok) break;
            tc_fence_after();
            pv(1, kt + j, j > 0);
            if (more) qk(1, kt + j + 1);
            done(1);
          }
          mma_commit(one, &bars.v_empty[st]);
          if (more) mma_commit(one, &bars.k_empty[next]);
        }
        kt += n;
      }
      mma_commit(one, &bars.idle);  // (and all arrivals of the tensor cores have been made: the block may end)
      all(&bars.idle, 0);
    }
  } else if (warp >= 8) {
    // ------------------------------- convert -------------------------------
    Setmax<kConvertRegs>::dec();
    // 128 threads, a 16-byte piece (16 dims of a position) of each page each.
    const int tid = threadIdx.x - 256;
    const int strip = tid >> 4, slot = tid & 15;
    const uint32_t chunk = (strip & 3) * 2;  // of 16 bytes, xor-swizzled by the row (its low bits: the slot's)
    const uint32_t to0 = (strip >> 2) * 16384 + slot * 128 + ((chunk ^ (slot & 7)) << 4);
    const uint32_t to1 = (strip >> 2) * 16384 + slot * 128 + (((chunk + 1) ^ (slot & 7)) << 4);
    // one tile's K (which = 0) or V
    auto convert = [&](int which, const uint8_t *from, uint8_t *to, uint64_t *empty, uint64_t *full, int left,
                       int pages, int free_phase) {
      ok = __all_sync(0xffffffffu, wait(empty, free_phase));
      if (!ok) return;
#pragma unroll 1
      for (int p = 0; p < kTilePages; ++p) {
        uint4 v = *reinterpret_cast<const uint4 *>(from + p * kInt8CodeBytes + tid * 16);
        // what lies behind the length, or of a page that was not copied, may hold anything
        if (p * kPage + slot >= left || !((pages >> p) & 1)) v = make_uint4(0u, 0u, 0u, 0u);
        uint32_t o[8];
        code_pairs<F, false>(v.x, o[0], o[1]);
        code_pairs<F, false>(v.y, o[2], o[3]);
        code_pairs<F, false>(v.z, o[4], o[5]);
        code_pairs<F, false>(v.w, o[6], o[7]);
        *reinterpret_cast<uint4 *>(to + p * 2048 + to0) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(to + p * 2048 + to1) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(full);
        mbar_arrive(&bars.raw_empty[which]);
      }
    };
    for (int k = 0; ok; ++k) {
      ok = __all_sync(0xffffffffu, wait(&bars.raw_full[0], k & 1));
      if (!ok) break;
      const int left = slot_of(k).left, pages = slot_of(k).pages;
      if (left < 0) break;
      const int st = stage_of(k), free_phase = phase_of(k) ^ 1;
      convert(0, raw, k_tiles + st * kOperandBytes, &bars.k_empty[st], &bars.k_full[st], left, pages, free_phase);
      ok = ok && __all_sync(0xffffffffu, wait(&bars.raw_full[1], k & 1));
      if (ok)
        convert(1, raw + kRawBytes, v_tiles + st * kOperandBytes, &bars.v_empty[st], &bars.v_full[st], left, pages,
                free_phase);
    }
  } else {
    // ------------------------------- softmax -------------------------------
    Setmax<kSoftmaxRegs>::inc();
    const int row = threadIdx.x & 127;  // of the pipeline; its TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(warp & 3) << 21;  // lane 32 (warp % 4), bits 16+
    const uint32_t ts = tm_s + lane_off, to = tm_o + lane_off;
    int sp = 0;  // phases of s_full
    Seg sg;
    while (ok && read_seg(seg_no++, sg)) {
      const int n_tiles = sg.k1 - sg.k0;
      const int r0 = sg.u * kUnitRows + pipe * kTile;
      const int rows = sg.n * G;
      if (r0 >= rows) {  // (the MMA warp skips it too)
        kt += n_tiles;
        continue;
      }
      const int r = r0 + row;
      const bool live = r < rows;
      const int i = r / G;
      const size_t qr = static_cast<size_t>(sg.row0 + i) * H * G + sg.h * G + r % G;
      const int lim = live ? sg.L - sg.n + i : -1;  // last position the row sees
      float a;  // logit units: step of the fixed query times log2(e) / sqrt(128)
      {
        // Two of the warp's rows at a time, 16 lanes each: whole lines are read.
        uint4 v[16];
        float amax = 0.f;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int from = 2 * x + (lane >> 4);
          const size_t at = (static_cast<size_t>(sg.row0 + __shfl_sync(0xffffffffu, i, from)) * H + sg.h) * G +
                            __shfl_sync(0xffffffffu, r - i * G, from);
          v[x] = r - lane + from < rows ? reinterpret_cast<const uint4 *>(qs.q + at * kHeadDim)[lane & 15]
                                        : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
          float top = 0.f;
#pragma unroll
          for (int y = 0; y < 4; ++y)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[y] << 16)), fabsf(__uint_as_float(w[y] & 0xFFFF0000u))));
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          top = __shfl_sync(0xffffffffu, top, (lane & 1) << 4);
          if (lane >> 1 == x) amax = top;
        }
        int ex = 0;
        if (amax > 0.f) {
          frexpf(amax, &ex);
          ex -= 15;
        }
        const float step = fmaxf(ldexpf(1.0f, ex), 0x1p-120f);  // largest element in [2^14, 2^15)
        const float mine = 1.0f / step;
        a = step * kScaleLog2;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int from = 2 * x + (lane >> 4), to_row = 32 * (warp & 3) + from, ch = lane & 15;
          const float inv = __shfl_sync(0xffffffffu, mine, from);
          const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
          uint32_t o[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            o[y] = pack_h2(__uint_as_float(w[y] << 16) * inv, __uint_as_float(w[y] & 0xFFFF0000u) * inv);
          *reinterpret_cast<uint4 *>(q_tile + (ch >> 3) * 16384 + to_row * 128 + (((ch & 7) ^ (to_row & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.q_full[pipe]);

      float m = kNegBig, l = 0.f, vref = 0.f;
      for (int j = 0; ok && j < n_tiles; ++j, ++kt) {
        ok = wait(&bars.s_full[pipe], sp & 1);
        ++sp;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const TileScales &sl = slot_of(kt);
        const int tok0 = (sg.k0 + j) * kTile;
        const bool masked = __any_sync(0xffffffffu, tok0 + kTile - 1 > lim) || sl.any_bad;
        // ---- the row's logits, and their maximum ----
        uint32_t s[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, s[q]);
        tmem_wait_ld();
        if (masked) mask_logits(s, sl, lim + 1 - tok0);
        // (-inf * 0 would be no logit: a block of zero keys has scale 0)
        auto scale_of = [&](int x) { return fmaxf(a * sl.ks[x], 0x1p-126f); };
        float mx = -CUDART_INF_F;
#pragma unroll
        for (int x = 0; x < kTilePages; ++x) {
          const uint32_t *z = s[x >> 1] + 16 * (x & 1);
          float mb = __uint_as_float(z[0]);
#pragma unroll
          for (int y = 1; y < 15; y += 2) mb = fmaxf(fmaxf(mb, __uint_as_float(z[y])), __uint_as_float(z[y + 1]));
          mx = fmaxf(mx, fmaxf(mb, __uint_as_float(z[15])) * scale_of(x));
        }
        vref = sl.vref;
        const float moved = sl.moved;
        if (__any_sync(0xffffffffu, mx > m + kLazy) || moved != 0.f) {
          const float mn = mx > m + kLazy ? mx : m;
          const float drop = fast_exp2(m - mn);
          if (j > 0) {
            const float f = drop * fast_exp2(moved);
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {  // (16 columns at a time: the logits are in registers)
              uint32_t o[16];
              tmem_ld16(to + 16 * q, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
              tmem_st16(to + 16 * q, o);
            }
            tmem_wait_st();
          }
          l *= drop;
          m = mn;
        }
        // ---- weights ----
        float2 l2 = make_float2(0.f, 0.f);
        const float2 m2 = make_float2(-m, -m);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t p[16];
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            const float cv = sl.cv[2 * q + hb];
            const float ak = scale_of(2 * q + hb);
            const float2 ak2 = make_float2(ak, ak);
            const float2 cv2 = make_float2(cv, cv);
#pragma unroll
            for (int x = 0; x < 16; x += 2) {
              const uint32_t *at = s[q] + 16 * hb + x;
              float2 z = ffma2(make_float2(__uint_as_float(at[0]), __uint_as_float(at[1])), ak2, m2);
              z.x = fast_exp2(z.x);
              z.y = fast_exp2(z.y);
              l2 = fadd2(l2, z);
              z = fmul2(z, cv2);
              p[8 * hb + x / 2] = pack_h2(z.x, z.y);
            }
          }
          tmem_st16(ts + 16 * q, p);
        }
        l += l2.x + l2.y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[pipe]);
      }
      ok = ok && wait(&bars.s_full[pipe], sp & 1);  // O is complete
      ++sp;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      // ---- out ----
      const bool whole = sg.k0 == 0 && sg.k1 == sg.nt;
      const float undo = fast_exp2(vref - kPShift);
      const float scale = whole ? (l > 0.f ? undo / l : 0.f) : undo;
      float *rec = partials + (static_cast<size_t>(2 * me + (sg.first ? 0 : 1)) * kUnitRows +
                               pipe * kTile + row) * kRecordFloats;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t o[32];
        tmem_ld32(to + 32 * q, o);
        tmem_wait_ld();
        float v[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) v[x] = l > 0.f ? __uint_as_float(o[x]) * scale : 0.f;
        if (live && whole) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const __nv_bfloat162 t = __floats2bfloat162_rn(v[8 * x + 2 * y], v[8 * x + 2 * y + 1]);
              w[y] = *reinterpret_cast<const uint32_t *>(&t);
            }
            reinterpret_cast<uint4 *>(out.out + qr * kHeadDim + 32 * q)[x] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        float *f32 = whole ? (out.out_f32 ? out.out_f32 + qr * kHeadDim : nullptr) : rec;
        if (live && f32 != nullptr)
#pragma unroll
          for (int x = 0; x < 8; ++x)
            reinterpret_cast<float4 *>(f32 + 32 * q)[x] =
                make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
      }
      if (live && whole && out.lse) out.lse[qr] = l > 0.f ? m * kLn2 + logf(l) : -CUDART_INF_F;
      if (live && !whole) *reinterpret_cast<float2 *>(rec + kHeadDim) = make_float2(m, l);
      tc_fence_before();
    }
    if (!ok) {
      // This warp's rows of the segment where it gave up, and of all that follow: empty.
      Segments rest(c, qs, find_share(c.num_seqs, me, workers, kTileMinShare, split, items));
      for (int no = 0; rest.next(); ++no) {
        const int r = rest.u * kUnitRows + pipe * kTile + row;
        if (no < seg_no - 1 || r >= rest.sq.n * G) continue;
        if (rest.k0 == 0 && rest.k1 == rest.nt) {
          const size_t qr = static_cast<size_t>(rest.sq.row0 + r / G) * H * G + rest.h * G + r % G;
          for (int x = 0; x < kHeadDim / 8; ++x)
            reinterpret_cast<uint4 *>(out.out + qr * kHeadDim)[x] = make_uint4(0u, 0u, 0u, 0u);
          for (int x = 0; out.out_f32 && x < kHeadDim / 4; ++x)
            reinterpret_cast<float4 *>(out.out_f32 + qr * kHeadDim)[x] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (out.lse) out.lse[qr] = -CUDART_INF_F;
        } else {
          float *rec = partials + (static_cast<size_t>(2 * me + (rest.first ? 0 : 1)) * kUnitRows +
                                   pipe * kTile + row) * kRecordFloats;
          *reinterpret_cast<float2 *>(rec + kHeadDim) = make_float2(kNegBig, 0.f);
        }
      }
    }
  }
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// Blocks (blockIdx.x, *) join the unit that the share of worker blockIdx.x + 1 starts inside of,
// where that worker is the unit's second (its note says so); rows over blockIdx.y and the warps.
__global__ void __launch_bounds__(256) block8_tile_merge_kernel(Outputs out, const float *partials,
                                                                const Crossing *notes, int H, int G) {
  wait_for_launch_before();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = blockIdx.x + 1;
  const Crossing x = read_note(notes + me);
  for (int i = blockIdx.y * 8 + warp; i < x.rows; i += gridDim.y * 8) {
    const int r = x.first_row + i;
    const size_t qr = static_cast<size_t>(x.row0 + r / G) * H * G + x.h * G + r % G;
    join_records(partials, kUnitRows, i, me - 1, x.last, [&](int w) { return w == me - 1 ? x.slot0 : 0; }, out, qr,
                 lane);
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
// CTAs for at most this many key tiles.
static int tile_ctas(int num_seqs, int total_q, int max_seq_len, int H, int G) {
  const long long units = (static_cast<long long>(total_q) * G + kUnitRows - 1) / kUnitRows + num_seqs;
  const long long tiles = units * H * (max_seq_len / kTile + 1);
  return static_cast<int>(std::max(1LL, std::min<long long>(kTileCtas, tiles)));
}

size_t tile_workspace_bytes(int num_seqs, int total_q, int max_seq_len, int H, int G) {
  const size_t ctas = tile_ctas(num_seqs, total_q, max_seq_len, H, G);
  return notes_bytes(ctas) + ctas * 2 * kUnitRows * kRecordFloats * sizeof(float);  // two records each
}

template <int F>
static cudaError_t launch_tile_t(const CacheView &c, const Queries &qs, int max_seq_len, const Outputs &out,
                                 void *workspace, const Waits &waits, int32_t *err, cudaStream_t s) {
  static PerDevice sms;
  int n_sm = 0;
  cudaError_t e = once_per_device(sms, [](int dev, int *g) {
    cudaError_t r = cudaFuncSetAttribute(block8_tile_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kTileSmem);
    return r == cudaSuccess ? cudaDeviceGetAttribute(g, cudaDevAttrMultiProcessorCount, dev) : r;
  }, &n_sm);
  if (e != cudaSuccess) return e;
  const int ctas = std::min(n_sm, tile_ctas(c.num_seqs, qs.total, max_seq_len, c.num_kv_heads, c.gqa));
  Crossing *notes = static_cast<Crossing *>(workspace);
  float *partials = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + notes_bytes(ctas));
  block8_tile_kernel<F><<<ctas, kTileThreads, kTileSmem, s>>>(c, qs, out, partials, notes, waits, err);
  e = cudaGetLastError();
  if (e != cudaSuccess || ctas == 1) return e;
  return launch_after(block8_tile_merge_kernel, dim3(ctas - 1, 8), 256, s, out,
                      static_cast<const float *>(partials), static_cast<const Crossing *>(notes), c.num_kv_heads,
                      c.gqa);
}

cudaError_t launch_tile_attention(int fmt, const CacheView &c, const Queries &qs, int max_seq_len,
                                  const Outputs &out, void *workspace, const Waits &waits, int32_t *err,
                                  cudaStream_t s) {
  Waits own = waits;
  if (own.limit == 0) own.limit = kTileWait;
  auto launch = fmt == kFmtInt8 ? launch_tile_t<kFmtInt8> : launch_tile_t<kFmtE4m3>;
  return launch(c, qs, max_seq_len, out, workspace, own, err, s);
}

}  // namespace kv4
