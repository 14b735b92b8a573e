// The 8-bit block-scaled cache: pages of 16 positions held as INT8 or e4m3 codes with one
// fp16 scale per (page, kv head), for K and for V. Value = code * scale.
//
//   block8_append_token_kernel  one new row per sequence: one warp per (sequence, kv head).
//   block8_append_rows_kernel   CSR rows: one warp per (page touched, kv head, K or V).
//   block8_attn_kernel          attention with 8 or 16 query rows (a kv head's query heads of
//                               one or more positions) per warp, split over the pages.
//   block8_merge_kernel         the exact merge of the units that several warps share.
//   (kv4_block8_tile.cu: attention of more than kWarpRows query rows of a kv head)
//
// Block scale. A block's scale is the largest row magnitude it has seen over the largest
// code (127, or 448 for e4m3), rounded UP to fp16, so that no code saturates (rounding to
// nearest would lose up to half the range where fp16 is subnormal). A row that raises it
// has the codes already in the block rounded again: code' = rne(code * s_old / s).
#include <algorithm>

#include "kv4_block8.cuh"

namespace kv4 {

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
// fp16 scale of a block whose largest magnitude is amax, rounded up, at most 65504.
template <int F>
__device__ __forceinline__ __half block_scale(float amax) {
  const float s = quotient_rn(fminf(amax, 3.0e38f), Fmt8<F>::kMax, Fmt8<F>::kRcp);
  return __float2half_ru(fminf(s, 65504.0f));
}

// Four values over the scale (y = 1/s; 0 when s = 0) to four codes. The quotient is the
// IEEE one (quotient_rn: the scale has 11 significant bits), so a code is the nearest one
// to the exact quotient: bf16 rows and stored code * scale products have at most 18.
template <int F>
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float s, float y) {
  if constexpr (F == kFmtInt8) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = max(-127, min(127, __float2int_rn(quotient_rn(x[i], s, y))));
      w |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * i);
    }
    return w;
  } else {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(quotient_rn(x[0], s, y), quotient_rn(x[1], s, y)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(quotient_rn(x[2], s, y), quotient_rn(x[3], s, y)), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
}

template <int F>
__device__ __forceinline__ void values4(uint32_t w, float s, float (&x)[4]) {
  if constexpr (F == kFmtInt8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = static_cast<float>(static_cast<int8_t>((w >> (8 * i)) & 0xFFu)) * s;
  } else {
    const float2 a = __half22float2(
        __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), __NV_E4M3)));
    const float2 b = __half22float2(
        __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3)));
    x[0] = a.x * s; x[1] = a.y * s; x[2] = b.x * s; x[3] = b.y * s;
  }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// The codes of rows [0, rows) of a block rounded again from scale s_old to s.
template <int F>
__device__ __forceinline__ void rescale_block(uint8_t *block, int rows, float s_old, float s, float y,
                                              int lane) {
  for (int i = lane; i < rows * 8; i += 32) {  // 16-byte pieces: strip i / rows, row i % rows
    uint4 *p = reinterpret_cast<uint4 *>(block + (i / rows) * (kPage * 16) + (i % rows) * 16);
    uint4 v = *p;
    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x[4];
      values4<F>(w[k], s_old, x);
      w[k] = codes4<F>(x, s, y);
    }
    *p = v;
  }
}

// The scale of a block that gets rows of magnitude amax from slot `slot` on; the codes already
// there are rounded again where it grows. (Lanes of one warp, all with the same arguments.)
template <int F>
__device__ __forceinline__ float grow_scale(uint8_t *block, uint16_t *scale, float amax, int slot, int lane) {
  const __half sh = block_scale<F>(amax);
  float s = __half2float(sh);
  if (slot > 0) {  // (a block's first slot starts its scale anew)
    const float s_old = __half2float(__ushort_as_half(*scale));
    if (s <= s_old) return s_old;
    rescale_block<F>(block, slot, s_old, s, __frcp_rn(s), lane);
    __syncwarp();  // every lane has read the old scale
  }
  if (lane == 0) *scale = __half_as_ushort(sh);
  return s;
}

// Four bf16 values with infinities as the largest finite number: the remainder of an infinite
// quotient is NaN. (Asked for only where a row's magnitude is infinite.)
__device__ __forceinline__ uint2 finite_bf16x4(uint2 raw) {
  raw.x -= __vcmpeq2(raw.x & 0x7fff7fffu, 0x7f807f80u) & 0x00010001u;
  raw.y -= __vcmpeq2(raw.y & 0x7fff7fffu, 0x7f807f80u) & 0x00010001u;
  return raw;
}

__device__ __forceinline__ float amax4(const float (&x)[4]) {
  return fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
}

// One warp per (sequence, kv head, K or V); lane l holds dims 4l .. 4l+3. Bound by its chain of
// loads (length, page id, scale), so the row is asked for first: 1024 sequences x 8 kv heads take
// 4.8 us in graph replays (10.4 a call through the binding), of which the bytes are 1.
template <int F>
__global__ void __launch_bounds__(256) block8_append_token_kernel(
    CacheView c, const uint16_t *__restrict__ k_new, const uint16_t *__restrict__ v_new,
    int32_t *err) {
  const int lane = threadIdx.x & 31;
  const int H = c.num_kv_heads;
  const long long warp = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (warp >= 2LL * c.num_seqs * H) return;
  const bool v = (warp & 1) != 0;
  const int unit = static_cast<int>(warp >> 1), b = unit / H, h = unit - b * H;
  const uint2 raw = *reinterpret_cast<const uint2 *>((v ? v_new : k_new) +
                                                     static_cast<size_t>(unit) * kHeadDim + 4 * lane);
  const int L = c.seq_lens[b], pos = L - 1;
  if (pos < 0 || L > c.max_pages * kPage) {
    if (lane == 0) set_err(err, KV4_DEVERR_SEQ_LEN);
    return;
  }
  const int page = c.page_table[static_cast<size_t>(b) * c.max_pages + pos / kPage];
  if (page < 0 || page >= c.num_pages) {
    if (lane == 0) set_err(err, KV4_DEVERR_PAGE_ID);
    return;
  }
  const int slot = pos % kPage;
  const size_t blk = static_cast<size_t>(page) * H + h;
  uint8_t *block = (v ? c.v_codes : c.k_codes) + blk * kInt8CodeBytes;
  float x[4];
  unpack_bf16x4(raw, x);
  const float amax = warp_max(amax4(x));
  if (amax == CUDART_INF_F) unpack_bf16x4(finite_bf16x4(raw), x);
  const float s = grow_scale<F>(block, (v ? c.v_params : c.k_params) + blk, amax, slot, lane);
  // [8 strips of 16 dims][16 slots][16 bytes]: lane l -> strip l / 4, bytes 4 (l % 4)
  *reinterpret_cast<uint32_t *>(block + (lane >> 2) * (kPage * 16) + slot * 16 + 4 * (lane & 3)) =
      codes4<F>(x, s, s == 0.f ? 0.f : __frcp_rn(s));
}

// 4 x 4 words over the four lanes of a group (lane % 4), transposed: lane t gets word t of each.
__device__ __forceinline__ uint4 transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, int t) {
  // words of lanes t ^ 2 first, then of t ^ 1: after both, lane t holds (a, b, c, d)[t] of lanes 0-3
  const bool hi2 = (t & 2) != 0, hi1 = (t & 1) != 0;
  const uint32_t x = __shfl_xor_sync(0xffffffffu, hi2 ? a : c, 2);
  const uint32_t y = __shfl_xor_sync(0xffffffffu, hi2 ? b : d, 2);
  // lanes 0, 1: words 0, 1 of themselves (a, b) and of lanes 2, 3 (x, y); lanes 2, 3: words 2, 3
  const uint32_t p0 = hi2 ? x : a, p1 = hi2 ? y : b;  // from lane t & 1
  const uint32_t q0 = hi2 ? c : x, q1 = hi2 ? d : y;  // from lane (t & 1) + 2
  const uint32_t u = __shfl_xor_sync(0xffffffffu, hi1 ? p0 : p1, 1);
  const uint32_t w = __shfl_xor_sync(0xffffffffu, hi1 ? q0 : q1, 1);
  return hi1 ? make_uint4(u, p1, w, q1) : make_uint4(p0, u, q0, w);
}

// CSR rows. A CTA looks over `span` rows; the first row of the call in each page leads that
// page's rows (they may reach past the CTA's). One warp per (led page, kv head, K or V): its rows
// (up to 16 x 256 bytes) in registers, the block's largest magnitude, the codes, and full 64-byte
// runs of each strip out. Bound by HBM (512 bytes of rows in, 256 of codes out per position and
// head) and the latency of a page's loads; the search for a row's sequence is shared by the CTA's
// ~4 pages and all heads. Prefill of 64 sequences of up to 1500 rows (47k rows x 8 kv heads), graph
// replays: 64 rows per CTA, three CTAs per SM, 63 us in e4m3 (4.6 TB/s), 73 in INT8 (whose codes take
// more instructions); 16 rows per CTA 80 us. Fewer rows than that fills the GPU with are dealt to more
// CTAs: 1024 sequences of 1 to 3 rows 87 -> 22 us, 64 of 2 to 9 rows 39 -> 7.5, one of 300 rows 18 -> 7.
constexpr int kRowsPerCta = 64;  // at most
constexpr int kAppendCtas = 148 * 3;
template <int F>
__global__ void __launch_bounds__(256, 3) block8_append_rows_kernel(
    CacheView c, const uint16_t *__restrict__ k_new, const uint16_t *__restrict__ v_new,
    const int32_t *__restrict__ indptr, int32_t total_new, int span, int32_t *err) {
  __shared__ int4 lead[kRowsPerCta];  // (first row, rows, slot, page)
  __shared__ int n_lead;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = c.num_kv_heads;
  if (threadIdx.x == 0) n_lead = 0;
  __syncthreads();
  if (threadIdx.x < span) {
    const int row = blockIdx.x * span + threadIdx.x;
    if (row < total_new) {
      int b, pos, L;
      locate_new_token(c.seq_lens, c.num_seqs, indptr, row, b, pos, L);
      const int i = row - indptr[b], n = indptr[b + 1] - indptr[b];
      if (i >= 0 && i < n) {  // (rows behind the last sequence belong to none)
        if (pos < 0 || pos >= L || L > c.max_pages * kPage || indptr[b + 1] > total_new) {
          set_err(err, KV4_DEVERR_SEQ_LEN);
        } else if (i == 0 || pos % kPage == 0) {
          const int page = c.page_table[static_cast<size_t>(b) * c.max_pages + pos / kPage];
          if (page < 0 || page >= c.num_pages)
            set_err(err, KV4_DEVERR_PAGE_ID);
          else  // (the order of the led pages is of no consequence)
            lead[atomicAdd(&n_lead, 1)] = make_int4(row, min(n - i, kPage - pos % kPage), pos % kPage, page);
        }
      }
    }
  }
  __syncthreads();
  const int tasks = n_lead * H * 2;
  const size_t stride = static_cast<size_t>(H) * kHeadDim;
  for (int t = warp; t < tasks; t += blockDim.x >> 5) {
    const int4 e = lead[t / (2 * H)];
    const int r = t % (2 * H), h = r >> 1, n = e.y, slot = e.z;
    const bool v = (r & 1) != 0;
    const size_t blk = static_cast<size_t>(e.w) * H + h;
    const uint16_t *rows = (v ? v_new : k_new) + e.x * stride + h * kHeadDim + 4 * lane;
    uint2 raw[kPage];
#pragma unroll
    for (int i = 0; i < kPage; ++i)
      raw[i] = i < n ? *reinterpret_cast<const uint2 *>(rows + i * stride) : make_uint2(0u, 0u);
    __nv_bfloat162 top = __float2bfloat162_rn(0.f);  // of |x|, on pairs
#pragma unroll
    for (int i = 0; i < kPage; ++i) {
      const uint32_t a = raw[i].x & 0x7fff7fffu, z = raw[i].y & 0x7fff7fffu;
      top = __hmax2(top, __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                 *reinterpret_cast<const __nv_bfloat162 *>(&z)));
    }
    const float amax = warp_max(fmaxf(__low2float(top), __high2float(top)));
    uint8_t *block = (v ? c.v_codes : c.k_codes) + blk * kInt8CodeBytes;
    const float s = grow_scale<F>(block, (v ? c.v_params : c.k_params) + blk, amax, slot, lane);
    const float y = s == 0.f ? 0.f : __frcp_rn(s);
    uint8_t *strip = block + (lane >> 2) * (kPage * 16) + slot * 16;
    if (amax == CUDART_INF_F) {  // apart, so that finite rows pay a branch only (in their loop: 5 us of 67)
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        float x[4];
        unpack_bf16x4(finite_bf16x4(*reinterpret_cast<const uint2 *>(rows + i * stride)), x);
        *reinterpret_cast<uint32_t *>(strip + i * 16 + 4 * (lane & 3)) = codes4<F>(x, s, y);
      }
      continue;
    }
#pragma unroll
    for (int q = 0; q < kPage; q += 4) {
      if (q >= n) break;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[4];
        unpack_bf16x4(raw[q + i], x);
        w[i] = codes4<F>(x, s, y);
      }
      const uint4 row = transpose4(w[0], w[1], w[2], w[3], lane & 3);  // row q + lane % 4
      if (q + (lane & 3) < n) *reinterpret_cast<uint4 *>(strip + (q + (lane & 3)) * 16) = row;
    }
  }
}

// ---------------------------------------------------------------------------
// attention: the split of a batch over warps
// ---------------------------------------------------------------------------
// A unit is 8 (or 16) query rows of one (sequence, kv head): row r = position i * G + query head g
// of the sequence's last n positions. Every unit reads the sequence's pages, so the batch
// is T = sum over sequences of units * pages; warp w takes the w-th of W contiguous, equal
// shares (to one page). A unit inside one warp's share is finished there; of a unit that
// several warps share, each writes a partial record and the merge kernel joins them in
// order. A warp has at most two such units: its first (record 2w) and its last (2w + 1).
constexpr int kAttnCtas = 148 * 3;            // resident CTAs of the largest grid
constexpr int kAttnWarps = kAttnCtas * kWarps;
constexpr int kMinShare = 4;                  // pages per warp, at least (~1 us: a record's join)
// Units of at most kUnitCtas CTAs (two per SM) whose warps then get at most kUnitPages pages each have
// clusters of their own, which saves the scan and the merge launch. Clusters / equal shares, us:
// 4 x 500 positions 8 / 14, 1 x 16000 25 / 43, 4 x 8000 20 / 27, 36 x 2000 31 / 39 (100 to 2000: 25 /
// 23). With more pages the longest sequence decides: 64 per warp 50 / 57, but ragged (512 to 4096)
// 47 / 42; 128 per warp and ragged 114 / 74.
constexpr int kUnitCtas = 296;
constexpr int kUnitPages = 32;
constexpr int kCols = 8;                      // query rows of a unit (MMA N)

struct Seq8 : SeqRows {
  int pages;  // pages a unit of it takes (1 for an empty sequence: it writes zeros)
  int units;  // per kv head
};

__device__ __forceinline__ Seq8 seq_of(const CacheView &c, const Queries &qs, int unit_rows, int b,
                                       int32_t *err) {
  Seq8 s;
  static_cast<SeqRows &>(s) = rows_of(c, qs, b, err);
  s.pages = max(1, (s.L + kPage - 1) / kPage);
  s.units = static_cast<int>((static_cast<long long>(s.n) * c.gqa + unit_rows - 1) / unit_rows);
  return s;
}

// ---------------------------------------------------------------------------
// attention: codes to tensor-core operands
// ---------------------------------------------------------------------------
// 8 x 8 fp16 matrix held as MMA fragments, transposed in registers.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

constexpr int kPair = 2;                                  // pages a warp takes at a time
constexpr int kStages8 = 2;                               // pairs in flight per warp
constexpr int kPage8Bytes = 2 * kInt8CodeBytes;           // K then V of one (page, kv head)
constexpr int kStage8Bytes = kPair * kPage8Bytes;
constexpr int kWarp8Smem = kStages8 * kStage8Bytes;
constexpr int kCta8Smem = kWarps * kWarp8Smem;
// The weights p = 2^(s - m) enter PV in fp16 as p * 2^14 * vs / 2^vref, vref the exponent of
// the largest value scale so far (at most 2^14; 11 significant bits down to 2^-14): the tensor
// cores take 16-bit operands, and a weight's 2^-11 is an eighth of what the bf16 output rounds by.
// The running maximum is kept as m - 14, which makes (m - 14, l 2^14, acc 2^14) the same state.
constexpr float kLift8 = 14.0f;

// One warp's share of a batch. NT groups of 8 query rows share each page's operands.
//   QK^T  INT8: integer MMAs on the codes as they are; the query as 23-bit fixed point (its
//         largest element at least 2^21 and below 2^22 steps) in three limbs: an element below
//         2^-14 of the largest is off by up to 2^-22 of it, the products' sums are exact. e4m3: fp16
//         MMAs, codes converted, the query a power of two from its bf16 value; both exact but for
//         the fp32 sums.
//   PV    fp16 MMAs on the converted codes, fp32 accumulators.
// Two pages (32 positions) per softmax step, so that the cross-lane maximum, the waits and the
// copies' bookkeeping are paid once for 8 KB. NT = 1 (up to 8 rows of a kv head: decode steps) is
// bound by the reading of the pages: 128 sequences of up to 16384, 382 us (e4m3, 6.0 TB/s) and 390
// (INT8). NT = 2 by the issue of MMAs, exponentials and conversions: 32 x 4096 positions 59 us with 8
// rows, 71 with 16 (one unit), 119 with 32 (two units) in INT8, 1 to 3 % less in e4m3 (graph replays).
//
// UNIT: few units, each given to the warps of a cluster (`parts` of them, equal runs of its pages),
// which join their records themselves behind a cluster barrier: no scan of the batch and no merge
// launch. `per_head`: units of a kv head of a sequence, at most.
template <int F, int NT, bool UNIT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 3 : 2) block8_attn_kernel(
    CacheView c, Queries qs, Outputs out, float *partials, Crossing *__restrict__ notes, int parts,
    int per_head, Waits waits, int32_t *err) {
  constexpr int ROWS = kCols * NT;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ SplitSmem split;
  __shared__ uint64_t bars_all[kWarps][kStages8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int G = c.gqa, H = c.num_kv_heads, B = c.num_seqs;
  uint8_t *stage0 = smem + warp * kWarp8Smem;
  uint64_t *bars = bars_all[warp];
  if (lane == 0) {
    for (int s = 0; s < kStages8; ++s) mbar_init(&bars[s], 1);
    fence_barrier_init();
  }
  auto items = [&](const Seq8 &s) { return static_cast<long long>(s.units) * s.pages * H; };
  const int me = blockIdx.x * kWarps + warp;
  Share share{0, 1, 0, 0};
  const int unit0 = UNIT ? me / parts : 0, part = UNIT ? me - unit0 * parts : 0;
  if constexpr (!UNIT) {
    share = take_share(B, me, gridDim.x * kWarps, kMinShare, split, [&](int i, bool check) {
      return items(seq_of(c, qs, ROWS, i, check && blockIdx.x == 0 ? err : nullptr));
    });
    if (share.begin >= share.end) {
      if (lane == 0) notes[me].rows = 0;
      return;
    }
  } else {
    share.b = unit0 / (H * per_head);
  }
  const long long t_begin = share.begin, t_end = share.end;
  int b = share.b;
  long long seq_first = share.seq_first;  // first item of sequence b
  Seq8 sq = seq_of(c, qs, ROWS, b, UNIT && part == 0 && unit0 % (H * per_head) == 0 ? err : nullptr);
  if (UNIT && unit0 % per_head >= sq.units) return;  // (the whole cluster)

  uint32_t parity = 0;
  bool dead = false;  // a wait gave up: its unit's part and all that follow are empty, and copy nothing
  const int mi = lane >> 3, r8 = lane & 7;
  // ldmatrix lane addresses of two strips: (strip 2pr | slots 0-7), (| slots 8-15), strip 2pr+1
  const int ld8 = ((mi >> 1) * 256) + (mi & 1) * 128 + r8 * 16;
  for (long long t = t_begin; t < t_end;) {
    int h, u, pg0, pg1;  // unit u of kv head h; its pages pg0 .. pg1-1 are this warp's
    if constexpr (UNIT) {
      const int in_seq = unit0 % (H * per_head);
      h = in_seq / per_head;
      u = in_seq - h * per_head;
      pg0 = static_cast<int>(static_cast<long long>(sq.pages) * part / parts);
      pg1 = static_cast<int>(static_cast<long long>(sq.pages) * (part + 1) / parts);
    } else {
      while (t >= seq_first + items(sq)) {
        seq_first += items(sq);
        sq = seq_of(c, qs, ROWS, ++b, nullptr);
      }
      const long long in_seq = t - seq_first;
      const int unit = static_cast<int>(in_seq / sq.pages);
      pg0 = static_cast<int>(in_seq - static_cast<long long>(unit) * sq.pages);
      pg1 = static_cast<int>(min(static_cast<long long>(sq.pages), pg0 + (t_end - t)));
      h = unit / sq.units;
      u = unit - h * sq.units;
    }
    const bool whole = !UNIT && pg0 == 0 && pg1 == sq.pages;
    const int np = sq.L > 0 && !dead ? pg1 - pg0 : 0, pairs = (np + kPair - 1) / kPair;
    const int32_t *pt = c.page_table + static_cast<size_t>(b) * c.max_pages + pg0;

    if (!UNIT && t == t_begin && lane == 0)
      notes[me] = crossing(Shares(split.scan[kSplitThreads], gridDim.x * kWarps, kMinShare), me, t_begin - pg0,
                           sq.pages, pg0, sq.row0, h, u * ROWS, min(ROWS, sq.n * G - u * ROWS));

    // page ids and scales of 32 pages at a time, page k in lane k % 32; the ids of the next 32
    // are there early, for the copies that start ahead
    int pid = -1, pid_next = -1, block0 = 0;
    float ks_l = 0.f, cv_l = 0.f, vref = -30.f;
    auto load_ids = [&](int k0) {
      int p = -1;
      if (k0 + lane < np) {
        p = pt[k0 + lane];
        if (p < 0 || p >= c.num_pages) {
          set_err(err, KV4_DEVERR_PAGE_ID);
          p = -1;  // the page's positions are left out
        }
      }
      return p;
    };
    auto issue = [&](int j) {  // the copies of pair j
      const int k = kPair * j, st = j % kStages8;
      const int from = k - block0 < 32 ? pid : pid_next;
      const int p0 = __shfl_sync(0xffffffffu, from, k & 31), p1 = __shfl_sync(0xffffffffu, from, (k & 31) + 1);
      if (lane == 0) {
        uint8_t *dst = stage0 + st * kStage8Bytes;
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(&bars[st], ((p0 >= 0) + (p1 >= 0)) * kPage8Bytes);
        if (p0 >= 0) {
          const size_t off = (static_cast<size_t>(p0) * H + h) * kInt8CodeBytes;
          bulk_g2s(dst, c.k_codes + off, kInt8CodeBytes, &bars[st]);
          bulk_g2s(dst + kInt8CodeBytes, c.v_codes + off, kInt8CodeBytes, &bars[st]);
        }
        if (p1 >= 0) {
          const size_t off = (static_cast<size_t>(p1) * H + h) * kInt8CodeBytes;
          bulk_g2s(dst + kPage8Bytes, c.k_codes + off, kInt8CodeBytes, &bars[st]);
          bulk_g2s(dst + kPage8Bytes + kInt8CodeBytes, c.v_codes + off, kInt8CodeBytes, &bars[st]);
        }
      }
    };
    pid = load_ids(0);
    int issued = min(pairs, kStages8);
    const int withheld = t == t_begin && me == waits.withheld ? 1 : 0;  // (the testing hook)
    for (int j = withheld; j < issued; ++j) issue(j);
    pid_next = load_ids(32);

    // ---- query operands: column gid of group g = query row u * ROWS + 8g + gid ----
    const int rows = sq.n * G;
    uint32_t q8[NT][F == kFmtInt8 ? 3 : 1][F == kFmtInt8 ? 4 : 8][2];
    float kq[NT][2];
    int lim[NT][2], lim_least = sq.L - 1;  // last position the columns 2tig, 2tig + 1 see
#pragma unroll
    for (int g = 0; g < NT; ++g) {
      const int r = u * ROWS + 8 * g + gid;
      const bool live = r < rows;
      const uint16_t *qrow = qs.q + (static_cast<size_t>(sq.row0 + r / G) * H * G + h * G + r % G) * kHeadDim;
      float qv[8][4];
      float amax = 0.f;
#pragma unroll
      for (int cc = 0; cc < 8; ++cc) {
        const uint2 v = live ? *reinterpret_cast<const uint2 *>(qrow + 16 * cc + 4 * tig) : make_uint2(0u, 0u);
        unpack_bf16x4(v, qv[cc]);
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fabsf(qv[cc][i]));
      }
      // the largest element over half_range_step is in [2^14, 2^15): 2^7 times finer for INT8
      const float step = F == kFmtInt8 ? half_range_step(amax) * 0.0078125f : half_range_step(amax);
      const float inv = 1.0f / step;  // a power of two: exact
#pragma unroll
      for (int cc = 0; cc < 8; ++cc) {
        if constexpr (F == kFmtInt8) {
          uint32_t w[3] = {0u, 0u, 0u};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int qi = __float2int_rn(qv[cc][i] * inv);
            w[0] |= (static_cast<uint32_t>(qi) & 0xFFu) << (8 * i);
            w[1] |= (static_cast<uint32_t>(qi >> 8) & 0xFFu) << (8 * i);
            w[2] |= (static_cast<uint32_t>(qi >> 16) & 0xFFu) << (8 * i);
          }
#pragma unroll
          for (int x = 0; x < 3; ++x) q8[g][x][cc >> 1][cc & 1] = w[x];
        } else {
          q8[g][0][cc][0] = pack_h2(qv[cc][0] * inv, qv[cc][1] * inv);
          q8[g][0][cc][1] = pack_h2(qv[cc][2] * inv, qv[cc][3] * inv);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        kq[g][e] = __shfl_sync(0xffffffffu, step, 4 * (2 * tig + e)) * kScaleLog2;
        const int rc = u * ROWS + 8 * g + 2 * tig + e;
        lim[g][e] = rc < rows ? sq.L - sq.n + rc / G : -1;
        lim_least = rc < rows ? min(lim_least, lim[g][e]) : lim_least;
      }
    }
    lim_least = __reduce_min_sync(0xffffffffu, lim_least);
    float m[NT][2], l[NT][2];
    float o[NT][8][4];
#pragma unroll
    for (int g = 0; g < NT; ++g) {
      m[g][0] = m[g][1] = kNegBig;
      l[g][0] = l[g][1] = 0.f;
#pragma unroll
      for (int cc = 0; cc < 8; ++cc) o[g][cc][0] = o[g][cc][1] = o[g][cc][2] = o[g][cc][3] = 0.f;
    }

    for (int j = 0; j < pairs; ++j) {
      const int k = kPair * j;
      if ((k & 31) == 0) {  // the next 32 pages' scales
        if (k > 0) {
          block0 = k;
          pid = pid_next;
          pid_next = load_ids(k + 32);
        }
        ks_l = cv_l = 0.f;
        if (pid >= 0) {
          ks_l = __half2float(__ushort_as_half(c.k_params[static_cast<size_t>(pid) * H + h]));
          cv_l = __half2float(__ushort_as_half(c.v_params[static_cast<size_t>(pid) * H + h]));
        }
        // fp16 scales are non-negative: their order is that of their fp32 bits
        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(cv_l));
        const float e = static_cast<float>(static_cast<int>(top >> 23) - 126);  // all below 2^e
        if (e > vref) {
          const float f = fast_exp2(vref - e);
#pragma unroll
          for (int g = 0; g < NT; ++g)
#pragma unroll
            for (int cc = 0; cc < 8; ++cc)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[g][cc][i] *= f;
          vref = e;
        }
        cv_l *= fast_exp2(-vref);
      }
      const int st = j % kStages8;
      if (!mbar_wait_bounded(&bars[st], (parity >> st) & 1u, waits.limit)) {
        if (lane == 0) set_err(err, KV4_DEVERR_TIMEOUT);
        const uint32_t longer = waits.limit > 0x0FFFFFFFu ? 0xFFFFFFFFu : waits.limit * 16u;
        for (int i = j + withheld; i < issued; ++i)  // let its copies in flight land before it ends
          mbar_wait_bounded(&bars[i % kStages8], (parity >> (i % kStages8)) & 1u, longer);
        dead = true;
#pragma unroll
        for (int g = 0; g < NT; ++g) {
          m[g][0] = m[g][1] = kNegBig;
          l[g][0] = l[g][1] = 0.f;
        }
        break;
      }
      parity ^= 1u << st;
      const uint32_t sa = smem_u32(stage0 + st * kStage8Bytes);
      const int tok0 = (pg0 + k) * kPage;
      float s[NT][kPair][2][2], cv[kPair];
      bool there[kPair];  // the page was copied
#pragma unroll
      for (int pp = 0; pp < kPair; ++pp) {
        there[pp] = __shfl_sync(0xffffffffu, pid, (k & 31) + pp) >= 0;
        const float ks = __shfl_sync(0xffffffffu, ks_l, (k & 31) + pp);
        cv[pp] = __shfl_sync(0xffffffffu, cv_l, (k & 31) + pp);
        float d[NT][4];
        const uint32_t sk = sa + pp * kPage8Bytes + ld8;
        if constexpr (F == kFmtInt8) {
          int32_t a2[NT][4] = {}, a1[NT][4] = {}, a0[NT][4] = {};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t kw[4];
            ldsm_x4(kw, sk + x * 512);
#pragma unroll
            for (int g = 0; g < NT; ++g) {
              mma_s8s8(a2[g], kw[0], kw[1], kw[2], kw[3], q8[g][2][x][0], q8[g][2][x][1]);
              mma_s8u8(a1[g], kw[0], kw[1], kw[2], kw[3], q8[g][1][x][0], q8[g][1][x][1]);
              mma_s8u8(a0[g], kw[0], kw[1], kw[2], kw[3], q8[g][0][x][0], q8[g][0][x][1]);
            }
          }
#pragma unroll
          for (int g = 0; g < NT; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i)  // (the low limbs' sums stay below 2^31: 255 * 127 * 128 * 257)
              d[g][i] = fmaf(static_cast<float>(a2[g][i]), 65536.f, static_cast<float>(a1[g][i] * 256 + a0[g][i]));
        } else {
#pragma unroll
          for (int g = 0; g < NT; ++g) d[g][0] = d[g][1] = d[g][2] = d[g][3] = 0.f;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t kw[4];
            ldsm_x4(kw, sk + x * 512);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t a01, a23, a45, a67;
              code_pairs<F, false>(kw[2 * hf], a01, a45);
              code_pairs<F, false>(kw[2 * hf + 1], a23, a67);
#pragma unroll
              for (int g = 0; g < NT; ++g)
                mma_f16(d[g], a01, a23, a45, a67, q8[g][0][2 * x + hf][0], q8[g][0][2 * x + hf][1]);
            }
          }
        }
#pragma unroll
        for (int g = 0; g < NT; ++g) {
          const float f0 = ks * kq[g][0], f1 = ks * kq[g][1];
          s[g][pp][0][0] = d[g][0] * f0;
          s[g][pp][0][1] = d[g][1] * f1;
          s[g][pp][1][0] = d[g][2] * f0;
          s[g][pp][1][1] = d[g][3] * f1;
        }
      }
      const bool tail = tok0 + kPair * kPage > sq.L || !there[0] || !there[1];
      if (tail || tok0 + kPair * kPage - 1 > lim_least) {
#pragma unroll
        for (int g = 0; g < NT; ++g)
#pragma unroll
          for (int pp = 0; pp < kPair; ++pp)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (!there[pp] || tok0 + kPage * pp + 8 * hf + gid > lim[g][e]) s[g][pp][hf][e] = -CUDART_INF_F;
      }
      uint32_t pb[NT][kPair][2];  // the weights as B operands
#pragma unroll
      for (int g = 0; g < NT; ++g) {
        float al[2];
        bool moved = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(fmaxf(s[g][0][0][e], s[g][0][1][e]), fmaxf(s[g][1][0][e], s[g][1][1][e]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float mn = fmaxf(m[g][e], x - kLift8);  // running maximum kept as max - 14
          al[e] = fast_exp2(m[g][e] - mn);
          moved |= mn != m[g][e];
          m[g][e] = mn;
          float sum = 0.f;
#pragma unroll
          for (int pp = 0; pp < kPair; ++pp)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              s[g][pp][hf][e] = fast_exp2(s[g][pp][hf][e] - mn);
              sum += s[g][pp][hf][e];
            }
          l[g][e] = fmaf(l[g][e], al[e], sum);
        }
        if (__any_sync(0xffffffffu, moved)) {
          const float2 a2 = make_float2(al[0], al[1]);
#pragma unroll
          for (int cc = 0; cc < 8; ++cc) {
            const float2 x = fmul2(make_float2(o[g][cc][0], o[g][cc][1]), a2);
            const float2 y = fmul2(make_float2(o[g][cc][2], o[g][cc][3]), a2);
            o[g][cc][0] = x.x; o[g][cc][1] = x.y; o[g][cc][2] = y.x; o[g][cc][3] = y.y;
          }
        }
        // P (tokens x columns) to the B operand (columns' tokens in pairs)
#pragma unroll
        for (int pp = 0; pp < kPair; ++pp)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            pb[g][pp][hf] = transpose8x8(pack_h2(s[g][pp][hf][0] * cv[pp], s[g][pp][hf][1] * cv[pp]));
      }
#pragma unroll
      for (int pp = 0; pp < kPair; ++pp) {
        // e4m3: the slots behind the length, and a page that was not copied, may hold NaN codes
        uint32_t keep_lo = 0xffffffffu, keep_hi = 0xffffffffu;  // tokens 2tig, +1 and 8 + those
        if (F == kFmtE4m3 && tail) {
          const int left = there[pp] ? sq.L - tok0 - kPage * pp : 0;
          keep_lo = (2 * tig < left ? 0xFFFFu : 0u) | (2 * tig + 1 < left ? 0xFFFF0000u : 0u);
          keep_hi = (2 * tig + 8 < left ? 0xFFFFu : 0u) | (2 * tig + 9 < left ? 0xFFFF0000u : 0u);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t vw[4];
          ldsm_x4_t(vw, sa + pp * kPage8Bytes + kInt8CodeBytes + x * 512 + ld8);
          if (F == kFmtE4m3 && tail) {
            vw[0] &= keep_lo; vw[1] &= keep_hi; vw[2] &= keep_lo; vw[3] &= keep_hi;
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t a01, a23, a45, a67;
            code_pairs<F, true>(vw[2 * hf], a01, a23);
            code_pairs<F, true>(vw[2 * hf + 1], a45, a67);
#pragma unroll
            for (int g = 0; g < NT; ++g)
              mma_f16(o[g][2 * x + hf], a01, a23, a45, a67, pb[g][pp][0], pb[g][pp][1]);
          }
        }
      }
      __syncwarp();
      if (issued < pairs) issue(issued++);  // the stage is free again
    }

    const float undo = fast_exp2(vref);
#pragma unroll
    for (int g = 0; g < NT; ++g)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[g][e] += __shfl_xor_sync(0xffffffffu, l[g][e], off);
        const int col = 8 * g + 2 * tig + e, rc = u * ROWS + col;
        if (rc >= rows) continue;
        if (whole) {
          const size_t qr = static_cast<size_t>(sq.row0 + rc / G) * H * G + h * G + rc % G;
          const float inv = l[g][e] > 0.f ? undo / l[g][e] : 0.f;
#pragma unroll
          for (int cc = 0; cc < 8; ++cc) {  // C rows gid, gid + 8: dims 16cc + 2gid, + 1
            const float x = o[g][cc][e] * inv, y = o[g][cc][2 + e] * inv;
            *reinterpret_cast<__nv_bfloat162 *>(out.out + qr * kHeadDim + 16 * cc + 2 * gid) =
                __floats2bfloat162_rn(x, y);
            if (out.out_f32)
              *reinterpret_cast<float2 *>(out.out_f32 + qr * kHeadDim + 16 * cc + 2 * gid) = make_float2(x, y);
          }
          if (out.lse && gid == 0) out.lse[qr] = l[g][e] > 0.f ? m[g][e] * kLn2 + logf(l[g][e]) : -CUDART_INF_F;
        } else {
          float *rec = partials + (static_cast<size_t>(2 * me + (UNIT || t == t_begin ? 0 : 1)) * ROWS + col) *
                                      kRecordFloats;
#pragma unroll
          for (int cc = 0; cc < 8; ++cc)
            st_rec(reinterpret_cast<float2 *>(rec + 16 * cc + 2 * gid),
                   make_float2(o[g][cc][e] * undo, o[g][cc][2 + e] * undo));
          if (gid == 0) st_rec(reinterpret_cast<float2 *>(rec + kHeadDim), make_float2(m[g][e], l[g][e]));
        }
      }
    if constexpr (UNIT) {
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
      for (int col = part; col < min(ROWS, rows - u * ROWS); col += parts) {
        const int r = u * ROWS + col;
        const size_t qr = static_cast<size_t>(sq.row0 + r / G) * H * G + h * G + r % G;
        join_records(partials, ROWS, col, me - part, me - part + parts - 1, [](int) { return 0; }, out, qr, lane);
      }
      return;
    }
    t += pg1 - pg0;
  }
}

// Block blockIdx.x joins the unit that the share of warp blockIdx.x + 1 starts inside of, where
// that warp is the unit's second (its note says so).
template <int NT>
__global__ void __launch_bounds__(256) block8_merge_kernel(Outputs out, const float *partials, const Crossing *notes,
                                                           int H, int G) {
  constexpr int ROWS = kCols * NT;
  wait_for_launch_before();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = blockIdx.x + 1;
  const Crossing x = read_note(notes + me);
  for (int col = warp; col < x.rows; col += 8) {
    const int r = x.first_row + col;
    const size_t qr = static_cast<size_t>(x.row0 + r / G) * H * G + x.h * G + r % G;
    // a warp's record of the unit is its first, but for the unit's first warp where the unit
    // starts inside its share
    join_records(partials, ROWS, col, me - 1, x.last, [&](int w) { return w == me - 1 ? x.slot0 : 0; }, out, qr,
                 lane);
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
template <int F>
static cudaError_t launch_block8_append_t(const CacheView &c, const uint16_t *k_new,
                                          const uint16_t *v_new, const int32_t *indptr,
                                          int32_t total_new, int32_t *err, cudaStream_t s) {
  if (indptr == nullptr) {
    const long long warps = 2LL * c.num_seqs * c.num_kv_heads;
    const unsigned blocks = static_cast<unsigned>((warps + 7) / 8);
    block8_append_token_kernel<F><<<blocks, 256, 0, s>>>(c, k_new, v_new, err);
  } else {
    const int span = std::min(kRowsPerCta, (total_new - 1) / kAppendCtas + 1);
    const unsigned blocks = static_cast<unsigned>((total_new - 1) / span + 1);
    block8_append_rows_kernel<F><<<blocks, 256, 0, s>>>(c, k_new, v_new, indptr, total_new, span, err);
  }
  return cudaGetLastError();
}

cudaError_t launch_block8_append(int fmt, const CacheView &c, const uint16_t *k_new,
                                 const uint16_t *v_new, const int32_t *indptr, int32_t total_new,
                                 int32_t *err, cudaStream_t s) {
  return fmt == kFmtInt8 ? launch_block8_append_t<kFmtInt8>(c, k_new, v_new, indptr, total_new, err, s)
                         : launch_block8_append_t<kFmtE4m3>(c, k_new, v_new, indptr, total_new, err, s);
}

// Warps of the attention grid for a batch of at most t_max items.
static int attn_warps(long long t_max) {
  const long long w = std::max(1LL, std::min<long long>(kAttnWarps, t_max / kMinShare));
  return static_cast<int>((w + kWarps - 1) / kWarps * kWarps);
}

// Pages of n positions (any n: n + 15 may not fit).
static int pages_of(int n) { return n / kPage + (n % kPage != 0); }

static long long items_bound(int num_seqs, int total_q, int max_seq_len, int H, int G, int rows) {
  const long long units = (static_cast<long long>(total_q) * G + rows - 1) / rows + num_seqs;
  return units * H * std::max(1, pages_of(max_seq_len));
}

// A note and two records of each warp, of the larger of the two unit sizes; or, for few units, two
// records of each warp of their clusters (at most kUnitCtas CTAs, so bounded by the units alone).
static size_t warp_workspace_bytes(int num_seqs, int total_q, int max_q_len, int max_seq_len, int H, int G) {
  size_t bytes = 0;
  for (int rows = kCols; rows <= 2 * kCols; rows += kCols) {
    const size_t n = attn_warps(items_bound(num_seqs, total_q, max_seq_len, H, G, rows));
    const long long units = static_cast<long long>(num_seqs) * H *
                            ((static_cast<long long>(max_q_len) * G + rows - 1) / rows);
    const size_t u = static_cast<size_t>(std::min<long long>(kUnitCtas, 8 * units)) * kWarps;
    const size_t record = 2u * rows * kRecordFloats * sizeof(float);
    bytes = std::max(bytes, std::max(notes_bytes(n) + n * record, u * record));
  }
  return (bytes + 255) / 256 * 256;
}

size_t block8_workspace_bytes(int num_seqs, int total_q, int max_q_len, int max_seq_len, int H, int G) {
  const size_t bytes = warp_workspace_bytes(num_seqs, total_q, max_q_len, max_seq_len, H, G);
  if (static_cast<long long>(max_q_len) * G <= kWarpRows) return bytes;
  return std::max(bytes, tile_workspace_bytes(num_seqs, total_q, max_seq_len, H, G));
}

// Resident CTAs of a form of the attention kernel on the current device.
template <int F, int NT, bool UNIT>
static cudaError_t resident_ctas(int *most) {
  static PerDevice grids;
  return once_per_device(grids, [](int dev, int *g) {
    cudaError_t r = cudaFuncSetAttribute(block8_attn_kernel<F, NT, UNIT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kCta8Smem);
    int sms = 0, per_sm = 0;
    if (r == cudaSuccess) r = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (r == cudaSuccess)
      r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, block8_attn_kernel<F, NT, UNIT>,
                                                        kWarps * 32, kCta8Smem);
    *g = sms * (per_sm > 0 ? per_sm : 1);
    return r;
  }, most);
}

// CTAs of a cluster that takes one unit (0: the batch is split by pages instead). A cluster's warps
// get two pairs of pages at least of the longest sequence.
static int unit_cluster(int num_seqs, int max_q_len, int max_seq_len, int H, int G, int rows) {
  const long long units = static_cast<long long>(num_seqs) * H *
                          ((static_cast<long long>(max_q_len) * G + rows - 1) / rows);
  if (units > kUnitCtas) return 0;
  const int pages = pages_of(max_seq_len);
  int ctas = 1;
  while (ctas < 8 && units * ctas * 2 <= kUnitCtas && pages >= 2 * kWarps * ctas * kPair) ctas *= 2;
  return pages > kUnitPages * kWarps * ctas ? 0 : ctas;
}

template <int F, int NT>
static cudaError_t launch_block8_attn_t(const CacheView &c, const Queries &qs, int max_seq_len,
                                        const Outputs &out, void *workspace, const Waits &waits,
                                        int32_t *err, cudaStream_t s) {
  int most = 0;
  constexpr int ROWS = kCols * NT;
  if (const int ctas = unit_cluster(c.num_seqs, qs.max_n, max_seq_len, c.num_kv_heads, c.gqa, ROWS)) {
    cudaError_t e = resident_ctas<F, NT, true>(&most);  // (sets the kernel's attributes)
    if (e != cudaSuccess) return e;
    const int per_head = (qs.max_n * c.gqa + ROWS - 1) / ROWS;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(c.num_seqs) * c.num_kv_heads * per_head * ctas);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = kCta8Smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, block8_attn_kernel<F, NT, true>, c, qs, out, static_cast<float *>(workspace),
                              static_cast<Crossing *>(nullptr), ctas * kWarps, per_head, waits, err);
  }
  cudaError_t e = resident_ctas<F, NT, false>(&most);
  if (e != cudaSuccess) return e;
  const long long bound = items_bound(c.num_seqs, qs.total, max_seq_len, c.num_kv_heads, c.gqa, ROWS);
  const int grid = std::min(attn_warps(bound) / kWarps, most);
  Crossing *notes = static_cast<Crossing *>(workspace);
  float *partials = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + notes_bytes(grid * kWarps));
  block8_attn_kernel<F, NT, false><<<grid, kWarps * 32, kCta8Smem, s>>>(c, qs, out, partials, notes, 0, 0, waits,
                                                                        err);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(block8_merge_kernel<NT>, dim3(grid * kWarps - 1), 256, s, out,
                      static_cast<const float *>(partials), static_cast<const Crossing *>(notes), c.num_kv_heads,
                      c.gqa);
}

cudaError_t launch_block8_attention(int fmt, const CacheView &c, const uint16_t *q,
                                    const int32_t *q_indptr, int total_q, int max_q_len,
                                    int max_seq_len, const Outputs &out, void *workspace,
                                    const Waits &waits, int32_t *err, cudaStream_t s) {
  const Queries qs{q, q_indptr, total_q, max_q_len};
  Waits warp_waits = waits;
  if (warp_waits.limit == 0) warp_waits.limit = kWaitLimit;
  const long long rows = static_cast<long long>(max_q_len) * c.gqa;
  if (rows > kWarpRows) return launch_tile_attention(fmt, c, qs, max_seq_len, out, workspace, waits, err, s);
  const bool one = rows <= kCols;
  auto launch = fmt == kFmtInt8 ? (one ? launch_block8_attn_t<kFmtInt8, 1> : launch_block8_attn_t<kFmtInt8, 2>)
                                : (one ? launch_block8_attn_t<kFmtE4m3, 1> : launch_block8_attn_t<kFmtE4m3, 2>);
  return launch(c, qs, max_seq_len, out, workspace, warp_waits, err, s);
}

}  // namespace kv4
