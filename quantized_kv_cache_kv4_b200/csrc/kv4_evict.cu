// Eviction from the KV4 cache by accumulated attention weight.
//
//   weights_kernel       the attention weight of every cached position in a decode step,
//                        summed over the query heads of its kv head and added to a total:
//                        acc_out[b][h][p] = acc_in[b][h][p] + sum_g exp(s_g(p) - lse_g).
//   select_kernel        per (sequence, kv head): the sinks, the recent window and the
//                        largest totals of the rest, in ascending order of position.
//   compact_kernel       the kept rows' INT4 codes, parameters and totals to the front of
//                        other pages; compact_in_place_kernel of the sequence's own.
//                        Both also move the recent window's INT8 copies to the slots of their
//                        new positions.
#include "kv4_attn_common.cuh"
#include "kv4_split.cuh"

namespace kv4 {

// ---------------------------------------------------------------------------
// attention weights
// ---------------------------------------------------------------------------
// A sequence's tiles per kv head: the INT4 pages that hold [S, L - R), then the sink tiles,
// then the ring tiles. A warp takes a contiguous share of all (sequence, kv head, tile).
struct Tiles {
  int L, int4_pages, sink, ring;
  __device__ __forceinline__ int n() const { return int4_pages + sink + ring; }
};

__device__ __forceinline__ Tiles tiles_of(const CacheView &c, int acc_stride, int b, int32_t *err) {
  Tiles t;
  t.L = c.seq_lens[b];
  if (t.L < 0 || t.L > c.max_pages * kPage || t.L > acc_stride) {
    set_err(err, KV4_DEVERR_SEQ_LEN);
    t.L = 0;
  }
  const int S = c.num_sinks, R = c.num_recent;
  t.int4_pages = t.L - R > S ? (t.L - R - 1) / kPage - S / kPage + 1 : 0;
  t.sink = (min(S, t.L) + kPage - 1) / kPage;
  t.ring = max(S, t.L - R) < t.L ? c.ring_tiles : 0;
  return t;
}

constexpr int kWMinShare = 4;  // tiles per warp, at least (~1 us: as much as a warp's start)
constexpr int kWStages = 4;
// a stage: the K codes of two kv heads (INT8: 2 x 2048 bytes), then their scales or parameters
constexpr int kWOffPar = 2 * kInt8CodeBytes;
constexpr int kWStageBytes = kWOffPar + 2 * kInt4ParamBytes;
constexpr int kWWarpSmem = kWStages * kWStageBytes;
constexpr int kWCtaSmem = kWarps * kWWarpSmem;

// D = A B, the accumulators' start being zero without registers for it.
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], uint32_t a01, uint32_t a23, uint32_t a45,
                                             uint32_t a67, uint32_t b01, uint32_t b23) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a01), "r"(a23), "r"(a45), "r"(a67), "r"(b01), "r"(b23), "f"(0.f));
}

// A warp serves HPW kv heads, the MMA's 8 columns split between them: with G <= 4 query heads
// each two heads fill them (a head's operand is zero in the other's columns, so that both heads'
// products meet in one accumulator), and the scaling, exponentials and bookkeeping of a tile are
// paid once for both. The query is scaled by a power of two to [2^14, 2^15) at its largest element
// and enters as fp16, in which its bf16 elements are exact; the codes are exact in fp16 too, so the
// only rounding of a logit is the fp32 accumulation. INT4 codes enter as fp16 subnormals (c * 2^-24,
// or 16 c * 2^-24 for the odd dims, whose query elements carry the factor 1/16); a group's scale and
// minimum multiply its product and its query sum, s = kk sum_g (scale_g (q c)_g + min_g sum(q)_g / kk).
// 64 x 2048 positions, 32 query and 8 kv heads, graph replays: 33 us with two heads per warp, 42 with
// one; 48 long tails 85 (3.7 TB/s) and 114 us; 4 x 500 positions 8.9 and 7.7. 64 query heads (one head
// per warp): 44 and 122. Bound by the chain of a tile (codes to MMAs to exponentials to the sum, 146 to
// 165 registers a thread allow three warps per scheduler) next to the reading of K; two to six CTAs per
// SM with fewer stages are no faster.
// HOOK: a call with the testing hook armed; without, the constant wait limit folds into the code (as
// an argument it costs 2 to 4 %).
template <int HPW, bool HOOK>
__global__ void __launch_bounds__(kWarps * 32, 3) weights_kernel(
    CacheView c, const uint16_t *__restrict__ q, const float *__restrict__ lse, const float *acc_in,
    float *acc_out, int acc_stride, Waits waits, int32_t *err) {
  constexpr int CPH = 8 / HPW;  // columns per head
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ SplitSmem split;
  __shared__ uint64_t bars_all[kWarps][kWStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int G = c.gqa, H = c.num_kv_heads, S = c.num_sinks, R = c.num_recent;
  const int slots = (H + HPW - 1) / HPW;
  uint8_t *stage0 = smem + warp * kWWarpSmem;
  uint64_t *bars = bars_all[warp];
  if (lane == 0) {
    for (int s = 0; s < kWStages; ++s) mbar_init(&bars[s], 1);
    fence_barrier_init();
  }
  const int me = blockIdx.x * kWarps + warp;
  const Share share = take_share(c.num_seqs, me, gridDim.x * kWarps, kWMinShare, split, [&](int i, bool check) {
    return static_cast<long long>(slots) *
           tiles_of(c, acc_stride, i, check && blockIdx.x == 0 ? err : nullptr).n();
  });
  if (share.begin >= share.end) return;
  int b = share.b;
  long long seq_first = share.seq_first;
  Tiles ti = tiles_of(c, acc_stride, b, nullptr);
  uint32_t parity = 0;
  const int mi = lane >> 3, r8 = lane & 7;
  const int ld = ((mi >> 1) * 256) + (mi & 1) * 128 + r8 * 16;  // two 16-byte strips of 16 slots

  for (long long t = share.begin; t < share.end;) {
    while (t >= seq_first + static_cast<long long>(slots) * ti.n()) {
      seq_first += static_cast<long long>(slots) * ti.n();
      ti = tiles_of(c, acc_stride, ++b, nullptr);
    }
    const long long in_seq = t - seq_first;
    const int n_tiles = ti.n();
    const int h = static_cast<int>(in_seq / n_tiles) * HPW;  // first of the warp's heads
    const int k0 = static_cast<int>(in_seq - static_cast<long long>(h / HPW) * n_tiles);
    const int k1 = static_cast<int>(min(static_cast<long long>(n_tiles), k0 + (share.end - t)));
    const int heads = min(HPW, H - h);
    const int L = ti.L, p0 = S / kPage, n4 = ti.int4_pages, n48 = ti.int4_pages + ti.sink;
    const int set = ti.sink ? (c.sink_idx ? c.sink_idx[b] : b) : 0;
    const int ring = ti.ring ? (c.ring_idx ? c.ring_idx[b] : b) : 0;
    const bool set_ok = set >= 0 && set < c.num_sink_sets, ring_ok = ring >= 0 && ring < c.num_rings;
    if (lane == 0 && ((ti.sink && !set_ok) || (ti.ring && !ring_ok))) set_err(err, KV4_DEVERR_SIDE_IDX);
    const int32_t *pt = c.page_table + static_cast<size_t>(b) * c.max_pages + p0;

    // INT4 page ids of 32 tiles at a time, tile k0 + i in lane i % 32, and of the next 32
    int pid = -1, pid_next = -1, block0 = k0;
    auto load_pages = [&](int at) {
      int p = -1;
      if (at + lane < min(k1, n4)) {
        p = pt[at + lane];
        if (p < 0 || p >= c.num_pages) {
          set_err(err, KV4_DEVERR_PAGE_ID);
          p = -1;
        }
      }
      return p;
    };
    // Tile k's K codes, and its parameters or scales, of the warp's heads: an INT4 page's heads are
    // adjacent, a side tile's are not. A tile that cannot be read only arrives, and its positions
    // are left out.
    auto issue = [&](int k) {
      const int at = (k - block0) & 31;
      const int a = __shfl_sync(0xffffffffu, pid, at), z = __shfl_sync(0xffffffffu, pid_next, at);
      if (lane != 0) return;
      const int st = (k - k0) % kWStages;
      uint8_t *dst = stage0 + st * kWStageBytes;
      fence_proxy_async_smem();
      if (k < n4) {
        const int p = k - block0 < 32 ? a : z;
        mbar_arrive_expect_tx(&bars[st], p < 0 ? 0 : heads * (kInt4CodeBytes + kInt4ParamBytes));
        if (p < 0) return;
        const size_t blk = static_cast<size_t>(p) * H + h;
        bulk_g2s(dst, c.k_codes + blk * kInt4CodeBytes, heads * kInt4CodeBytes, &bars[st]);
        bulk_g2s(dst + kWOffPar, reinterpret_cast<const uint8_t *>(c.k_params) + blk * kInt4ParamBytes,
                 heads * kInt4ParamBytes, &bars[st]);
      } else {
        const bool sink = k < n48, there = sink ? set_ok : ring_ok;
        mbar_arrive_expect_tx(&bars[st], there ? heads * (kInt8CodeBytes + kInt8ScaleBytes) : 0);
        if (!there) return;
        for (int i = 0; i < heads; ++i) {
          const size_t x = sink ? (static_cast<size_t>(set) * H + h + i) * c.sink_tiles + (k - n4)
                                : (static_cast<size_t>(ring) * H + h + i) * c.ring_tiles + (k - n48);
          bulk_g2s(dst + i * kInt8CodeBytes, (sink ? c.sink_k : c.ring_k) + x * kInt8CodeBytes, kInt8CodeBytes,
                   &bars[st]);
          bulk_g2s(dst + kWOffPar + i * kInt8ScaleBytes, (sink ? c.sink_ks : c.ring_ks) + x * kPage,
                   kInt8ScaleBytes, &bars[st]);
        }
      }
    };
    pid = load_pages(k0);
    int issued = min(k1, k0 + kWStages);
    const int withheld = HOOK && t == share.begin && me == waits.withheld ? 1 : 0;
    for (int k = k0 + withheld; k < issued; ++k) issue(k);
    pid_next = load_pages(k0 + 32);

    // ---- query fragments: column gid = (head gid / CPH, query gid % CPH) ----
    const int head_b = gid / CPH, head_c = (2 * tig) / CPH;  // of the B and of the C columns
    const bool live = gid % CPH < G && head_b < heads;
    const uint16_t *qrow = q + (static_cast<size_t>(b) * H * G + (h + head_b) * G + gid % CPH) * kHeadDim;
    uint32_t q8[8][2];  // INT8 strip s: dims 16s + 4tig + (0,1), (2,3)
    uint32_t q4[4][4];  // INT4 group g: dims 32g + 8tig + (0,4), (2,6), then (1,5), (3,7) / 16
    float2 qs[4];       // group sums of the columns 2tig, 2tig + 1, over kk
    float2 kq, kk, ls;  // logit factors of the INT8 and the INT4 products; -lse in log2 units
    {
      float amax = 0.f;
      float v[4][8];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint4 w = load_q8(qrow, 32 * g + 8 * tig, live);
        const uint32_t w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[g][2 * i] = __uint_as_float(w4[i] << 16);
          v[g][2 * i + 1] = __uint_as_float(w4[i] & 0xFFFF0000u);
          amax = fmaxf(amax, fmaxf(fabsf(v[g][2 * i]), fabsf(v[g][2 * i + 1])));
        }
      }
      const float step = half_range_step(amax);
      const float inv = 1.0f / step;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += v[g][i];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= inv * (1.0f / kSubUnscale);  // powers of two
        qs[g].x = __shfl_sync(0xffffffffu, sum, 4 * (2 * tig));
        qs[g].y = __shfl_sync(0xffffffffu, sum, 4 * (2 * tig + 1));
        const float odd = inv * 0.0625f;
        q4[g][0] = pack_h2(v[g][0] * inv, v[g][4] * inv);
        q4[g][1] = pack_h2(v[g][2] * inv, v[g][6] * inv);
        q4[g][2] = pack_h2(v[g][1] * odd, v[g][5] * odd);
        q4[g][3] = pack_h2(v[g][3] * odd, v[g][7] * odd);
      }
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const uint2 w = live ? *reinterpret_cast<const uint2 *>(qrow + 16 * s + 4 * tig) : make_uint2(0u, 0u);
        q8[s][0] = pack_h2(__uint_as_float(w.x << 16) * inv, __uint_as_float(w.x & 0xFFFF0000u) * inv);
        q8[s][1] = pack_h2(__uint_as_float(w.y << 16) * inv, __uint_as_float(w.y & 0xFFFF0000u) * inv);
      }
      kq.x = __shfl_sync(0xffffffffu, step, 4 * (2 * tig)) * kScaleLog2;
      kq.y = __shfl_sync(0xffffffffu, step, 4 * (2 * tig + 1)) * kScaleLog2;
      kk = make_float2(kq.x * kSubUnscale, kq.y * kSubUnscale);
      // a column without a query weighs nothing
      const int j = (2 * tig) % CPH;
      const float *ll = lse + (static_cast<size_t>(b) * H + h + head_c) * G + j;
      ls.x = head_c < heads && j < G ? -ll[0] * kLog2e : -CUDART_INF_F;
      ls.y = head_c < heads && j + 1 < G ? -ll[1] * kLog2e : -CUDART_INF_F;
    }
    // the slot whose total this lane moves (HPW = 1: lanes of tig < 2 move all)
    const int mine = gid + 8 * (tig & 1);
    const bool moves = HPW == 1 ? tig < 2 : head_c < heads;
    const size_t acc0 = (static_cast<size_t>(b) * H + h + (HPW == 1 ? 0 : min(head_c, heads - 1))) * acc_stride;
    const int par_at = kWOffPar + min(head_c, heads - 1) * kInt4ParamBytes;

    bool dead = false;
    for (int k = k0; k < k1; ++k) {
      if (k - block0 == 32) {
        block0 += 32;
        pid = pid_next;
        pid_next = load_pages(block0 + 32);
      }
      int pos;  // of this lane's total; whether it is one of the tile's, and the tile was read
      bool in;
      const bool copied = __shfl_sync(0xffffffffu, pid, (k - block0) & 31) >= 0;
      if (k < n4) {
        pos = (p0 + k) * kPage + mine;
        in = pos >= S && pos < L - R && copied;
      } else if (k < n48) {
        pos = (k - n4) * kPage + mine;
        in = pos < min(S, L) && set_ok;
      } else {
        const int slot = (k - n48) * kPage + mine;
        const int lastp = L - 1, base = lastp - lastp % R + slot;  // the last p < L with p mod R = slot
        pos = base > lastp ? base - R : base;
        in = slot < R && pos >= max(S, L - R) && ring_ok;
      }
      in = in && moves;
      const float old = in && acc_in != nullptr ? acc_in[acc0 + pos] : 0.f;
      const int st = (k - k0) % kWStages;
      const uint32_t limit = HOOK ? waits.limit : kWaitLimit;
      if (!mbar_wait_bounded(&bars[st], (parity >> st) & 1u, limit)) {
        if (lane == 0) set_err(err, KV4_DEVERR_TIMEOUT);
        const uint32_t longer = limit > 0x0FFFFFFFu ? 0xFFFFFFFFu : limit * 16u;
        for (int i = k + withheld; i < issued; ++i)  // let its copies in flight land before it ends
          mbar_wait_bounded(&bars[(i - k0) % kWStages], (parity >> ((i - k0) % kWStages)) & 1u, longer);
        dead = true;
        break;
      }
      parity ^= 1u << st;
      const uint8_t *sp = stage0 + st * kWStageBytes;
      const uint32_t sa = smem_u32(sp) + ld;
      float2 s[2];  // logits of the slots gid, gid + 8 in log2 units, less lse
      if (k < n4) {
        float z[2][2] = {};
        const uint4 par[2] = {*reinterpret_cast<const uint4 *>(sp + par_at + gid * 16),
                              *reinterpret_cast<const uint4 *>(sp + par_at + (gid + 8) * 16)};
#pragma unroll
        for (int gp = 0; gp < 2; ++gp) {  // two groups per ldmatrix
          float d[2][4];
#pragma unroll
          for (int hs = 0; hs < HPW; ++hs) {
            if (hs > 0 && heads < HPW) break;
            uint32_t w[4];
            ldsm_x4(w, sa + hs * kInt4CodeBytes + gp * 512);
#pragma unroll
            for (int gg = 0; gg < 2; ++gg) {
              const int g = 2 * gp + gg;
              uint32_t lo[4], hi[4], bq[4];
              nib_pairs_v_sub(w[2 * gg], lo);
              nib_pairs_v_sub(w[2 * gg + 1], hi);
#pragma unroll
              for (int i = 0; i < 4; ++i) bq[i] = HPW == 1 || head_b == hs ? q4[g][i] : 0u;
              if (hs == 0) mma_f16_zero(d[gg], lo[0], hi[0], lo[2], hi[2], bq[0], bq[1]);
              else mma_f16(d[gg], lo[0], hi[0], lo[2], hi[2], bq[0], bq[1]);
              mma_f16(d[gg], lo[1], hi[1], lo[3], hi[3], bq[2], bq[3]);
            }
          }
#pragma unroll
          for (int gg = 0; gg < 2; ++gg) {
            const int g = 2 * gp + gg;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t pw = g == 0 ? par[hf].x : g == 1 ? par[hf].y : g == 2 ? par[hf].z : par[hf].w;
              const float2 sm = h2_to_f2(pw);  // (scale, min)
              z[hf][0] = fmaf(d[gg][2 * hf], sm.x, z[hf][0]);
              z[hf][1] = fmaf(d[gg][2 * hf + 1], sm.x, z[hf][1]);
              z[hf][0] = fmaf(qs[g].x, sm.y, z[hf][0]);
              z[hf][1] = fmaf(qs[g].y, sm.y, z[hf][1]);
            }
          }
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          s[hf].x = fmaf(z[hf][0], kk.x, ls.x);
          s[hf].y = fmaf(z[hf][1], kk.y, ls.y);
        }
      } else {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int hs = 0; hs < HPW; ++hs) {
          if (hs > 0 && heads < HPW) break;
#pragma unroll
          for (int pr = 0; pr < 4; ++pr) {
            uint32_t w[4];
            ldsm_x4(w, sa + hs * kInt8CodeBytes + pr * 512);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t ulo = w[2 * hf] ^ 0x80808080u, uhi = w[2 * hf + 1] ^ 0x80808080u;
              const bool on = HPW == 1 || head_b == hs;
              mma_f16(d, s8_pair<0x4140>(ulo), s8_pair<0x4140>(uhi), s8_pair<0x4342>(ulo), s8_pair<0x4342>(uhi),
                      on ? q8[2 * pr + hf][0] : 0u, on ? q8[2 * pr + hf][1] : 0u);
            }
          }
        }
        const uint16_t *sc =
            reinterpret_cast<const uint16_t *>(sp + kWOffPar + min(head_c, heads - 1) * kInt8ScaleBytes);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float ks = __half2float(__ushort_as_half(sc[gid + 8 * hf]));
          s[hf].x = fmaf(d[2 * hf] * ks, kq.x, ls.x);
          s[hf].y = fmaf(d[2 * hf + 1] * ks, kq.y, ls.y);
        }
      }
      const float w0 = fast_exp2(s[0].x) + fast_exp2(s[0].y), w1 = fast_exp2(s[1].x) + fast_exp2(s[1].y);
      // sums over a head's lanes of a slot: one exchange gives each lane one of its two slots
      const float give = (tig & 1) ? w0 : w1, keep = (tig & 1) ? w1 : w0;
      float w = keep + __shfl_xor_sync(0xffffffffu, give, 1);
      if (HPW == 1) w += __shfl_xor_sync(0xffffffffu, w, 2);
      if (in) acc_out[acc0 + pos] = old + w;
      __syncwarp();
      if (issued < k1) issue(issued++);
    }
    if (dead) return;
    t += k1 - k0;
  }
}

// ---------------------------------------------------------------------------
// select
// ---------------------------------------------------------------------------
// Totals in their order as unsigned keys from 1 on: NaN below everything, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 1u;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 + 0 = +0
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}

// The 32 x 32 bit matrix whose row l is lane l's word, transposed: lane i gets bit i of every lane.
__device__ __forceinline__ uint32_t transpose_bits(uint32_t v, int lane) {
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    // the columns whose number has bit j clear
    const uint32_t m = j == 16 ? 0x0000ffffu : j == 8 ? 0x00ff00ffu : j == 4 ? 0x0f0f0f0fu : j == 2 ? 0x33333333u
                                                                                                  : 0x55555555u;
    const uint32_t x = __shfl_xor_sync(0xffffffffu, v, j);
    v = (lane & j) ? (v & ~m) | ((x >> j) & m) : (v & m) | ((x & m) << j);
  }
  return v;
}

// One CTA per (sequence, kv head); a thread holds K keys of the row in registers, striped over the
// block (position i * 512 + thread), so the row is read once. Sinks and recent positions have the
// largest key of all, so that the `budget` largest keys are what stays. The key at the border by
// digits of 11, 11 and 10 bits from the top: a histogram of the keys that agree with the digits so
// far, its sums from the largest digit down, until a digit's keys are all to be taken or all three
// digits are known; then of the keys equal to the border the lowest positions. One scan over the
// (stripe, warp) counts of taken and of equal keys gives every kept position its place. Bound by
// the integer pipe: about 30 of its instructions per key.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;  // four per thread

template <int K>
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(
    CacheView c, int longest, const float *__restrict__ acc, int acc_stride, int budget, int32_t *keep,
    int32_t *new_lens, int32_t *err) {
  __shared__ __align__(16) int hist[kBins];
  __shared__ uint32_t cnt[K * kSelWarps];  // taken keys, equal keys << 16, of a stripe's warp
  __shared__ uint32_t part[kSelWarps];
  __shared__ uint32_t s_border;
  __shared__ int s_need, s_done;
  const int H = c.num_kv_heads, S = c.num_sinks, R = c.num_recent;
  const int b = blockIdx.x / H, h = blockIdx.x - b * H;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int L = c.seq_lens[b];
  int32_t *out = keep + static_cast<size_t>(blockIdx.x) * budget;
  const float *row = acc + static_cast<size_t>(blockIdx.x) * acc_stride;
  if (L < 0 || L > longest) {  // (at most K * 512)
    if (tid == 0) set_err(err, KV4_DEVERR_SEQ_LEN);
    L = 0;
  }
  if (h == 0 && tid == 0) new_lens[b] = min(L, budget);
  if (L <= budget) {
    for (int j = tid; j < budget; j += kSelThreads) out[j] = j < L ? j : -1;
    return;
  }
  int need = budget;
  uint32_t key[K];  // 0: no position
#pragma unroll
  for (int i = 0; i < K; ++i)  // (the index kept in the row, so that no load waits for a branch)
    key[i] = __float_as_uint(__ldg(row + min(i * kSelThreads + tid, L - 1)));
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int p = i * kSelThreads + tid;
    key[i] = order_key(__uint_as_float(key[i]));
    // (whole stripes of candidates need no look at their positions)
    if (i * kSelThreads < S || (i + 1) * kSelThreads > L - R)
      key[i] = p >= L ? 0u : p < S || p >= L - R ? 0xffffffffu : key[i];
  }
  uint32_t border = 0u;  // its digits so far
  bool whole = false;    // every key from the border on is taken
#pragma unroll
  for (int digit = 0; digit < 3; ++digit) {
    if (whole) break;
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
    reinterpret_cast<int4 *>(hist)[tid] = make_int4(0, 0, 0, 0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      // a key agrees with the border's digits where key - border is below the digits' step
      const uint32_t off = key[i] - border;
      const bool agrees = digit == 0 ? key[i] != 0u : off < (digit == 1 ? 1u << 21 : 1u << 10);
      if (agrees) atomicAdd(&hist[off >> shift], 1);
    }
    __syncthreads();
    const int first = kBins - 4 - 4 * tid;  // this thread's bins, the largest digits first
    const int4 v = *reinterpret_cast<const int4 *>(&hist[first]);
    const int n[4] = {v.w, v.z, v.y, v.x};
    const int sum = n[0] + n[1] + n[2] + n[3];
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int above = incl - sum;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) above += w < warp ? static_cast<int>(part[w]) : 0;
    if (above < need && need <= above + sum) {
      int at = -1, size = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (at < 0 && above + n[i] >= need) at = i, size = n[i];
        if (at < 0) above += n[i];
      }
      s_border = border + (static_cast<uint32_t>(first + 3 - at) << shift);
      s_need = need - above;
      s_done = size == need - above;
    }
    __syncthreads();
    border = s_border;
    need = s_need;
    whole = s_done != 0;
  }
  // taken: keys above the border (from it on where `whole`, and a key is at least 1); equal: at it
  const uint32_t above = whole ? border - 1u : border;
  uint32_t own_t = 0u, own_e = 0u;  // bit i: this thread's key of stripe i
#pragma unroll
  for (int i = 0; i < K; ++i) own_t |= key[i] > above ? 1u << i : 0u;
  if (!whole)
#pragma unroll
    for (int i = 0; i < K; ++i) own_e |= key[i] == border ? 1u << i : 0u;
  // lane i: the warp's 32 keys of stripe i
  const uint32_t all_t = transpose_bits(own_t, lane), all_e = whole ? 0u : transpose_bits(own_e, lane);
  if (lane < K) cnt[lane * kSelWarps + warp] = __popc(all_t) | (__popc(all_e) << 16);
  __syncthreads();
  // exclusive scan of the K * 16 counts, at most one per thread
  const uint32_t mine = tid < K * kSelWarps ? cnt[tid] : 0u;
  uint32_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  uint32_t base = incl - mine;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) base += w < warp ? part[w] : 0u;
  if (tid < K * kSelWarps) cnt[tid] = base;
  __syncthreads();
  const uint32_t before = lane < K ? cnt[lane * kSelWarps + warp] : 0u;
  const unsigned below = (1u << lane) - 1u;
  // (a place is below `budget`: the taken keys and the first `need` equal ones are that many)
  if (whole) {
    const int first = static_cast<int>(before & 0xffffu);
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const unsigned m = __shfl_sync(0xffffffffu, all_t, i);
      const int at = __shfl_sync(0xffffffffu, first, i) + __popc(m & below);
      if (own_t & (1u << i)) out[at] = i * kSelThreads + tid;
    }
  } else {
#pragma unroll 4
    for (int i = 0; i < K; ++i) {
      const unsigned mt = __shfl_sync(0xffffffffu, all_t, i), me = __shfl_sync(0xffffffffu, all_e, i);
      const uint32_t bf = __shfl_sync(0xffffffffu, before, i);
      const int eq = static_cast<int>(bf >> 16) + __popc(me & below);  // equal keys before this one
      const int at = static_cast<int>(bf & 0xffffu) + __popc(mt & below) + min(eq, need);
      if (((mt >> lane) & 1u) || (((me >> lane) & 1u) && eq < need)) out[at] = i * kSelThreads + tid;
    }
  }
}

// Rows too long for the registers: the same selection, the row read again for each digit and in
// order for the places.
constexpr int kLongThreads = 1024;
__global__ void __launch_bounds__(kLongThreads) select_long_kernel(
    CacheView c, int longest, const float *__restrict__ acc, int acc_stride, int budget, int32_t *keep,
    int32_t *new_lens, int32_t *err) {
  __shared__ int hist[256];
  __shared__ int warp_cnt[2][32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int H = c.num_kv_heads, S = c.num_sinks, R = c.num_recent;
  const int b = blockIdx.x / H, h = blockIdx.x - b * H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int L = c.seq_lens[b];
  int32_t *out = keep + static_cast<size_t>(blockIdx.x) * budget;
  const float *row = acc + static_cast<size_t>(blockIdx.x) * acc_stride;
  const bool bad = L < 0 || L > longest;
  if (bad) {
    if (threadIdx.x == 0) set_err(err, KV4_DEVERR_SEQ_LEN);
    L = 0;
  }
  if (h == 0 && threadIdx.x == 0) new_lens[b] = min(L, budget);
  if (L <= budget) {
    for (int j = threadIdx.x; j < budget; j += blockDim.x) out[j] = j < L ? j : -1;
    return;
  }
  const int lo = S, hi = L - R;  // candidates (hi - lo > budget - S - R)
  int need = budget - S - R;     // how many of them stay
  uint32_t prefix = 0u;          // the border key's bits so far
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();
    for (int p = lo + threadIdx.x; p < hi; p += blockDim.x) {
      const uint32_t key = order_key(row[p]);
      if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(key >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {  // lane l: bins 255 - 8l .. 248 - 8l, from the largest down
      int cnt[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cnt[i] = hist[255 - 8 * lane - i];
        sum += cnt[i];
      }
      int incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
      }
      int above = incl - sum;
      const bool mine = need > 0 ? above < need && need <= incl : lane == 0;
      if (mine) {
        int i = 0;
        while (need > 0 && above + cnt[i] < need) above += cnt[i++];
        s_prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - i) << shift);
        s_need = need - above;
      }
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    __syncthreads();
  }
  const bool none = budget == S + R;  // no candidate stays
  // positions in order: above the border, or at it while `need` of those last
  int base_keep = 0, base_tie = 0;
  for (int p0 = 0; p0 < L; p0 += blockDim.x) {
    const int p = p0 + threadIdx.x;
    bool tie = false, take = false;
    if (p < L) {
      if (p < lo || p >= hi) {
        take = true;
      } else if (!none) {
        const uint32_t key = order_key(row[p]);
        take = key > prefix;
        tie = key == prefix;
      }
    }
    const unsigned mt = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) warp_cnt[0][warp] = __popc(mt);
    __syncthreads();
    int ties = base_tie, all_ties = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) ties += warp_cnt[0][w];
      all_ties += warp_cnt[0][w];
    }
    ties += __popc(mt & ((1u << lane) - 1u));
    if (tie && ties < need) take = true;
    const unsigned mk = __ballot_sync(0xffffffffu, take);
    if (lane == 0) warp_cnt[1][warp] = __popc(mk);
    __syncthreads();
    int at = base_keep, all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) at += warp_cnt[1][w];
      all += warp_cnt[1][w];
    }
    at += __popc(mk & ((1u << lane) - 1u));
    if (take && at < budget) out[at] = p;
    base_keep += all;
    base_tie += all_ties;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
// Where the kept rows go.
struct Moves {
  const int32_t *keep;  // [B][H][budget]
  int32_t budget;
  const int32_t *new_lens;
  const int32_t *dst_table;  // nullptr: the sequence's own pages
  int32_t dst_max_pages;
  const int32_t *dst_ring;  // nullptr: the sequence's own ring
  const float *acc_in;
  float *acc_out;
  int32_t in_stride, out_stride;
};

// Rows kept of sequence b (0, flagged, where its counts do not fit).
__device__ __forceinline__ int kept_rows(const CacheView &c, const Moves &mv, int b, int L, int32_t *err) {
  const int n = mv.new_lens[b];
  const int cap = mv.dst_table ? mv.dst_max_pages : c.max_pages;
  if (L < 0 || L > c.max_pages * kPage || n < 0 || n > L || n > mv.budget || n > cap * kPage ||
      (mv.acc_in && (L > mv.in_stride || n > mv.out_stride))) {
    set_err(err, KV4_DEVERR_SEQ_LEN);
    return 0;
  }
  return n;
}

// Whether position src of L may go to place j: kept positions ascend, so src >= j, and the sinks keep
// their places (their INT8 copies do not move).
__device__ __forceinline__ bool may_move(const CacheView &c, int src, int j, int L) {
  return src >= j && src < L && (j >= c.num_sinks || src == j);
}

// 16-byte piece i of a row: K groups 0-3, V groups 0-3, K parameters, V parameters.
__device__ __forceinline__ uint4 *row_piece(const CacheView &c, size_t blk, int slot, int i) {
  if (i < 8) {
    uint8_t *codes = (i < 4 ? c.k_codes : c.v_codes) + blk * kInt4CodeBytes;
    return reinterpret_cast<uint4 *>(codes + (i & 3) * (kPage * 16) + slot * 16);
  }
  uint16_t *par = (i == 8 ? c.k_params : c.v_params) + blk * (kInt4ParamBytes / 2);
  return reinterpret_cast<uint4 *>(par + slot * 8);
}

// The recent window's INT8 copies: position p (before) is p - (L - n) afterwards, so slot p mod R
// moves to slot (p - (L - n)) mod R, of the same ring or another. kRingThreads threads of a CTA (its
// others gone) per (sequence, kv head); all rows (at most 144, 16 pieces of 16 bytes each) are held in registers
// before any is written.
constexpr int kRingThreads = 256;
__device__ __forceinline__ void move_ring(const CacheView &c, const Moves &mv, int b, int h, int32_t *err) {
  constexpr int kPieces = KV4_MAX_PROTECTED * 16 / kRingThreads;  // 9 per thread
  const int H = c.num_kv_heads, S = c.num_sinks, R = c.num_recent;
  const int L = c.seq_lens[b];
  const int n = kept_rows(c, mv, b, L, nullptr);
  const int lo = max(S, n - R);  // first position of the window afterwards
  if (lo >= n) return;
  const int from = c.ring_idx ? c.ring_idx[b] : b;
  const int to = mv.dst_ring ? mv.dst_ring[b] : from;
  if (from < 0 || from >= c.num_rings || to < 0 || to >= c.num_rings) {
    if (threadIdx.x == 0) set_err(err, KV4_DEVERR_SIDE_IDX);
    return;
  }
  const int gone = L - n, cnt = n - lo;
  if (from == to && gone % R == 0) return;
  const int32_t *keep = mv.keep + (static_cast<size_t>(b) * H + h) * mv.budget;
  // the window must have been kept whole
  const bool bad = threadIdx.x < cnt && keep[lo + threadIdx.x] != lo + static_cast<int>(threadIdx.x) + gone;
  const size_t src = (static_cast<size_t>(from) * H + h) * c.ring_tiles;
  const size_t dst = (static_cast<size_t>(to) * H + h) * c.ring_tiles;
  const int s0 = (lo + gone) % R, d0 = lo % R;  // slots of the window's first row
  const int x = threadIdx.x & 15;               // piece: 8 strips of K, 8 of V
  const int8_t *codes = x < 8 ? c.ring_k : c.ring_v;
  const uint16_t *scales = x < 8 ? c.ring_ks : c.ring_vs;
  uint4 v[kPieces];
  uint16_t sc[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int r = i * 16 + (threadIdx.x >> 4);
    int slot = s0 + r;
    slot -= slot >= R ? R : 0;
    if (r < cnt) {
      v[i] = *reinterpret_cast<const uint4 *>(codes + (src + slot / kPage) * kInt8CodeBytes +
                                              (x & 7) * (kPage * 16) + (slot % kPage) * 16);
      if ((x & 7) == 0) sc[i] = scales[src * kPage + slot];
    }
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_err(err, KV4_DEVERR_KEEP);
    return;
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int r = i * 16 + (threadIdx.x >> 4);
    int slot = d0 + r;
    slot -= slot >= R ? R : 0;
    if (r < cnt) {
      *reinterpret_cast<uint4 *>((x < 8 ? c.ring_k : c.ring_v) + (dst + slot / kPage) * kInt8CodeBytes +
                                 (x & 7) * (kPage * 16) + (slot % kPage) * 16) = v[i];
      if ((x & 7) == 0) (x < 8 ? c.ring_ks : c.ring_vs)[dst * kPage + slot] = sc[i];
    }
  }
}

// To other pages. Of a sequence's blocks the first H move its ring, a kv head each; the others have a
// warp per (page of kept rows, kv head), where lane l moves piece l / 16 + 2i of the row in slot l % 16,
// so that every store instruction fills 256-byte runs. Bound by HBM, where the rows of a page that
// are kept share 32-byte sectors with the ones that are not.
__global__ void __launch_bounds__(256) compact_kernel(CacheView c, Moves mv, int page_blocks, int32_t *err) {
  const int lane = threadIdx.x & 31;
  const int H = c.num_kv_heads;
  const int b = blockIdx.x / (H + page_blocks), at = blockIdx.x - b * (H + page_blocks);
  if (at < H) {
    if (c.num_recent > 0) move_ring(c, mv, b, at, err);
    return;
  }
  const int task = (at - H) * 8 + (threadIdx.x >> 5);
  const int dp = task / H, h = task - dp * H;
  if (dp >= (mv.budget + kPage - 1) / kPage) return;
  const size_t unit = static_cast<size_t>(b) * H + h;
  const int j = dp * kPage + (lane & 15);
  // (what the row's own loads need is asked for at once)
  const int src = j < mv.budget ? mv.keep[unit * mv.budget + j] : -1;
  const int dpage = dp < mv.dst_max_pages ? mv.dst_table[static_cast<size_t>(b) * mv.dst_max_pages + dp] : -1;
  const int L = c.seq_lens[b];
  const int n = kept_rows(c, mv, b, L, dp == 0 && h == 0 ? err : nullptr);
  if (dp * kPage >= n) return;
  if (dpage < 0 || dpage >= c.num_pages) {
    if (lane == 0) set_err(err, KV4_DEVERR_PAGE_ID);
    return;
  }
  if (j >= n) return;
  if (!may_move(c, src, j, L)) {
    set_err(err, KV4_DEVERR_KEEP);
    return;
  }
  const int spage = c.page_table[static_cast<size_t>(b) * c.max_pages + src / kPage];
  if (spage < 0 || spage >= c.num_pages) {
    set_err(err, KV4_DEVERR_PAGE_ID);
    return;
  }
  const size_t sb = static_cast<size_t>(spage) * H + h, db = static_cast<size_t>(dpage) * H + h;
  const int half = lane >> 4;
  const bool totals = mv.acc_in && half == 0;
  const float a = totals ? mv.acc_in[unit * mv.in_stride + src] : 0.f;
  uint4 v[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = *row_piece(c, sb, src % kPage, 2 * i + half);
#pragma unroll
  for (int i = 0; i < 5; ++i) *row_piece(c, db, lane & 15, 2 * i + half) = v[i];
  if (totals) mv.acc_out[unit * mv.out_stride + j] = a;
}

// In the sequence's own pages: one CTA per (sequence, kv head), 16 rows per warp and round.
// Row j comes from a position >= j, so what a round writes was read in it or before it: one
// barrier between a round's loads and its stores is all the order there is to keep. The second half
// of the grid, where there is a recent window, moves the rings
// (graph replays: one sequence of 777 rows to 500 in 5 us, 64 of 2048 to 1024 in 43; with a launch of
// its own 4 and 3 us more).
constexpr int kInPlaceThreads = 512;
__global__ void __launch_bounds__(kInPlaceThreads) compact_in_place_kernel(CacheView c, Moves mv,
                                                                          int32_t *err) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = c.num_kv_heads, units = c.num_seqs * H;
  const int unit0 = blockIdx.x < units ? blockIdx.x : blockIdx.x - units;
  const int b = unit0 / H, h = unit0 - b * H;
  if (blockIdx.x >= units) {
    if (threadIdx.x < kRingThreads) move_ring(c, mv, b, h, err);
    return;
  }
  const int L = c.seq_lens[b];
  const int n = kept_rows(c, mv, b, L, h == 0 && threadIdx.x == 0 ? err : nullptr);
  const size_t unit = unit0;
  const int32_t *pt = c.page_table + static_cast<size_t>(b) * c.max_pages;
  const int half = lane >> 4;
  for (int j0 = 0; j0 < n; j0 += kInPlaceThreads / 2) {
    const int j = j0 + warp * kPage + (lane & 15);
    bool move = false;
    uint4 v[5];
    float a = 0.f;
    int dpage = -1, src = -1;
    if (j < n) {
      src = mv.keep[unit * mv.budget + j];
      if (!may_move(c, src, j, L)) {
        set_err(err, KV4_DEVERR_KEEP);
      } else {
        const int spage = pt[src / kPage];
        dpage = pt[j / kPage];
        if (spage < 0 || spage >= c.num_pages || dpage < 0 || dpage >= c.num_pages) {
          set_err(err, KV4_DEVERR_PAGE_ID);
        } else {
          move = true;
          const size_t sb = static_cast<size_t>(spage) * H + h;
#pragma unroll
          for (int i = 0; i < 5; ++i) v[i] = *row_piece(c, sb, src % kPage, 2 * i + half);
          if (mv.acc_in && half == 0) a = mv.acc_in[unit * mv.in_stride + src];
        }
      }
    }
    __syncthreads();
    if (move) {
      const size_t db = static_cast<size_t>(dpage) * H + h;
      if (src != j)
#pragma unroll
        for (int i = 0; i < 5; ++i) *row_piece(c, db, j % kPage, 2 * i + half) = v[i];
      if (mv.acc_in && half == 0) mv.acc_out[unit * mv.out_stride + j] = a;
    }
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
template <int HPW, bool HOOK>
static cudaError_t launch_weights_t(const CacheView &c, int max_seq_len, const uint16_t *q, const float *lse,
                                    const float *acc_in, float *acc_out, int acc_stride, const Waits &waits,
                                    int32_t *err, cudaStream_t s) {
  static PerDevice grids;
  int most = 0;
  cudaError_t e = once_per_device(grids, [](int dev, int *g) {
    cudaError_t r = cudaFuncSetAttribute(weights_kernel<HPW, HOOK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kWCtaSmem);
    int sms = 0, per_sm = 0;
    if (r == cudaSuccess) r = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (r == cudaSuccess)
      r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, weights_kernel<HPW, HOOK>, kWarps * 32, kWCtaSmem);
    *g = sms * (per_sm > 0 ? per_sm : 1);
    return r;
  }, &most);
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>(c.num_seqs) * ((c.num_kv_heads + HPW - 1) / HPW) *
                          (max_seq_len / kPage + 2 + c.sink_tiles + c.ring_tiles);
  const long long want = (tiles / kWMinShare + kWarps) / kWarps;
  const int grid = static_cast<int>(want < most ? want : most);
  weights_kernel<HPW, HOOK><<<grid, kWarps * 32, kWCtaSmem, s>>>(c, q, lse, acc_in, acc_out, acc_stride, waits, err);
  return cudaGetLastError();
}

cudaError_t launch_weights(const CacheView &c, int max_seq_len, const uint16_t *q, const float *lse,
                           const float *acc_in, float *acc_out, int acc_stride, const Waits &waits,
                           int32_t *err, cudaStream_t s) {
  Waits own = waits;
  if (own.limit == 0) own.limit = kWaitLimit;
  auto launch = own.withheld >= 0 ? (c.gqa <= 4 ? launch_weights_t<2, true> : launch_weights_t<1, true>)
                                  : (c.gqa <= 4 ? launch_weights_t<2, false> : launch_weights_t<1, false>);
  return launch(c, max_seq_len, q, lse, acc_in, acc_out, acc_stride, own, err, s);
}

cudaError_t launch_select(const CacheView &c, int max_seq_len, const float *acc, int acc_stride, int budget,
                          int32_t *keep, int32_t *new_lens, int32_t *err, cudaStream_t s) {
  const int units = c.num_seqs * c.num_kv_heads;
  const int longest = max_seq_len < acc_stride ? max_seq_len : acc_stride;
  // the fewest keys per thread that hold the longest row (graph replays, 64 x 8 rows of 2048: 10 us
  // with 4 keys, 25 with 32; of 4096: 17 with 16; of 8192: 18 with 16, 26 with 32, 83 with the row read
  // again; 128 x 8 of up to 16384: 45 with 32, 240 with the row read again)
  if (longest <= 4 * kSelThreads)
    select_kernel<4><<<units, kSelThreads, 0, s>>>(c, longest, acc, acc_stride, budget, keep, new_lens, err);
  else if (longest <= 16 * kSelThreads)
    select_kernel<16><<<units, kSelThreads, 0, s>>>(c, longest, acc, acc_stride, budget, keep, new_lens, err);
  else if (longest <= 32 * kSelThreads)
    select_kernel<32><<<units, kSelThreads, 0, s>>>(c, longest, acc, acc_stride, budget, keep, new_lens, err);
  else
    select_long_kernel<<<units, kLongThreads, 0, s>>>(c, longest, acc, acc_stride, budget, keep, new_lens, err);
  return cudaGetLastError();
}

cudaError_t launch_compact(const CacheView &c, const int32_t *keep, int budget, const int32_t *new_lens,
                           const int32_t *dst_table, int dst_max_pages, const int32_t *dst_ring,
                           const float *acc_in, int in_stride, float *acc_out, int out_stride,
                           int32_t *err, cudaStream_t s) {
  const Moves mv{keep, budget, new_lens, dst_table, dst_max_pages, dst_ring, acc_in, acc_out, in_stride, out_stride};
  const int units = c.num_seqs * c.num_kv_heads;
  if (dst_table) {
    const int pages = (budget + kPage - 1) / kPage;
    const int blocks = (pages * c.num_kv_heads + 7) / 8;
    compact_kernel<<<static_cast<unsigned>(c.num_seqs) * (c.num_kv_heads + blocks), 256, 0, s>>>(c, mv, blocks, err);
    return cudaGetLastError();
  }
  compact_in_place_kernel<<<c.num_recent > 0 ? 2 * units : units, kInPlaceThreads, 0, s>>>(c, mv, err);
  return cudaGetLastError();
}

}  // namespace kv4
