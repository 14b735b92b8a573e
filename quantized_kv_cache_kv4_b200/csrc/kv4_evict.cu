// Eviction from the KV4 cache by accumulated attention weight.
//
//   weights_kernel       the attention weight of every cached position in a decode step,
//                        summed over the query heads of its kv head and added to a total:
//                        acc_out[b][h][p] = acc_in[b][h][p] + sum_g exp(s_g(p) - lse_g).
//   select_kernel        per (sequence, kv head): the sinks, the recent window and the
//                        largest totals of the rest, in ascending order of position.
//   compact_kernel       the kept rows' INT4 codes, parameters and totals to the front of
//                        other pages; compact_in_place_kernel of the sequence's own.
//   ring_kernel          the recent window's INT8 copies to the slots of their new positions.
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

constexpr int kWMinShare = 4;  // tiles per warp, at least
constexpr int kWStages = 8;
constexpr int kWStageBytes = 2304;  // K codes (at most 2048), then K scales or parameters
constexpr int kWWarpSmem = kWStages * kWStageBytes;
constexpr int kWCtaSmem = kWarps * kWWarpSmem;

// One warp serves one kv head's G <= 8 query heads (MMA columns). The query is scaled by a
// power of two to [2^14, 2^15) at its largest element and enters as fp16, in which its bf16
// elements are exact; the codes are exact in fp16 too, so the only rounding of a logit is
// the fp32 accumulation. INT4 codes enter as fp16 subnormals (c * 2^-24, or 16 c * 2^-24
// for the odd dims, whose query elements carry the factor 1/16).
__global__ void __launch_bounds__(kWarps * 32, 3) weights_kernel(
    CacheView c, const uint16_t *__restrict__ q, const float *__restrict__ lse, const float *acc_in,
    float *acc_out, int acc_stride, int32_t *err) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ SplitSmem split;
  __shared__ uint64_t bars_all[kWarps][kWStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int G = c.gqa, H = c.num_kv_heads, S = c.num_sinks, R = c.num_recent;
  uint8_t *stage0 = smem + warp * kWWarpSmem;
  uint64_t *bars = bars_all[warp];
  if (lane == 0) {
    for (int s = 0; s < kWStages; ++s) mbar_init(&bars[s], 1);
    fence_barrier_init();
  }
  const int me = blockIdx.x * kWarps + warp;
  const Share share = take_share(c.num_seqs, me, gridDim.x * kWarps, kWMinShare, split, [&](int i, bool check) {
    return static_cast<long long>(H) *
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
    while (t >= seq_first + static_cast<long long>(H) * ti.n()) {
      seq_first += static_cast<long long>(H) * ti.n();
      ti = tiles_of(c, acc_stride, ++b, nullptr);
    }
    const long long in_seq = t - seq_first;
    const int n_tiles = ti.n();
    const int h = static_cast<int>(in_seq / n_tiles);
    const int k0 = static_cast<int>(in_seq - static_cast<long long>(h) * n_tiles);
    const int k1 = static_cast<int>(min(static_cast<long long>(n_tiles), k0 + (share.end - t)));
    const int L = ti.L, p0 = S / kPage;
    const int set = ti.sink ? (c.sink_idx ? c.sink_idx[b] : b) : 0;
    const int ring = ti.ring ? (c.ring_idx ? c.ring_idx[b] : b) : 0;
    const bool set_ok = set >= 0 && set < c.num_sink_sets, ring_ok = ring >= 0 && ring < c.num_rings;
    const int32_t *pt = c.page_table + static_cast<size_t>(b) * c.max_pages + p0;

    // Whether tile k can be read (else its positions are left out), and its copies
    int pid = -1, pid_next = -1, block0 = k0;
    auto load_pages = [&](int at) {
      int p = -1;
      if (at + lane < min(k1, ti.int4_pages)) {
        p = pt[at + lane];
        if (p < 0 || p >= c.num_pages) {
          set_err(err, KV4_DEVERR_PAGE_ID);
          p = -1;
        }
      }
      return p;
    };
    // (K codes, K scales or parameters, bytes of each) of tile k; no bytes: it is left out
    auto issue = [&](int k) {
      const int a = __shfl_sync(0xffffffffu, pid, (k - block0) & 31);
      const int z = __shfl_sync(0xffffffffu, pid_next, (k - block0) & 31);
      if (lane != 0) return;
      const int st = (k - k0) % kWStages;
      uint8_t *dst = stage0 + st * kWStageBytes;
      const uint8_t *codes = nullptr;
      const void *par = nullptr;
      uint32_t nc = kInt8CodeBytes, np = kInt8ScaleBytes;
      if (k < ti.int4_pages) {
        const int p = k - block0 < 32 ? a : z;
        if (p >= 0) {
          const size_t blk = static_cast<size_t>(p) * H + h;
          codes = c.k_codes + blk * kInt4CodeBytes;
          par = reinterpret_cast<const uint8_t *>(c.k_params) + blk * kInt4ParamBytes;
          nc = kInt4CodeBytes;
          np = kInt4ParamBytes;
        }
      } else if (k < ti.int4_pages + ti.sink) {
        if (set_ok) {
          const size_t x = (static_cast<size_t>(set) * H + h) * c.sink_tiles + (k - ti.int4_pages);
          codes = reinterpret_cast<const uint8_t *>(c.sink_k) + x * kInt8CodeBytes;
          par = c.sink_ks + x * kPage;
        } else {
          set_err(err, KV4_DEVERR_SIDE_IDX);
        }
      } else if (ring_ok) {
        const size_t x = (static_cast<size_t>(ring) * H + h) * c.ring_tiles + (k - ti.int4_pages - ti.sink);
        codes = reinterpret_cast<const uint8_t *>(c.ring_k) + x * kInt8CodeBytes;
        par = c.ring_ks + x * kPage;
      } else {
        set_err(err, KV4_DEVERR_SIDE_IDX);
      }
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(&bars[st], codes ? nc + np : 0);
      if (codes) {
        bulk_g2s(dst, codes, nc, &bars[st]);
        bulk_g2s(dst + kInt8CodeBytes, par, np, &bars[st]);
      }
    };
    pid = load_pages(k0);
    pid_next = load_pages(k0 + 32);
    int issued = min(k1, k0 + kWStages);
    for (int k = k0; k < issued; ++k) issue(k);

    // ---- query fragments, column gid = query head gid ----
    const bool live = gid < G;
    const uint16_t *qrow = q + (static_cast<size_t>(b) * H * G + h * G + gid) * kHeadDim;
    uint32_t q8[8][2];  // INT8 strip s: dims 16s + 4tig + (0,1), (2,3)
    uint32_t q4[4][4];  // INT4 group g: dims 32g + 8tig + (0,4), (2,6), then (1,5), (3,7) / 16
    float qs[4][2];     // group sums of the columns 2tig, 2tig + 1 (true values)
    float kq[2], ls[2];
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
        qs[g][0] = __shfl_sync(0xffffffffu, sum, 4 * (2 * tig)) * kScaleLog2;
        qs[g][1] = __shfl_sync(0xffffffffu, sum, 4 * (2 * tig + 1)) * kScaleLog2;
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
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 2 * tig + e;
        kq[e] = __shfl_sync(0xffffffffu, step, 4 * col) * kScaleLog2;
        // a column without a query weighs nothing
        ls[e] = col < G ? lse[(static_cast<size_t>(b) * H + h) * G + col] * kLog2e : CUDART_INF_F;
      }
    }
    const size_t acc0 = (static_cast<size_t>(b) * H + h) * acc_stride;

    bool dead = false;
    for (int k = k0; k < k1; ++k) {
      if (k - block0 == 32) {
        block0 += 32;
        pid = pid_next;
        pid_next = load_pages(block0 + 32);
      }
      // position of this lane's tokens (slots gid, gid + 8) and whether the tile holds them
      int pos[2];
      bool in[2];
      bool ok;
      if (k < ti.int4_pages) {
        ok = __shfl_sync(0xffffffffu, pid, (k - block0) & 31) >= 0;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          pos[hf] = (p0 + k) * kPage + gid + 8 * hf;
          in[hf] = pos[hf] >= S && pos[hf] < L - R;
        }
      } else if (k < ti.int4_pages + ti.sink) {
        ok = set_ok;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          pos[hf] = (k - ti.int4_pages) * kPage + gid + 8 * hf;
          in[hf] = pos[hf] < min(S, L);
        }
      } else {
        ok = ring_ok;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int slot = (k - ti.int4_pages - ti.sink) * kPage + gid + 8 * hf;
          // the last position p < L with p mod R = slot
          const int back = slot < R ? (L - 1 - slot + R) % R : 0;
          pos[hf] = L - 1 - back;
          in[hf] = slot < R && pos[hf] >= max(S, L - R) && pos[hf] >= 0;
        }
      }
      float old[2] = {0.f, 0.f};
      if (tig == 0 && acc_in != nullptr)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          if (in[hf]) old[hf] = acc_in[acc0 + pos[hf]];
      const int st = (k - k0) % kWStages;
      if (!mbar_wait_bounded(&bars[st], (parity >> st) & 1u)) {
        if (lane == 0) set_err(err, KV4_DEVERR_TIMEOUT);
        for (int i = k; i < issued; ++i)
          mbar_wait_bounded(&bars[(i - k0) % kWStages], (parity >> ((i - k0) % kWStages)) & 1u,
                            kWaitLimit * 16u);
        dead = true;
        break;
      }
      parity ^= 1u << st;
      const uint8_t *sp = stage0 + st * kWStageBytes;
      const uint32_t sa = smem_u32(sp);
      float s[2][2];  // logits in log2 units, less lse
      if (ok && k < ti.int4_pages) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) s[hf][0] = -ls[0], s[hf][1] = -ls[1];
        const uint4 par[2] = {*reinterpret_cast<const uint4 *>(sp + kInt8CodeBytes + gid * 16),
                              *reinterpret_cast<const uint4 *>(sp + kInt8CodeBytes + (gid + 8) * 16)};
#pragma unroll
        for (int gp = 0; gp < 2; ++gp) {  // two groups per ldmatrix
          uint32_t w[4];
          ldsm_x4(w, sa + gp * 512 + ld);
#pragma unroll
          for (int gg = 0; gg < 2; ++gg) {
            const int g = 2 * gp + gg;
            uint32_t lo[4], hi[4];
            nib_pairs_v_sub(w[2 * gg], lo);
            nib_pairs_v_sub(w[2 * gg + 1], hi);
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(d, lo[0], hi[0], lo[2], hi[2], q4[g][0], q4[g][1]);
            mma_f16(d, lo[1], hi[1], lo[3], hi[3], q4[g][2], q4[g][3]);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t pw = g == 0 ? par[hf].x : g == 1 ? par[hf].y : g == 2 ? par[hf].z : par[hf].w;
              const float2 sm = h2_to_f2(pw);  // (scale, min)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                s[hf][e] = fmaf(d[2 * hf + e] * (kSubUnscale * kq[e]), sm.x, s[hf][e]);
                s[hf][e] = fmaf(qs[g][e], sm.y, s[hf][e]);
              }
            }
          }
        }
      } else if (ok) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int pr = 0; pr < 4; ++pr) {
          uint32_t w[4];
          ldsm_x4(w, sa + pr * 512 + ld);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t ulo = w[2 * hf] ^ 0x80808080u, uhi = w[2 * hf + 1] ^ 0x80808080u;
            mma_f16(d, s8_pair<0x4140>(ulo), s8_pair<0x4140>(uhi), s8_pair<0x4342>(ulo),
                    s8_pair<0x4342>(uhi), q8[2 * pr + hf][0], q8[2 * pr + hf][1]);
          }
        }
        const uint16_t *sc = reinterpret_cast<const uint16_t *>(sp + kInt8CodeBytes);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float ks = __half2float(__ushort_as_half(sc[gid + 8 * hf]));
#pragma unroll
          for (int e = 0; e < 2; ++e) s[hf][e] = fmaf(d[2 * hf + e] * ks, kq[e], -ls[e]);
        }
      }
      if (ok) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float w = fast_exp2(s[hf][0]) + fast_exp2(s[hf][1]);
          w += __shfl_xor_sync(0xffffffffu, w, 1);
          w += __shfl_xor_sync(0xffffffffu, w, 2);
          if (tig == 0 && in[hf]) acc_out[acc0 + pos[hf]] = old[hf] + w;
        }
      }
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
constexpr int kSelThreads = 1024;

// Totals in their order as unsigned keys: NaN below everything, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 + 0 = +0
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}

// One CTA per (sequence, kv head). The k-th largest key of the candidates [S, L - R) by
// four passes over 8 bits each; equal keys at the border are taken from the lowest position
// on.
__global__ void __launch_bounds__(kSelThreads) select_kernel(
    CacheView c, const float *__restrict__ acc, int acc_stride, int budget, int32_t *keep,
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
  const bool bad = L < 0 || L > acc_stride;
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

// 16-byte piece i of a row: K groups 0-3, V groups 0-3, K parameters, V parameters.
__device__ __forceinline__ uint4 *row_piece(const CacheView &c, size_t blk, int slot, int i) {
  if (i < 8) {
    uint8_t *codes = (i < 4 ? c.k_codes : c.v_codes) + blk * kInt4CodeBytes;
    return reinterpret_cast<uint4 *>(codes + (i & 3) * (kPage * 16) + slot * 16);
  }
  uint16_t *par = (i == 8 ? c.k_params : c.v_params) + blk * (kInt4ParamBytes / 2);
  return reinterpret_cast<uint4 *>(par + slot * 8);
}

// A warp per (sequence, page of kept rows, kv head): lane l moves piece l / 16 + 2i of the
// row in slot l % 16, so that every store instruction fills 256-byte runs.
__global__ void __launch_bounds__(256) compact_kernel(CacheView c, Moves mv, int32_t *err) {
  const int lane = threadIdx.x & 31;
  const int H = c.num_kv_heads;
  const int per_seq = (mv.budget + kPage - 1) / kPage;
  const long long task = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int h = static_cast<int>(task % H);
  const long long rest = task / H;
  const int dp = static_cast<int>(rest % per_seq);
  const int b = static_cast<int>(rest / per_seq);
  if (b >= c.num_seqs) return;
  const int L = c.seq_lens[b];
  const int n = kept_rows(c, mv, b, L, dp == 0 && h == 0 ? err : nullptr);
  const int j = dp * kPage + (lane & 15);
  if (dp * kPage >= n) return;
  const int dpage = mv.dst_table[static_cast<size_t>(b) * mv.dst_max_pages + dp];
  if (dpage < 0 || dpage >= c.num_pages) {
    if (lane == 0) set_err(err, KV4_DEVERR_PAGE_ID);
    return;
  }
  if (j >= n) return;
  const size_t unit = static_cast<size_t>(b) * H + h;
  const int src = mv.keep[unit * mv.budget + j];
  if (src < j || src >= L) {  // (ascending positions have src >= j)
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
  uint4 v[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = *row_piece(c, sb, src % kPage, 2 * i + half);
#pragma unroll
  for (int i = 0; i < 5; ++i) *row_piece(c, db, lane & 15, 2 * i + half) = v[i];
  if (mv.acc_in && half == 0) mv.acc_out[unit * mv.out_stride + j] = mv.acc_in[unit * mv.in_stride + src];
}

// In the sequence's own pages: one CTA per (sequence, kv head), 16 rows per warp and round.
// Row j comes from a position >= j, so what a round writes was read in it or before it: one
// barrier between a round's loads and its stores is all the order there is to keep.
constexpr int kInPlaceThreads = 512;
__global__ void __launch_bounds__(kInPlaceThreads) compact_in_place_kernel(CacheView c, Moves mv,
                                                                          int32_t *err) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = c.num_kv_heads;
  const int b = blockIdx.x / H, h = blockIdx.x - b * H;
  const int L = c.seq_lens[b];
  const int n = kept_rows(c, mv, b, L, h == 0 && threadIdx.x == 0 ? err : nullptr);
  const size_t unit = blockIdx.x;
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
      if (src < j || src >= L) {
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

// The recent window's INT8 copies: position p (before) is p - (L - n) afterwards, so slot
// p mod R moves to slot (p - (L - n)) mod R, of the same ring or another. One CTA per
// (sequence, kv head); all rows are read before any is written.
__global__ void __launch_bounds__(256) ring_kernel(CacheView c, Moves mv, int32_t *err) {
  extern __shared__ __align__(16) uint8_t rows[];  // [2][R][128] codes, then [2][R] scales
  const int H = c.num_kv_heads, S = c.num_sinks, R = c.num_recent;
  const int b = blockIdx.x / H, h = blockIdx.x - b * H;
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
  if (from == to && (L - n) % R == 0) return;
  uint16_t *scales = reinterpret_cast<uint16_t *>(rows + 2 * R * kHeadDim);
  const int32_t *keep = mv.keep + static_cast<size_t>(blockIdx.x) * mv.budget;
  const size_t src = (static_cast<size_t>(from) * H + h) * c.ring_tiles;
  const size_t dst = (static_cast<size_t>(to) * H + h) * c.ring_tiles;
  const int cnt = n - lo;
  bool bad = false;  // the window must have been kept whole
  for (int i = threadIdx.x; i < cnt; i += blockDim.x) bad |= keep[lo + i] != lo + i + (L - n);
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_err(err, KV4_DEVERR_KEEP);
    return;
  }
  for (int i = threadIdx.x; i < cnt * 16; i += blockDim.x) {  // 16-byte pieces: 8 of K, 8 of V
    const int r = i >> 4, x = i & 15, slot = (lo + r + (L - n)) % R;
    const int8_t *codes = x < 8 ? c.ring_k : c.ring_v;
    const size_t tile = src + slot / kPage;
    reinterpret_cast<uint4 *>(rows)[i] = *reinterpret_cast<const uint4 *>(
        codes + tile * kInt8CodeBytes + (x & 7) * (kPage * 16) + (slot % kPage) * 16);
    if (x == 0) scales[2 * r] = c.ring_ks[src * kPage + slot];
    if (x == 8) scales[2 * r + 1] = c.ring_vs[src * kPage + slot];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < cnt * 16; i += blockDim.x) {
    const int r = i >> 4, x = i & 15, slot = (lo + r) % R;
    int8_t *codes = x < 8 ? c.ring_k : c.ring_v;
    const size_t tile = dst + slot / kPage;
    *reinterpret_cast<uint4 *>(codes + tile * kInt8CodeBytes + (x & 7) * (kPage * 16) + (slot % kPage) * 16) =
        reinterpret_cast<const uint4 *>(rows)[i];
    if (x == 0) c.ring_ks[dst * kPage + slot] = scales[2 * r];
    if (x == 8) c.ring_vs[dst * kPage + slot] = scales[2 * r + 1];
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
cudaError_t launch_weights(const CacheView &c, int max_seq_len, const uint16_t *q, const float *lse,
                           const float *acc_in, float *acc_out, int acc_stride, int32_t *err,
                           cudaStream_t s) {
  static PerDevice grids;
  int most = 0;
  cudaError_t e = once_per_device(grids, [](int dev, int *g) {
    cudaError_t r = cudaFuncSetAttribute(weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kWCtaSmem);
    int sms = 0, per_sm = 0;
    if (r == cudaSuccess) r = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (r == cudaSuccess)
      r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, weights_kernel, kWarps * 32, kWCtaSmem);
    *g = sms * (per_sm > 0 ? per_sm : 1);
    return r;
  }, &most);
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>(c.num_seqs) * c.num_kv_heads *
                          (max_seq_len / kPage + 2 + c.sink_tiles + c.ring_tiles);
  const long long want = (tiles / kWMinShare + kWarps) / kWarps;
  const int grid = static_cast<int>(want < most ? want : most);
  weights_kernel<<<grid, kWarps * 32, kWCtaSmem, s>>>(c, q, lse, acc_in, acc_out, acc_stride, err);
  return cudaGetLastError();
}

cudaError_t launch_select(const CacheView &c, const float *acc, int acc_stride, int budget,
                          int32_t *keep, int32_t *new_lens, int32_t *err, cudaStream_t s) {
  select_kernel<<<c.num_seqs * c.num_kv_heads, kSelThreads, 0, s>>>(c, acc, acc_stride, budget, keep,
                                                                   new_lens, err);
  return cudaGetLastError();
}

cudaError_t launch_compact(const CacheView &c, const int32_t *keep, int budget, const int32_t *new_lens,
                           const int32_t *dst_table, int dst_max_pages, const int32_t *dst_ring,
                           const float *acc_in, int in_stride, float *acc_out, int out_stride,
                           int32_t *err, cudaStream_t s) {
  const Moves mv{keep, budget, new_lens, dst_table, dst_max_pages, dst_ring, acc_in, acc_out, in_stride, out_stride};
  const int units = c.num_seqs * c.num_kv_heads;
  if (dst_table) {
    const long long warps = static_cast<long long>(units) * ((budget + kPage - 1) / kPage);
    compact_kernel<<<static_cast<unsigned>((warps + 7) / 8), 256, 0, s>>>(c, mv, err);
  } else {
    compact_in_place_kernel<<<units, kInPlaceThreads, 0, s>>>(c, mv, err);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || c.num_recent == 0) return e;
  const size_t smem = static_cast<size_t>(c.num_recent) * (2 * kHeadDim + 4);
  ring_kernel<<<units, 256, smem, s>>>(c, mv, err);
  return cudaGetLastError();
}

}  // namespace kv4
