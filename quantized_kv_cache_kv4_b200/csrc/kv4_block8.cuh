// Pieces shared by the kernels of the 8-bit block-scaled cache (kv4_block8.cu: append and
// the attention of few query rows; kv4_block8_tile.cu: the attention of many).
#pragma once

#include <cuda_fp8.h>

#include "kv4_attn_common.cuh"
#include "kv4_split.cuh"

namespace kv4 {

constexpr int kFmtInt8 = KV4_BLOCK8_INT8;
constexpr int kFmtE4m3 = KV4_BLOCK8_E4M3;

template <int F>
struct Fmt8 {
  static constexpr float kMax = F == KV4_BLOCK8_INT8 ? 127.0f : 448.0f;
  static constexpr float kRcp = 1.0f / (F == KV4_BLOCK8_INT8 ? 127.0f : 448.0f);
};

__device__ __forceinline__ void unpack_bf16x4(uint2 raw, float (&x)[4]) {
  x[0] = __uint_as_float(raw.x << 16);
  x[1] = __uint_as_float(raw.x & 0xFFFF0000u);
  x[2] = __uint_as_float(raw.y << 16);
  x[3] = __uint_as_float(raw.y & 0xFFFF0000u);
}

// The queries of a call: CSR rows (indptr nullptr: one per sequence), at most max_n of one
// sequence.
struct Queries {
  const uint16_t *q;
  const int32_t *indptr;
  int32_t total, max_n;
};

// Length, queries and first query row of sequence b (wrong ones are flagged: a wrong length
// counts as 0, wrong rows as none).
struct SeqRows {
  int L, n, row0;
};
__device__ __forceinline__ SeqRows rows_of(const CacheView &c, const Queries &qs, int b, int32_t *err) {
  SeqRows s;
  s.L = c.seq_lens[b];
  if (s.L < 0 || s.L > c.max_pages * kPage) {
    set_err(err, KV4_DEVERR_SEQ_LEN);
    s.L = 0;
  }
  s.row0 = b;
  s.n = 1;
  if (qs.indptr != nullptr) {
    s.row0 = qs.indptr[b];
    const int end = qs.indptr[b + 1];
    if (s.row0 < 0 || end < s.row0 || end > qs.total || end - s.row0 > qs.max_n) {
      set_err(err, KV4_DEVERR_SEQ_LEN);
      s.n = 0;
    } else {
      s.n = end - s.row0;
    }
  }
  return s;
}

// A 32-bit word of four codes (bytes 0..3) as two fp16 pairs: (0, 1), (2, 3) for K and
// (0, 2), (1, 3) for V, whose transposed ldmatrix words hold two dims of two tokens.
// Both formats are exact in fp16.
template <int F, bool V>
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t &a, uint32_t &b) {
  if constexpr (F == kFmtInt8) {
    const uint32_t u = w ^ 0x80808080u;
    a = V ? s8_pair<0x4240>(u) : s8_pair<0x4140>(u);
    b = V ? s8_pair<0x4341>(u) : s8_pair<0x4342>(u);
  } else {
    const uint32_t u = V ? prmt(w, 0u, 0x3120) : w;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(u));
  }
}

// A worker's note for the merge: its share starts inside a unit that starts in the share before
// it, whose records workers (this one - 1) .. last hold (rows = 0: it does not).
struct alignas(16) Crossing {
  int rows;       // query rows of the unit
  int first_row;  // its first among the sequence's
  int row0, h;    // the sequence's first query row; the kv head
  int last;       // last worker of the unit
  int slot0;      // which of its two records the unit's first worker wrote
  int pad[2];
};

// The note of worker `me`, whose share starts `inside` items after the unit's first item t0 of n.
__device__ __forceinline__ Crossing crossing(const Shares &sh, int me, long long t0, int n, int inside, int row0,
                                             int h, int first_row, int rows) {
  Crossing x{};
  if (inside > 0 && sh.begin(me - 1) <= t0) {
    x.rows = rows;
    x.first_row = first_row;
    x.row0 = row0;
    x.h = h;
    x.last = sh.owner(t0 + n - 1);
    x.slot0 = sh.begin(me - 1) == t0 ? 0 : 1;
  }
  return x;
}

// A note as the kernel before it left it in L2.
__device__ __forceinline__ Crossing read_note(const Crossing *note) {
  const int4 *p = reinterpret_cast<const int4 *>(note);
  const int4 a = __ldcg(p), b = __ldcg(p + 1);
  return Crossing{a.x, a.y, a.z, a.w, b.x, b.y, {0, 0}};
}

inline size_t notes_bytes(size_t workers) { return (workers * sizeof(Crossing) + 255) / 256 * 256; }

// A kernel that may be resident before the launch before it has ended, and waits for that here.
__device__ __forceinline__ void wait_for_launch_before() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class... P, class... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Joins the partial records (max in log2 units, sum, weighted values) of one row of a unit that
// workers w0 .. w1 share, in that order, and writes the row. Records: [2 per worker][rows][132];
// slot(w): which of worker w's two. 32 records at a time: their maxima and sums by the lanes
// first, so that the loads of the values wait for nothing but their own batch.
template <class Slot>
__device__ __forceinline__ void join_records(const float *partials, int rows, int x, int w0,
                                             int w1, Slot slot, const Outputs &out, size_t qr, int lane) {
  float mm = kNegBig, ll = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int w = w0; w <= w1; w += 32) {
    const int n = min(32, w1 - w + 1);
    size_t at = 0;
    float2 ml = make_float2(kNegBig, 0.f);
    if (lane < n) {
      at = ((2 * static_cast<size_t>(w + lane) + slot(w + lane)) * rows + x) * kRecordFloats;
      ml = __ldcg(reinterpret_cast<const float2 *>(partials + at + kHeadDim));
      if (ml.y <= 0.f) ml.x = kNegBig;  // nothing visible there
    }
    float mx = ml.x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    const float mn = fmaxf(mm, mx);
    const float a = fast_exp2(mm - mn);
    const float e = ml.y > 0.f ? fast_exp2(ml.x - mn) : 0.f;
    float sum = ml.y * e;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    ll = ll * a + sum;
    acc.x *= a; acc.y *= a; acc.z *= a; acc.w *= a;
    mm = mn;
    for (int i = 0; i < n; i += 8) {  // eight records' values in flight
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const size_t r = __shfl_sync(0xffffffffu, at, min(i + k, n - 1));
        v[k] = __ldcg(reinterpret_cast<const float4 *>(partials + r + 4 * lane));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float f = i + k < n ? __shfl_sync(0xffffffffu, e, i + k) : 0.f;
        if (f > 0.f) {
          acc.x = fmaf(v[k].x, f, acc.x); acc.y = fmaf(v[k].y, f, acc.y);
          acc.z = fmaf(v[k].z, f, acc.z); acc.w = fmaf(v[k].w, f, acc.w);
        }
      }
    }
  }
  const float inv = ll > 0.f ? 1.0f / ll : 0.f;
  acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
  *reinterpret_cast<uint2 *>(out.out + qr * kHeadDim + 4 * lane) =
      make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
  if (out.out_f32) *reinterpret_cast<float4 *>(out.out_f32 + qr * kHeadDim + 4 * lane) = acc;
  if (out.lse && lane == 0) out.lse[qr] = ll > 0.f ? mm * kLn2 + logf(ll) : -CUDART_INF_F;
}

// Launches of the many-rows attention (kv4_block8_tile.cu).
size_t tile_workspace_bytes(int num_seqs, int total_q, int max_seq_len, int H, int G);
cudaError_t launch_tile_attention(int fmt, const CacheView &c, const Queries &qs, int max_seq_len,
                                  const Outputs &out, void *workspace, const Waits &waits, int32_t *err,
                                  cudaStream_t s);

// Up to this many query rows (positions x query heads of a kv head) of a sequence the warp
// kernel takes the call, beyond it the tile kernel, whose time hardly depends on the rows up to
// 128. Warp kernel / tile kernel, INT8, graph replays, us: 32 x 4096 positions 32 rows 117 / 168, 48
// rows 162 / 168, 64 rows 212 / 171; 4 x 8000 32 rows 36 / 52, 48 rows 53 / 52, 64 rows 64 / 53; 128 x
// 1000 48 rows 179 / 203, 64 rows 231 / 207. By time the border is at 48 rows; it is at 64 because
// the warp kernel keeps the weights to 2^-38 of the largest, the tile kernel to 2^-31.
constexpr int kWarpRows = 64;

}  // namespace kv4
