// What the kernels of seppaged_attn share: arguments, sequences, number formats.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "sep_common.cuh"
#include "sep_launch.h"

namespace sep {

struct PagedAttnParams {
  const uint8_t *k_pages, *v_pages;
  const float *k_scale, *v_scale;
  const uint8_t* flags;
  const void* q;
  long long q_tok, q_head;
  void* o;
  float* lse;
  const int32_t *table, *lens, *indptr;
  long long* base;  // [S + 1] first tile of each sequence (workspace)
  float* part;      // parts of row tiles that several warps share (workspace)
  int* chunk_plan;    // kernel of chunks: items, parts per item, then first item of each sequence (workspace)
  float* chunk_part;  // parts of its items (workspace)
  unsigned* err;
  int T, S, Hq, Hkv, G, num_pages, max_pages, log_page, a, n, bf16, nwarps;
  int chunks;  // sequences with more than kLongRows rows are left to the chunk kernel
  float scale_log2;
};

// One sequence of the call, its index values brought into range.
struct SeqInfo {
  int len;       // tokens in the pages that may be read
  int tok0, nq;  // first query token and count
  int lead;      // position of query 0 (negative: padding queries, which keep nothing)
  bool bad;      // an index was out of range
};
constexpr int kMaxLen = 1 << 30;
__device__ __forceinline__ SeqInfo seq_info(const PagedAttnParams& p, int s) {
  SeqInfo q;
  const int i0 = __ldg(p.indptr + s), i1 = __ldg(p.indptr + s + 1);
  q.tok0 = max(0, min(i0, p.T));
  q.nq = max(0, min(i1, p.T) - q.tok0);
  const int len = __ldg(p.lens + s);
  q.len = (int)min((long long)min(max(len, 0), kMaxLen), (long long)p.max_pages << p.log_page);
  q.lead = q.len - q.nq;
  q.bad = i0 != q.tok0 || i1 != q.tok0 + q.nq || len != q.len;
  return q;
}
// (token, head in group) rows from which a sequence is a chunk
constexpr int kLongRows = 32;
__device__ __forceinline__ bool is_chunk(const PagedAttnParams& p, const SeqInfo& q) {
  return p.chunks && q.len > 0 && (long long)q.nq * p.G > kLongRows;
}

__device__ __forceinline__ uint32_t cvt_e4m3x2(uint32_t w) {  // low 16 bits: two e4m3 -> two fp16
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t cvt_e4m3x2_hi(uint32_t w) {  // high 16 bits
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Byte masks of the NaN bytes (0x7f, 0xff) of four e4m3 values: 0x80 in each such byte.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

constexpr uint32_t kNoRow = 0xffffffffu;

// The exponent fields of a page's scales (powers of two, or 0 while the page holds only zeros), and the
// key scale and the log2 of the value scale (-inf for 0) from them.
__device__ __forceinline__ uint32_t scale_exponents(float ks, float vs) {
  return (__float_as_uint(ks) >> 23 & 0xffu) | (__float_as_uint(vs) >> 23 & 0xffu) << 8;
}
__device__ __forceinline__ float key_scale(uint32_t ex) { return __uint_as_float((ex & 0xffu) << 23); }
__device__ __forceinline__ float value_log2(uint32_t ex) {
  return ex >> 8 ? (float)((int)(ex >> 8) - 127) : -INFINITY;
}

__device__ __forceinline__ void store_out(const PagedAttnParams& p, long long at, float a, float b) {
  uint32_t w;
  if (p.bf16) w = pack_bf16x2(a, b);
  else w = pack_half2(a, b);
  *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + at) = w;
}
constexpr float kLn2 = 0.69314718055994531f;

// ------------------------------------------------------------------ items of the chunk kernel
// 256 rows of one sequence and KV head. With few items each is cut along its keys into parts, one per CTA,
// that leave their results, maxima and sums for the join.
constexpr int kRowsPerItem = 256;
constexpr int kScanStep = 1024;  // positions examined per refill of the list of kept keys
constexpr int kChunkCtas = 148;
struct Item {
  SeqInfo q;
  int seq, h, r0, rows;  // first row, rows of the sequence
  int w0, kend;          // window keys [w0, kend); listed keys left of w0
  int scan0, scan1, win0, win1;  // this part's share of both
};
__device__ __forceinline__ int chunk_items(const PagedAttnParams& p, const SeqInfo& q) {
  if (!is_chunk(p, q)) return 0;
  return p.Hkv * (int)(((long long)q.nq * p.G + kRowsPerItem - 1) / kRowsPerItem);
}
// Steps (window tiles of 128 keys, scan steps) of a sequence's last item.
__device__ __forceinline__ int chunk_steps(const PagedAttnParams& p, const SeqInfo& q) {
  const int w0 = max(0, q.len - (q.nq < kRowsPerItem ? q.nq : kRowsPerItem) - max(p.n, 1) + 1) & ~127;
  return (w0 + kScanStep - 1) / kScanStep + (q.len - w0 + 127) / 128;
}
// Part x % parts of item x / parts; within a sequence the latest (longest) rows first.
__device__ __forceinline__ Item chunk_item(const PagedAttnParams& p, const int* base, int x, int parts) {
  Item it;
  const int item = x / parts, part = x - item * parts;
  int lo = 0, hi = p.S;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (base[mid] <= item) lo = mid;
    else hi = mid;
  }
  it.seq = lo;
  it.q = seq_info(p, lo);
  it.rows = it.q.nq * p.G;
  const int nrt = (it.rows + kRowsPerItem - 1) / kRowsPerItem, y = item - base[lo];
  const int rt = nrt - 1 - y / p.Hkv;
  it.h = y % p.Hkv;
  it.r0 = rt * kRowsPerItem;
  const int lo_pos = max(0, it.q.lead + it.r0 / p.G);
  const int hi_pos = it.q.lead + min(it.q.nq - 1, (it.r0 + kRowsPerItem - 1) / p.G);
  it.kend = max(0, hi_pos + 1);
  it.w0 = min(max(0, lo_pos - max(p.n, 1) + 1), it.kend) & ~127;
  const int ns = (it.w0 + kScanStep - 1) / kScanStep, steps = ns + (it.kend - it.w0 + 127) / 128;
  const int a = (int)((long long)steps * part / parts), b = (int)((long long)steps * (part + 1) / parts);
  it.scan0 = min(it.w0, a * kScanStep);
  it.scan1 = min(it.w0, b * kScanStep);
  it.win0 = min(it.kend, it.w0 + max(0, a - ns) * 128);
  it.win1 = min(it.kend, it.w0 + max(0, b - ns) * 128);
  return it;
}
// The output row's elements become NaN where a kept key's value is NaN (the products took those as 0).
template <int D>
__device__ __forceinline__ void restore_nan(const PagedAttnParams& p, const Item& it, int pos, uint16_t* out) {
  const int32_t* table = p.table + (long long)it.seq * p.max_pages;
  for (int j = 0; j <= pos; ++j) {
    const int id = __ldg(table + (j >> p.log_page));
    if (id < 0 || id >= p.num_pages) continue;
    const int off = j & ((1 << p.log_page) - 1);
    if (!(pos - j < p.n || j < p.a || __ldg(p.flags + ((size_t)id << p.log_page) + off) != 0)) continue;
    const uint8_t* v = p.v_pages + ((((size_t)id * p.Hkv + it.h) << p.log_page) + off) * D;
    for (int c = 0; c < D / 4; ++c) {
      const uint32_t b = nan_bytes(__ldg(reinterpret_cast<const uint32_t*>(v) + c));
      for (int y = 0; y < 4; ++y)
        if (b >> (8 * y) & 0x80u) out[4 * c + y] = 0x7fffu;  // NaN in bf16 and fp16
    }
  }
}
// Part of an item in the workspace: [256][D] results, then [256][4] of maximum, sum, NaN flag.
template <int D>
__device__ __forceinline__ float* chunk_part_of(const PagedAttnParams& p, int x) {
  return p.chunk_part + (size_t)x * (kRowsPerItem * (D + 4));
}
// Row r of item `item`, by one warp.
template <int D>
__device__ __forceinline__ void chunk_join_row(const PagedAttnParams& p, int item, int r, int parts, int lane) {
  constexpr int F = D / 32;  // columns per lane
  const Item it = chunk_item(p, p.chunk_plan + 2, item * parts, parts);
  if (it.r0 + r >= it.rows) return;
  const int tok = (it.r0 + r) / p.G, hq = it.h * p.G + (it.r0 + r) - tok * p.G;
  auto stats = [&](int i) {
    return *reinterpret_cast<const float4*>(chunk_part_of<D>(p, item * parts + i) + kRowsPerItem * D + r * 4);
  };
  float m = -INFINITY;
  bool bad = false;
  for (int i = 0; i < parts; ++i) {
    const float4 st = stats(i);
    m = fmaxf(m, st.x);
    bad |= st.z != 0.f;
  }
  const float mr = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[F];
#pragma unroll
  for (int y = 0; y < F; ++y) acc[y] = 0.f;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const float4 st = stats(i);
    const float f = st.y * ex2(st.x - mr);  // the part's share of the sum
    l += f;
    const float* a = chunk_part_of<D>(p, item * parts + i) + (size_t)r * D + lane * F;
#pragma unroll
    for (int y = 0; y < F; y += 2) {
      const float2 v = *reinterpret_cast<const float2*>(a + y);
      acc[y] = fmaf(v.x, f, acc[y]);
      acc[y + 1] = fmaf(v.y, f, acc[y + 1]);
    }
  }
  const bool none = m == -INFINITY && !(l != l);
  const float f = none ? 0.f : 1.f / l;
  const long long row = (long long)(it.q.tok0 + tok) * p.Hq + hq;
#pragma unroll
  for (int y = 0; y < F; y += 2)
    store_out(p, row * D + lane * F + y, none ? 0.f : acc[y] * f, none ? 0.f : acc[y + 1] * f);
  if (lane == 0 && p.lse) p.lse[row] = none ? -INFINITY : (m + log2f(l)) * kLn2;
  if (bad) {
    __syncwarp();
    if (lane == 0) restore_nan<D>(p, it, it.q.lead + tok, static_cast<uint16_t*>(p.o) + row * D);
  }
}

cudaError_t launch_paged_chunks(const PagedAttnParams& p, int d, cudaStream_t stream);

}  // namespace sep
