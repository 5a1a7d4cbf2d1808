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

cudaError_t launch_paged_chunks(const PagedAttnParams& p, int d, cudaStream_t stream);

}  // namespace sep
