// seppaged_append: new keys and values into the paged e4m3 cache, keys rotated on the way.
//
// Each (page, KV head) holds its rows as e4m3 values times one power-of-two scale, for K and for V:
//   s = 2^e, e the smallest integer with amax <= 448 * 2^e over the finite values of the page's rows
//   (0 while all of them are 0), stored value = nearest e4m3 of x / s, ties to even.
// A power of two, because e4m3 is a floating format: a mantissa in the scale would not add
// precision, while x / s, the return to 16 bits in the attention and the re-expression of a page
// in a larger scale stay exact (the last down to e4m3's subnormals, which are rounded again).
// Rows arrive in order: a page's scale starts with its slot 0 and then only grows, and the rows
// that it holds already are re-expressed when it does. Values that are not finite are stored as
// NaN (e4m3 has no infinity), so that they show in the attention instead of passing as numbers.
//
// Work: one team of P * d / 32 threads per (page touched, KV head), 32 elements of K and of V per
// thread, kept in fp32 registers from the load over the maximum to the store: one read of the
// 16-bit rows, one write of the bytes; HBM bounds it. The (cos, sin) table of the page's new rows
// is formed once per CTA and used by all its heads.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "sep_common.cuh"
#include "sep_launch.h"
#include "sep_rope.cuh"

namespace sep {

namespace {

struct AppendParams {
  SepPagedState st;
  const void* k;
  const void* v;
  long long k_tok, k_head, v_tok, v_head;  // element strides
  const uint8_t* sep;
  const int32_t *table, *lens, *indptr;
  unsigned* err;
  int T, S, max_pages, log_page;
  int by_token;     // units are numbered by token (one CTA column per token) instead of by page
  int heads_per_cta;
};

// First unit of sequence s. A sequence with c new tokens touches at most min(c, c / P + 2) pages, so
// both numberings leave every sequence room for its pages; units past them have nothing to do.
__device__ __forceinline__ long long unit_start(const AppendParams& p, int s, int ip) {
  return p.by_token ? ip : (long long)(ip >> p.log_page) + 2ll * s;
}

// Exponent e of the scale of a page whose largest finite magnitude is amax > 0: the smallest e >= -100
// with amax <= 448 * 2^e = 1.75 * 2^(8 + e).
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127;  // fp32 subnormals give -127 and end at the limit
  return max(e - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0), -100);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;  // false for NaN too
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// x / s; infinities become NaN (the conversion would saturate them)
__device__ __forceinline__ float scaled(float x, float inv) {
  return fabsf(x) <= 3.402823466e38f ? x * inv : __uint_as_float(0x7fc00000u);
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t w, int hi) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(hi ? w >> 16 : w & 0xffffu),
                                                   __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Four e4m3 values times a power of two <= 1, rounded again.
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float ratio) {
  const float2 a = e4m3x2_to_float2(w, 0), b = e4m3x2_to_float2(w, 1);
  return to_e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}

constexpr int kChunks = 4;  // 8-element chunks of K and of V per thread

template <typename T>
struct __align__(16) Vec8 {
  T v[8];
};

template <typename T, int D>
__global__ void __launch_bounds__(512) paged_append_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ float2 s_cs[];  // [P][d_rot / 2]
  __shared__ float s_max[2][16];    // per warp: K, V
  const SepPagedState& st = p.st;
  const int P = 1 << p.log_page, nthr = blockDim.x, tid = threadIdx.x;
  constexpr int CPR = D / 8;  // chunks per row
  grid_dep_wait();
  grid_dep_launch_next();

  // ---- the sequence and page of this unit
  const long long unit = blockIdx.x;
  int seq = -1;
  for (int s0 = 0; s0 < p.S; s0 += nthr) {
    const int s = s0 + tid;
    const int hit = __syncthreads_count(s < p.S && unit_start(p, s, __ldg(p.indptr + s)) <= unit);
    seq += hit;
    if (hit < min(nthr, p.S - s0)) break;
  }
  if (seq < 0) return;
  const int i0 = __ldg(p.indptr + seq), i1 = __ldg(p.indptr + seq + 1);
  const long long len = __ldg(p.lens + seq);
  const long long lead = len - ((long long)i1 - i0);  // position of token i0; negative: padding
  const long long first = max(lead, 0ll);
  const long long pg = (first >> p.log_page) + (unit - unit_start(p, seq, i0));
  const long long r0 = max(first, pg << p.log_page), r1 = min(len, (pg + 1) << p.log_page);
  if (r0 >= r1) return;
  const long long tok0 = i0 + (r0 - lead);  // token of row r0
  int id = -1;
  if (pg < p.max_pages) id = __ldg(p.table + (long long)seq * p.max_pages + pg);
  if (id < 0 || id >= st.num_pages || tok0 < 0 || tok0 + (r1 - r0) > p.T) {
    if (tid == 0) record_failure(p.err, nullptr, SEP_ERR_INDEX);
    return;
  }
  const int slot0 = (int)(r0 & (P - 1)), nrow = (int)(r1 - r0);

  const int h = st.rope.d_rot >> 1;
  for (int e = tid; e < nrow * h; e += nthr) {
    float c, s;
    rope_angle(r0 + e / h, __ldg(st.rope.freq + e % h), &c, &s);
    s_cs[e] = make_float2(c * st.rope.magnitude, s * st.rope.magnitude);
  }
  if (blockIdx.y == 0)
    for (int r = tid; r < nrow; r += nthr)
      st.flags[(size_t)id * P + slot0 + r] = p.sep ? p.sep[tok0 + r] : 0;
  __syncthreads();

  const int team_size = P * CPR / kChunks, teams = nthr / team_size;
  const int team = tid / team_size, tt = tid - team * team_size;
  const int h_end = min(st.Hkv, (int)(blockIdx.y + 1) * p.heads_per_cta);
  for (int hb = blockIdx.y * p.heads_per_cta; hb < h_end; hb += teams) {
    const int head = hb + team;
    const bool on = head < h_end;
    float kx[kChunks][8], vx[kChunks][8];
    float km = 0.f, vm = 0.f;
    const T* kb = static_cast<const T*>(p.k) + tok0 * p.k_tok + (long long)head * p.k_head;
    const T* vb = static_cast<const T*>(p.v) + tok0 * p.v_tok + (long long)head * p.v_head;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int ch = tt + c * team_size, row = ch / CPR - slot0, e0 = (ch % CPR) * 8;
      const bool live = on && row >= 0 && row < nrow;
      Vec8<T> a = {}, b = {};
      if (live) {
        a = *reinterpret_cast<const Vec8<T>*>(kb + row * p.k_tok + e0);
        b = *reinterpret_cast<const Vec8<T>*>(vb + row * p.v_tok + e0);
      }
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        kx[c][z] = to_float(a.v[z]);
        vx[c][z] = to_float(b.v[z]);
      }
      if (live && e0 < st.rope.d_rot) {
        const float2* cs = s_cs + row * h;
        const T* kr = kb + row * p.k_tok;
        if (st.rope.interleaved) {
#pragma unroll
          for (int z = 0; z < 8; z += 2) {
            if (e0 + z < st.rope.d_rot) {
              const float2 w = cs[(e0 + z) >> 1];
              const float x1 = kx[c][z], x2 = kx[c][z + 1];
              kx[c][z] = __fmaf_rn(x1, w.x, -__fmul_rn(x2, w.y));
              kx[c][z + 1] = __fmaf_rn(x2, w.x, __fmul_rn(x1, w.y));
            }
          }
        } else if ((h & 7) == 0) {  // the partners are one 16-byte group
          const bool upper = e0 >= h;
          const Vec8<T> o = *reinterpret_cast<const Vec8<T>*>(kr + (upper ? e0 - h : e0 + h));
          const float2* ce = cs + (upper ? e0 - h : e0);
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            const float2 w = ce[z];
            const float part = to_float(o.v[z]);
            kx[c][z] = upper ? __fmaf_rn(kx[c][z], w.x, __fmul_rn(part, w.y))
                             : __fmaf_rn(kx[c][z], w.x, -__fmul_rn(part, w.y));
          }
        } else {
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            const int e = e0 + z;
            if (e < st.rope.d_rot) {
              const bool upper = e >= h;
              const float2 w = cs[upper ? e - h : e];
              const float part = to_float(kr[upper ? e - h : e + h]);
              kx[c][z] = upper ? __fmaf_rn(kx[c][z], w.x, __fmul_rn(part, w.y))
                               : __fmaf_rn(kx[c][z], w.x, -__fmul_rn(part, w.y));
            }
          }
        }
      }
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        km = fmaxf(km, finite_abs(kx[c][z]));
        vm = fmaxf(vm, finite_abs(vx[c][z]));
      }
    }
    // ---- largest magnitudes of the team's rows
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, o));
      vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
    }
    if ((tid & 31) == 0) {
      s_max[0][tid >> 5] = km;
      s_max[1][tid >> 5] = vm;
    }
    const size_t sc = (size_t)id * st.Hkv + (on ? head : 0);
    const float old_k = slot0 > 0 && on ? st.k_scale[sc] : 0.f;
    const float old_v = slot0 > 0 && on ? st.v_scale[sc] : 0.f;
    __syncthreads();  // every thread has read the old scales and written its maximum
    const int w0 = team * team_size >> 5, w1 = (team + 1) * team_size >> 5;
    for (int w = w0; w < w1; ++w) {
      km = fmaxf(km, s_max[0][w]);
      vm = fmaxf(vm, s_max[1][w]);
    }
    const float new_k = fmaxf(old_k, km > 0.f ? pow2(scale_exponent(km)) : 0.f);
    const float new_v = fmaxf(old_v, vm > 0.f ? pow2(scale_exponent(vm)) : 0.f);
    if (on) {
      if (tt == 0) {
        st.k_scale[sc] = new_k;
        st.v_scale[sc] = new_v;
      }
      // 1 / 0 for a page of zeros: 0, so that zeros stay zeros and NaN stays NaN
      const float inv_k = new_k > 0.f ? 1.f / new_k : 0.f, inv_v = new_v > 0.f ? 1.f / new_v : 0.f;
      const bool grow_k = old_k > 0.f && new_k > old_k, grow_v = old_v > 0.f && new_v > old_v;
      uint8_t* kp = st.k_pages + sc * P * D;
      uint8_t* vp = st.v_pages + sc * P * D;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int ch = tt + c * team_size, slot = ch / CPR, row = slot - slot0;
        uint2* kd = reinterpret_cast<uint2*>(kp + (size_t)ch * 8);
        uint2* vd = reinterpret_cast<uint2*>(vp + (size_t)ch * 8);
        if (row >= 0 && row < nrow) {
          const float* a = kx[c];
          const float* b = vx[c];
          *kd = make_uint2(to_e4m3x4(scaled(a[0], inv_k), scaled(a[1], inv_k), scaled(a[2], inv_k),
                                     scaled(a[3], inv_k)),
                           to_e4m3x4(scaled(a[4], inv_k), scaled(a[5], inv_k), scaled(a[6], inv_k),
                                     scaled(a[7], inv_k)));
          *vd = make_uint2(to_e4m3x4(scaled(b[0], inv_v), scaled(b[1], inv_v), scaled(b[2], inv_v),
                                     scaled(b[3], inv_v)),
                           to_e4m3x4(scaled(b[4], inv_v), scaled(b[5], inv_v), scaled(b[6], inv_v),
                                     scaled(b[7], inv_v)));
        } else if (slot < slot0) {
          if (grow_k) {
            const uint2 w = *kd;
            const float ratio = old_k * inv_k;
            *kd = make_uint2(rescale_e4m3x4(w.x, ratio), rescale_e4m3x4(w.y, ratio));
          }
          if (grow_v) {
            const uint2 w = *vd;
            const float ratio = old_v * inv_v;
            *vd = make_uint2(rescale_e4m3x4(w.x, ratio), rescale_e4m3x4(w.y, ratio));
          }
        }
      }
    }
    __syncthreads();  // s_max is reused by the next heads
  }
}

template <typename T, int D>
cudaError_t launch_append_t(AppendParams p, cudaStream_t stream) {
  const int P = p.st.page;
  const int team = P * D / 8 / kChunks;  // 32 .. 512
  const int threads = std::max(team, 256), teams = threads / team;
  const long long by_page = p.T / P + 2ll * p.S;
  p.by_token = p.T <= by_page;
  const long long units = p.by_token ? p.T : by_page;
  // Few pages: one round of teams per CTA, so that the heads spread over the SMs. Many pages: all
  // heads of a page in one CTA, which then forms its angle table once.
  p.heads_per_cta = units >= 148 * 8 ? p.st.Hkv : std::min(teams, p.st.Hkv);
  const size_t smem = (size_t)P * (p.st.rope.d_rot / 2) * sizeof(float2);
  if (smem > 48 * 1024) {
    static std::atomic<bool> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !set[dev].load()) {
      e = cudaFuncSetAttribute(paged_append_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               128 * (D / 2) * (int)sizeof(float2));
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) set[dev].store(true);
    }
  }
  const dim3 grid((unsigned)units, (p.st.Hkv + p.heads_per_cta - 1) / p.heads_per_cta);
  return launch_chained(paged_append_kernel<T, D>, grid, dim3(threads), smem, stream, p);
}

}  // namespace

cudaError_t launch_paged_append(const SepPagedState& st, int dtype, const void* k, long long k_tok,
                                long long k_head, const void* v, long long v_tok, long long v_head,
                                const uint8_t* sep, int T, int S, int max_pages, const int32_t* table,
                                const int32_t* lens, const int32_t* indptr, cudaStream_t stream) {
  AppendParams p = {};
  p.st = st;
  p.k = k;
  p.v = v;
  p.k_tok = k_tok;
  p.k_head = k_head;
  p.v_tok = v_tok;
  p.v_head = v_head;
  p.sep = sep;
  p.table = table;
  p.lens = lens;
  p.indptr = indptr;
  p.err = device_error_word();
  p.T = T;
  p.S = S;
  p.max_pages = max_pages;
  p.log_page = 31 - __builtin_clz((unsigned)st.page);
  if (dtype == SEP_DTYPE_BF16)
    return st.d == 128 ? launch_append_t<__nv_bfloat16, 128>(p, stream)
                       : launch_append_t<__nv_bfloat16, 64>(p, stream);
  return st.d == 128 ? launch_append_t<__half, 128>(p, stream) : launch_append_t<__half, 64>(p, stream);
}

}  // namespace sep
