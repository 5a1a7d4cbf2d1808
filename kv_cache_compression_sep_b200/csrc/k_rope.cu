// sep_rope_fwd / sep_rope_bwd: rotary positions on queries and keys, in front of the attention.
//
// Pair z of the first d_rot elements of a head, at position p, turns by the angle p * w_z:
//   y1 = m (x1 cos - x2 sin),   y2 = m (x2 cos + x1 sin)
// with pairs (z, z + d_rot/2) (half layout) or (2z, 2z + 1) (interleaved) and m the magnitude
// factor of the scaled frequencies. The map is m times an orthogonal matrix, so its gradient is
// the same kernel with the sign of sin flipped: dx1 = m (g1 cos + g2 sin), dx2 = m (g2 cos - g1
// sin). Elements from d_rot on pass through.
//
// The data is read and written once and nothing else of size moves, so HBM bounds it. The angle of
// a (token, pair) is shared by every query and key head: a CTA takes a run of tokens with all their
// heads, forms the (cos, sin) table of its tokens in shared memory (angles in fp64, reduced to
// [-pi, pi], see rope_angle) and then streams the rows, 16 bytes per access.
#include <cuda_runtime.h>

#include <algorithm>

#include "sep_common.cuh"
#include "sep_launch.h"
#include "sep_rope.cuh"

namespace sep {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTokens = 16;  // tokens per CTA

struct RopeSide {
  const void* x;
  void* y;
  long long xs[3], ys[3];  // element strides: batch, token, head
  int H;
};
struct RopeParams {
  RopeSide side[2];  // q, k (H = 0: absent)
  const void* pos;
  long long pos_stride;  // positions of batch b start at b * pos_stride
  const double* freq;
  long long ntok;  // B * L
  int L, d, d_rot, interleaved, pos64, tokens, copy_rest;
  float magnitude, sign;
};

// One 16-byte (VEC > 1) or one-element access group of a row. A group of the rotated part holds
// VEC elements and, in the half layout, their partners.
template <typename T, int VEC>
struct __align__(sizeof(T) * VEC) Group {
  T v[VEC];
};

template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void rope_row_group(const RopeParams& p, const T* x, T* y, int u,
                                               const float2* cs) {
  using Gr = Group<T, VEC>;
  const int h = p.d_rot >> 1;
  const int nrot = INTER ? p.d_rot / VEC : h / VEC;  // groups of the rotated part
  if (VEC > 1 || !INTER) {
    if (u < nrot) {
      if (INTER) {
        Gr a = *reinterpret_cast<const Gr*>(x + u * VEC), r;
#pragma unroll
        for (int z = 0; z + 1 < VEC; z += 2) {
          const float2 c = cs[(u * VEC + z) >> 1];
          const float x1 = to_float(a.v[z]), x2 = to_float(a.v[z + 1]);
          r.v[z] = from_float<T>(__fmaf_rn(x1, c.x, -__fmul_rn(x2, c.y)));
          r.v[z + 1] = from_float<T>(__fmaf_rn(x2, c.x, __fmul_rn(x1, c.y)));
        }
        *reinterpret_cast<Gr*>(y + u * VEC) = r;
      } else {
        Gr a = *reinterpret_cast<const Gr*>(x + u * VEC);
        Gr b = *reinterpret_cast<const Gr*>(x + h + u * VEC);
#pragma unroll
        for (int z = 0; z < VEC; ++z) {
          const float2 c = cs[u * VEC + z];
          const float x1 = to_float(a.v[z]), x2 = to_float(b.v[z]);
          a.v[z] = from_float<T>(__fmaf_rn(x1, c.x, -__fmul_rn(x2, c.y)));
          b.v[z] = from_float<T>(__fmaf_rn(x2, c.x, __fmul_rn(x1, c.y)));
        }
        *reinterpret_cast<Gr*>(y + u * VEC) = a;
        *reinterpret_cast<Gr*>(y + h + u * VEC) = b;
      }
    } else {
      const int e = p.d_rot + (u - nrot) * VEC;
      *reinterpret_cast<Gr*>(y + e) = *reinterpret_cast<const Gr*>(x + e);
    }
  } else {  // interleaved, element by element: a group is one pair, then single elements
    if (u < h) {
      const float2 c = cs[u];
      const float x1 = to_float(x[2 * u]), x2 = to_float(x[2 * u + 1]);
      y[2 * u] = from_float<T>(__fmaf_rn(x1, c.x, -__fmul_rn(x2, c.y)));
      y[2 * u + 1] = from_float<T>(__fmaf_rn(x2, c.x, __fmul_rn(x1, c.y)));
    } else {
      y[p.d_rot + u - h] = x[p.d_rot + u - h];
    }
  }
}

template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float2 s_cs[];  // [tokens][d_rot / 2]
  __shared__ int s_b[kRopeMaxTokens], s_l[kRopeMaxTokens];
  const int h = p.d_rot >> 1;
  const long long t0 = (long long)blockIdx.x * p.tokens;
  const int nt = (int)min((long long)p.tokens, p.ntok - t0);
  grid_dep_wait();
  grid_dep_launch_next();
  if (threadIdx.x < nt) {
    s_b[threadIdx.x] = (int)((t0 + threadIdx.x) / p.L);
    s_l[threadIdx.x] = (int)((t0 + threadIdx.x) % p.L);
  }
  for (int e = threadIdx.x; e < nt * h; e += kRopeThreads) {
    const long long t = t0 + e / h;
    const long long at = (t / p.L) * p.pos_stride + t % p.L;
    const long long pos = p.pos64 ? static_cast<const long long*>(p.pos)[at]
                                  : (long long)static_cast<const int*>(p.pos)[at];
    float c, s;
    rope_angle(pos, __ldg(p.freq + e % h), &c, &s);
    s_cs[e] = make_float2(c * p.magnitude, s * p.magnitude * p.sign);
  }
  __syncthreads();
  const int nrot = (VEC == 1 || !INTER) ? h / VEC : p.d_rot / VEC;
  const int U = nrot + (p.copy_rest ? (p.d - p.d_rot) / VEC : 0);
  const int H = p.side[0].H + p.side[1].H;
  const int rows = nt * H;
  const unsigned items = (unsigned)rows * U;
  for (unsigned i = threadIdx.x; i < items; i += kRopeThreads) {
    const unsigned row = i / (unsigned)U, u = i - row * U;
    const unsigned tok = row / (unsigned)H;
    int head = row - tok * H;
    const int sd = head >= p.side[0].H;
    head -= sd ? p.side[0].H : 0;
    const RopeSide& s = p.side[sd];
    const T* x = static_cast<const T*>(s.x) + s_b[tok] * s.xs[0] + s_l[tok] * s.xs[1] + head * s.xs[2];
    T* y = static_cast<T*>(s.y) + s_b[tok] * s.ys[0] + s_l[tok] * s.ys[1] + head * s.ys[2];
    rope_row_group<T, VEC, INTER>(p, x, y, u, s_cs + tok * h);
  }
}

template <typename T>
cudaError_t launch_rope_t(const RopeParams& p, bool vec, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  const long long grid = (p.ntok + p.tokens - 1) / p.tokens;
  const size_t smem = (size_t)p.tokens * (p.d_rot / 2) * sizeof(float2);
  auto go = [&](auto kernel) {
    return launch_chained(kernel, dim3((unsigned)grid), dim3(kRopeThreads), smem, stream, p);
  };
  if (vec) return p.interleaved ? go(rope_kernel<T, V, true>) : go(rope_kernel<T, V, false>);
  return p.interleaved ? go(rope_kernel<T, 1, true>) : go(rope_kernel<T, 1, false>);
}

}  // namespace

cudaError_t launch_rope(const SepRope& r, int dtype, int B, int L, int d, const void* pos, int pos64,
                        long long pos_stride, const SepRopeTensor* q, const SepRopeTensor* k,
                        float sign, cudaStream_t stream) {
  RopeParams p = {};
  const size_t es = dtype == SEP_DTYPE_F32 ? 4 : 2;
  const int V = (int)(16 / es);
  // 16-byte accesses need every group 16-byte aligned: bases, strides, the start of the second
  // half and of the part that passes through. Otherwise the same kernel goes element by element.
  bool vec = d % V == 0 && r.d_rot % V == 0 && (r.interleaved || (r.d_rot / 2) % V == 0);
  bool inplace = true;
  const SepRopeTensor* side[2] = {q, k};
  for (int s = 0; s < 2; ++s) {
    if (!side[s]) continue;
    RopeSide& o = p.side[s];
    o.x = side[s]->x;
    o.y = side[s]->y;
    o.H = side[s]->H;
    bool same = o.x == o.y;
    for (int z = 0; z < 3; ++z) {
      o.xs[z] = side[s]->x_stride[z];
      o.ys[z] = side[s]->y_stride[z];
      vec = vec && o.xs[z] % V == 0 && o.ys[z] % V == 0;
      same = same && o.xs[z] == o.ys[z];
    }
    vec = vec && ((reinterpret_cast<uintptr_t>(o.x) | reinterpret_cast<uintptr_t>(o.y)) & 15) == 0;
    inplace = inplace && same;
  }
  p.pos = pos;
  p.pos64 = pos64;
  p.pos_stride = pos_stride;
  p.freq = r.freq;
  p.ntok = (long long)B * L;
  p.L = L;
  p.d = d;
  p.d_rot = r.d_rot;
  p.interleaved = r.interleaved;
  p.copy_rest = !inplace;
  p.magnitude = r.magnitude;
  p.sign = sign;
  // enough CTAs for every SM a few times over, then up to 16 tokens each
  p.tokens = (int)std::min<long long>(kRopeMaxTokens, std::max<long long>(1, p.ntok / (148 * 6)));
  if (dtype == SEP_DTYPE_BF16) return launch_rope_t<__nv_bfloat16>(p, vec, stream);
  if (dtype == SEP_DTYPE_F16) return launch_rope_t<__half>(p, vec, stream);
  return launch_rope_t<float>(p, vec, stream);
}

}  // namespace sep
