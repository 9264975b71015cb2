// RMS norm of every query and key head and the rotation by position, in one
// pass over the projections' output.
//
//   y = x * rsqrt(mean(x^2) + eps) * w        over the head's d elements,
//   (a, b) -> (a cos - b sin, b cos + a sin)  for each rotated pair,
//   angle = (positions[j] + pos_offset) * inv_freq[i].
// All in float32, rounded once into the output's type. The angle of a far
// position has more turns than float32 can count: the number of turns is
// formed in float64, its whole part dropped there, and only the remaining
// fraction of a turn goes to float32 (error below 2^-25 turns plus the
// float64 product's, 2^-53 of the turns).
//
// A block takes TOK tokens. Its threads first work out each token's cosines
// and sines once, into shared memory, for all the token's heads; then groups
// of lanes with 16 bytes each take the heads in turn.
#include "oda_internal.cuh"

using namespace oda;

namespace {

constexpr int kThreads = 256;

struct RopeArgs {
  const void* q;
  const void* k;                // or null
  const void* q_weight;         // [d] of the context's type, or null: no norm
  const void* k_weight;
  const float* inv_freq;        // [rot / 2]
  const int32_t* positions;     // [n]
  void* q_out;
  void* k_out;
  long long q_stride, k_stride, q_out_stride, k_out_stride;   // elements between tokens
  long long n;
  float eps;
  int pos_offset, rot, hq, hkv;
};

template <typename T>
__device__ __forceinline__ void widen(const uint4 v, float* x);
template <>
__device__ __forceinline__ void widen<__nv_bfloat16>(const uint4 v, float* x) {
  bf16x2_to_f32(v.x, x[0], x[1]);
  bf16x2_to_f32(v.y, x[2], x[3]);
  bf16x2_to_f32(v.z, x[4], x[5]);
  bf16x2_to_f32(v.w, x[6], x[7]);
}
template <>
__device__ __forceinline__ void widen<float>(const uint4 v, float* x) {
  x[0] = __uint_as_float(v.x);
  x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z);
  x[3] = __uint_as_float(v.w);
}
template <typename T>
__device__ __forceinline__ uint4 narrow(const float* x);
template <>
__device__ __forceinline__ uint4 narrow<__nv_bfloat16>(const float* x) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 e = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    r[i] = *reinterpret_cast<const uint32_t*>(&e);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
template <>
__device__ __forceinline__ uint4 narrow<float>(const float* x) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                    __float_as_uint(x[3]));
}

template <typename T, int D, int TOK, bool NEIGHBOURS>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int EPL = 16 / (int)sizeof(T);          // elements per lane
  constexpr int LPH = D / EPL;                      // lanes per head
  constexpr int GROUPS = kThreads / LPH;
  __shared__ float2 turn[TOK][D / 2];               // (cos, sin)
  pdl_wait();
  pdl_launch_dependents();
  const int half = a.rot / 2;
  const long long j0 = (long long)blockIdx.x * TOK;
  const int ntok = (int)min((long long)TOK, a.n - j0);
  for (int i = threadIdx.x; i < ntok * half; i += kThreads) {
    const int tk = i / half, f = i - tk * half;
    const double pos = (double)((long long)a.positions[j0 + tk] + a.pos_offset);
    const double turns = pos * ((double)a.inv_freq[f] * 0.15915494309189533577);
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    turn[tk][f] = make_float2(c, s);
  }
  __syncthreads();
  const int li = threadIdx.x % LPH, grp = threadIdx.x / LPH;
  const int e0 = li * EPL;
  const int heads = a.hq + (a.k ? a.hkv : 0);
  const int lane = threadIdx.x & 31;
  const bool rotated = e0 < a.rot;
  const bool first = e0 < half;
  // the lane of the same head that holds the other half of this lane's pairs
  const int other = rotated ? lane + (first ? half / EPL : -(half / EPL)) : lane;
  for (int base = 0; base < ntok * heads; base += GROUPS) {     // uniform over the block
    const int it = base + grp;
    const bool in = it < ntok * heads;
    const int tk = in ? it / heads : 0;
    const int h = in ? it - tk * heads : 0;
    const bool is_k = h >= a.hq;
    const T* src = is_k ? static_cast<const T*>(a.k) + (j0 + tk) * a.k_stride + (h - a.hq) * D
                        : static_cast<const T*>(a.q) + (j0 + tk) * a.q_stride + h * D;
    const T* wsrc = static_cast<const T*>(is_k ? a.k_weight : a.q_weight);
    float x[EPL];
    uint4 v = make_uint4(0, 0, 0, 0);
    if (in) v = *reinterpret_cast<const uint4*>(src + e0);
    widen<T>(v, x);
    // (every lane reduces: a warp may hold a head with a weight and one without)
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, LPH);
    if (wsrc) {
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      float w[EPL];
      widen<T>(*reinterpret_cast<const uint4*>(wsrc + e0), w);
#pragma unroll
      for (int i = 0; i < EPL; ++i) x[i] = x[i] * r * w[i];
    }
    float y[EPL];
    if (NEIGHBOURS) {
#pragma unroll
      for (int i = 0; i < EPL; i += 2) {
        const float2 cs = rotated ? turn[tk][(e0 + i) / 2] : make_float2(1.f, 0.f);
        y[i] = x[i] * cs.x - x[i + 1] * cs.y;
        y[i + 1] = x[i + 1] * cs.x + x[i] * cs.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float p = __shfl_sync(0xffffffffu, x[i], other);
        const float2 cs = rotated ? turn[tk][first ? e0 + i : e0 + i - half] : make_float2(1.f, 0.f);
        y[i] = first ? x[i] * cs.x - p * cs.y : x[i] * cs.x + p * cs.y;
        if (!rotated) y[i] = x[i];
      }
    }
    if (in) {
      T* dst = is_k ? static_cast<T*>(a.k_out) + (j0 + tk) * a.k_out_stride + (h - a.hq) * D
                    : static_cast<T*>(a.q_out) + (j0 + tk) * a.q_out_stride + h * D;
      *reinterpret_cast<uint4*>(dst + e0) = narrow<T>(y);
    }
  }
}

template <typename T, int D>
oda_status launch_td(const RopeArgs& a, bool neighbours, cudaStream_t st) {
  constexpr int TOK = 1;
  const long long grid = ceil_div64(a.n, TOK);
  if (grid >= (1ll << 31)) return ODA_ERR_SHAPE;
  auto k = neighbours ? qk_norm_rope_kernel<T, D, TOK, true> : qk_norm_rope_kernel<T, D, TOK, false>;
  return launch_pdl(k, dim3((unsigned)grid), dim3(kThreads), 0, st, a) == cudaSuccess ? ODA_OK
                                                                                      : ODA_ERR_CUDA;
}

}  // namespace

namespace oda_impl {

oda_status launch_qk_norm_rope(oda_ctx* ctx, const void* q, int64_t q_stride, const void* k,
                               int64_t k_stride, const void* q_weight, const void* k_weight,
                               float eps, const float* inv_freq, int rot, bool neighbours,
                               const int32_t* positions, int pos_offset, int64_t n, void* q_out,
                               int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                               cudaStream_t st) {
  const oda_config& c = ctx->cfg;
  RopeArgs a;
  a.q = q;
  a.k = k;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.n = n;
  a.eps = eps;
  a.pos_offset = pos_offset;
  a.rot = rot;
  a.hq = c.hq;
  a.hkv = c.hkv;
  if (c.dtype == ODA_BF16)
    return c.head_dim == 128 ? launch_td<__nv_bfloat16, 128>(a, neighbours, st)
                             : launch_td<__nv_bfloat16, 64>(a, neighbours, st);
  return c.head_dim == 128 ? launch_td<float, 128>(a, neighbours, st)
                           : launch_td<float, 64>(a, neighbours, st);
}

}  // namespace oda_impl
