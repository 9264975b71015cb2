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
// Every element is read once and written once; 16K tokens of 24 heads of 128 (201 MB)
// take 34 us, 5.9 TB/s, with most of the issue slots in use. Each
// lane owns both elements of its pairs (two 16-byte chunks half a rotated part
// apart), so the rotation needs no exchange and the norm's sum is one
// butterfly over the D / 16 lanes (bf16) of a head. A block takes `tok` tokens:
// its loads are issued first, kItems heads a lane, and the tokens' cosines and
// sines are worked out once, into shared memory, for all their heads while the
// loads fly.
#include "oda_internal.cuh"

using namespace oda;

namespace {

constexpr int kItems = 3;        // heads of a lane in flight
constexpr int kMaxTok = 8;       // tokens of a block

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
  int pos_offset, rot, hq, hkv, tok;
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

template <typename T, int D, bool NEIGHBOURS, int kThreads>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int EPL = 16 / (int)sizeof(T);          // elements of a chunk
  constexpr int NL = D / EPL / 2;                   // lanes per head, two chunks each
  constexpr int GROUPS = kThreads / NL;
  // (cos, sin) of two pairs in 16 bytes; a lane reads M of them a chunk, stored
  // M apart so that neighbouring lanes read neighbouring 16 bytes
  constexpr int M = NEIGHBOURS ? EPL / 4 : EPL / 2;
  constexpr int UNITS = D / 4;
  __shared__ float4 turn[kMaxTok][UNITS];
  const auto slot = [](int u) { return u % M * (UNITS / M) + u / M; };
  pdl_wait();
  pdl_launch_dependents();
  const int half = a.rot / 2;
  const long long j0 = (long long)blockIdx.x * a.tok;
  const int ntok = (int)min((long long)a.tok, a.n - j0);
  const int heads = a.hq + (a.k ? a.hkv : 0);
  const int li = threadIdx.x % NL, grp = threadIdx.x / NL;
  // this lane's chunks: a pair of halves of the rotated part, or two behind it
  const int pairs = half / EPL;
  const bool rotated = li < pairs;
  const int c0 = rotated ? li * EPL : a.rot + (li - pairs) * 2 * EPL;
  const int c1 = rotated ? c0 + half : c0 + EPL;
  int tk = grp / heads, h = grp - tk * heads;       // the group's first (token, head)
  const int step_tk = GROUPS / heads, step_h = GROUPS - step_tk * heads;
  bool first = true;
  do {
    uint4 v[kItems][2];
    int itk[kItems], ih[kItems];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      itk[u] = tk;
      ih[u] = h;
      // (behind the last head the last token's again: no branch between the loads)
      const long long j = j0 + min(tk, ntok - 1);
      const T* src = h >= a.hq ? static_cast<const T*>(a.k) + j * a.k_stride + (h - a.hq) * D
                               : static_cast<const T*>(a.q) + j * a.q_stride + h * D;
      v[u][0] = *reinterpret_cast<const uint4*>(src + c0);
      v[u][1] = *reinterpret_cast<const uint4*>(src + c1);
      tk += step_tk;
      h += step_h;
      if (h >= heads) {
        h -= heads;
        ++tk;
      }
    }
    if (first) {
      first = false;
      for (int i = threadIdx.x; i < ntok * half; i += kThreads) {
        const int t = i / half, f = i - t * half;
        const double pos = (double)((long long)a.positions[j0 + t] + a.pos_offset);
        const double turns = pos * ((double)a.inv_freq[f] * 0.15915494309189533577);
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        reinterpret_cast<float2*>(&turn[t][slot(f / 2)])[f & 1] = make_float2(c, s);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      float x[2][EPL];
      widen<T>(v[u][0], x[0]);
      widen<T>(v[u][1], x[1]);
      const bool is_k = ih[u] >= a.hq;
      const T* w = static_cast<const T*>(is_k ? a.k_weight : a.q_weight);
      // (every lane reduces: a warp may hold heads with a weight and without, or none)
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) ss = fmaf(x[0][i], x[0][i], fmaf(x[1][i], x[1][i], ss));
#pragma unroll
      for (int o = 1; o < NL; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, NL);
      if (itk[u] >= ntok) continue;
      if (w) {
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float wf[EPL];
          widen<T>(*reinterpret_cast<const uint4*>(w + (p ? c1 : c0)), wf);
#pragma unroll
          for (int i = 0; i < EPL; ++i) x[p][i] = x[p][i] * r * wf[i];
        }
      }
      if (rotated) {
        const float4* tt = turn[itk[u]];
        if (NEIGHBOURS) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int u0 = (p ? c1 : c0) / 4;
#pragma unroll
            for (int m = 0; m < M; ++m) {
              const float4 cs = tt[slot(u0 + m)];
              float* y = x[p] + 4 * m;
              const float y0 = y[0], y1 = y[1], y2 = y[2], y3 = y[3];
              y[0] = y0 * cs.x - y1 * cs.y;
              y[1] = y1 * cs.x + y0 * cs.y;
              y[2] = y2 * cs.z - y3 * cs.w;
              y[3] = y3 * cs.z + y2 * cs.w;
            }
          }
        } else {
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const float4 cs = tt[slot(li * M + m)];
            const float a0 = x[0][2 * m], a1 = x[0][2 * m + 1], b0 = x[1][2 * m], b1 = x[1][2 * m + 1];
            x[0][2 * m] = a0 * cs.x - b0 * cs.y;
            x[1][2 * m] = b0 * cs.x + a0 * cs.y;
            x[0][2 * m + 1] = a1 * cs.z - b1 * cs.w;
            x[1][2 * m + 1] = b1 * cs.z + a1 * cs.w;
          }
        }
      }
      T* dst = is_k ? static_cast<T*>(a.k_out) + (j0 + itk[u]) * a.k_out_stride + (ih[u] - a.hq) * D
                    : static_cast<T*>(a.q_out) + (j0 + itk[u]) * a.q_out_stride + ih[u] * D;
      *reinterpret_cast<uint4*>(dst + c0) = narrow<T>(x[0]);
      *reinterpret_cast<uint4*>(dst + c1) = narrow<T>(x[1]);
    }
  } while (__any_sync(0xffffffffu, tk < ntok));
}

template <typename T, int D, int kThreads>
oda_status launch_threads(RopeArgs& a, bool neighbours, int sms, cudaStream_t st) {
  constexpr int GROUPS = kThreads / (D * (int)sizeof(T) / 32);
  const int heads = a.hq + (a.k ? a.hkv : 0);
  // twice the tokens that a block's lanes hold at once (16K tokens of 24 heads: 34.2 us;
  // once 35.7, three times 36.5), while every SM has a block (1537 tokens of 6
  // heads: 3.0 us; with four blocks for every SM 4.2)
  a.tok = 2 * kItems * GROUPS / heads;
  a.tok = a.tok < 1 ? 1 : a.tok > kMaxTok ? kMaxTok : a.tok;
  while (a.tok > 1 && ceil_div64(a.n, a.tok) < sms) --a.tok;
  const long long grid = ceil_div64(a.n, a.tok);
  if (grid >= (1ll << 31)) return ODA_ERR_SHAPE;
  auto k = neighbours ? qk_norm_rope_kernel<T, D, true, kThreads> : qk_norm_rope_kernel<T, D, false, kThreads>;
  return launch_pdl(k, dim3((unsigned)grid), dim3(kThreads), 0, st, a) == cudaSuccess ? ODA_OK
                                                                                      : ODA_ERR_CUDA;
}

// Fewer tokens than SMs: a block has an SM to itself, the larger one is quicker
// (16 tokens of 24 heads: 2.2 against 2.6 us). More: smaller blocks leave fewer
// loads waiting for a block's last (16K tokens, once: 36.0 against 37.0 us).
template <typename T, int D>
oda_status launch_td(RopeArgs& a, bool neighbours, int sms, cudaStream_t st) {
  return a.n < sms ? launch_threads<T, D, 256>(a, neighbours, sms, st)
                   : launch_threads<T, D, 128>(a, neighbours, sms, st);
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
    return c.head_dim == 128 ? launch_td<__nv_bfloat16, 128>(a, neighbours, ctx->num_sms, st)
                             : launch_td<__nv_bfloat16, 64>(a, neighbours, ctx->num_sms, st);
  return c.head_dim == 128 ? launch_td<float, 128>(a, neighbours, ctx->num_sms, st)
                           : launch_td<float, 64>(a, neighbours, ctx->num_sms, st);
}

}  // namespace oda_impl
