// Quantising K/V into the paged 8-bit cache as it is written, and reading it
// back (formats and formula: kv8.cuh).
//
// Both work on "items": the (row, block column) pairs that a call touches. A
// row's new (or read) tokens are the n_b = tok_start[b+1] - tok_start[b] last
// positions up to seq_lens[b]; they touch at most n_b / 16 + 2 blocks, so item
// numbers tok_start[b] / 16 + 2 b + (0, 1, ...) never overlap between rows and
// the grid follows from n_tokens and B on the host, with no device count. A
// warp takes one (item, layer, KV head, K or V): it owns that block's 16 x d
// codes and its scale, so no two warps write the same bytes and the largest
// magnitude is one warp reduction.
#include "kv8.cuh"
#include "plan.cuh"

using namespace oda;

namespace {

struct Kv8Args {
  const void* k_new;            // append: [nl][n_tokens][hkv][d]
  const void* v_new;
  void* k_out;                  // read: the same layout, either may be null
  void* v_out;
  const int32_t* tok_start;     // [B+1], or null: one token per row
  const int32_t* seq_lens;
  const int32_t* block_table;
  uint8_t* codes;               // layer 0 base
  float* scales;
  void* ring;                   // layer 0 base, or null
  long long n_tokens;
  long long items;
  long long warps;              // warps with a unit of work
  long long num_blocks;
  long long ring_layer_elems;
  int max_blocks, B, hkv, lb, nl;
  int sink, window, ring_blocks;
  int* err;
};

struct Item {
  int b, col;          // row, block column
  int s0, s1;          // slots [s0, s1) of the block
  int t;
  long long tok;       // token (of n_tokens) in slot s0
  long long blk;       // physical block
};

// Work out item `it`; false: nothing to do (or a bad argument, recorded).
__device__ __forceinline__ bool find_item(const Kv8Args& a, long long it, Item& m) {
  int j = 0;
  long long ts = it, n = 1;
  m.b = (int)it;
  if (a.tok_start) {
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {                           // largest b with start(b) <= it
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)__ldg(a.tok_start + mid) / ODA_TILE + 2ll * mid <= it) lo = mid; else hi = mid - 1;
    }
    m.b = lo;
    ts = __ldg(a.tok_start + lo);
    const long long te = __ldg(a.tok_start + lo + 1);
    n = te - ts;
    if (ts < 0 || n < 0 || te > a.n_tokens) {
      record_error(a.err, ODA_ERR_BOUNDS);
      return false;
    }
    if (n == 0) return false;
    j = (int)(it - (ts / ODA_TILE + 2ll * lo));
  }
  m.t = __ldg(a.seq_lens + m.b);
  const long long past = m.t - n;               // positions before the call's
  if (m.t < 1 || past < 0) {
    record_error(a.err, ODA_ERR_BOUNDS);
    return false;
  }
  m.col = (int)(past / ODA_TILE) + j;
  if (j < 0 || m.col > (m.t - 1) / ODA_TILE) return false;
  const long long p0 = (long long)m.col * ODA_TILE;
  const long long first = past > p0 ? past : p0;
  m.s0 = (int)(first - p0);
  m.s1 = (int)min((long long)ODA_TILE, m.t - p0);
  m.tok = ts + (first - past);
  m.blk = m.col < a.max_blocks ? __ldg(a.block_table + (long long)m.b * a.max_blocks + m.col) : -1;
  if (m.blk < 0 || m.blk >= a.num_blocks) {
    record_error(a.err, ODA_ERR_BOUNDS);
    return false;
  }
  return true;
}

// This warp's unit: (layer, item, KV head, K or V), K/V and heads fastest so
// that neighbouring warps read neighbouring rows of the new tokens.
__device__ __forceinline__ bool find_unit(const Kv8Args& a, int& l, int& g, int& kv, Item& m) {
  const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (w >= a.warps) return false;
  const int u = (int)(w % (2 * a.hkv));
  const long long r = w / (2 * a.hkv);
  kv = u & 1;
  g = u >> 1;
  l = (int)(r / a.items);
  return find_item(a, r % a.items, m);
}

template <typename T, int D>
struct Rows {
  static constexpr int EPL = 16 / (int)sizeof(T);     // elements per lane and row
  static constexpr int LPR = D / EPL;                 // lanes per row
  static constexpr int RPP = 32 / LPR;                // rows per pass of the warp
  static constexpr int PASSES = ODA_TILE / RPP;
};

template <typename T>
__device__ __forceinline__ uint32_t abs_bits_max(const uint4 v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(T) == 2) {
      m = max(m, (w[i] << 16) & 0x7fffffffu);
      m = max(m, w[i] & 0x7fff0000u);
    } else {
      m = max(m, w[i] & 0x7fffffffu);
    }
  }
  return m;
}

// The codes of a lane's 16 bytes of one row, at dst.
template <typename T, int FMT>
__device__ __forceinline__ void store_codes(uint8_t* dst, const uint4 v, float inv) {
  if (sizeof(T) == 2) {
    float x[8];
    bf16x2_to_f32(v.x, x[0], x[1]);
    bf16x2_to_f32(v.y, x[2], x[3]);
    bf16x2_to_f32(v.z, x[4], x[5]);
    bf16x2_to_f32(v.w, x[6], x[7]);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], inv);
    *reinterpret_cast<uint2*>(dst) = make_uint2(Fmt8<FMT>::pack(x[0], x[1], x[2], x[3]),
                                                Fmt8<FMT>::pack(x[4], x[5], x[6], x[7]));
  } else {
    *reinterpret_cast<uint32_t*>(dst) = Fmt8<FMT>::pack(
        __fmul_rn(__uint_as_float(v.x), inv), __fmul_rn(__uint_as_float(v.y), inv),
        __fmul_rn(__uint_as_float(v.z), inv), __fmul_rn(__uint_as_float(v.w), inv));
  }
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(256) append_kv8_kernel(const Kv8Args a) {
  using R = Rows<T, D>;
  pdl_wait();
  pdl_launch_dependents();
  int l, g, kv;
  Item m;
  if (!find_unit(a, l, g, kv, m)) return;
  const int lane = threadIdx.x & 31;
  const int rr = lane / R::LPR, li = lane % R::LPR;
  const T* src = static_cast<const T*>(kv ? a.v_new : a.k_new) +
                 (((long long)l * a.n_tokens + m.tok) * a.hkv + g) * D + li * R::EPL;
  const long long half = (((long long)(a.lb + l) * a.num_blocks + m.blk) * a.hkv + g) * 2 + kv;
  uint8_t* tile = a.codes + half * (ODA_TILE * D);
  const float old = m.s0 > 0 ? a.scales[half] : 0.f;
  uint4 x[R::PASSES];
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < R::PASSES; ++p) {
    const int s = p * R::RPP + rr;
    x[p] = make_uint4(0, 0, 0, 0);
    if (s >= m.s0 && s < m.s1)
      x[p] = __ldcs(reinterpret_cast<const uint4*>(src + (long long)(s - m.s0) * a.hkv * D));
  }
#pragma unroll
  for (int p = 0; p < R::PASSES; ++p) top = abs_bits_max<T>(x[p], top);
  top = __reduce_max_sync(0xffffffffu, top);
  float scale = fmaxf(__fdiv_rn(__uint_as_float(top), Fmt8<FMT>::kTop), old);
  if (scale < 0x1p-107f) scale = 0.f;
  // a value that is not finite (or was, earlier in this block) leaves no
  // scale that could stand for the block: it reads back as NaN
  if (top >= 0x7f800000u || old != old) scale = __uint_as_float(0x7fc00000u);
  const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
  if (m.s0 > 0 && scale > old) {
    // the scale grew: the codes held before move to the new one
    const float ratio = __fmul_rn(old, inv);
    uint32_t* w = reinterpret_cast<uint32_t*>(tile);
    for (int i = lane; i < m.s0 * (D / 4); i += 32) {
      const float4 c = codes_to_f32<FMT>(w[i]);
      w[i] = Fmt8<FMT>::pack(__fmul_rn(c.x, ratio), __fmul_rn(c.y, ratio), __fmul_rn(c.z, ratio),
                             __fmul_rn(c.w, ratio));
    }
  }
  if (lane == 0) a.scales[half] = scale;
#pragma unroll
  for (int p = 0; p < R::PASSES; ++p) {
    const int s = p * R::RPP + rr;
    if (s >= m.s0 && s < m.s1) store_codes<T, FMT>(tile + s * D + li * R::EPL, x[p], inv);
  }
  if (a.ring) {
    T* ring = static_cast<T*>(a.ring) + (long long)(a.lb + l) * a.ring_layer_elems +
              ((long long)m.b * a.hkv + g) * a.ring_blocks * 2 * ODA_TILE * D + li * R::EPL;
#pragma unroll
    for (int p = 0; p < R::PASSES; ++p) {
      const int s = p * R::RPP + rr;
      const long long pos = (long long)m.col * ODA_TILE + s;      // 0-indexed
      if (s < m.s0 || s >= m.s1) continue;
      if (pos >= (long long)m.t - a.window) {
        const int w = a.sink + (int)(pos % a.window);
        *reinterpret_cast<uint4*>(ring + ((long long)(w / ODA_TILE * 2 + kv) * ODA_TILE +
                                          w % ODA_TILE) * D) = x[p];
      }
      if (pos < a.sink)
        *reinterpret_cast<uint4*>(ring + ((pos / ODA_TILE * 2 + kv) * ODA_TILE + pos % ODA_TILE) * D) =
            x[p];
    }
  }
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(256) read_kv8_kernel(const Kv8Args a) {
  using R = Rows<T, D>;
  pdl_wait();
  pdl_launch_dependents();
  int l, g, kv;
  Item m;
  if (!find_unit(a, l, g, kv, m)) return;
  T* out = static_cast<T*>(kv ? a.v_out : a.k_out);
  if (!out) return;
  const int lane = threadIdx.x & 31;
  const int rr = lane / R::LPR, li = lane % R::LPR;
  out += (((long long)l * a.n_tokens + m.tok) * a.hkv + g) * D + li * R::EPL;
  const long long half = (((long long)(a.lb + l) * a.num_blocks + m.blk) * a.hkv + g) * 2 + kv;
  const uint8_t* tile = a.codes + half * (ODA_TILE * D) + li * R::EPL;
  const float scale = a.scales[half];
  uint32_t w[R::PASSES][R::EPL / 4];
#pragma unroll
  for (int p = 0; p < R::PASSES; ++p) {
    const int s = p * R::RPP + rr;
    const bool in = s >= m.s0 && s < m.s1;
#pragma unroll
    for (int i = 0; i < R::EPL / 4; ++i)
      w[p][i] = in ? reinterpret_cast<const uint32_t*>(tile + s * D)[i] : 0u;
  }
#pragma unroll
  for (int p = 0; p < R::PASSES; ++p) {
    const int s = p * R::RPP + rr;
    if (s < m.s0 || s >= m.s1) continue;
    T* dst = out + (long long)(s - m.s0) * a.hkv * D;
    uint4 v;
    if (sizeof(T) == 2) {
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < R::EPL / 4; ++i) {
        const float4 c = codes_to_f32<FMT>(w[p][i]);
        const __nv_bfloat162 e = __floats2bfloat162_rn(__fmul_rn(c.x, scale), __fmul_rn(c.y, scale));
        const __nv_bfloat162 f = __floats2bfloat162_rn(__fmul_rn(c.z, scale), __fmul_rn(c.w, scale));
        r[2 * i] = *reinterpret_cast<const uint32_t*>(&e);
        r[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&f);
      }
      v = make_uint4(r[0], r[1], r[2], r[3]);
    } else {
      const float4 c = codes_to_f32<FMT>(w[p][0]);
      v = make_uint4(__float_as_uint(__fmul_rn(c.x, scale)), __float_as_uint(__fmul_rn(c.y, scale)),
                     __float_as_uint(__fmul_rn(c.z, scale)), __float_as_uint(__fmul_rn(c.w, scale)));
    }
    __stcs(reinterpret_cast<uint4*>(dst), v);
  }
}

template <typename F>
oda_status dispatch(const oda_config& c, int format, F&& f) {
#define ODA_CASE(TT, DT, DD, FF)                                     \
  if (c.dtype == DT && c.head_dim == DD && format == FF) return f.template operator()<TT, DD, FF>();
  ODA_CASE(__nv_bfloat16, ODA_BF16, 128, kInt8) ODA_CASE(__nv_bfloat16, ODA_BF16, 128, kE4m3)
  ODA_CASE(__nv_bfloat16, ODA_BF16, 64, kInt8) ODA_CASE(__nv_bfloat16, ODA_BF16, 64, kE4m3)
  ODA_CASE(float, ODA_F32, 128, kInt8) ODA_CASE(float, ODA_F32, 128, kE4m3)
  ODA_CASE(float, ODA_F32, 64, kInt8) ODA_CASE(float, ODA_F32, 64, kE4m3)
#undef ODA_CASE
  return ODA_ERR_SHAPE;
}

struct Launch {
  const Kv8Args* a;
  bool append;
  cudaStream_t st;
  template <typename T, int D, int FMT>
  oda_status operator()() {
    const long long grid = ceil_div64(a->warps, 8);
    if (grid >= (1ll << 31)) return ODA_ERR_SHAPE;
    auto k = append ? append_kv8_kernel<T, D, FMT> : read_kv8_kernel<T, D, FMT>;
    return launch_pdl(k, dim3((unsigned)grid), dim3(256), 0, st, *a) == cudaSuccess ? ODA_OK
                                                                                    : ODA_ERR_CUDA;
  }
};

oda_status launch(oda_ctx* ctx, bool append, int format, int lb, int le, Kv8Args& a, int B,
                  long long n_tokens, cudaStream_t st) {
  const oda_config& c = ctx->cfg;
  a.n_tokens = n_tokens;
  a.items = a.tok_start ? n_tokens / ODA_TILE + 2ll * B : B;
  a.warps = a.items * (le - lb) * 2 * c.hkv;
  a.num_blocks = c.num_blocks;
  a.ring_layer_elems = ctx->lay.ring_layer_elems;
  a.max_blocks = c.max_blocks_per_seq;
  a.B = B;
  a.hkv = c.hkv;
  a.lb = lb;
  a.nl = le - lb;
  a.sink = c.sink;
  a.window = c.window;
  a.ring_blocks = (int)ctx->lay.ring_blocks;
  a.err = ctx->err;
  return dispatch(c, format, Launch{&a, append, st});
}

}  // namespace

namespace oda_impl {

oda_status launch_append_kv8(oda_ctx* ctx, int format, int lb, int le, const void* k_new,
                             const void* v_new, const int32_t* tok_start, long long n_tokens,
                             const int32_t* seq_lens, const int32_t* block_table, void* codes,
                             float* scales, void* ring, int B, cudaStream_t st) {
  Kv8Args a = {};
  a.k_new = k_new;
  a.v_new = v_new;
  a.tok_start = tok_start;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.ring = ring;
  return launch(ctx, true, format, lb, le, a, B, n_tokens, st);
}

oda_status launch_read_kv8(oda_ctx* ctx, int format, int lb, int le, const int32_t* tok_start,
                           long long n_tokens, const int32_t* seq_lens, const int32_t* block_table,
                           const void* codes, const float* scales, void* k_out, void* v_out, int B,
                           cudaStream_t st) {
  Kv8Args a = {};
  a.k_out = k_out;
  a.v_out = v_out;
  a.tok_start = tok_start;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
  a.scales = const_cast<float*>(scales);
  return launch(ctx, false, format, lb, le, a, B, n_tokens, st);
}

}  // namespace oda_impl
