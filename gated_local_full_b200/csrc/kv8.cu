// Quantising K/V into the paged 8-bit cache as it is written, and reading it
// back (formats and formula: kv8.cuh).
//
// Both work on "items": the (row, block column) pairs that a call touches. A
// row's new (or read) tokens are the n_b = tok_start[b+1] - tok_start[b] last
// positions up to seq_lens[b]; they touch at most n_b / 16 + 2 blocks, so item
// numbers tok_start[b] / 16 + 2 b + (0, 1, ...) never overlap between rows and
// the grid follows from n_tokens and B on the host, with no device count. An
// item has 2 hkv units (KV head, K or V) a layer: 16 x d codes and a scale each,
// one after another in memory. A unit belongs to one warp (or half of one), so
// no two write the same bytes and the largest magnitude is one reduction.
//   append, one token a row: a quarter to a whole warp a unit, all of them in
//     one wave; bound by the latency of lengths -> block id -> scale (28 layers of 32
//     rows, 8 KV heads: 5 us).
//   append, any number: a warp a unit, the new tokens requested before the
//     block id; bound by HBM (16K tokens, 100 MB: about 17 us).
//   read: a warp takes kReadUnits units of an item, whose codes are all
//     requested before the first is turned into values: more than half of the
//     item numbers may be empty, and finding an item costs two round trips. Bound by
//     HBM (8 x 16K tokens, 805 MB: 126 us, 6.4 TB/s).
#include "kv8.cuh"

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
  long long num_blocks;
  long long ring_layer_elems;
  unsigned items, groups;       // groups: of units, the work of one warp
  int max_blocks, B, hkv, lb;
  int sink, window, ring_blocks;
  int* err;
};

// Blocks of 64, 128 and 256 threads: 28 layers x 32 rows written and read back 16.0, 14.0
// and 14.8 us, a 16K prefill 32.4, 32.4 and 33.8, ragged float32 chunks 5.2, 5.7 and 6.8.
constexpr int kThreads = 128;
// One, two and four units (in blocks of 256 threads): 28 layers x 32 rows written and
// read back 17.2, 14.7 and 15.6 us, 8 x 16K tokens read 124.6, 126.2 and 126.1 us.
constexpr int kReadUnits = 2;

struct Item {
  int b, col;          // row, block column
  int s0, s1;          // slots [s0, s1) of the block
  int t;
  long long tok;       // token (of n_tokens) in slot s0
};

// Work out item `it` (a whole warp); false: nothing to do, or a bad argument
// (recorded).
__device__ __forceinline__ bool find_item(const Kv8Args& a, unsigned it, Item& m) {
  const int lane = threadIdx.x & 31;
  int j = 0;
  long long ts = it, n = 1;
  m.b = (int)it;
  if (a.tok_start) {
    // the last row that starts at or before it; all that is needed of a row is
    // asked for at once. The numbers hold as long as the stretches are in order: the first row
    // whose is not is the last that is looked at (the last item, if no other, gets
    // there), and neither it nor a row behind has an item.
    int b = 0, r_ts = 0, r_te = 0, r_t = 0;
    bool ordered = true;
    for (int base = 0; base < a.B; base += 32) {
      const int r = base + lane;
      int v_ts = 0, v_te = 0, v_t = 0;
      if (r < a.B) {
        v_ts = load_int(a.tok_start + r);
        v_te = load_int(a.tok_start + r + 1);
        v_t = load_int(a.seq_lens + r);
      }
      const unsigned wrong = __ballot_sync(0xffffffffu, v_ts < 0 || v_te < v_ts || v_te > a.n_tokens);
      const unsigned who = ((wrong & (0u - wrong)) * 2u - 1u) &    // up to the first wrong one
          __ballot_sync(0xffffffffu, r < a.B && (long long)v_ts / ODA_TILE + 2ll * r <= (long long)it);
      if (wrong) record_error(a.err, ODA_ERR_BOUNDS);
      if (!who) break;
      const int at = 31 - __clz(who);
      b = base + at;
      r_ts = __shfl_sync(0xffffffffu, v_ts, at);
      r_te = __shfl_sync(0xffffffffu, v_te, at);
      r_t = __shfl_sync(0xffffffffu, v_t, at);
      ordered = !((wrong >> at) & 1u);
      if (wrong) break;
    }
    if (!ordered) return false;
    m.b = b;
    m.t = r_t;
    ts = r_ts;
    n = (long long)r_te - ts;
    if (n == 0) return false;
    j = (int)((long long)it - (ts / ODA_TILE + 2ll * b));
  } else {
    m.t = load_int(a.seq_lens + m.b);
  }
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
  return true;
}

// The physical block of a row's column, or -1 (recorded).
__device__ __forceinline__ long long find_block(const Kv8Args& a, int b, int col) {
  const long long blk =
      col < a.max_blocks ? load_int(a.block_table + (long long)b * a.max_blocks + col) : -1;
  if (blk >= 0 && blk < a.num_blocks) return blk;
  record_error(a.err, ODA_ERR_BOUNDS);
  return -1;
}

template <typename T, int D>
struct Rows {
  static constexpr int EPL = 16 / (int)sizeof(T);     // elements per lane and row
  static constexpr int LPR = D / EPL;                 // lanes per row
  static constexpr int RPP = 32 / LPR;                // rows per pass of the warp
  static constexpr int PASSES = ODA_TILE / RPP;
};

// Running maximum of |x| as bits: of float32, or of each half of a bf16 pair
// (sign-free bits order as the magnitudes do, NaN above infinity).
template <typename T>
__device__ __forceinline__ uint32_t abs_bits_max(const uint4 v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = sizeof(T) == 2 ? __vmaxu2(m, w[i] & 0x7fff7fffu) : max(m, w[i] & 0x7fffffffu);
  return m;
}

// ... and as float32 bits.
template <typename T>
__device__ __forceinline__ uint32_t abs_bits_f32(uint32_t m) {
  return sizeof(T) == 2 ? max(m << 16, m & 0xffff0000u) : m;
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

// A block's scale once values of magnitude `top` (float32 bits) join it.
template <int FMT>
__device__ __forceinline__ float new_scale(uint32_t top, float old) {
  float scale = fmaxf(__fdiv_rn(__uint_as_float(top), Fmt8<FMT>::kTop), old);
  if (scale < 0x1p-107f) scale = 0.f;
  // a value that is not finite (or was, earlier in this block) leaves no
  // scale that could stand for the block: it reads back as NaN
  if (top >= 0x7f800000u || old != old) scale = __uint_as_float(0x7fc00000u);
  return scale;
}

// The codes held before move to a grown scale: `words` of them by `lanes` lanes.
template <int FMT>
__device__ __forceinline__ void rescale_codes(uint8_t* tile, int words, int lane, int lanes, float old,
                                              float inv) {
  const float ratio = __fmul_rn(old, inv);
  uint32_t* w = reinterpret_cast<uint32_t*>(tile);
  for (int i = lane; i < words; i += lanes) {
    const float4 c = codes_to_f32<FMT>(w[i]);
    w[i] = Fmt8<FMT>::pack(__fmul_rn(c.x, ratio), __fmul_rn(c.y, ratio), __fmul_rn(c.z, ratio),
                           __fmul_rn(c.w, ratio));
  }
}

// A token's chunk of one head into the ring: its slot of the window, and of the
// sinks. pos is 0-indexed, t the row's last position, ring the head's chunk.
template <typename T, int D>
__device__ __forceinline__ void store_ring(const Kv8Args& a, T* ring, int pos, int t, int kv,
                                           const uint4 x) {
  if (pos >= (long long)t - a.window) {
    const int w = a.sink + pos % a.window;
    *reinterpret_cast<uint4*>(ring + ((long long)(w / ODA_TILE * 2 + kv) * ODA_TILE + w % ODA_TILE) * D) = x;
  }
  if (pos < a.sink)
    *reinterpret_cast<uint4*>(ring + ((long long)(pos / ODA_TILE * 2 + kv) * ODA_TILE + pos % ODA_TILE) * D) = x;
}

template <typename T, int D>
__device__ __forceinline__ T* ring_chunk(const Kv8Args& a, int l, int b, int g, int li) {
  return static_cast<T*>(a.ring) + (long long)(a.lb + l) * a.ring_layer_elems +
         ((long long)b * a.hkv + g) * a.ring_blocks * 2 * ODA_TILE * D + li * Rows<T, D>::EPL;
}

// One token a row: LPR lanes a unit, one chunk of 16 bytes each.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kThreads) append_one_kv8_kernel(const Kv8Args a) {
  using R = Rows<T, D>;
  pdl_wait();
  pdl_launch_dependents();
  const unsigned idx = blockIdx.x * (kThreads / R::LPR) + threadIdx.x / R::LPR;
  const unsigned units = 2u * a.hkv;
  const unsigned b = idx / units, unit = idx - b * units;
  if (b >= (unsigned)a.B) return;               // LPR lanes together
  const int kv = unit & 1, g = unit >> 1, l = blockIdx.y;
  const int li = threadIdx.x % R::LPR;
  const unsigned lanes = (R::LPR == 32 ? 0xffffffffu : (1u << (R::LPR & 31)) - 1u)
                         << ((threadIdx.x & 31) / R::LPR * R::LPR);
  const T* src = static_cast<const T*>(kv ? a.v_new : a.k_new) +
                 (((long long)l * a.n_tokens + b) * a.hkv + g) * D + li * R::EPL;
  const uint4 x = load_stream(reinterpret_cast<const uint4*>(src));
  const int t = load_int(a.seq_lens + b);
  if (t < 1) {
    record_error(a.err, ODA_ERR_BOUNDS);
    return;
  }
  const long long blk = find_block(a, (int)b, (t - 1) / ODA_TILE);
  if (blk < 0) return;
  const int s = (t - 1) % ODA_TILE;
  const long long half = (((long long)(a.lb + l) * a.num_blocks + blk) * a.hkv + g) * 2 + kv;
  uint8_t* tile = a.codes + half * (ODA_TILE * D);
  const float old = s > 0 ? a.scales[half] : 0.f;
  uint32_t top = abs_bits_max<T>(x, 0u);
  top = __reduce_max_sync(lanes, abs_bits_f32<T>(top));
  const float scale = new_scale<FMT>(top, old);
  const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
  if (s > 0 && scale > old) rescale_codes<FMT>(tile, s * (D / 4), li, R::LPR, old, inv);
  __syncwarp(lanes);                            // every lane has read the old scale
  if (li == 0) a.scales[half] = scale;
  store_codes<T, FMT>(tile + s * D + li * R::EPL, x, inv);
  if (a.ring) store_ring<T, D>(a, ring_chunk<T, D>(a, l, (int)b, g, li), t - 1, t, kv, x);
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kThreads, (sizeof(T) == 2 ? 1024 : 512) / kThreads) append_kv8_kernel(const Kv8Args a) {
  using R = Rows<T, D>;
  pdl_wait();
  pdl_launch_dependents();
  const unsigned w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const unsigned it = w / a.groups, unit = w - it * a.groups;
  if (it >= a.items) return;
  Item m;
  if (!find_item(a, it, m)) return;
  const int kv = unit & 1, g = unit >> 1, l = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int rr = lane / R::LPR, li = lane % R::LPR;
  const T* src = static_cast<const T*>(kv ? a.v_new : a.k_new) +
                 (((long long)l * a.n_tokens + m.tok) * a.hkv + g) * D + li * R::EPL;
  uint4 x[R::PASSES];
#pragma unroll
  for (int p = 0; p < R::PASSES; ++p) {
    // (a slot outside reads the first token again: no branch between the loads,
    // and the largest magnitude stays)
    const int s = p * R::RPP + rr;
    const int i = s >= m.s0 && s < m.s1 ? s - m.s0 : 0;
    x[p] = load_stream(reinterpret_cast<const uint4*>(src + (long long)i * a.hkv * D));
  }
  const long long blk = find_block(a, m.b, m.col);
  if (blk < 0) return;
  const long long half = (((long long)(a.lb + l) * a.num_blocks + blk) * a.hkv + g) * 2 + kv;
  uint8_t* tile = a.codes + half * (ODA_TILE * D);
  const float old = m.s0 > 0 ? a.scales[half] : 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < R::PASSES; ++p) top = abs_bits_max<T>(x[p], top);
  top = __reduce_max_sync(0xffffffffu, abs_bits_f32<T>(top));
  const float scale = new_scale<FMT>(top, old);
  const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
  if (m.s0 > 0 && scale > old) rescale_codes<FMT>(tile, m.s0 * (D / 4), lane, 32, old, inv);
  __syncwarp();                                 // every lane has read the old scale
  if (lane == 0) a.scales[half] = scale;
#pragma unroll
  for (int p = 0; p < R::PASSES; ++p) {
    const int s = p * R::RPP + rr;
    if (s >= m.s0 && s < m.s1) store_codes<T, FMT>(tile + s * D + li * R::EPL, x[p], inv);
  }
  // (most blocks of a long chunk lie before the window)
  if (a.ring && (m.col * ODA_TILE < a.sink || (m.col + 1ll) * ODA_TILE > (long long)m.t - a.window)) {
    T* ring = ring_chunk<T, D>(a, l, m.b, g, li);
#pragma unroll
    for (int p = 0; p < R::PASSES; ++p) {
      const int s = p * R::RPP + rr;
      if (s >= m.s0 && s < m.s1)
        store_ring<T, D>(a, ring, m.col * ODA_TILE + s, m.t, kv, x[p]);
    }
  }
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kThreads, (D * sizeof(T) <= 256 ? 1024 : 768) / kThreads) read_kv8_kernel(const Kv8Args a) {
  using R = Rows<T, D>;
  constexpr int U = kReadUnits, NW = R::EPL / 4;
  pdl_wait();
  pdl_launch_dependents();
  const unsigned w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const unsigned it = w / a.groups;
  const int unit0 = (int)(w - it * a.groups) * U, units = 2 * a.hkv;
  if (it >= a.items) return;
  Item m;
  if (!find_item(a, it, m)) return;
  const long long blk = find_block(a, m.b, m.col);
  if (blk < 0) return;
  const int l = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int rr = lane / R::LPR, li = lane % R::LPR;
  const long long half = ((long long)(a.lb + l) * a.num_blocks + blk) * units + unit0;
  const uint8_t* tile = a.codes + half * (ODA_TILE * D) + li * R::EPL;
  uint32_t c[U][R::PASSES][NW];
  float scale[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool there = unit0 + u < units;
    scale[u] = there ? a.scales[half + u] : 0.f;
#pragma unroll
    for (int p = 0; p < R::PASSES; ++p) {
      const int s = p * R::RPP + rr;
      // (what is not wanted reads a wanted slot again: no branch between the loads)
      const uint8_t* src = tile + ((there ? u : 0) * ODA_TILE + (s >= m.s0 && s < m.s1 ? s : m.s0)) * D;
      if (NW == 2) {
        const uint2 v = load_stream(reinterpret_cast<const uint2*>(src));
        c[u][p][0] = v.x;
        c[u][p][NW - 1] = v.y;
      } else {
        c[u][p][0] = load_stream(reinterpret_cast<const uint32_t*>(src));
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int unit = unit0 + u, kv = unit & 1, g = unit >> 1;
    T* out = static_cast<T*>(kv ? a.v_out : a.k_out);
    if (!out || unit >= units) continue;
    out += (((long long)l * a.n_tokens + m.tok) * a.hkv + g) * D + li * R::EPL;
#pragma unroll
    for (int p = 0; p < R::PASSES; ++p) {
      const int s = p * R::RPP + rr;
      if (s < m.s0 || s >= m.s1) continue;
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const float4 f = codes_to_f32<FMT>(c[u][p][i]);
        const float y[4] = {__fmul_rn(f.x, scale[u]), __fmul_rn(f.y, scale[u]), __fmul_rn(f.z, scale[u]),
                            __fmul_rn(f.w, scale[u])};
        if (sizeof(T) == 2) {
          const __nv_bfloat162 e = __floats2bfloat162_rn(y[0], y[1]), h = __floats2bfloat162_rn(y[2], y[3]);
          r[2 * i] = *reinterpret_cast<const uint32_t*>(&e);
          r[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) r[k] = __float_as_uint(y[k]);
        }
      }
      __stcs(reinterpret_cast<uint4*>(out + (long long)(s - m.s0) * a.hkv * D),
             make_uint4(r[0], r[1], r[2], r[3]));
    }
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
  Kv8Args* a;
  bool append;
  int layers;
  cudaStream_t st;
  template <typename T, int D, int FMT>
  oda_status operator()() {
    const bool one = append && !a->tok_start;
    const int units = 2 * a->hkv;
    const long long items = a->tok_start ? a->n_tokens / ODA_TILE + 2ll * a->B : a->B;
    const long long groups = append ? units : ceil_div64(units, kReadUnits);
    const long long lanes = items * groups * (one ? Rows<T, D>::LPR : 32);
    const long long grid = ceil_div64(lanes, kThreads);
    if (grid >= (1ll << 31) || items * groups >= (1ll << 32) - kThreads || layers > 65535)
      return ODA_ERR_SHAPE;
    a->items = (unsigned)items;
    a->groups = (unsigned)groups;
    auto k = one ? append_one_kv8_kernel<T, D, FMT>
                 : append ? append_kv8_kernel<T, D, FMT> : read_kv8_kernel<T, D, FMT>;
    return launch_pdl(k, dim3((unsigned)grid, (unsigned)layers), dim3(kThreads), 0, st, *a) == cudaSuccess
               ? ODA_OK
               : ODA_ERR_CUDA;
  }
};

oda_status launch(oda_ctx* ctx, bool append, int format, int lb, int le, Kv8Args& a, int B,
                  long long n_tokens, cudaStream_t st) {
  const oda_config& c = ctx->cfg;
  a.n_tokens = n_tokens;
  a.num_blocks = c.num_blocks;
  a.ring_layer_elems = ctx->lay.ring_layer_elems;
  a.max_blocks = c.max_blocks_per_seq;
  a.B = B;
  a.hkv = c.hkv;
  a.lb = lb;
  a.sink = c.sink;
  a.window = c.window;
  a.ring_blocks = (int)ctx->lay.ring_blocks;
  a.err = ctx->err;
  return dispatch(c, format, Launch{&a, append, le - lb, st});
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
