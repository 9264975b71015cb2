// Decode attention of the listed rows over a paged cache held in 8 bits.
//
// For a row with query heads h of KV head g, over its positions j (all, or
// one region):
//   s_j = (q_h . kcode_j) * kscale_blk / sqrt(d),
//   o_h = sum_j softmax_j(s) vscale_blk vcode_j,  lse_h = log sum_j exp(s_j).
// The scales stay outside the products: a block's 16 tokens share them, so
// kscale multiplies 16 scores and vscale 16 weights, never a code.
//
// Arithmetic. The codes (int8 or e4m3) are exact in f16, so both contractions
// run as mma.sync m16n8k16 with f16 inputs and float32 sums, one 16-token block
// (tile) at a time and one warp per tile:
//   * q is brought into f16 exactly: a power of two per head puts its largest
//     element into [1, 2) (an element below 2^-17 of that may lose its last
//     bits, 2^-25 of the largest). A float32 q is split into two f16 parts.
//   * the softmax weight w_j = 2^(s_j + log2 vscale - M + 14) is split into an
//     f16 part and the f16 rest, 22 bits in all: columns 0-3 of the second
//     product take the first parts of the (up to four) heads, columns 4-7 the
//     rests. M is the running maximum of s_j + log2 vscale (what the value
//     accumulators are relative to), kept apart from the maximum m of s_j (what
//     the sum l is relative to): a block with a tiny scale then cannot push
//     another block's weights out of f16.
// Fragments come straight from 16-byte loads, with no transposition:
//   * K (second operand, 16 dims x 8 columns): lane (n = lane / 4, tg = lane % 4)
//     takes 16-byte chunk lane % 8 of row lane / 8. With d = 128 the two
//     columns 2r, 2r+1 are the two halves of row r; rows 0-7 of the query
//     operand hold the heads' first 64 dims and rows 8-15 the last 64, and a
//     score is the sum of two accumulators of one lane. With d = 64 a 128-byte
//     line holds two tokens, one per column.
//   * V (first operand, 16 dims x 16 tokens): lane (g, tg) takes dims 16 g .. of
//     its four tokens; token and dim orders are free as long as the weights
//     and the output use the same ones.
//   * the score accumulators of a lane are the weights it needs in the second
//     product: probabilities never leave their lane.
#include "kv8.cuh"
#include "plan.cuh"
#include "tiles.cuh"

using namespace oda;

namespace {

constexpr int W = 8;                     // warps per CTA
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per barrier wait

struct Attn8Args {
  const void* q;
  void* out;
  float* lse;
  const int32_t* seq_lens;
  const uint8_t* codes;                  // layer base
  const float* scales;                   // layer base
  const int32_t* block_table;
  const int32_t* idx;
  const int32_t* count;
  const int32_t* range_lo;
  const int32_t* range_hi;
  long long num_blocks;
  int max_blocks, B, hkv, G, max_batch, ns;
  int early;                             // stage the first tiles before the dependency wait
  float qscale;                          // log2(e) / sqrt(d)
  float* partials;                       // [max_parts][G][d], then [max_parts][G][2]
  int max_parts;
  int* tickets;
  int* err;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 bytes from global to shared memory whose arrival counts on a barrier.
__device__ __forceinline__ void cp_async8_arrive(uint32_t dst, const void* src, uint32_t bar) {
  asm volatile(
      "cp.async.ca.shared.global [%0], [%1], 8;\n\t"
      "cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%2];" ::"r"(dst), "l"(src), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }

// A lane's share of one tile: NI chunks of K, and four tokens' V.
template <int D>
struct Tile {
  static constexpr int NI = D / 32;      // K loads (lines of 128 bytes: 16 or 8 a tile)
  static constexpr int VW = D / 32;      // 32-bit words of V per token and lane
  static constexpr int MT = D / 16;      // 16-dim slices of the output
  uint32_t k[NI][4];
  uint32_t v[4][VW];
};

// The token (slot of the tile) of a lane's j-th score.
template <int D>
__device__ __forceinline__ int token_of(int tg, int j) {
  return D == 128 ? tg + 4 * j : 2 * tg + (j & 1) + 8 * (j >> 1);
}

template <int D>
__device__ __forceinline__ void load_tile(Tile<D>& t, const uint8_t* tile, int lane) {
#pragma unroll
  for (int i = 0; i < Tile<D>::NI; ++i) {
    const uint4 x = *reinterpret_cast<const uint4*>(tile + i * 512 + lane * 16);
    t.k[i][0] = x.x; t.k[i][1] = x.y; t.k[i][2] = x.z; t.k[i][3] = x.w;
  }
  const uint8_t* v = tile + ODA_TILE * D + (lane >> 2) * (D / 8);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint8_t* p = v + token_of<D>(lane & 3, j) * D;
    if (D == 128) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      t.v[j][0] = x.x; t.v[j][1] = x.y; t.v[j][2 % Tile<D>::VW] = x.z; t.v[j][3 % Tile<D>::VW] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      t.v[j][0] = x.x; t.v[j][1] = x.y;
    }
  }
}

// A warp's running state for one segment (row, KV head). Lane (g, tg): head
// g % 4 for the statistics; of the accumulators, D / 8 dims of columns 2 tg, 2 tg + 1.
template <typename T, int D, int FMT>
struct State {
  uint32_t qf[4][4];                     // query operand: 4 slices of 16 dims a chunk
  float qs;                              // score scale of this lane's head
  float m, M, l;
  float acc[Tile<D>::MT][4];

  __device__ __forceinline__ void reset() {
    m = M = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < Tile<D>::MT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;
  }

  // q: the G query heads of the segment, [G][D]
  __device__ __forceinline__ void load_q(const T* q, int G, float qscale, int lane) {
    const int g = lane >> 2, tg = lane & 3, h = g & 3;
    constexpr int HALVES = D / 64;
    float x[HALVES][16];
    float top = 0.f;
#pragma unroll
    for (int p = 0; p < HALVES; ++p)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[p][e] = h < G ? to_f32<T>(q[h * D + p * 64 + tg * 16 + e]) : 0.f;
        top = fmaxf(top, fabsf(x[p][e]));
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^e <= top < 2^(e+1); no power for zeros and for what is not finite
    int e = (int)((__float_as_uint(top) >> 23) & 255u) - 127;
    e = e == 128 ? 0 : max(e, -100);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    qs = qscale * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int p = 0; p < HALVES; ++p)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float y = x[p][i] * down;
        // rows 4-7 repeat the heads; for a float32 query they hold the rest
        if (sizeof(T) == 4 && g >= 4) y -= __half2float(__float2half_rn(y));
        x[p][i] = y;
      }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      qf[s][0] = pack_f16(x[0][4 * s], x[0][4 * s + 1]);
      qf[s][2] = pack_f16(x[0][4 * s + 2], x[0][4 * s + 3]);
      qf[s][1] = HALVES == 2 ? pack_f16(x[HALVES - 1][4 * s], x[HALVES - 1][4 * s + 1]) : 0u;
      qf[s][3] = HALVES == 2 ? pack_f16(x[HALVES - 1][4 * s + 2], x[HALVES - 1][4 * s + 3]) : 0u;
    }
  }

  // One tile; `mask`: which of its 16 tokens take part (at least one).
  __device__ __forceinline__ void tile(Tile<D>& t, uint32_t mask, float kscale, float vscale,
                                       int lane) {
    const int g = lane >> 2, tg = lane & 3;
    float s[4];
#pragma unroll
    for (int i = 0; i < Tile<D>::NI; ++i) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t b0, b1;
        Fmt8<FMT>::to_f16(t.k[i][w], b0, b1);
        mma16816(c, qf[w][0], qf[w][1], qf[w][2], qf[w][3], b0, b1);
      }
      if (D == 128) {
        s[i] = c[0] + c[3];
      } else {
        s[2 * (i & 1)] = c[0];
        s[2 * (i & 1) + 1] = c[1];
      }
    }
    if (sizeof(T) == 4) {                // the two parts of a float32 query
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], 16);
    }
    const float sc = qs * kscale;
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] *= sc;
    if (mask != 0xffffu) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!((mask >> token_of<D>(tg, j)) & 1u)) {
          s[j] = -INFINITY;
          // a slot outside may hold anything: a weight of 0 must not meet a NaN
#pragma unroll
          for (int w = 0; w < Tile<D>::VW; ++w) t.v[j][w] = 0u;
        }
    }
    float top = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float lv = fast_log2(vscale);
    const float m_new = fmaxf(m, top), M_new = fmaxf(M, top + lv);
    const float ms = m_new == -INFINITY ? 0.f : m_new;
    const float Ms = M_new == -INFINITY ? 0.f : M_new;
    if (__any_sync(0xffffffffu, M_new > M)) {
      const float alpha = fast_exp2(M - Ms);              // M = -inf: 0
      const float a0 = __shfl_sync(0xffffffffu, alpha, ((2 * tg) & 3) * 4);
      const float a1 = __shfl_sync(0xffffffffu, alpha, ((2 * tg + 1) & 3) * 4);
#pragma unroll
      for (int i = 0; i < Tile<D>::MT; ++i) {
        acc[i][0] *= a0; acc[i][1] *= a1;
        acc[i][2] *= a0; acc[i][3] *= a1;
      }
    }
    l *= fast_exp2(m - ms);
    m = m_new;
    M = M_new;
    float w[4];
    const float shift = lv - Ms + 14.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      l += fast_exp2(s[j] - ms);
      w[j] = fast_exp2(s[j] + shift);
    }
    // columns 0-3: the weights' f16 parts; 4-7: the rests
    uint32_t b0 = pack_f16(w[0], w[1]), b1 = pack_f16(w[2], w[3]);
    if (g >= 4) {
      const float2 h0 = __half22float2(*reinterpret_cast<__half2*>(&b0));
      const float2 h1 = __half22float2(*reinterpret_cast<__half2*>(&b1));
      b0 = pack_f16(w[0] - h0.x, w[1] - h0.y);
      b1 = pack_f16(w[2] - h1.x, w[3] - h1.y);
    }
#pragma unroll
    for (int x = 0; x < Tile<D>::VW; ++x) {
      // bytes of tokens 0 and 1 (2 and 3) of this lane side by side, per dim
      const uint32_t p = __byte_perm(t.v[0][x], t.v[1][x], 0x5140);
      const uint32_t q2 = __byte_perm(t.v[0][x], t.v[1][x], 0x7362);
      const uint32_t r = __byte_perm(t.v[2][x], t.v[3][x], 0x5140);
      const uint32_t u = __byte_perm(t.v[2][x], t.v[3][x], 0x7362);
      uint32_t a0, a1, a2, a3;
      Fmt8<FMT>::to_f16(p, a0, a1);
      Fmt8<FMT>::to_f16(r, a2, a3);
      mma16816(acc[2 * x], a0, a1, a2, a3, b0, b1);
      Fmt8<FMT>::to_f16(q2, a0, a1);
      Fmt8<FMT>::to_f16(u, a2, a3);
      mma16816(acc[2 * x + 1], a0, a1, a2, a3, b0, b1);
    }
  }

  // This warp's (acc, M, m, l) for every head: ws [G][D + 4].
  __device__ __forceinline__ void store(float* ws, int G, int lane) {
    const int g = lane >> 2, tg = lane & 3;
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
#pragma unroll
    for (int i = 0; i < Tile<D>::MT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float x = acc[i][c] + __shfl_xor_sync(0xffffffffu, acc[i][c], 2);
        const int h = 2 * tg + (c & 1);
        if (tg < 2 && h < G) ws[h * (D + 4) + g * (D / 8) + 2 * i + (c >> 1)] = x;
      }
    if (tg == 0 && g < G) {
      ws[g * (D + 4) + D] = M;
      ws[g * (D + 4) + D + 1] = m;
      ws[g * (D + 4) + D + 2] = l;
    }
  }
};

// Shared memory of a launch, in order.
struct Smem {
  size_t wstate, rows, bars, scale, tile, bad, total;
  __host__ __device__ Smem(int G, int d, int max_batch, int ns) {
    const size_t state = (size_t)W * G * (d + 4) * 4, merge = (size_t)W * 32 * 6 * 4;
    size_t at = (size_t)W * ns * 2 * ODA_TILE * d;           // stages
    wstate = at;                                             // [W][G][d + 4], or the merge's
    at += state > merge ? state : merge;
    bars = at;                                               // [W][ns]
    at += (size_t)W * ns * 8;
    scale = at;                                              // [W][ns] float2
    at += (size_t)W * ns * 8;
    tile = at;                                               // [W][ns] tile of each stage
    at += (size_t)W * ns * 4;
    bad = at;                                                // [W][ns] its block is out of range
    at += (size_t)W * ns * 4;
    rows = at;                                               // 5 arrays by row slot
    at += (size_t)(5 * max_batch + 2) * 4;
    total = (at + 15) & ~(size_t)15;
  }
};

// The last CTA of a segment puts its parts together. A thread takes four
// output elements and every SPLIT-th part, U of them in one round trip.
template <typename T, int D>
__device__ __forceinline__ void merge_parts(const Attn8Args& a, float* sm, int b, int g, int pbase,
                                            int nparts) {
  constexpr int U = 10;
  const int tid = threadIdx.x, G = a.G;
  const int nch = G * D / 4;                                 // 16 .. 128 chunks
  const int split = W * 32 / nch;
  const int ch = tid % nch, part = tid / nch;
  const int h = ch * 4 / D;
  const float* pml = a.partials + (size_t)a.max_parts * G * D;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = part; j0 < nparts; j0 += U * split) {
    float2 ml[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * split;
      ml[u] = make_float2(-INFINITY, 0.f);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < nparts) {
        ml[u] = __ldcg(reinterpret_cast<const float2*>(pml) + (long long)(pbase + j) * G + h);
        v[u] = __ldcg(reinterpret_cast<const float4*>(a.partials + (long long)(pbase + j) * G * D) + ch);
      }
    }
    float mt = m;
#pragma unroll
    for (int u = 0; u < U; ++u) mt = fmaxf(mt, ml[u].x);
    if (l != 0.f) {
      const float f = fast_exp2(m - mt);
      l *= f; acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (ml[u].y == 0.f) continue;                          // no token (a NaN is not left out)
      const float f = fast_exp2(ml[u].x - mt);
      l = fmaf(ml[u].y, f, l);
      acc.x = fmaf(v[u].x, f, acc.x); acc.y = fmaf(v[u].y, f, acc.y);
      acc.z = fmaf(v[u].z, f, acc.z); acc.w = fmaf(v[u].w, f, acc.w);
    }
    m = mt;
  }
  // the threads of one chunk, through shared memory: [6][W * 32]
  float* s = sm + tid;
  s[0] = m; s[W * 32] = l;
  s[2 * W * 32] = acc.x; s[3 * W * 32] = acc.y; s[4 * W * 32] = acc.z; s[5 * W * 32] = acc.w;
  __syncthreads();
  if (part == 0) {
    float mt = m;
    for (int p = 1; p < split; ++p) mt = fmaxf(mt, sm[p * nch + ch]);
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = 0; p < split; ++p) {
      const float* x = sm + p * nch + ch;
      if (x[W * 32] == 0.f) continue;
      const float f = fast_exp2(x[0] - mt);
      l += x[W * 32] * f;
      acc.x += x[2 * W * 32] * f; acc.y += x[3 * W * 32] * f;
      acc.z += x[4 * W * 32] * f; acc.w += x[5 * W * 32] * f;
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const long long head = (long long)b * a.hkv * G + g * G + h;
    T* o = static_cast<T*>(a.out) + head * D + ch * 4 % D;
    o[0] = (T)(acc.x * inv); o[1] = (T)(acc.y * inv); o[2] = (T)(acc.z * inv); o[3] = (T)(acc.w * inv);
    if (ch * 4 % D == 0 && a.lse)
      a.lse[head] = l != 0.f ? (mt + fast_log2(l)) * 0.69314718055994531f : -INFINITY;
  }
}

// A persistent grid takes the tiles as plan.cuh divides them; a CTA's share
// may lie in one segment (row, KV head) or span several. Each warp streams
// its own tiles, every W-th of the share, through a.ns stages of shared memory
// with bulk copies, and runs ahead of its arithmetic across segments.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(W * 32, 2) attn_kv8_kernel(const Attn8Args a) {
  constexpr int TILE = 2 * ODA_TILE * D;
  extern __shared__ __align__(128) unsigned char smem[];
  const int G = a.G, ns = a.ns;
  const Smem lay(G, D, a.max_batch, ns);
  float* wstate = reinterpret_cast<float*>(smem + lay.wstate);
  int* rowstart = reinterpret_cast<int*>(smem + lay.rows);             // [max_batch + 1]
  int* rowcs = rowstart + a.max_batch + 1;                             // [max_batch + 1]
  int* rowb = rowcs + a.max_batch + 1;                                 // [max_batch] each
  int* rowt = rowb + a.max_batch;
  int* rowlo = rowt + a.max_batch;
  __shared__ int sinfo[9];
  __shared__ int slast;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* stages = smem + (size_t)warp * ns * TILE;
  const uint32_t bars = smem_addr(smem + lay.bars + (size_t)warp * ns * 8);
  float2* sscale = reinterpret_cast<float2*>(smem + lay.scale) + warp * ns;
  int* stile = reinterpret_cast<int*>(smem + lay.tile) + warp * ns;
  int* sbad = reinterpret_cast<int*>(smem + lay.bad) + warp * ns;
  if (lane < ns) mbar_init(bars + 8 * lane, 2);    // the codes' bytes, the scales
  fence_mbar_init();
  if (!a.early) {
    pdl_wait();
    pdl_launch_dependents();
  }
  if (warp == 0) {
    PlanIn p = {};
    p.B = a.B;
    p.count = a.count;
    p.idx = a.idx;
    p.seq_lens = a.seq_lens;
    p.hkv = a.hkv;
    p.max_blocks = a.max_blocks;
    p.min_tiles = W;
    p.grid = (int)gridDim.x;
    p.err = a.err;
    p.report = blockIdx.x == 0;
    p.range_lo = a.range_lo;
    p.range_hi = a.range_hi;
    const PlanHead h = plan_rows(p, rowb, rowt, rowstart, rowcs, rowlo);
    if (lane == 0) {
      int o[5];
      plan_cta((int)blockIdx.x, h, rowstart, rowcs, a.hkv, o);
      sinfo[0] = h.nr; sinfo[1] = h.tot; sinfo[2] = h.P; sinfo[3] = h.al;
      for (int i = 0; i < 5; ++i) sinfo[4 + i] = o[i];
    }
  }
  __syncthreads();
  const int nr = sinfo[0], total = sinfo[1], P = sinfo[2], aligned = sinfo[3];
  const int lo = sinfo[4], hi = sinfo[5];
  const bool work = nr > 0 && total > 0 && lo < hi;
  if (!work) {
    if (a.early) {
      pdl_wait();
      pdl_launch_dependents();
    }
    return;
  }
  const uint64_t policy = l2_policy_evict_first();           // K/V is read once a launch

  // ---- producer: the tiles of this warp, in order
  Cursor prod;
  prod.k = lo;
  locate(rowstart, nr, a.hkv, lo, prod);
  prod.k = min(lo + warp, hi);
  normalize(rowstart, a.hkv, hi, warp, prod);
  int bc_row = -1, bc_base = 0, bc_val = -1;                 // blocks of its next 32 tiles, one a lane
  int pstage = 0, cstage = 0, flying = 0;
  uint32_t parity = 0;
  auto issue = [&]() {                                       // the next tile into stage pstage
    const int jt = prod.k - (rowstart[prod.i] + prod.g * prod.nt);
    if (prod.i != bc_row || jt < bc_base || jt >= bc_base + 32 * W || (jt - bc_base) % W != 0) {
      bc_row = prod.i;
      bc_base = jt;
      const int jl = jt + lane * W;
      bc_val = jl < prod.nt ? a.block_table[(long long)rowb[prod.i] * a.max_blocks +
                                            (rowlo[prod.i] - 1) / ODA_TILE + jl]
                            : -1;
    }
    const int blk = __shfl_sync(0xffffffffu, bc_val, (jt - bc_base) / W);
    if (lane == 0) {
      const uint32_t bar = bars + 8 * pstage;
      const bool bad = blk < 0 || (long long)blk >= a.num_blocks;
      stile[pstage] = prod.k;
      sbad[pstage] = bad;
      if (bad) {
        record_error(a.err, ODA_ERR_BOUNDS);
        mbar_arrive(bar);
        mbar_arrive(bar);
      } else {
        const long long th = (long long)blk * a.hkv + prod.g;
        mbar_arrive_expect_tx(bar, TILE);
        bulk_g2s(smem_addr(stages + (size_t)pstage * TILE), a.codes + th * TILE, TILE, bar, policy);
        cp_async8_arrive(smem_addr(sscale + pstage), a.scales + th * 2, bar);
      }
    }
    pstage = pstage + 1 == ns ? 0 : pstage + 1;
    ++flying;
    prod.k += W;
    normalize(rowstart, a.hkv, hi, warp, prod);
  };
  for (int s = 0; s < ns && prod.k < hi; ++s) issue();
  if (a.early) {
    pdl_wait();
    pdl_launch_dependents();
  }
  float* pacc = a.partials;
  float* pml = a.partials + (size_t)a.max_parts * G * D;
  const int hq = a.hkv * G;
  bool aborted = false;
  __syncwarp();

  // ---- segments of this CTA's share
  Cursor seg;
  seg.k = lo;
  locate(rowstart, nr, a.hkv, lo, seg);
  while (true) {
    const int b = rowb[seg.i], g = seg.g;
    const int s0 = seg.s1 - seg.nt, s1 = seg.s1;
    const int first = rowlo[seg.i], last = rowt[seg.i];
    const int base = (first - 1) / ODA_TILE * ODA_TILE;
    const int plo = first - 1 - base, phi = last - base;
    State<T, D, FMT> st;
    st.reset();
    st.load_q(static_cast<const T*>(a.q) + ((long long)b * hq + g * G) * D, G, a.qscale, lane);
    while (flying > 0) {
      const int k = stile[cstage];
      if (k >= s1) break;                                    // of a later segment
      if (!aborted) {
        const bool ok = __all_sync(0xffffffffu,
                                   mbar_wait_bounded(bars + 8 * cstage, parity, kWaitLimitNs));
        if (!ok) {
          aborted = true;
          if (lane == 0) record_error(a.err, ODA_ERR_TIMEOUT);
        }
      }
      if (aborted) break;
      const float2 sc = sscale[cstage];
      const uint32_t mask = sbad[cstage] ? 0u : range_bits(plo, phi, (k - s0) * ODA_TILE);
      Tile<D> t;
      load_tile<D>(t, stages + (size_t)cstage * TILE, lane);
      __syncwarp();                                          // every lane has its share
      if (++cstage == ns) {
        cstage = 0;
        parity ^= 1u;
      }
      --flying;
      if (prod.k < hi) issue();
      if (mask) st.tile(t, mask, sc.x, sc.y, lane);
      __syncwarp();                                          // stile, sbad of the tile just issued
    }
    st.store(wstate + warp * G * (D + 4), G, lane);
    __syncthreads();
    const int sigma = seg.i * a.hkv + g;
    int pbase, nparts, mypart;
    if (aligned) {
      pbase = sinfo[6];
      nparts = sinfo[7];
      mypart = pbase + sinfo[8];
    } else {
      const int c_first = (int)(((long long)(s0 + 1) * P - 1) / total);
      const int c_last = (int)(((long long)s1 * P - 1) / total);
      pbase = c_first + sigma;
      nparts = c_last - c_first + 1;
      mypart = (int)blockIdx.x + sigma;
    }
    for (int o = tid; o < G * D; o += W * 32) {
      const int h = o / D, dd = o % D;
      float mt = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) mt = fmaxf(mt, wstate[(w * G + h) * (D + 4) + D + 1]);
      float lt = 0.f, at = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float* ws = wstate + (w * G + h) * (D + 4);
        if (ws[D + 2] == 0.f) continue;                // no token (a NaN is not left out)
        lt += ws[D + 2] * fast_exp2(ws[D + 1] - mt);
        at += ws[dd] * fast_exp2(ws[D] - 14.f - mt);   // M = -inf: 0, or the NaN of a NaN scale
      }
      if (nparts == 1) {
        static_cast<T*>(a.out)[((long long)b * hq + g * G + h) * D + dd] =
            (T)(lt != 0.f ? at / lt : 0.f);
        if (dd == 0 && a.lse)
          a.lse[(long long)b * hq + g * G + h] =
              lt != 0.f ? (mt + fast_log2(lt)) * 0.69314718055994531f : -INFINITY;
      } else {
        const long long px = (long long)mypart * G + h;
        pacc[px * D + dd] = at;
        if (dd == 0) { pml[px * 2] = mt; pml[px * 2 + 1] = lt; }
      }
    }
    if (nparts > 1) {
      __syncthreads();
      if (tid == 0) slast = ticket_add(&a.tickets[sigma], 1) == nparts - 1;
      __syncthreads();
      if (slast) {
        merge_parts<T, D>(a, wstate, b, g, pbase, nparts);
        if (tid == 0) a.tickets[sigma] = 0;
      }
    }
    __syncthreads();
    if (s1 >= hi) break;
    // the next segment with tiles
    do {
      if (++seg.g == a.hkv) {
        seg.g = 0;
        ++seg.i;
        seg.nt = (rowstart[seg.i + 1] - rowstart[seg.i]) / a.hkv;
      }
    } while (seg.nt == 0);
    seg.s1 = s1 + seg.nt;
  }
  // never leave a copy landing in shared memory after exit (after a timeout
  // the copies still flying are waited for once more, within the limit)
  while (flying > 0) {
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(bars + 8 * cstage, parity, kWaitLimitNs))) break;
    if (++cstage == ns) {
      cstage = 0;
      parity ^= 1u;
    }
    --flying;
  }
}

// Stages per warp: three where two CTAs of them fit an SM beside the row
// arrays of a large batch, else two.
int stages_for(const oda_config& c) {
  const int G = c.hq / c.hkv;
  return Smem(G, c.head_dim, c.max_batch, 3).total <= 112 * 1024 ? 3 : 2;
}

size_t smem_bytes(const oda_config& c) {
  return Smem(c.hq / c.hkv, c.head_dim, c.max_batch, stages_for(c)).total;
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

struct Setup {
  oda_ctx* ctx;
  int* ctas;
  template <typename T, int D, int FMT>
  oda_status operator()() {
    const void* k = reinterpret_cast<const void*>(attn_kv8_kernel<T, D, FMT>);
    const size_t sm = smem_bytes(ctx->cfg);
    ODA_CUDA_TRY(raise_smem_limit(k, sm));
    int occ = 0;
    ODA_CUDA_TRY(occupancy_cached(&occ, k, W * 32, sm));
    if (occ < 1) return ODA_ERR_SHAPE;
    *ctas = ctx->num_sms * occ;
    return ODA_OK;
  }
};

struct Launch {
  oda_ctx* ctx;
  const Attn8Args* a;
  cudaStream_t st;
  template <typename T, int D, int FMT>
  oda_status operator()() {
    return launch_pdl(attn_kv8_kernel<T, D, FMT>, dim3(ctx->attn_kv8_ctas), dim3(W * 32),
                      smem_bytes(ctx->cfg), st, *a) == cudaSuccess
               ? ODA_OK
               : ODA_ERR_CUDA;
  }
};

}  // namespace

namespace oda_impl {

// The grid fits both formats; the context's partials hold one per CTA and segment.
oda_status attn_kv8_setup(oda_ctx* ctx) {
  int x = 0, y = 0;
  oda_status s = dispatch(ctx->cfg, kInt8, Setup{ctx, &x});
  if (s == ODA_OK) s = dispatch(ctx->cfg, kE4m3, Setup{ctx, &y});
  ctx->attn_kv8_ctas = x < y ? x : y;
  return s;
}

oda_status launch_attn_kv8(oda_ctx* ctx, int format, int layer, const void* q,
                           const int32_t* seq_lens, const int32_t* range_lo,
                           const int32_t* range_hi, const int32_t* block_table, const void* codes,
                           const float* scales, const int32_t* idx, const int32_t* count, void* out,
                           float* lse, int B, bool early, cudaStream_t st) {
  const oda_config& c = ctx->cfg;
  Attn8Args a;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.seq_lens = seq_lens;
  a.codes = static_cast<const uint8_t*>(codes) + (size_t)layer * (size_t)ctx->lay.cache_layer_elems;
  a.scales = scales + (size_t)layer * (size_t)c.num_blocks * c.hkv * 2;
  a.block_table = block_table;
  a.idx = idx;
  a.count = count;
  a.range_lo = range_lo;
  a.range_hi = range_hi;
  a.num_blocks = c.num_blocks;
  a.max_blocks = c.max_blocks_per_seq;
  a.B = B;
  a.hkv = c.hkv;
  a.G = c.hq / c.hkv;
  a.max_batch = c.max_batch;
  a.ns = stages_for(c);
  a.early = early ? 1 : 0;
  a.qscale = 1.4426950408889634f / sqrtf((float)c.head_dim);
  a.partials = ctx->partials;
  a.max_parts = ctx->max_parts;
  a.tickets = ctx->tickets;
  a.err = ctx->err;
  return dispatch(c, format, Launch{ctx, &a, st});
}

}  // namespace oda_impl
