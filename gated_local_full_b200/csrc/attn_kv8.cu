// Decode attention of the listed rows over a paged cache held in 8 bits.
//
// For a row with query heads h of KV head g, over its positions j (all, or
// one region):
//   s_j = (q_h . kcode_j) * kscale_blk / sqrt(d),
//   o_h = sum_j softmax_j(s) vscale_blk vcode_j,  lse_h = log sum_j exp(s_j).
// The scales stay outside the products: a block's 16 tokens share them, so
// kscale multiplies 16 scores and vscale 16 weights, never a code.
//
// Arithmetic, one 16-token block (tile) at a time and one warp per tile, with
// the tokens as the products' 16 rows (scores) or depth (values):
//   * Scores, e4m3: the codes become f16, exactly, and mma.sync m16n8k16 sums in
//     float32. A power of two per head puts the query's largest element into
//     [1, 2); an element is then one f16 number and a second, 2^11 times what is left, in
//     columns of their own: within 2^-22 of itself, or 2^-36 of the largest (bfloat16: exact
//     down to 2^-28 of the largest).
//   * Scores, int8: the codes go into mma.sync m16n8k32 as they are, so the query
//     is written in whole numbers: a power of two per head makes its largest
//     element 2^29 .. 2^30, and four balanced digits to the base 256 are four
//     columns. The sums are exact; 2^-30 of the largest element is lost.
//     (For e4m3 that instruction's e4m3 form measured 20 cycles, the two f16 products 16.)
//   * The softmax weight times the value's scale, w_j = 2^(s_j - m) R with R =
//     vscale 2^(m - M + 11), is split into an f16 part and 2^11 times the rest, in two
//     columns with accumulators of their own; the codes of V become f16. So w_j is within
//     2^-22 of itself or, more than 2^25 below the reference, 2^-47 of that: a block far above the
//     others in one dim leaves the others' shares of the rest. (With the rest unscaled it was 2^-36,
//     and a block 2^40 above lost all else.) M is a reference for
//     s_j + log2 vscale (what the value accumulators are relative to), kept apart
//     from the reference m of s_j (what the sum l is relative to): a block with
//     a tiny scale then cannot push another block's weights out of f16. Both are
//     maxima when they are set, and set anew once a weight exceeds 16 times its
//     reference, so most tiles need neither a maximum over lanes nor a rescaling.
//   * A lane (g = lane / 4, tg = lane % 4) holds scores of one head and of the
//     two tokens in rows g and g + 8; its columns of the second product are that
//     head's, so references, sums and accumulators never leave their lane. The
//     weights reach the second product's layout by an 8 x 8 transposition.
// Fragments come straight from 16-byte loads:
//   * K (first operand): chunks tg and tg + 4 (d = 128) of the lane's two tokens.
//   * V (first operand, 16 dims x 16 tokens): D / 8 dims of tokens 4 tg .. 4 tg + 3,
//     the tokens in rows 2 tg, 2 tg + 1, 2 tg + 8, 2 tg + 9. The eight lanes that
//     shared memory serves together read four tokens, four rows apart, at the
//     same 32 bytes of their rows: V's second half is a copy of its own, 64
//     bytes further than it would be, so that no more than two lanes meet in a
//     bank. (Tiles in one copy, two and four, the last with no two lanes in a
//     bank: 8 rows of 16K tokens 49.2, 48.2 and 50.8 us, the mixed batch 188, 187
//     and 195: the copy engine's time against shared memory's.)
//
// Bound by HBM for long rows (one of 128K tokens, 8 KV heads, d = 128: 49.6 us
// for 269 MB, 5.4 TB/s with the start and the merge; 15 rows of 4K to 64K: 187 us,
// 6.2 TB/s), by latency for short ones (two rows of 64: 4.0 us).
#define ODA_PLAN_ROLLED

#include "kv8.cuh"
#include "plan.cuh"
#include "tiles.cuh"

using namespace oda;

namespace {

constexpr int W = 6;                     // warps per CTA
constexpr int kCopies = 2;               // copies of a tile, a lane each (above)
constexpr int kRows = 16 / kCopies;      // rows of V of each
constexpr int kSkew = 128 / kCopies;     // bytes that each lies further than it would
constexpr int kBatch = 16 / kCopies;     // pairs of tiles of a warp looked up together
constexpr int kAhead = 16;               // tiles of a CTA put into L2 before the dependency wait
constexpr float kNone = -3.402823466e38f;  // a reference before any token: no finite score is below
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

__device__ __forceinline__ void mma16832(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transposed 8 x 8 matrix of 16-bit elements, two of a row in each lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 8 bytes from global to shared memory whose arrival counts on a barrier.
__device__ __forceinline__ void cp_async8_arrive(uint32_t dst, const void* src, uint32_t bar) {
  asm volatile(
      "cp.async.ca.shared.global [%0], [%1], 8;\n\t"
      "cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%2];" ::"r"(dst), "l"(src), "r"(bar)
      : "memory");
}

// The whole warp waits for a barrier's phase; false: it gave up.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kWaitLimitNs));
}
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_long(bar, parity);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// V of a lane's four tokens; p: its place in the stage.
template <int D>
__device__ __forceinline__ void load_v(uint32_t (&v)[4][D / 32], const unsigned char* p, uint32_t mask,
                                       int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (D == 128) {
      const uint4 x = *reinterpret_cast<const uint4*>(p + j * D);
      v[j][0] = x.x; v[j][1] = x.y; v[j][2] = x.z; v[j][3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(p + j * D);
      v[j][0] = x.x; v[j][1] = x.y;
    }
  }
  if (mask != 0xffffu) {
    // a slot outside may hold anything: a weight of 0 must not meet a NaN
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (!((mask >> (4 * (lane & 3) + j)) & 1u)) {
#pragma unroll
        for (int x = 0; x < D / 32; ++x) v[j][x] = 0u;
      }
  }
}

// 16 elements of a query head, as they lie in memory, in float32.
template <typename T>
__device__ __forceinline__ void widen16(const uint4* r, float* x) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      bf16x2_to_f32(r[i].x, x[8 * i], x[8 * i + 1]);
      bf16x2_to_f32(r[i].y, x[8 * i + 2], x[8 * i + 3]);
      bf16x2_to_f32(r[i].z, x[8 * i + 4], x[8 * i + 5]);
      bf16x2_to_f32(r[i].w, x[8 * i + 6], x[8 * i + 7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = __uint_as_float(r[i].x); x[4 * i + 1] = __uint_as_float(r[i].y);
      x[4 * i + 2] = __uint_as_float(r[i].z); x[4 * i + 3] = __uint_as_float(r[i].w);
    }
  }
}

template <int D>
struct Tile {
  static constexpr int KC = D / 64;      // chunks of K per lane and column
  static constexpr int VW = D / 32;      // 32-bit words of V per token and lane
  static constexpr int MT = D / 16;      // 16-dim slices of the output
  static constexpr int VG = kRows * D + kSkew;  // V's pitch of a copy's rows in a stage
  static constexpr int BYTES = 2 * ODA_TILE * D;               // in the cache
  static constexpr int STAGE = ODA_TILE * D + kCopies * VG;    // in shared memory
};

constexpr float kLift = 11.f;            // weights are at most 2^15 < 65504
constexpr float kUnlift = 0x1p-11f;

// The head of a lane's scores: of up to two a segment, or (wide) of up to four.
__device__ __forceinline__ int head_of(int tg, bool wide) { return (tg >> 1) + (wide ? 2 * (tg & 1) : 0); }

// A warp's running state for one segment (row, KV head).
template <typename T, int D, int FMT, bool WIDE>
struct State {
  static constexpr int KC = Tile<D>::KC;
  static constexpr int SETS = WIDE ? 2 : 1;   // int8: of digit columns, two heads each
  // second operand of the scores: products (int8: of two words, a set for two
  // heads; e4m3: of one word)
  uint32_t qf[FMT == kInt8 ? 2 * KC * SETS : 4 * KC][2];
  float qs;                              // this lane's head: what its sums count for, times the scores' scale
  float m, M, l, K;                      // K = 2^(m - M + kLift), infinite past float32 or while M is kNone
  float acc[Tile<D>::MT][4];             // [0] + [1] 2^-11: one dim of this lane's head, [2] + [3] 2^-11: the next

  __device__ __forceinline__ void reset() {
    m = M = kNone;
    l = 0.f;
    K = INFINITY;
#pragma unroll
    for (int i = 0; i < Tile<D>::MT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;
  }

  // The elements that this lane's columns need, asked for before they are wanted.
  struct Query {
    static constexpr int SETS = FMT == kInt8 ? State::SETS : 1;
    uint4 r[SETS][KC][sizeof(T)];
    // q: the G query heads of the segment, [G][D]
    __device__ __forceinline__ void fetch(const T* q, int G, int lane) {
      const int g = lane >> 2, tg = lane & 3;
#pragma unroll
      for (int set = 0; set < SETS; ++set) {
        const int h = FMT == kInt8 ? 2 * set + (g >> 2) : head_of(g >> 1, WIDE);
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int i = 0; i < (int)sizeof(T); ++i) {
            r[set][c][i] = make_uint4(0, 0, 0, 0);
            if (h < G) r[set][c][i] = reinterpret_cast<const uint4*>(q + h * D + (tg + 4 * c) * 16)[i];
          }
      }
    }
  };

  // A head's elements of this lane's chunks over a power of two, 2^e <= largest < 2^(e+1), times
  // 2^lift; returns 2^e.
  __device__ __forceinline__ float scale_head(const uint4 (&r)[KC][sizeof(T)], int lift, float (&x)[KC][16]) {
    uint32_t top = 0;                    // |x| as bits: a NaN counts as the largest
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      widen16<T>(r[c], x[c]);
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[c][i]) & 0x7fffffffu);
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // (a query below 2^-97 counts from there; what is not finite makes every score NaN)
    const int e = min(max((int)(top >> 23) - 127, -97), 127);
    const float down = lift - e < -126 ? 0x1p-127f : __uint_as_float((uint32_t)(127 + lift - e) << 23);
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[c][i] *= down;
    return top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 + e) << 23);
  }

  __device__ __forceinline__ void set_q(const Query& q, int G, float qscale, int lane) {
    const int g = lane >> 2, tg = lane & 3;
    float x[KC][16];
    if constexpr (FMT == kInt8) {        // column g: digit g % 4 of head g / 4, and of head 2 + g / 4
#pragma unroll
      for (int set = 0; set < SETS; ++set) {
        const float up = scale_head(q.r[set], 29, x);
        // y = d0 + 256 d1 + 256^2 d2 + 256^3 d3, each within -128 .. 127: digit k is byte k of
        // y plus half of what the digits below it can hold
        const int k = g & 3;
        const int carry = (int)(0x00808080u & ((1u << (8 * k)) - 1u));
        const uint32_t two = 0x40u + 0x11u * k;              // byte k of each of two words
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = (uint32_t)(__float2int_rn(x[c][4 * w + i]) + carry);
            qf[2 * KC * set + 2 * c + w / 2][w & 1] =
                __byte_perm(__byte_perm(y[0], y[1], two), __byte_perm(y[2], y[3], two), 0x5410);
          }
        // scores of the set's head tg / 2 come from the columns of g = 4 (tg / 2) ..
        const float mine = __shfl_sync(0xffffffffu, up, (tg >> 1) * 16);
        if (set == 0 || (tg & 1)) qs = qscale * 0x1p-29f * mine;
      }
    } else {                             // columns 2 t, 2 t + 1: the head of lanes tg = t, and its rest
      const float up = scale_head(q.r[0], 0, x);
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float y0 = x[c][4 * w + 2 * i], y1 = x[c][4 * w + 2 * i + 1];
            if (g & 1) {
              y0 = (y0 - __half2float(__float2half_rn(y0))) * 0x1p11f;
              y1 = (y1 - __half2float(__float2half_rn(y1))) * 0x1p11f;
            }
            qf[4 * c + w][i] = pack_f16(y0, y1);
          }
      qs = qscale * __shfl_sync(0xffffffffu, up, tg * 8);
    }
  }

  // The scores of this lane's head with the tokens in rows g and g + 8, before the block's scale.
  // (p_k: this lane's place in the stage's K)
  __device__ __forceinline__ void scores(float (&s)[2], const unsigned char* p_k, int tg) const {
    uint32_t k[2][KC][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint4 x = *reinterpret_cast<const uint4*>(p_k + 2 * i * D + 64 * c);
        k[i][c][0] = x.x; k[i][c][1] = x.y; k[i][c][2] = x.z; k[i][c][3] = x.w;
      }
    if constexpr (FMT == kInt8) {
      // |sum| <= 2^21: the accumulators start at the bits of 1.5 * 2^23, and are floats as they stand
      const float f = tg & 1 ? 65536.f : 1.f;
      float v[SETS][2];
#pragma unroll
      for (int set = 0; set < SETS; ++set) {
        int c[4] = {0x4b400000, 0x4b400000, 0x4b400000, 0x4b400000};
#pragma unroll
        for (int p = 0; p < 2 * KC; ++p)
          mma16832(c, k[0][p / 2][p % 2 * 2], k[1][p / 2][p % 2 * 2], k[0][p / 2][p % 2 * 2 + 1],
                   k[1][p / 2][p % 2 * 2 + 1], qf[2 * KC * set + p][0], qf[2 * KC * set + p][1]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          v[set][i] = f * fmaf(__int_as_float(c[2 * i + 1]) - 0x1.8p23f, 256.f,
                               __int_as_float(c[2 * i]) - 0x1.8p23f);
      }
      // the other two digits are the neighbour's
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float keep = v[0][i], send = v[0][i];
        if (WIDE) {
          if (tg & 1) keep = v[SETS - 1][i]; else send = v[SETS - 1][i];
        }
        s[i] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
      }
    } else {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < 4 * KC; ++p) {
        uint32_t a0, a1, a2, a3;
        Fmt8<FMT>::to_f16(k[0][p / 4][p % 4], a0, a2);
        Fmt8<FMT>::to_f16(k[1][p / 4][p % 4], a1, a3);
        mma16816(c, a0, a1, a2, a3, qf[p][0], qf[p][1]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        s[i] = fmaf(c[2 * i + 1], 0x1p-11f, c[2 * i]);
    }
  }

  // Two tiles' weights, as the second operand of the values' product; mask: which
  // of a tile's 16 tokens take part.
  __device__ __forceinline__ void weights(const float (&raw)[2][2], const uint32_t (&mask)[2],
                                          const float2 (&scale)[2], uint32_t (&b)[2][2], int g) {
    float s[2][2], e[2][2], w[2][2], R[2];
    const bool whole = (mask[0] & mask[1]) == 0xffffu;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float sc = qs * scale[t].x;
#pragma unroll
      for (int i = 0; i < 2; ++i) s[t][i] = raw[t][i] * sc;
      R[t] = scale[t].y == 0.f ? 0.f : scale[t].y * K;
    }
    if (!whole) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t mine = mask[t] >> (4 * (g >> 1) + (g & 1));
        if (!(mine & 1u)) s[t][0] = -INFINITY;
        if (!(mine & 4u)) s[t][1] = -INFINITY;
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        e[t][i] = fast_exp2(s[t][i] - m);
        w[t][i] = e[t][i] * R[t];
      }
    const bool anew = fmaxf(fmaxf(e[0][0], e[0][1]), fmaxf(e[1][0], e[1][1])) > 16.f ||
                      fmaxf(fmaxf(w[0][0], w[0][1]), fmaxf(w[1][0], w[1][1])) > 32768.f ||
                      fmaxf(R[0], R[1]) > 0x1p100f;
    if (__any_sync(0xffffffffu, anew)) {
      float lv[2], top[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        lv[t] = fast_log2(scale[t].y);
        top[t] = fmaxf(s[t][0], s[t][1]);
        top[t] = fmaxf(top[t], __shfl_xor_sync(0xffffffffu, top[t], 4));
        top[t] = fmaxf(top[t], __shfl_xor_sync(0xffffffffu, top[t], 8));
        top[t] = fmaxf(top[t], __shfl_xor_sync(0xffffffffu, top[t], 16));
      }
      const float m_new = fmaxf(m, fmaxf(top[0], top[1]));
      const float M_new = fmaxf(M, fmaxf(top[0] + lv[0], top[1] + lv[1]));
      const float alpha = fast_exp2(M - M_new);
#pragma unroll
      for (int i = 0; i < Tile<D>::MT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][c] *= alpha;
      l *= fast_exp2(m - m_new);
      m = m_new;
      M = M_new;
      // (infinite where it leaves float32, since only blocks of zeros reach m: the exact way each time)
      K = M == kNone || m - M + kLift > 126.f ? INFINITY : fast_exp2(fmaxf(m - M + kLift, -126.f));
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          e[t][i] = fast_exp2(s[t][i] - m);
          w[t][i] = fast_exp2(s[t][i] + (lv[t] - M + kLift));      // R may be out of range
        }
    }
    l += (e[0][0] + e[0][1]) + (e[1][0] + e[1][1]);
    // row g: this lane's two columns are the weight's f16 part and 2^11 times its rest
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        b[t][i] = transpose8x8(pack_f16(w[t][i], (w[t][i] - __half2float(__float2half_rn(w[t][i]))) * 0x1p11f));
  }

  __device__ __forceinline__ void values(const uint32_t (&v)[4][Tile<D>::VW], const uint32_t (&b)[2]) {
#pragma unroll
    for (int x = 0; x < Tile<D>::VW; ++x) {
      // bytes of tokens 0 and 1 (2 and 3) of this lane side by side, per dim
      const uint32_t p = __byte_perm(v[0][x], v[1][x], 0x5140);
      const uint32_t q2 = __byte_perm(v[0][x], v[1][x], 0x7362);
      const uint32_t r = __byte_perm(v[2][x], v[3][x], 0x5140);
      const uint32_t u = __byte_perm(v[2][x], v[3][x], 0x7362);
      uint32_t a0, a1, a2, a3;
      Fmt8<FMT>::to_f16(p, a0, a1);
      Fmt8<FMT>::to_f16(r, a2, a3);
      mma16816(acc[2 * x], a0, a1, a2, a3, b[0], b[1]);
      Fmt8<FMT>::to_f16(q2, a0, a1);
      Fmt8<FMT>::to_f16(u, a2, a3);
      mma16816(acc[2 * x + 1], a0, a1, a2, a3, b[0], b[1]);
    }
  }

  // This warp's (acc 2^-kLift, M, m, l) for every head: ws [G][D + 4].
  __device__ __forceinline__ void store(float* ws, int G, int lane) {
    const int g = lane >> 2, tg = lane & 3;
    l += __shfl_xor_sync(0xffffffffu, l, 4);
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    const int h = head_of(tg, WIDE);
    if (h >= G || (!WIDE && (tg & 1))) return;
    float* w = ws + h * (D + 4);
#pragma unroll
    for (int i = 0; i < Tile<D>::MT; ++i) {
      w[g * (D / 8) + 2 * i] = fmaf(acc[i][1], kUnlift * 0x1p-11f, acc[i][0] * kUnlift);
      w[g * (D / 8) + 2 * i + 1] = fmaf(acc[i][3], kUnlift * 0x1p-11f, acc[i][2] * kUnlift);
    }
    if (g == 0) {
      w[D] = M;
      w[D + 1] = m;
      w[D + 2] = l;
    }
  }
};

// Shared memory of a launch, in order.
struct Smem {
  size_t wstate, full, meta, rows, total;
  // ns: stages of a pair of tiles per warp
  __host__ __device__ Smem(int G, int d, int max_batch, int ns) {
    const size_t state = (size_t)W * G * (d + 4) * 4, merge = (size_t)W * 32 * 6 * 4;
    size_t at = (size_t)W * ns * 2 * (d == 128 ? Tile<128>::STAGE : Tile<64>::STAGE);
    wstate = at;                                             // [W][G][d + 4], or the merge's
    at += state > merge ? state : merge;
    meta = at;                                               // [W][ns][2] Meta
    at += (size_t)W * ns * 2 * 16;
    full = at;                                               // [W][ns] barriers: a pair has landed
    at += (size_t)W * ns * 8;
    rows = at;                                               // 5 arrays by row slot
    at += (size_t)(5 * max_batch + 2) * 4;
    total = (at + 15) & ~(size_t)15;
  }
};

// What comes with a tile: its scales and which of its 16 tokens take part (0: none;
// its block is out of range, or the pair has one tile only).
struct __align__(16) Meta {
  float2 scale;
  uint32_t mask, unused;
};

// The last CTA of a segment puts its parts together. A thread takes four
// output elements and every SPLIT-th part, U of them in one round trip.
template <typename T, int D>
__device__ __forceinline__ void merge_parts(const Attn8Args& a, float* sm, int b, int g, int pbase,
                                            int nparts) {
  // (13 saves a 128K row's 37 parts a round, 0.3 us, and costs shorter rows as much. At G = 4,
  // d = 128 `split` is 1: a region of 10K tokens beside shorter ones, cut into 53, takes 7 rounds.)
  constexpr int U = 8;
  const int tid = threadIdx.x, G = a.G;
  const int nch = G * D / 4;                                 // 16 .. 128 chunks
  const int split = W * 32 / nch;
  const int ch = tid % nch, part = tid / nch;
  const int h = ch * 4 / D;
  const float* pml = a.partials + (size_t)a.max_parts * G * D;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int j0 = part; part < split && j0 < nparts; j0 += U * split) {
    float2 ml[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // (past the last part the last one again, left out below: no branch between the loads)
      const int j = min(j0 + u * split, nparts - 1);
      ml[u] = __ldcg(reinterpret_cast<const float2*>(pml) + (long long)(pbase + j) * G + h);
      v[u] = __ldcg(reinterpret_cast<const float4*>(a.partials + (long long)(pbase + j) * G * D) + ch);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j0 + u * split >= nparts) ml[u].y = 0.f;
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
#pragma unroll 1
    for (int p = 1; p < split; ++p) mt = fmaxf(mt, sm[p * nch + ch]);
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
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

// A walk over a CTA's share [lo, hi): the segment at hand (row slot i, KV head g, its
// tiles [s1 - nt, s1) and those of them in the share, [x0, x1)), taken in pairs of
// tiles, the last of which may hold one; `before`: the pairs of earlier segments.
struct Walk {
  int i, g, nt, s1, x0, x1, before;
  __device__ __forceinline__ void start(const int* rowstart, int nr, int hkv, int lo, int hi) {
    Cursor c;
    locate(rowstart, nr, hkv, lo, c);
    i = c.i; g = c.g; nt = c.nt; s1 = c.s1;
    x0 = lo;
    x1 = min(s1, hi);
    before = 0;
  }
  __device__ __forceinline__ int pairs() const { return (x1 - x0 + 1) >> 1; }
  // on to the next segment (there is one: x1 < hi)
  __device__ __forceinline__ void next(const int* rowstart, int hkv, int hi) {
    before += pairs();
    do {
      if (++g == hkv) {
        g = 0;
        ++i;
        nt = (rowstart[i + 1] - rowstart[i]) / hkv;
      }
    } while (nt == 0);
    x0 = s1;
    s1 += nt;
    x1 = min(s1, hi);
  }
  // on to pair p, which is not before this segment; false: there is none
  __device__ __forceinline__ bool seek(const int* rowstart, int hkv, int hi, int p) {
#pragma unroll 1
    while (p - before >= pairs()) {
      if (x1 >= hi) return false;
      next(rowstart, hkv, hi);
    }
    return true;
  }
};

// The rows of a launch, worked out by one warp: the partition's head, and this
// CTA's share in sinfo: {rows, tiles, CTAs, aligned, lo, hi, pbase, nparts, part,
// pairs}, and the walk at its start.
__device__ __forceinline__ void partition(const Attn8Args& a, bool report, int* sinfo, Walk* walk, int* rowb,
                                          int* rowt, int* rowstart, int* rowcs, int* rowlo) {
  PlanIn p = {};
  p.B = a.B;
  p.count = a.count;
  p.idx = a.idx;
  p.seq_lens = a.seq_lens;
  p.hkv = a.hkv;
  p.max_blocks = a.max_blocks;
  p.min_tiles = 2 * W;                   // a pair for every warp
  p.slack = 6 * W;
  p.grid = (int)gridDim.x;
  p.err = a.err;
  p.report = report && blockIdx.x == 0;
  p.range_lo = a.range_lo;
  p.range_hi = a.range_hi;
  const PlanHead h = plan_rows(p, rowb, rowt, rowstart, rowcs, rowlo);
  if ((threadIdx.x & 31) == 0) {
    int o[5];
    plan_cta((int)blockIdx.x, h, rowstart, rowcs, a.hkv, o);
    sinfo[0] = h.nr; sinfo[1] = h.tot; sinfo[2] = h.P; sinfo[3] = h.al;
    for (int i = 0; i < 5; ++i) sinfo[4 + i] = o[i];
    if (h.nr > 0 && h.nr <= a.B && o[0] >= 0 && o[0] < o[1] && o[1] <= h.tot) {
      Walk w;
      w.start(rowstart, h.nr, a.hkv, o[0], o[1]);
      *walk = w;
#pragma unroll 1
      while (w.x1 < o[1]) w.next(rowstart, a.hkv, o[1]);
      sinfo[9] = w.before + w.pairs();
    }
  }
  __syncwarp();
}

// One warp: whether the lists still are those the partition was worked out from, and
// raise no error. One round trip, since it needs no value to ask for the next.
__device__ __forceinline__ bool same_lists(const Attn8Args& a, const int* sinfo, const int* rowb,
                                           const int* rowt, const int* rowlo) {
  const int nr = sinfo[0];
  bool same = load_list(a.count) == nr;
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < nr; i += 32) {
    const int b = rowb[i];
    const int id = load_list(a.idx + i), t = load_list(a.seq_lens + b);
    int first = 1, last = t;
    if (a.range_lo) {
      first = load_list(a.range_lo + b);
      last = load_list(a.range_hi + b) - 1;
    }
    same = same && id == b && t >= 1 && first == rowlo[i] && last == rowt[i] &&
           first >= 1 && last >= first && last <= t && (last - 1) / ODA_TILE < a.max_blocks;
  }
  return __all_sync(0xffffffffu, same);
}

// A persistent grid takes the tiles as plan.cuh divides them; a CTA's share
// may lie in one segment (row, KV head) or span several. Warp w takes the share's
// pairs of tiles w, w + W, ... and streams them through a.ns stages of shared memory
// with bulk copies, running ahead of its arithmetic across segments. Two tiles at
// a time are two independent chains of arithmetic: one alone left a warp waiting
// for its own results two cycles of three (128K tokens: 57 us with 8 warps of one
// tile at a time, 52 with 6 warps of two). What a copy needs is worked out for
// kBatch pairs at once, four lanes a pair, one for each of its copies; the block ids
// are looked up a batch ahead. (Tile by tile this cost as many instructions as
// the arithmetic.) Which tile a warp takes depends on the lists alone, so equal
// calls give equal bits. Loops that are not unrolled for their arrays are kept
// rolled: fetching instructions is a quarter of a warp's time (a row of 700
// tokens 9.7 -> 9.4 us, 32 rows of 1500 20.5 -> 20.1).
template <typename T, int D, int FMT, bool WIDE>
__global__ void __launch_bounds__(W * 32, 2) attn_kv8_kernel(const Attn8Args a) {
  constexpr int TILE = Tile<D>::BYTES, STAGE = Tile<D>::STAGE;
  extern __shared__ __align__(128) unsigned char smem[];
  const int G = a.G, ns = a.ns;
  const Smem lay(G, D, a.max_batch, ns);
  float* wstate = reinterpret_cast<float*>(smem + lay.wstate);
  int* rowstart = reinterpret_cast<int*>(smem + lay.rows);             // [max_batch + 1]
  int* rowcs = rowstart + a.max_batch + 1;                             // [max_batch + 1]
  int* rowb = rowcs + a.max_batch + 1;                                 // [max_batch] each
  int* rowt = rowb + a.max_batch;
  int* rowlo = rowt + a.max_batch;
  __shared__ int sinfo[10];
  __shared__ Walk swalk;
  __shared__ int slast;
  __shared__ int waited;                                     // the dependency wait is over
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t full = smem_addr(smem + lay.full) + 8 * warp * ns;
  if (lane < ns) mbar_init(full + 8 * lane, 4);              // the codes' bytes and the scales of two tiles
  fence_mbar_init();
  if (tid == 0) waited = 0;
  __syncthreads();
  if (warp == 0) {
    // Before the dependency wait: the partition from lists that the launch before may
    // still be writing (every value is checked before it is used as an index), and
    // this CTA's first tiles into L2. A prefetch reads no value, and after the wait
    // the lists are compared, so a stale guess costs only time.
    // (One loop for the guess and the partition proper: their code is large.)
#pragma unroll 1
    for (int pass = a.early ? 1 : 0; pass < 2; ++pass) {
      if (pass == 1 && !a.early) {
        pdl_wait();
        pdl_launch_dependents();
        if (same_lists(a, sinfo, rowb, rowt, rowlo)) break;
      }
      partition(a, pass == 1, sinfo, &swalk, rowb, rowt, rowstart, rowcs, rowlo);
      const int k = sinfo[4] + lane;
      // (a CTA that started late, the wait already over, leaves the prefetch out)
      if (pass == 0 && !*const_cast<volatile int*>(&waited) && sinfo[0] > 0 && k < sinfo[5] && lane < kAhead) {
        Cursor c;
        locate(rowstart, sinfo[0], a.hkv, k, c);
        const int col = (rowlo[c.i] - 1) / ODA_TILE + k - (c.s1 - c.nt);
        const int blk = col < a.max_blocks ? load_list(a.block_table + (long long)rowb[c.i] * a.max_blocks + col) : -1;
        if (blk >= 0 && (long long)blk < a.num_blocks) {
          const long long th = (long long)blk * a.hkv + c.g;
          bulk_prefetch_l2(a.codes + th * TILE, TILE);
          asm volatile("prefetch.global.L2 [%0];" ::"l"(a.scales + th * 2));
        }
      }
      __syncwarp();
    }
  } else if (!a.early) {
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 32) *const_cast<volatile int*>(&waited) = 1;
  }
  __syncthreads();
  const int nr = sinfo[0], total = sinfo[1], P = sinfo[2], aligned = sinfo[3];
  const int lo = sinfo[4], hi = sinfo[5];
  if (!(nr > 0 && total > 0 && lo < hi)) {
    if (a.early) {
      pdl_wait();
      pdl_launch_dependents();
    }
    return;
  }

  // ---- copies
  const int tile = (lane / kCopies) & 1, piece = lane % kCopies;   // this lane's copy of its pair
  const uint64_t policy = l2_policy_evict_first();           // K/V is read once a launch
  const unsigned char* stages = smem + (uint32_t)(warp * ns * 2 * STAGE);
  Meta* meta = reinterpret_cast<Meta*>(smem + lay.meta) + warp * ns * 2;
  const uint32_t to = smem_addr(stages) + tile * STAGE + (piece ? ODA_TILE * D + piece * Tile<D>::VG : 0);
  const uint32_t from = piece ? ODA_TILE * D + piece * kRows * D : 0;
  const uint32_t bytes = (piece ? kRows : ODA_TILE + kRows) * D;   // the first: K too
  Walk at;
  int pair = warp + W * (lane / (2 * kCopies)), blk = -1, jt = 0;       // of the next batch
  bool there;
  auto lookup = [&]() {
    there = at.seek(rowstart, a.hkv, hi, pair);
    const int k = at.x0 + 2 * (pair - at.before) + tile;
    there = there && k < at.x1;
    jt = k - (at.s1 - at.nt);
    if (there)
      blk = a.block_table[(long long)rowb[at.i] * a.max_blocks + (rowlo[at.i] - 1) / ODA_TILE + jt];
  };
  at = swalk;
  const int count = (sinfo[9] - warp + W - 1) / W;           // this warp's pairs
  Walk seg = swalk;
  const int hq = a.hkv * G;
  typename State<T, D, FMT, WIDE>::Query query;
  auto fetch = [&]() {
    query.fetch(static_cast<const T*>(a.q) + ((long long)rowb[seg.i] * hq + seg.g * G) * D, G, lane);
  };
  if (!a.early) fetch();                                     // before the lookup: it is wanted no later
  lookup();
  const uint8_t* src = nullptr;                              // of this batch
  const float* ssrc = nullptr;
  uint32_t mask = 0;
  int issued = 0, islot = 0;
  auto issue = [&]() {
    if (issued % kBatch == 0) {
      mask = 0;
      if (there) {
        const int first = rowlo[at.i], last = rowt[at.i];
        const int base = (first - 1) / ODA_TILE * ODA_TILE;
        const bool bad = blk < 0 || (long long)blk >= a.num_blocks;
        const long long th = (long long)blk * a.hkv + at.g;
        src = a.codes + th * TILE + from;
        ssrc = a.scales + th * 2;
        mask = bad ? 0u : range_bits(first - 1 - base, last - base, jt * ODA_TILE);
        if (bad) record_error(a.err, ODA_ERR_BOUNDS);
      }
      pair += W * kBatch;
      lookup();
    }
    if (lane / (2 * kCopies) == issued % kBatch) {
      const uint32_t bar = full + 8 * islot;
      if (piece == 0) {
        Meta& mt = meta[2 * islot + tile];
        mt.mask = mask;
        if (mask) {
          mbar_arrive_expect_tx(bar, TILE);
          cp_async8_arrive(smem_addr(&mt.scale), ssrc, bar);
        } else {
          mt.scale = make_float2(0.f, 0.f);
          mbar_arrive(bar);
          mbar_arrive(bar);
        }
      }
      if (mask) bulk_g2s(to + islot * 2 * STAGE, src, bytes, bar, policy);
    }
    ++issued;
    islot = islot + 1 == ns ? 0 : islot + 1;
  };
#pragma unroll 1
  while (issued < ns && issued < count) issue();
  if (a.early) {
    pdl_wait();
    pdl_launch_dependents();
    fetch();
  }

  // ---- segments of this CTA's share
  float* pacc = a.partials;
  float* pml = a.partials + (size_t)a.max_parts * G * D;
  const int lg = lane >> 2, tg = lane & 3;
  const uint32_t k_at = (4 * (lg >> 1) + (lg & 1)) * D + tg * 16;
  const uint32_t v_at = ODA_TILE * D + tg * 4 * D + tg * 4 / kRows * kSkew + lg * (D / 8);
  int slot = 0, used = 0;
  uint32_t parity = 0;
  bool aborted = false;
#pragma unroll 1
  while (true) {
    const int b = rowb[seg.i], g = seg.g, s0 = seg.s1 - seg.nt, s1 = seg.s1;
    State<T, D, FMT, WIDE> st;
    st.reset();
    st.set_q(query, G, a.qscale, lane);
#pragma unroll 1
    for (const int end = seg.before + seg.pairs(); used * W + warp < end; ++used) {
      if (aborted || !wait_phase(full + 8 * slot, parity)) {
        if (!aborted && lane == 0) record_error(a.err, ODA_ERR_TIMEOUT);
        aborted = true;
        break;
      }
      const Meta ma = meta[2 * slot], mb = meta[2 * slot + 1];
      const unsigned char* stage = stages + (uint32_t)(slot * 2 * STAGE);
      const uint32_t masks[2] = {ma.mask, mb.mask};
      const float2 scales[2] = {ma.scale, mb.scale};
      float raw[2][2];
      uint32_t w[2][2], v[2][4][Tile<D>::VW];
      st.scores(raw[0], stage + k_at, tg);
      st.scores(raw[1], stage + STAGE + k_at, tg);
      load_v<D>(v[0], stage + v_at, masks[0], lane);
      load_v<D>(v[1], stage + STAGE + v_at, masks[1], lane);
      __syncwarp();                                          // every lane has its share
      if (++slot == ns) {
        slot = 0;
        parity ^= 1u;
      }
      if (issued < count) issue();
      st.weights(raw, masks, scales, w, lg);
      st.values(v[0], w[0]);
      st.values(v[1], w[1]);
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
    if (tid < G * D / 4) {
      const int h = tid * 4 / D, dd = tid * 4 % D;
      const float* ws = wstate + h * (D + 4);
      float4 tail[W];                                        // M, m, l of a warp
      float mt = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        tail[w] = *reinterpret_cast<const float4*>(ws + w * G * (D + 4) + D);
        mt = fmaxf(mt, tail[w].y);
      }
      float lt = 0.f;
      float4 at4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(ws + w * G * (D + 4) + dd);
        if (tail[w].z == 0.f) continue;                      // no token (a NaN is not left out)
        lt += tail[w].z * fast_exp2(tail[w].y - mt);
        // M = kNone: 0, or the NaN of a NaN scale. (M may lie further below mt than float32 reaches: in
        // two halves what counts is the product.)
        const float f = fast_exp2(0.5f * (tail[w].x - mt));
        at4.x += x.x * f * f; at4.y += x.y * f * f; at4.z += x.z * f * f; at4.w += x.w * f * f;
      }
      if (nparts == 1) {
        const float inv = lt != 0.f ? 1.f / lt : 0.f;
        const long long head = (long long)b * hq + g * G + h;
        T* o = static_cast<T*>(a.out) + head * D + dd;
        o[0] = (T)(at4.x * inv); o[1] = (T)(at4.y * inv); o[2] = (T)(at4.z * inv); o[3] = (T)(at4.w * inv);
        if (dd == 0 && a.lse)
          a.lse[head] = lt != 0.f ? (mt + fast_log2(lt)) * 0.69314718055994531f : -INFINITY;
      } else {
        const long long px = (long long)mypart * G + h;
        *reinterpret_cast<float4*>(pacc + px * D + dd) = at4;
        if (dd == 0) *reinterpret_cast<float2*>(pml + px * 2) = make_float2(mt, lt);
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
    if (s1 >= hi) break;
    __syncthreads();
    seg.next(rowstart, a.hkv, hi);
    fetch();
  }
  // never leave a copy landing in shared memory after exit: after a timeout
  // those still flying are waited for once more, within the limit
  if (aborted) {
#pragma unroll 1
    for (; used < issued; ++used) {
      if (!wait_phase(full + 8 * slot, parity)) break;
      if (++slot == ns) {
        slot = 0;
        parity ^= 1u;
      }
    }
  }
}

// Stages per warp: two where two CTAs of them fit an SM beside the row arrays
// of a large batch, else one. (32 heads over 8, d = 128, contexts for 52 rows and for 53: 8 rows
// of 16K 43.4 and 44.7 us in e4m3, 46.9 and 47.3 in int8, 15 rows of 4K to 64K 142 and 134.)
int stages_for(const oda_config& c) {
  const int G = c.hq / c.hkv;
  return Smem(G, c.head_dim, c.max_batch, 2).total <= 113 * 1024 - 128 ? 2 : 1;
}

size_t smem_bytes(const oda_config& c) {
  return Smem(c.hq / c.hkv, c.head_dim, c.max_batch, stages_for(c)).total;
}

template <typename F>
oda_status dispatch(const oda_config& c, int format, F&& f) {
  const bool wide = c.hq / c.hkv > 2;
#define ODA_CASE(TT, DT, DD, FF)                                                   \
  if (c.dtype == DT && c.head_dim == DD && format == FF)                           \
    return wide ? f.template operator()<TT, DD, FF, true>() : f.template operator()<TT, DD, FF, false>();
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
  template <typename T, int D, int FMT, bool WIDE>
  oda_status operator()() {
    const void* k = reinterpret_cast<const void*>(attn_kv8_kernel<T, D, FMT, WIDE>);
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
  template <typename T, int D, int FMT, bool WIDE>
  oda_status operator()() {
    return launch_pdl(attn_kv8_kernel<T, D, FMT, WIDE>, dim3(ctx->attn_kv8_ctas), dim3(W * 32),
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
