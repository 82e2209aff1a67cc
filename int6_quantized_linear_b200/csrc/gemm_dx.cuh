// gemm_dx.cuh -- the input gradient of a quantized layer on the 5th-generation tensor core.
//
//   dx[M][K] = dy[M][N] . W[N][K],  dy bf16 (or the gated block's (dg | du)), W quantized, dx bf16
//
// The contraction runs over the weight rows n, along which the packed codes are strided, so the weight
// tile is wanted transposed: D[128 k][tokens] += W^T[128 k][64 n] x dy^T, W^T the MMA's A operand in tensor memory
// (lane = k, two n a column) and dy, as it lies, its B operand in shared memory.  The transposition costs
// nothing: a matrix load with transposition (ldmatrix .trans on 16-bit elements) of eight rows' packed codes
// gives each thread 16 bits of codes of two neighbouring rows n, n + 1 side by side -- four nibbles, two bytes or
// eight 2-bit fields of consecutive k -- and each mask of that word is a pair (n, n + 1) of one k: a TMEM word.
// (A first form decoded along the rows and let the tensor core transpose an M-major A tile in shared memory: 821
// cycles a stage of 256 tokens, all of them shared-memory traffic -- its stores, the tensor core's reads of it and of
// dy -- against the MMAs' 512; without the tile it is about 580.)
//
// Operands are fp16 with exact power-of-two scales, as in the forward GEMM (gemm_prep.cuh).  A weight row's
// scale 2^b_n cannot be undone after a sum over rows, so its inverse goes into the other operand:
//     dx[m][k] = 2^-(a_m + w_top) sum_n (dy[m][n] 2^(a_m + w_top - b_n)) (w[n][k] 2^b_n),
// with a_m chosen so that the row's largest scaled magnitude lies in [2^14, 2^15).
//
// Codes become weights as in the gated GEMM (gated_chunk_to_f16): 4-, 2- and 8-bit codes shifted to the top of a half's
// mantissa are subnormals, and one fused multiply-add with the inverse power in the scale makes a weight below 1; int6
// goes through 1024 + f.  A column of dx depends on that column of W alone, so the range below a row's largest weight
// matters here: a group whose largest weight is 2^-13 of it has its weights to 2^-11 of that one, a smaller group one bit
// less a power of two (int6: 2^-28).  (A subtraction from 1024 + q as in the forward GEMM reaches 2^-28 for all; equal at
// M = 2048, but K = 5120, N = 27648, M = 4 took 45.1 us against 41.5.)
//
// Passes: (1) row exponents b_n; (2) dy to scaled fp16 rows; (3) the scaled group metadata, transposed so that a
// stage's words are one TMA box; (4) the GEMM; (5) the sum of the parts of split tiles.
//
// One or two CTAs an SM (ctas_per_sm).  The tiles of whole waves (as many tiles as CTAs, again and again) are computed
// alone, all CTAs moving along n together so that each code row and each dy column is fetched from memory about once
// a wave; the tiles of the last, partial wave are cut along n into equal shares, one a CTA, whose fp32 sums
// go to the workspace and are added in a fixed order (a full last wave costs as much as the others however
// few tiles it has: at M = 2048, K = 5120 it would be a third wave for 24 of 148 CTAs).
//
// Workspace (256-byte aligned sections, Np = N rounded up to 64):
//   dy16   fp16 [M][Np]      scaled dy, zeros past N
//   dexp   s32  [M]          -(a_m + w_top)
//   rowexp u8   [Np]         exponent byte of 2^(w_top - b_n), 0 for rows of zeros
//   meta   u32  [K / gran][Np]  scaled metadata of a run of gran weights, two words for each two rows n, n + 1
//                            of fp16 pairs: their scales, then their offsets (int4 -Z S, affine b; int6 the scales
//                            of the run's two 16-groups); zeros past N
//   partial f32 [2 DX_CTAS ctas_per_sm][tokens a tile][128]
#pragma once
#include "gated.cuh"
#include "gemm_sm100.cuh"

namespace ql {
namespace dx {

constexpr int BN = 64;    // weight rows a stage (the contraction)
constexpr int BKT = 128;  // k a tile (the MMA's M)
constexpr int DX_CTAS = 148;       // SMs a launch uses at most: those of a B200
constexpr int MIN_SHARE = 8;       // stages a share of a split tile has at least
// Token tiles: the class (most tokens of a tile, which sizes the rings) and the tokens that a launch's tiles
// have, a multiple of 16 (the MMA's N) that spreads M evenly.
constexpr int TT_LARGE = 256, TT_MEDIUM = 64, TT_SMALL = 32;
// CTAs an SM: a CTA's chain of copy, decoding, MMA and release takes more than 500 cycles a stage, and up to 64
// tokens the MMAs themselves take 230 to 250, so two CTAs share the tensor core (int4, K = 5120, N = 27648, M = 4: 40.4
// us a call against 47.7, M = 64: 45.5 against 54.4; int6, K = 4096, N = 8192, M = 12: 23.7 against 24.2; with tiles of
// 128 tokens one CTA was faster, 67.2 against 75.2 at M = 128).
__host__ __device__ constexpr int ctas_per_sm(int tt) { return tt == TT_LARGE ? 1 : 2; }
inline int tile_class(int64_t M) { return M <= TT_SMALL ? TT_SMALL : M <= TT_MEDIUM ? TT_MEDIUM : TT_LARGE; }
inline int tile_tokens(int64_t M) {
  const int c = tile_class(M);
  const int64_t tiles = (M + c - 1) / c;
  return (int)(((M + tiles - 1) / tiles + 15) / 16 * 16);
}
inline int64_t padded_n(int64_t N) { return (N + 63) / 64 * 64; }
// weights a metadata word covers
__host__ __device__ constexpr int gran(int fmt, int group) { return fmt == FMT_AFFINE ? group : 32; }

struct Workspace {
  __half *dy16;
  int *dexp;
  uint8_t *rowexp;
  uint32_t *meta;
  float *partial;
  int w_top;  // of the layer's format
};

inline size_t workspace_bytes(int64_t M, int64_t N, int64_t K, int g) {
  const size_t np = (size_t)padded_n(N);
  return align256((size_t)M * np * 2) + align256((size_t)M * 4) + align256(np) + align256((size_t)(K / g) * np * 4) +
         (size_t)2 * DX_CTAS * ctas_per_sm(tile_class(M)) * tile_tokens(M) * BKT * 4;
}

inline Workspace carve(void *base, int64_t M, int64_t N, int64_t K, int g, int w_top) {
  const size_t np = (size_t)padded_n(N);
  uint8_t *p = static_cast<uint8_t *>(base);
  Workspace w;
  w.dy16 = reinterpret_cast<__half *>(p);
  p += align256((size_t)M * np * 2);
  w.dexp = reinterpret_cast<int *>(p);
  p += align256((size_t)M * 4);
  w.rowexp = p;
  p += align256(np);
  w.meta = reinterpret_cast<uint32_t *>(p);
  p += align256((size_t)(K / g) * np * 4);
  w.partial = reinterpret_cast<float *>(p);
  w.w_top = w_top;
  return w;
}

// The passes are a chain of programmatic dependents.  Pass 1 waits for what precedes the call before it
// lets pass 2 start, and pass 2 for pass 1 before it lets pass 3 start, so passes 2 and 3 find the call's
// inputs and the row exponents complete; pass 3 waits for pass 2 before it ends, and the GEMM for pass 3.
// With few tokens pass 2 has few CTAs, and passes 2 and 3 run side by side.

// ---- pass 1: row exponents ------------------------------------------------------------------------
// b_n puts the bound on row n's weights that its group words give (as the forward kernels', see gemm_prep.cuh) into
// [2^w_top, 2 2^w_top).  The row factor 2^(w_top - b_n) that multiplies dy, the power of two at or below that bound, is
// kept as its exponent byte: a product of dy and it is out of range only where dx is.  A row of zeros has the factor 0,
// so that its dy does not count in a token's scale.
//
// 16 lanes a row, or 32 where the rows are few for the GPU and a row has a word for each lane (int4, M = 4: N = 5120,
// K = 27648 39.6 us a call against 43.7, N = 27648, K = 5120 41.5 against 40.5; the call took 37.5 with bounds from
// the steps alone, which a large step that no group uses makes useless).
constexpr int RE_THREADS = 256;
__host__ __device__ constexpr int w_top(int fmt) { return fmt == FMT_INT6 || fmt == FMT_INT6P ? 14 : -1; }
__host__ __device__ constexpr int64_t meta_words(int fmt, int64_t K, int G) { return fmt == FMT_AFFINE ? K / G : K / 256; }
inline int row_exp_lanes(int fmt, int64_t N, int64_t K, int G) {
  return N <= DX_CTAS * 64 && meta_words(fmt, K, G) >= 32 ? 32 : 16;
}
constexpr int WP_ROWS = 64, WP_RUNS = 64, WP_THREADS = 256;

// Byte i of a word in the mantissa of 2^23
QL_DEVI float byte_of(uint32_t w, int i) { return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7650 | i)); }

// Group words and step word of one super-block (int4, int6: 16 bytes of group words) or group (affine) of a row,
// and a bound on its weights.  Words of zeros have the bound 0.
template <int FMT>
struct MetaWords {
  uint4 g;
  uint32_t s;
};
template <>
struct MetaWords<FMT_AFFINE> {
  uint32_t g;
};
template <int FMT>
QL_DEVI MetaWords<FMT> load_meta_words(const uint8_t *gmeta, const uint8_t *steps, int64_t at) {
  if constexpr (FMT == FMT_AFFINE) return {__ldg(reinterpret_cast<const uint32_t *>(gmeta) + at)};
  else if constexpr (FMT == FMT_INT4)
    return {__ldg(reinterpret_cast<const uint4 *>(gmeta) + at), __ldg(reinterpret_cast<const uint32_t *>(steps) + at)};
  else
    return {__ldg(reinterpret_cast<const uint4 *>(gmeta) + at),
            (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(steps) + at)};
}
template <int FMT, int BITS>
QL_DEVI float meta_bound(const MetaWords<FMT> &m) {
  if constexpr (FMT == FMT_AFFINE) {
    const float s = bf16_bits_to_f32(m.g), b = bf16_bits_to_f32(m.g >> 16);
    return fmaxf(fabsf(b), fabsf(fmaf((float)((1 << BITS) - 1), s, b)));
  } else {
    const uint32_t w[4] = {m.g.x, m.g.y, m.g.z, m.g.w};
    if constexpr (FMT == FMT_INT4) {
      const float zs = f16_bits_to_f32(m.s >> 16), nzs = -8388608.f * zs;
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float Z = fmaf(byte_of(w[j >> 1], 2 * (j & 1) + 1), zs, nzs);
        top = fmaxf(top, (byte_of(w[j >> 1], 2 * (j & 1)) - 8388608.f) * fmaxf(fabsf(Z), fabsf(15.f - Z)));
      }
      return top * fabsf(f16_bits_to_f32(m.s));
    } else {
      uint32_t hi = 0x00800080u, lo = 0x00800080u;  // of the codes plus 128, two a word
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = w[j] ^ 0x80808080u, a = c & 0x00FF00FFu, b = (c >> 8) & 0x00FF00FFu;
        hi = __vmaxu2(hi, __vmaxu2(a, b));
        lo = __vminu2(lo, __vminu2(a, b));
      }
      const int top = max((int)max(hi & 0xFFFFu, hi >> 16) - 128, 128 - (int)min(lo & 0xFFFFu, lo >> 16));
      return 32.f * (float)top * fabsf(f16_bits_to_f32(m.s));
    }
  }
}

template <int FMT, int BITS, int LANES>
__global__ void __launch_bounds__(RE_THREADS) row_exp_kernel(const uint8_t *gmeta, const uint8_t *steps, int64_t N,
                                                             int64_t K, int G, Workspace ws) {
  const int sub = threadIdx.x % LANES;
  const int64_t n = (int64_t)blockIdx.x * (RE_THREADS / LANES) + threadIdx.x / LANES;  // < Np
  const int64_t words = n < N ? meta_words(FMT, K, G) : 0, first = n * words;
  pdl_wait();
  pdl_launch_dependents();
  float top = 0.f;
#pragma unroll 1
  for (int64_t i = sub; i < words; i += LANES)
    top = fmaxf(top, meta_bound<FMT, BITS>(load_meta_words<FMT>(gmeta, steps, first + i)));
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  // b in [-126, 120], so that it and 127 + w_top - b are exponents: rows below 2^-106 lie lower, and affine weights of
  // 2^126 and more are out of range
  constexpr int TOP = w_top(FMT);
  if (sub == 0) ws.rowexp[n] = (uint8_t)(top == 0.f ? 0 : 127 + TOP - min(scale_exponent(top, TOP), 120));
}

// ---- pass 2: dy (or (dg | du)) to scaled fp16 rows ----------------------------------------------------
// One CTA a token row; an element enters the product as v 2^(w_top - b_n) 2^a, the row's a from a bound on
// its scaled magnitudes.

// The exponent bytes of four rows -> their factors, i = 0..3
QL_DEVI float row_factor(uint32_t bytes, int i) { return __uint_as_float(__byte_perm(bytes, 0u, 0x0444 | (i << 12)) >> 1); }

// The largest value of every thread's v over the CTA.
template <int THREADS>
QL_DEVI float block_max(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) v = fmaxf(v, red[w]);
  return v;
}

// Eight bf16 of a row from element i on, those from `end` on as zeros.  VEC: the row's elements are 16-byte
// aligned at every multiple of 8, and end is one.
template <bool VEC>
QL_DEVI uint4 load8(const __nv_bfloat16 *row, int64_t i, int64_t end) {
  if constexpr (VEC) {
    return __ldg(reinterpret_cast<const uint4 *>(row + i));
  } else {
    uint32_t u[4] = {0u, 0u, 0u, 0u};
    const uint16_t *src = reinterpret_cast<const uint16_t *>(row);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < end) u[j >> 1] |= (uint32_t)src[i + j] << (16 * (j & 1));
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
}
QL_DEVI void unpack8(uint4 q, float (&v)[8]) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(u[j] << 16);
    v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
  }
}

constexpr int DY_REGS = 4;
// threads a row: with 256 rows of up to 8192 stay in registers, with 1024 rows of up to 32768
inline int dy_threads(int64_t N) { return N <= 8 * DY_REGS * 256 ? 256 : 1024; }

// Rows of up to DY_REGS vectors of 8 a thread are read once and kept; longer rows are read again.
template <int DY_THREADS, bool VEC>
__global__ void __launch_bounds__(DY_THREADS) dy_prep_kernel(const __nv_bfloat16 *dy, int64_t N, int64_t np,
                                                             Workspace ws) {
  __shared__ float red[DY_THREADS / 32];
  const int64_t m = blockIdx.x, nv = (N + 7) / 8;
  const __nv_bfloat16 *row = dy + m * N;
  const uint2 *fac = reinterpret_cast<const uint2 *>(ws.rowexp);
  uint4 *out = reinterpret_cast<uint4 *>(ws.dy16 + m * np);
  auto top8 = [](uint4 q, uint2 f, float t) {
    float v[8];
    unpack8(q, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) t = fmaxf(t, fabsf(v[j] * row_factor(j < 4 ? f.x : f.y, j & 3)));
    return t;
  };
  auto put8 = [](uint4 q, uint2 f, float sc) {
    float v[8];
    unpack8(q, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * row_factor(j < 4 ? f.x : f.y, j & 3) * sc;
    return make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
  };
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const bool kept = nv <= (int64_t)DY_REGS * DY_THREADS;
  uint4 q[DY_REGS];
  uint2 f[DY_REGS];
  float top = 0.f;
  if (kept) {
#pragma unroll
    for (int r = 0; r < DY_REGS; ++r) {
      const int64_t i = threadIdx.x + r * DY_THREADS;
      q[r] = i < nv ? load8<VEC>(row, 8 * i, N) : zero;
    }
  }
  pdl_wait();  // the row exponents
  pdl_launch_dependents();
  if (kept) {
#pragma unroll
    for (int r = 0; r < DY_REGS; ++r) {
      const int64_t i = threadIdx.x + r * DY_THREADS;
      f[r] = i < nv ? fac[i] : make_uint2(0u, 0u);
    }
#pragma unroll
    for (int r = 0; r < DY_REGS; ++r) top = top8(q[r], f[r], top);
  } else {
    for (int64_t i = threadIdx.x; i < nv; i += DY_THREADS) top = top8(load8<VEC>(row, 8 * i, N), fac[i], top);
  }
  const int a = scale_exponent(block_max<DY_THREADS>(top, red), 14);
  const float sc = exp2i(a);
  if (kept) {
#pragma unroll
    for (int r = 0; r < DY_REGS; ++r) {
      const int64_t i = threadIdx.x + r * DY_THREADS;
      if (i < nv) out[i] = put8(q[r], f[r], sc);
    }
  } else {
    for (int64_t i = threadIdx.x; i < nv; i += DY_THREADS) out[i] = put8(load8<VEC>(row, 8 * i, N), fac[i], sc);
  }
  if (threadIdx.x < np / 8 - nv) out[nv + threadIdx.x] = zero;
  if (threadIdx.x == 0) ws.dexp[m] = -(a + ws.w_top);
}

struct GatedGrad {
  const int8_t *codes;   // checkpoint of (g, u)
  const uint8_t *exps;
  const __nv_bfloat16 *dh;  // [M][F]
  __nv_bfloat16 *dgu;       // [M][2F] or NULL
  int64_t F, np;
};

constexpr float MAX_SLOPE = 1.13f;  // of the activations; |act(g)| <= |g|

// Eight exponent bytes of rows n .. n + 7 (bytes from `end` on as zeros).  VEC: n is a multiple of 8.
template <bool VEC>
QL_DEVI uint2 load_rowexp(const uint8_t *e, int64_t n, int64_t end) {
  if constexpr (VEC) {
    return *reinterpret_cast<const uint2 *>(e + n);
  } else {
    uint32_t u[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (n + j < end) u[j >> 2] |= (uint32_t)e[n + j] << (8 * (j & 3));
    return make_uint2(u[0], u[1]);
  }
}

QL_DEVI uint32_t max_byte(uint2 v) {
  uint32_t m = __vmaxu4(v.x, v.y);
  m = __vmaxu4(m, m >> 16);
  return max(m & 0xFFu, (m >> 8) & 0xFFu);
}

// Eight 16-bit values -> row elements n .. n + 7 (those below `end`).  VEC: 16-byte aligned, all of them.
template <bool VEC>
QL_DEVI void store8(void *row, int64_t n, int64_t end, const uint32_t (&o)[4]) {
  uint16_t *dst = static_cast<uint16_t *>(row) + n;
  if constexpr (VEC) {
    *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (n + j < end) dst[j] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
  }
}

// A thread takes eight features (half a group of the checkpoint) at a time.  The row's scale comes from a bound that
// needs no activation -- the eight's largest |dh| times 127 steps of u (slope at most 1.13) or of g -- so every
// gradient is computed once; the bound's slack costs a few of the 29 powers of two that fp16 has below its
// top.  The int8 codes become floats by a byte permute and a subtraction.  VEC: F % 8 == 0.
template <int ACT, bool VEC, int THREADS>
__global__ void __launch_bounds__(THREADS) dgu_prep_kernel(GatedGrad p, Workspace ws) {
  __shared__ float red[THREADS / 32];
  const int64_t m = blockIdx.x, N = 2 * p.F, fp = save8_cols(p.F);
  const int units = (int)((p.F + 7) / 8);
  const __nv_bfloat16 *dh = p.dh + m * p.F;
  const uint2 *cg = reinterpret_cast<const uint2 *>(p.codes + 2 * m * fp), *cu = cg + fp / 8;
  const uint8_t *eg = p.exps + 2 * m * (fp / 16), *eu = eg + fp / 16;
  float top = 0.f;
  pdl_wait();  // the row exponents
  pdl_launch_dependents();
#pragma unroll 2
  for (int i = threadIdx.x; i < units; i += THREADS) {
    const int64_t f = 8 * (int64_t)i;
    const float dm = chunk_amax(load8<VEC>(dh, f, p.F), 0.f) * 127.f;
    const uint2 rg = load_rowexp<VEC>(ws.rowexp, f, p.F), ru = load_rowexp<VEC>(ws.rowexp + p.F, f, p.F);
    const float sg = save8_scale(__ldg(eg + (i >> 1))), su = save8_scale(__ldg(eu + (i >> 1)));
    top = fmaxf(top, dm * su * (MAX_SLOPE * __uint_as_float(max_byte(rg) << 23)));
    top = fmaxf(top, dm * sg * __uint_as_float(max_byte(ru) << 23));
  }
  // (the bound may pass the largest float where no gradient does)
  const int a = scale_exponent(fminf(block_max<THREADS>(top, red), 3.402823466e38f), 14);
  const float sc = exp2i(a);
  __half *out = ws.dy16 + m * p.np;
#pragma unroll 1
  for (int i = threadIdx.x; i < units; i += THREADS) {
    const int64_t f = 8 * (int64_t)i;
    const uint4 d = load8<VEC>(dh, f, p.F);
    const uint2 qg = __ldg(cg + i), qu = __ldg(cu + i);
    const uint2 rg = load_rowexp<VEC>(ws.rowexp, f, p.F), ru = load_rowexp<VEC>(ws.rowexp + p.F, f, p.F);
    const float sg = save8_scale(__ldg(eg + (i >> 1))), su = save8_scale(__ldg(eu + (i >> 1)));
    const uint32_t dw[4] = {d.x, d.y, d.z, d.w};
    const uint32_t gw[2] = {qg.x ^ 0x80808080u, qg.y ^ 0x80808080u}, uw[2] = {qu.x ^ 0x80808080u, qu.y ^ 0x80808080u};
    const uint32_t fg[2] = {rg.x, rg.y}, fu[2] = {ru.x, ru.y};
    uint32_t og[4], ou[4], bg[4], bu[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float dgv[2], duv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e = 2 * j + h;
        const float dv = h ? __uint_as_float(dw[j] & 0xffff0000u) : __uint_as_float(dw[j] << 16);
        // code c as the byte c + 128 in the mantissa of 2^23 (one FMA with (2^23 + 128) s would overflow from s = 2^105)
        const float g = (byte_of(gw[e >> 2], e & 3) - 8388736.f) * sg;
        const float u = (byte_of(uw[e >> 2], e & 3) - 8388736.f) * su;
        float av, ad;
        act_grad(ACT, g, av, ad);
        dgv[h] = dv * u * ad;
        duv[h] = dv * av;
      }
      if (p.dgu) {
        bg[j] = pack_bf16x2(dgv[0], dgv[1]);
        bu[j] = pack_bf16x2(duv[0], duv[1]);
      }
      const int e = 2 * j;
      og[j] = pack_f16x2(dgv[0] * row_factor(fg[e >> 2], e & 3) * sc, dgv[1] * row_factor(fg[e >> 2], (e & 3) + 1) * sc);
      ou[j] = pack_f16x2(duv[0] * row_factor(fu[e >> 2], e & 3) * sc, duv[1] * row_factor(fu[e >> 2], (e & 3) + 1) * sc);
    }
    store8<VEC>(out, f, p.F, og);
    store8<VEC>(out + p.F, f, p.F, ou);
    if (p.dgu) {
      store8<VEC>(p.dgu + m * N, f, p.F, bg);
      store8<VEC>(p.dgu + m * N + p.F, f, p.F, bu);
    }
  }
  if (threadIdx.x < p.np - N) out[N + threadIdx.x] = __float2half_rn(0.f);
  if (threadIdx.x == 0) ws.dexp[m] = -(a + ws.w_top);
}

// ---- pass 3: scaled metadata, transposed ------------------------------------------------------------
// Two neighbouring runs' metadata (gran weights each; int4 and int6: of one super-block) from their group words --
// the two in w0 (int4, int6) or one each in w0 and w1 (affine) -- and their step word, for a row with sc = 2^b_n:
// the scales times sc and what undoes the codes' place in a half, 2^code_up; -Z S and b times sc.  The powers of two
// are exact, so they go into the steps first.  Byte codes become floats by a permute into the mantissa of 2^23 (a
// conversion unit has a quarter of the rate).
__host__ __device__ constexpr int code_up(int fmt, int bits) {  // int6's codes are whole numbers
  return fmt == FMT_INT6 || fmt == FMT_INT6P ? 0 : 14 + bits;
}
template <int FMT, int BITS>
QL_DEVI void scaled_meta(uint32_t w0, uint32_t w1, uint32_t s, float sc, uint32_t (&o)[2]) {
  constexpr float UP = (float)(1 << code_up(FMT, BITS));
  if constexpr (FMT == FMT_INT4) {
    const float ss = f16_bits_to_f32(s) * sc * UP, zs = f16_bits_to_f32(s >> 16) * (-1.f / UP);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float S = __fmul_rn(byte_of(w0, 2 * i) - 8388608.f, ss);
      o[i] = pack_f16x2(S, __fmul_rn(byte_of(w0, 2 * i + 1) - 8388608.f, zs) * S);
    }
  } else if constexpr (FMT == FMT_INT6 || FMT == FMT_INT6P) {
    const float st = f16_bits_to_f32(s) * sc;
    w0 ^= 0x80808080u;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      o[i] = pack_f16x2(__fmul_rn(byte_of(w0, 2 * i) - 8388736.f, st), __fmul_rn(byte_of(w0, 2 * i + 1) - 8388736.f, st));
  } else {
    o[0] = pack_f16x2(bf16_bits_to_f32(w0) * sc * UP, bf16_bits_to_f32(w0 >> 16) * sc);
    o[1] = pack_f16x2(bf16_bits_to_f32(w1) * sc * UP, bf16_bits_to_f32(w1 >> 16) * sc);
  }
}

// A CTA turns the words of 64 rows x 64 runs through shared memory, read along the row and written along n.  About 10 us
// for 27648 x 160 runs (28 MB in and out; with a conversion a byte and a word a store it was 13.2), issue 70 %.
template <int FMT, int BITS>
__global__ void __launch_bounds__(WP_THREADS) meta_kernel(const uint8_t *gmeta, const uint8_t *steps, int64_t N,
                                                          int64_t K, int G, int64_t np, Workspace ws) {
  constexpr int RW = WP_ROWS / (WP_THREADS / 32);  // rows a warp
  __shared__ uint32_t turn[WP_ROWS][WP_RUNS + 1];  // even rows, then odd; even runs, then odd (no bank conflicts)
  static_assert(WP_ROWS == 64 && WP_RUNS == 64, "a lane a row pair and a run pair");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n0 = (int64_t)blockIdx.x * WP_ROWS, r0 = (int64_t)blockIdx.y * WP_RUNS, runs = K / gran(FMT, G);
  pdl_launch_dependents();
  // a lane takes runs 2 l and 2 l + 1 of its row: one word of 16-bit group words (int4, int6), two of affine
  static_assert(RW == 8, "a warp's exponent bytes are one load");
  const int64_t r = r0 + 2 * lane, first = n0 + RW * warp;
  const int rows = r < runs ? (int)(N - first < RW ? N - first : RW) : 0;  // rows of this lane that exist
  uint32_t c[RW][2], st[RW];
  constexpr int GB = FMT == FMT_AFFINE ? 4 : 2, SB = FMT == FMT_INT4 ? 4 : 2;  // bytes of a group word, of a step word
  const uint8_t *gsrc = gmeta + GB * (first * runs + r), *ssrc = steps + SB * (first * (K / 256) + (r >> 3));
#pragma unroll
  for (int j = 0; j < RW; ++j) {
    c[j][0] = c[j][1] = st[j] = 0u;
    if (j < rows) {
      c[j][0] = __ldg(reinterpret_cast<const uint32_t *>(gsrc));
      if constexpr (FMT == FMT_AFFINE) {
        if (r + 1 < runs) c[j][1] = __ldg(reinterpret_cast<const uint32_t *>(gsrc) + 1);
      } else {  // K % 256 == 0: eight runs a super-block
        st[j] = FMT == FMT_INT4 ? __ldg(reinterpret_cast<const uint32_t *>(ssrc))
                                : (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(ssrc));
      }
    }
    gsrc += GB * runs;
    ssrc += SB * (K / 256);
  }
  // (pass 2 waited for pass 1 before it let this one start; from L2, where its stores are)
  const uint2 eb = __ldcg(reinterpret_cast<const uint2 *>(ws.rowexp + first));
#pragma unroll
  for (int j = 0; j < RW; ++j) {
    // 2^b_n from the byte 127 + w_top - b_n, b_n in [-126, 120]; any for rows of zeros
    const uint32_t byte = ((j < 4 ? eb.x : eb.y) >> (8 * (j & 3))) & 0xFFu;
    const float sc = __uint_as_float((uint32_t)min(254 + w_top(FMT) - (int)byte, 254) << 23);
    uint32_t o[2];
    scaled_meta<FMT, BITS>(c[j][0], c[j][1], st[j], sc, o);
    const int row = RW * warp + j, at = (row >> 1) + WP_ROWS / 2 * (row & 1);
    turn[at][lane] = o[0];
    turn[at][WP_RUNS / 2 + lane] = o[1];
  }
  __syncthreads();
  uint32_t *out = ws.meta + (r0 + warp) * np + n0 + 2 * lane;
  const int left = (int)(runs - r0 < WP_RUNS ? runs - r0 : WP_RUNS) - warp;
#pragma unroll
  for (int i = 0; i < WP_RUNS / (WP_THREADS / 32); ++i) {
    if ((WP_THREADS / 32) * i < left) {  // rows n, n + 1: their low halves, then their high halves
      const int col = (warp >> 1) + WP_RUNS / 2 * (warp & 1) + (WP_THREADS / 64) * i;
      const uint32_t a = turn[lane][col], b = turn[WP_ROWS / 2 + lane][col];
      *reinterpret_cast<uint2 *>(out) = make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    }
    out += (WP_THREADS / 32) * np;
  }
  pdl_wait();  // for pass 2
}

// ---- pass 4: the GEMM ------------------------------------------------------------------------------
constexpr int WARP_TMA = 0, WARP_MMA = 1, WARP_EPI0 = 4, WARP_DEQ0 = 8, NPROD = 3;
constexpr int NG = 2;  // dequantiser groups
constexpr int NUM_THREADS = (WARP_DEQ0 + 4 * NG) * 32;

// What TMA brings -- the dy tile (B), the packed codes and the metadata words -- waits in a ring as deep as shared
// memory allows (up to 16): for few tokens the stream of codes bounds the kernel and needs bytes in flight.  The
// weight tiles (A, 32 columns each) have a ring of up to eight beside the accumulators in tensor memory: two
// accumulators (an epilogue beside the next tile's MMAs) of 32 columns, or one of 64 or 256.
__host__ __device__ constexpr int code_row(int fmt, int bits) { return BKT * gemm::code_bits(fmt, bits) / 8; }
__host__ __device__ constexpr int b_bytes(int tt) { return tt * BN * 2; }
__host__ __device__ constexpr int p_bytes(int fmt, int bits) { return BN * code_row(fmt, bits); }
constexpr int META_BYTES = BN * 4 * 4;  // up to four runs of 32 k
constexpr uint32_t A_COLS = BN / 2;
__host__ __device__ constexpr uint32_t tmem_cols(int tt) { return 512u / ctas_per_sm(tt); }
__host__ __device__ constexpr int num_acc(int tt) { return tt == TT_SMALL ? 2 : 1; }
// dynamic shared memory of a CTA: an SM's 228 KB less 1 KB a CTA
__host__ __device__ constexpr int smem_limit(int tt) { return 233472 / ctas_per_sm(tt) - 1024; }
__host__ __device__ constexpr int stage_bytes(int fmt, int bits, int tt) {
  return b_bytes(tt) + p_bytes(fmt, bits) + META_BYTES;
}
__host__ __device__ constexpr int smem_need(int fmt, int bits, int tt, int st) {
  return st * stage_bytes(fmt, bits, tt) + (3 * st + 5) * 8 + 16 + 1024;
}
__host__ __device__ constexpr int stages(int fmt, int bits, int tt) {
  int st = 16;
  while (smem_need(fmt, bits, tt, st) > smem_limit(tt)) --st;
  return st;
}
__host__ __device__ constexpr int a_stages(int fmt, int bits, int tt) {
  const int fit = (int)(tmem_cols(tt) - num_acc(tt) * tt) / (int)A_COLS, st = stages(fmt, bits, tt);
  return st < fit ? (st < 8 ? st : 8) : (fit < 8 ? fit : 8);
}
__host__ __device__ constexpr int smem_bytes(int fmt, int bits, int tt) {
  return smem_need(fmt, bits, tt, stages(fmt, bits, tt));
}

// How the tiles are dealt: `waves` whole waves of `ctas` tiles, then the `rest` tiles that are left, their
// rest * steps stages cut into `shares` equal ranges, one a CTA.
struct Deal {
  int m_tiles, k_tiles;
  int tokens;  // a tile
  int steps;   // stages a tile: Np / 64
  int ctas, waves, rest, shares;
  __host__ __device__ bool joins() const { return shares != rest; }  // else a share is a whole tile
  __host__ __device__ int64_t share_begin(int c) const { return (int64_t)rest * steps * c / shares; }
};

inline Deal deal(int64_t M, int64_t N, int64_t K, int sms) {  // the tile class is M's
  Deal d;
  d.tokens = tile_tokens(M);
  d.m_tiles = (int)((M + d.tokens - 1) / d.tokens);
  d.k_tiles = (int)((K + BKT - 1) / BKT);
  d.steps = (int)(padded_n(N) / BN);
  d.ctas = (sms < DX_CTAS ? sms : DX_CTAS) * ctas_per_sm(tile_class(M));
  const int64_t tiles = (int64_t)d.m_tiles * d.k_tiles;
  d.waves = (int)(tiles / d.ctas);
  d.rest = (int)(tiles % d.ctas);
  const int64_t left = (int64_t)d.rest * d.steps;
  int64_t s = left / MIN_SHARE;
  if (s > d.ctas) s = d.ctas;
  if (s < d.rest) s = d.rest;  // at most a tile a share
  d.shares = d.rest ? (int)s : 0;
  return d;
}

// A CTA's share of the rest: stages [step0, step1) of rest tile `tile` and [0, step2) of the next.  It is worked out
// once a CTA (three 64-bit divisions take about a microsecond), while the kernel before this one runs.
struct Share {
  int tile, step0, step1, step2;
};
QL_DEVI Share get_share(const Deal &d, int c) {
  if (c >= d.shares) return Share{0, 0, 0, 0};
  const int64_t b = d.share_begin(c), e = d.share_begin(c + 1), t0 = b / d.steps, left = e - t0 * d.steps;
  return Share{(int)t0, (int)(b - t0 * d.steps), (int)(left < d.steps ? left : d.steps),
               left > d.steps ? (int)(left - d.steps) : 0};
}

// The i-th piece of work of CTA c: stages [step0, step1) of a tile; slot < 0: the whole tile, stored as dx;
// otherwise the slot of its partial sums.  A share is at most a tile long, so it has at most two pieces.
struct Piece {
  uint32_t tile;
  int step0, step1, slot;
};
QL_DEVI bool get_piece(const Deal &d, const Share &sh, int c, int i, Piece &p) {
  if (i < d.waves) {
    p = Piece{(uint32_t)(i * d.ctas + c), 0, d.steps, -1};
    return true;
  }
  const uint32_t tile = (uint32_t)(d.waves * d.ctas + sh.tile);
  if (i == d.waves && sh.step0 < sh.step1) {
    p = Piece{tile, sh.step0, sh.step1, d.joins() ? 2 * c : -1};
    return true;
  }
  if (i == d.waves + 1 && sh.step2 > 0) {
    p = Piece{tile + 1, 0, sh.step2, 2 * c + 1};
    return true;
  }
  return false;
}

struct Params {
  int64_t M, N, K;
  int G;
  Deal deal;
  const int *dexp;
  float *partial;
  __nv_bfloat16 *dx;
};

// k of TMEM lane r of a tile, as the matrix loads deal them out (thread t of a warp holds codes of column t / 4):
// nibbles 4 (t / 4) + i in lane 8 i + t / 4 of the warp's 32, bytes 2 (t / 4) + i of its two 16-k halves, 2-bit
// fields 8 (t / 4) + i of 64 k, of which the warp takes four (i = 0..3 or 4..7); dense int6: see decode_stage.
template <int FMT, int BITS>
QL_DEVI int out_k(int r) {
  if (FMT == FMT_INT6) return (r & ~7) | ((r & 7) >> 1) | ((r & 1) << 2);
  if (FMT == FMT_AFFINE && BITS == 8) return (r & ~15) | ((r & 7) << 1) | ((r >> 3) & 1);
  if (FMT == FMT_AFFINE && BITS == 2) return (r & 64) | ((r & 7) << 3) | ((r >> 3) & 7);
  return (r & ~31) | ((r & 7) << 2) | ((r >> 3) & 3);
}

QL_DEVI uint32_t fma_h2(uint32_t q, __half2 s, __half2 o) {
  const __half2 w = __hfma2(*reinterpret_cast<const __half2 *>(&q), s, o);
  return *reinterpret_cast<const uint32_t *>(&w);
}
QL_DEVI __half2 as_h2(uint32_t u) { return *reinterpret_cast<const __half2 *>(&u); }
// Four 8 x 8 matrices of 16-bit elements, transposed; lane l gives the address of row l (16 bytes).
QL_DEVI void ldmatrix_x4_trans(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
QL_DEVI uint32_t movmatrix_trans(uint32_t v) {
  uint32_t o;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(o) : "r"(v));
  return o;
}
QL_DEVI uint2 lds_u2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
QL_DEVI uint32_t lds_u1(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
// 16 lanes x 32 columns: thread t's words 2 j and 2 j + 1 go to lanes t / 4 and t / 4 + 8, column 4 j + t % 4.
QL_DEVI void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// A warp's 32 k (quarter wq of the tile's 128) of a stage's 64 rows: its code tile at shared address `codes`, its
// metadata words at `meta` + the thread's offset -> the words of lanes 0-15 (lo) and 16-31 (hi) of the quarter.
template <int FMT, int BITS>
QL_DEVI void decode_stage(uint32_t codes, uint32_t meta, int wq, int lane, uint32_t (&lo)[16], uint32_t (&hi)[16]) {
  // codes at the top of a half's mantissa, its lowest bit bit TOP; int6 fields f = (q & 63) ^ 32 = q + 32 as 1024 + f
  constexpr int TOP = 10 - BITS;
  constexpr uint32_t MASK = 0x00010001u * (uint32_t)(1024 - (1 << TOP)), M6 = 0x64206420u;
  auto weight6 = [](uint32_t f, __half2 s) {
    const __half2 w = __hmul2(__hsub2(as_h2(f), __float2half2_rn(1056.f)), s);
    return *reinterpret_cast<const uint32_t *>(&w);
  };
  if constexpr (FMT == FMT_INT4 || (FMT == FMT_AFFINE && BITS == 4)) {  // rows of 64 bytes, 64-byte swizzle
    uint32_t c[8];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int n = 32 * x + lane;
      ldmatrix_x4_trans(codes + n * 64 + ((wq ^ ((n >> 1) & 3)) << 4), c + 4 * x);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint2 m = lds_u2(meta + 32 * j);
      const __half2 s = as_h2(m.x), z = as_h2(m.y);
      lo[2 * j] = fma_h2((c[j] << 6) & MASK, s, z);
      lo[2 * j + 1] = fma_h2((c[j] << 2) & MASK, s, z);
      hi[2 * j] = fma_h2((c[j] >> 2) & MASK, s, z);
      hi[2 * j + 1] = fma_h2((c[j] >> 6) & MASK, s, z);
    }
  } else if constexpr (FMT == FMT_AFFINE && BITS == 8) {  // rows of 128 bytes, 128-byte swizzle
    uint32_t c[2][8];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int n = 32 * x + lane;
        ldmatrix_x4_trans(codes + n * 128 + (((2 * wq + b) ^ (n & 7)) << 4), c[b] + 4 * x);
      }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint2 m = lds_u2(meta + 32 * j);
      const __half2 s = as_h2(m.x), z = as_h2(m.y);
      lo[2 * j] = fma_h2((c[0][j] << 2) & MASK, s, z);
      lo[2 * j + 1] = fma_h2((c[0][j] >> 6) & MASK, s, z);
      hi[2 * j] = fma_h2((c[1][j] << 2) & MASK, s, z);
      hi[2 * j + 1] = fma_h2((c[1][j] >> 6) & MASK, s, z);
    }
  } else if constexpr (FMT == FMT_AFFINE) {  // 2-bit: rows of 32 bytes, two 64-k halves
    uint32_t c[8];
#pragma unroll
    for (int x = 0; x < 2; ++x) ldmatrix_x4_trans(codes + (32 * x + lane) * 32 + 16 * (wq >> 1), c + 4 * x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint2 m = lds_u2(meta + 32 * j);
      const __half2 s = as_h2(m.x), z = as_h2(m.y);
      const uint32_t v = c[j] >> (8 * (wq & 1));
      lo[2 * j] = fma_h2((v << 8) & MASK, s, z);
      lo[2 * j + 1] = fma_h2((v << 6) & MASK, s, z);
      hi[2 * j] = fma_h2((v << 4) & MASK, s, z);
      hi[2 * j + 1] = fma_h2((v << 2) & MASK, s, z);
    }
  } else if constexpr (FMT == FMT_INT6P) {  // nibbles as int4, then the high plane, rows of 32 bytes for 128 k
    uint32_t c[8], h[8];
    const int g = lane >> 2;
    // thread t needs the high fields of nibble column t / 4: a byte of the high plane's column 4 (wq & 1) + t / 8
    const int src = 4 * (4 * (wq & 1) + (g >> 1)) + (lane & 3);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int n = 32 * x + lane;
      ldmatrix_x4_trans(codes + n * 64 + ((wq ^ ((n >> 1) & 3)) << 4), c + 4 * x);
      ldmatrix_x4_trans(codes + BN * 64 + n * 32 + 16 * (wq >> 1), h + 4 * x);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __half2 s = as_h2(lds_u1(meta + 32 * j + (g & 4)));  // 16-weight groups: g / 4
      const uint32_t hv = __shfl_sync(0xffffffffu, h[j], src) >> (8 * (g & 1));
      lo[2 * j] = weight6(((c[j] & 0x000F000Fu) | ((hv << 4) & 0x00300030u)) ^ M6, s);
      lo[2 * j + 1] = weight6((((c[j] >> 4) & 0x000F000Fu) | ((hv << 2) & 0x00300030u)) ^ M6, s);
      hi[2 * j] = weight6((((c[j] >> 8) & 0x000F000Fu) | (hv & 0x00300030u)) ^ M6, s);
      hi[2 * j + 1] = weight6((((c[j] >> 12) & 0x000F000Fu) | ((hv >> 2) & 0x00300030u)) ^ M6, s);
    }
  } else {
    // dense int6: thread t takes row t / 4 of eight and, of each 8 codes (two 24-bit units), codes t % 4 and 4 + t % 4
    // as the elements 2 (t % 4), + 1 of an 8 x 8 matrix, which movmatrix transposes: row p is k = p / 2 + 4 (p % 2)
    const int g = lane >> 2, sh = 6 * (lane & 3);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t row = codes + (8 * j + g) * code_row(FMT, BITS) + 24 * wq;
      const uint2 x = lds_u2(row), y = lds_u2(row + 8), w = lds_u2(row + 16);
      const uint32_t u[8] = {x.x, __funnelshift_r(x.x, x.y, 24), __funnelshift_r(x.y, y.x, 16), y.x >> 8,
                             y.y, __funnelshift_r(y.y, w.x, 24), __funnelshift_r(w.x, w.y, 16), w.y >> 8};
      const uint2 m = lds_u2(meta + 32 * j);
      const __half2 s[2] = {as_h2(m.x), as_h2(m.y)};
      uint32_t o[4];
#pragma unroll
      for (int b = 0; b < 4; ++b)
        o[b] = weight6(movmatrix_trans((__byte_perm(u[2 * b] >> sh, u[2 * b + 1] >> sh, 0x5410) & 0x003F003Fu) ^ M6),
                    s[b >> 1]);
      lo[2 * j] = o[0];
      lo[2 * j + 1] = o[1];
      hi[2 * j] = o[2];
      hi[2 * j + 1] = o[3];
    }
  }
}

// Warp roles: 0, 2 and 3 TMA producers, 1 tensor memory and MMA issue, 4-7 epilogue (one k a lane), 8..
// dequantisers in groups of four warps (one a quarter of the TMEM lanes) that take the stages in turn.
template <int FMT, int BITS, int TT>
__global__ void __launch_bounds__(NUM_THREADS, ctas_per_sm(TT))
    gemm_dx_kernel(const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ CUtensorMap map_codes,
                   const __grid_constant__ CUtensorMap map_codes_hi, const __grid_constant__ CUtensorMap map_meta,
                   Params p) {
  constexpr int STAGES = stages(FMT, BITS, TT), AST = a_stages(FMT, BITS, TT);
  constexpr int NACC = num_acc(TT);
  constexpr int PROW = code_row(FMT, BITS);
  constexpr int OFF_P = b_bytes(TT), OFF_M = OFF_P + p_bytes(FMT, BITS);  // in a stage, after the dy tile
  constexpr int STAGE = stage_bytes(FMT, BITS, TT);
  constexpr uint32_t A_COL0 = NACC * TT;
  static_assert(STAGE % 1024 == 0 && OFF_P % 1024 == 0, "swizzle atoms");
  static_assert(STAGES >= AST && NG <= STAGES && NPROD <= STAGES, "an A slot's previous MMAs are found by their stage");
  constexpr uint32_t TMEM_COLS = tmem_cols(TT);
  static_assert(A_COL0 + AST * A_COLS <= TMEM_COLS, "A ring beside the accumulators");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * STAGE);
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 2 * STAGES + AST + 5);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  auto bar_tma_full = [&](int s) { return smem_u32(bars + s); };
  auto bar_empty = [&](int s) { return smem_u32(bars + STAGES + s); };
  auto bar_a_full = [&](int s) { return smem_u32(bars + 2 * STAGES + s); };
  auto bar_acc_full = [&](int a) { return smem_u32(bars + 2 * STAGES + AST + a); };
  auto bar_acc_empty = [&](int a) { return smem_u32(bars + 2 * STAGES + AST + 2 + a); };
  const uint32_t bar_final = smem_u32(bars + 2 * STAGES + AST + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = (int)blockIdx.x;
  // runs of a tile and bytes of its metadata box
  const int runs = FMT == FMT_AFFINE ? (p.G >= BKT ? 1 : BKT / p.G) : 4;
  const int tokens = p.deal.tokens;
  const uint32_t stage_tx = (uint32_t)(b_bytes(tokens) + p_bytes(FMT, BITS) + runs * BN * 4);

  auto step_ring = [](int &slot, uint32_t &phase, int by, int depth) {
    slot += by;
    if (slot >= depth) {
      slot -= depth;
      phase ^= 1u;
    }
  };

  __shared__ Share own_share;
  if (threadIdx.x == WARP_EPI0 * 32) own_share = get_share(p.deal, cta);
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_tma_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int s = 0; s < AST; ++s) mbar_init(bar_a_full(s), 4);
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar_acc_full(a), 1);
      mbar_init(bar_acc_empty(a), 4);
    }
    mbar_init(bar_final, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == WARP_MMA) {
    tmem_alloc(smem_u32(tmem_holder), TMEM_COLS);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const Share share = own_share;
  pdl_launch_dependents();
  pdl_wait();  // the preparation passes' results

  // Warps 0, 2 and 3 bring the stages in turn: a thread needs 120 ns and more to wait for a stage and start its
  // copies (measured: 64 x 64-byte boxes, 123 ns a stage from one thread, 41 ns from four), whatever their size.
  if (warp != WARP_MMA && warp < WARP_EPI0) {
    if (lane == 0) {
      tma_prefetch_desc(&map_dy);
      tma_prefetch_desc(&map_codes);
      tma_prefetch_desc(&map_meta);
      if constexpr (FMT == FMT_INT6P) tma_prefetch_desc(&map_codes_hi);
      const int first = warp == WARP_TMA ? 0 : warp - 1;
      int s = first;
      uint32_t ph = 0;
      int64_t it = first;
      bool ok = true;
      const bool start = !copies_withheld();
      int st = first;  // this producer's next stage, counted from the piece's first
      Piece pc;
      for (int i = 0; ok && start && get_piece(p.deal, share, cta, i, pc); ++i) {
        const uint32_t k_tile = pc.tile / (uint32_t)p.deal.m_tiles;
        const int32_t m0 = (int32_t)(pc.tile - k_tile * p.deal.m_tiles) * tokens;
        const int32_t x = FMT == FMT_INT6P ? (int32_t)(192 * (k_tile >> 1) + 64 * (k_tile & 1)) : (int32_t)(k_tile * PROW);
        const int32_t xh = (int32_t)(192 * (k_tile >> 1) + 128 + 32 * (k_tile & 1));
        const int32_t run0 = (int32_t)(k_tile * BKT / gran(FMT, p.G));
        const int steps = pc.step1 - pc.step0;
        for (; st < steps; st += NPROD, it += NPROD) {
          if (!mbar_wait_bounded(bar_empty(s), ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t b = bar_tma_full(s), dst = sbase + s * STAGE;
          const int32_t n = (pc.step0 + st) * BN;
          mbar_arrive_expect_tx(b, stage_tx);
          tma_load_2d(dst + OFF_P, &map_codes, b, x, n);
          if constexpr (FMT == FMT_INT6P) tma_load_2d(dst + OFF_P + BN * 64, &map_codes_hi, b, xh, n);
          tma_load_2d(dst + OFF_M, &map_meta, b, n, run0);
          tma_load_2d(dst, &map_dy, b, n, m0);
          step_ring(s, ph, NPROD, STAGES);
        }
        st -= steps;
      }
      if (!ok) {  // let copies already issued land before the CTA can exit
        for (int64_t j = it - NPROD; j >= 0 && j >= it - STAGES; j -= NPROD) {
          const long long t0 = clock64();
          while (!mbar_try_wait(bar_tma_full((int)(j % STAGES)), (uint32_t)((j / STAGES) & 1)) &&
                 clock64() - t0 < QL_WAIT_LIMIT_CYCLES) {
          }
        }
      }
    }
  } else if (warp == WARP_MMA) {
    const uint32_t idesc = umma_idesc_f16_f32(BKT, tokens);
    const uint64_t bd0 = umma_desc_k_sw128(sbase);
    int s = 0, as = 0;
    uint32_t ph = 0, aph = 0;
    bool ok = true, issued = false;
    Piece pc;
    for (int i = 0; ok && get_piece(p.deal, share, cta, i, pc); ++i) {
      const int a = i % NACC;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar_acc_empty(a), ((i / NACC) & 1) ^ 1, abort_flag))) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + (uint32_t)(a * TT);
      for (int st = pc.step0; st < pc.step1; ++st) {
        // the dequantisers waited for this stage's copies, so the dy tile has landed too
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar_a_full(as), aph, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        // done: the stage and the A slot are free
        umma_stage_tmem_a(d_tmem, tmem_base + A_COL0 + (uint32_t)as * A_COLS, bd0 + (uint64_t)(s * (STAGE >> 4)), idesc,
                          st != pc.step0, bar_empty(s));
        issued = true;
        step_ring(s, ph, 1, STAGES);
        step_ring(as, aph, 1, AST);
      }
      if (ok) umma_commit_elected(bar_acc_full(a));
    }
    if (issued) {  // all MMAs retired before teardown
      umma_commit_elected(bar_final);
      const long long t0 = clock64();
      while (!mbar_try_wait(bar_final, 0) && clock64() - t0 < QL_WAIT_LIMIT_CYCLES) {
      }
    }
  } else if (warp >= WARP_EPI0 && warp < WARP_EPI0 + 4) {
    const int e = warp - WARP_EPI0;  // TMEM lane quarter
    Piece pc;
    for (int i = 0; get_piece(p.deal, share, cta, i, pc); ++i) {
      const int a = i % NACC;
      const uint32_t k_tile = pc.tile / (uint32_t)p.deal.m_tiles, m_tile = pc.tile - k_tile * p.deal.m_tiles;
      const int64_t k = (int64_t)k_tile * BKT + out_k<FMT, BITS>(32 * e + lane);
      const int64_t m0 = (int64_t)m_tile * tokens;
      const int valid = (int)(p.M - m0 < tokens ? p.M - m0 : tokens);
      if (!mbar_wait_suspend(bar_acc_full(a), (i / NACC) & 1, abort_flag)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < tokens / 16; ++c) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(tmem_base + ((uint32_t)(32 * e) << 16) + (uint32_t)(a * TT + 16 * c), r);
        tmem_ld_wait();
        if (c == tokens / 16 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_acc_empty(a));
        }
        if (pc.slot < 0) {
          if (k < p.K) {
            __nv_bfloat16 *dst = p.dx + (m0 + 16 * c) * p.K + k;
#pragma unroll
            for (int t = 0; t < 16; ++t) {
              if (16 * c + t < valid)
                *dst = __float2bfloat16_rn(mul_pow2(__uint_as_float(r[t]), __ldg(p.dexp + m0 + 16 * c + t)));
              dst += p.K;
            }
          }
        } else {
          float *dst = p.partial + ((int64_t)pc.slot * tokens + 16 * c) * BKT + out_k<FMT, BITS>(32 * e + lane);
#pragma unroll
          for (int t = 0; t < 16; ++t)
            if (16 * c + t < valid) dst[t * BKT] = __uint_as_float(r[t]);
        }
      }
    }
  } else if (warp >= WARP_DEQ0) {
    const int wd = warp - WARP_DEQ0, g = wd >> 2;
    const int wq = wd & 3;  // lane quarter
    // the thread's place in a stage's metadata: the run of its 32 k (2-bit: of its 8 of 64), rows 2 (t % 4), + 1
    const int run = BITS == 2 && FMT == FMT_AFFINE ? 2 * (wq >> 1) + (lane >> 4) : wq;
    const int run_shift = FMT != FMT_AFFINE || p.G == 32 ? 0 : p.G == 64 ? 1 : 2;
    const int meta0 = OFF_M + (run >> run_shift) * (BN * 4) + 8 * (lane & 3);
    const uint32_t t_row = tmem_base + ((uint32_t)(32 * wq) << 16) + A_COL0;
    int64_t total = 0;  // this CTA's stages
    Piece pc;
    for (int i = 0; get_piece(p.deal, share, cta, i, pc); ++i) total += pc.step1 - pc.step0;
    int s = g, as = g % AST;
    uint32_t ph = 0;
    // the stage of the step AST before, whose MMAs read this step's A slot, and its phase (the first AST steps
    // find their slots free: the phase before the first)
    int es = g + STAGES - AST;
    uint32_t eph = 1;
    if (es >= STAGES) {
      es -= STAGES;
      eph = 0;
    }
    for (int64_t it = g; it < total; it += NG) {
      // In this order: copies may land out of turn and other groups be behind, and a wait by parity is only
      // right while its barrier is at that phase or just past it.  The A slot's wait says that the MMAs of step
      // it - AST, and so of every step before, are done; the previous use of stage s (it - STAGES) is one of them.
      if (!__all_sync(0xffffffffu, mbar_wait_suspend(bar_empty(es), eph, abort_flag))) break;
      if (!__all_sync(0xffffffffu, mbar_wait_suspend(bar_tma_full(s), ph, abort_flag))) break;
      tc_fence_after();
      uint32_t lo[16], hi[16];
      decode_stage<FMT, BITS>(sbase + s * STAGE + OFF_P, sbase + s * STAGE + meta0, wq, lane, lo, hi);
      tmem_st_16x128b_x8(t_row + (uint32_t)as * A_COLS, lo);
      tmem_st_16x128b_x8(t_row + (uint32_t)as * A_COLS + (16u << 16), hi);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_a_full(as));
      step_ring(s, ph, NG, STAGES);
      step_ring(es, eph, NG, STAGES);
      as += NG;
      if (as >= AST) as %= AST;
    }
  }

  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ---- pass 5: the sums of the split tiles' parts -------------------------------------------------------
// A CTA takes 8 tokens of a tile, a thread 4 k of one of them; the parts are added in the order of the shares, four
// loads in flight (they come from L2 and their latency is what this pass takes).
constexpr int JOIN_THREADS = 256, JOIN_TOKENS = JOIN_THREADS / (BKT / 4), JOIN_LOADS = 4;

__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(Params p) {
  const Deal &d = p.deal;
  const int rest_tile = (int)blockIdx.x;
  const uint32_t tile = (uint32_t)(d.waves * d.ctas + rest_tile);
  // The shares that touch the tile: from the last one, first, that begins at or before its stage 0 (share c begins at
  // stage floor(all c / shares)) up to the first, end, that begins at or behind its last.
  const int64_t all = (int64_t)d.rest * d.steps, lo = (int64_t)rest_tile * d.steps;
  int first = rest_tile * d.shares / d.rest;
  while (all * (first + 1) < (lo + 1) * d.shares) ++first;
  const int end = ((rest_tile + 1) * d.shares + d.rest - 1) / d.rest;
  const bool second = all * first < lo * d.shares;  // share `first` began in the tile before: its second piece
  const uint32_t k_tile = tile / (uint32_t)d.m_tiles, m_tile = tile - k_tile * d.m_tiles;
  const int t = blockIdx.y * JOIN_TOKENS + threadIdx.x / (BKT / 4), r = 4 * (threadIdx.x % (BKT / 4));
  const int64_t m = (int64_t)m_tile * d.tokens + t, k = (int64_t)k_tile * BKT + r;
  pdl_launch_dependents();
  pdl_wait();  // the parts
  if (t >= d.tokens || m >= p.M || k >= p.K) return;
  const int e = __ldg(p.dexp + m);
  const float *src = p.partial + (int64_t)t * BKT + r;
  const int64_t slot = (int64_t)d.tokens * BKT;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = first; c < end; c += JOIN_LOADS) {
    float4 x[JOIN_LOADS];
#pragma unroll
    for (int j = 0; j < JOIN_LOADS; ++j)
      x[j] = c + j < end ? __ldcg(reinterpret_cast<const float4 *>(src + slot * (2 * (c + j) + (second && c + j == first))))
                         : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < JOIN_LOADS; ++j) {
      v.x += x[j].x; v.y += x[j].y; v.z += x[j].z; v.w += x[j].w;
    }
  }
  *reinterpret_cast<uint2 *>(p.dx + m * p.K + k) =
      make_uint2(pack_bf16x2(mul_pow2(v.x, e), mul_pow2(v.y, e)), pack_bf16x2(mul_pow2(v.z, e), mul_pow2(v.w, e)));
}

}  // namespace dx
}  // namespace ql
