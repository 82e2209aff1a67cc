// gemm_sm100.cuh -- prefill-shaped layer on the 5th-generation tensor core.
//
//   y[M][N] = x[M][K] . W^T,  x bf16, W quantized, y bf16, fp32 accumulation
//
// Persistent kernel, one CTA per SM, tiles of BN=128 weight rows x TT tokens,
// K streamed in BK=64 steps through a shared-memory ring of x and code tiles.
// The dequantised weight tile never touches shared memory: the dequantisers
// write it into tensor memory (TMEM), where the MMAs of M = 128 (weight rows,
// A read from TMEM) x N = TT (tokens, B = the x tile in shared memory) consume
// it.  Shared memory then carries only the x tile (written once by TMA, read
// once by the tensor core) and the packed codes: a shared-memory weight tile
// would add its store, and a second token half would read it again, roughly
// doubling the bytes shared memory moves per MMA.  Two token tiles:
//   TT = 256 (prefill): one M = 128, N = 256 MMA per 16-k slice.  The
//     accumulator (128 lanes x 256 columns) and a ring of A stages (32 columns
//     each) share the 512 TMEM columns, so there is one accumulator and the
//     epilogue of a tile runs between two tiles' MMAs.
//   TT = 32 (up to 32 tokens): one M = 128, N = 32 MMA per slice, two 32-column
//     accumulators (an epilogue overlaps the next tile), the A ring beside them.
// Warp roles:
//   warp 0      TMA producer: scaled fp16 x tile (TT x 64, 128-byte
//               swizzle) and the packed code tile (128 rows x BK codes)
//   warp 1      TMEM allocator; the whole warp runs the MMA loop and an elected
//               lane issues tcgen05.mma (f16 x f16 -> f32)
//   warps 2-3   (int4) copy each super-block's group and step words into a
//               metadata ring, MSLOTS super-blocks ahead
//   warps 4-7   epilogue: tcgen05.ld the accumulator (warp w reads TMEM lanes
//               32*(w%4).., one weight row per lane), undo the two
//               power-of-two scales (exponents added first), round to bf16,
//               store y
//   warps 8..    dequantisers: packed codes + metadata -> weight times 2^b_n
//               -> fp16, one whole 64-weight tile row per thread, into the
//               TMEM lanes of the warp's quarter.  Groups of four warps take
//               the stages in turn: two groups (warps 8-15) at TT = 256, four
//               (warps 8-23) at TT = 32.
// The operands are fp16 rather than bf16 because rounding every weight to
// bf16 costs ~1% of rms(y); fp16 costs ~0.1% (see gemm_prep.cuh for the
// scaling that keeps fp32 range).  Loop state advances by counters: no
// division runs per stage.
// Every mbarrier wait is bounded; a wait that gives up sets the device status
// word and makes every role leave its loop.
#pragma once
#include "gated.cuh"
#include "gemm_prep.cuh"
#include "pack_dequant.cuh"

namespace ql {
namespace gemm {

constexpr int BM = 256;  // tokens per tile of the prefill form (the MMA's N)
constexpr int BN = 128;  // weight rows per tile
constexpr int BK = 64;
constexpr int WARP_TMA = 0;
constexpr int WARP_MMA = 1;
constexpr int WARP_META0 = 2;    // int4: two warps copy each super-block's group and step words ahead
constexpr int NUM_META_WARPS = 2;
constexpr int WARP_EPI0 = 4;
constexpr int WARP_DEQ0 = 8;
// dequantising warps: groups of four (one per TMEM lane quarter) take turns on the stages.  CPS is the
// CTAs resident per SM.  The 32-token form, whose MMAs are short and whose pace is its stage chain, has
// four groups at one CTA an SM, or two at two CTAs an SM (a layer with more 128-row tiles than SMs
// then runs every tile at once); the 256-token form has two (its register budget).
__host__ __device__ constexpr int deq_warps(int tt, int cps = 1) { return tt == BM || cps == 2 ? 8 : 16; }
__host__ __device__ constexpr int num_threads(int tt, int cps = 1) { return (WARP_DEQ0 + deq_warps(tt, cps)) * 32; }
constexpr int TT_SMALL = 32;          // token tile for up to 32 tokens
// int4 metadata ring: one slot per 256-weight super-block (four k-stages): [BN rows][16 bytes] of group
// words (the u32 of stage kb holds its two 32-weight groups), then [BN rows][4 bytes] of step words.
// Whole super-blocks make a row's copy one 16-byte and one 4-byte cp.async, against two 4-byte copies a
// stage, each from another row's line (int4 K is a multiple of 256, so no super-block straddles tiles).
constexpr int MSLOTS = 3;
constexpr int META_SLOT_BYTES = BN * 16 + BN * 4;
constexpr int SMEM_LIMIT = 232448;        // dynamic shared memory a CTA may use

__host__ __device__ constexpr int code_bits(int fmt, int bits) {
  return fmt == FMT_INT4 ? 4 : ((fmt == FMT_INT6 || fmt == FMT_INT6P) ? 6 : bits);
}
__host__ __device__ constexpr int p_row_bytes(int fmt, int bits) { return BK * code_bits(fmt, bits) / 8; }
__host__ __device__ constexpr int p_bytes(int fmt, int bits) { return BN * p_row_bytes(fmt, bits); }

// TT is the token tile: BM = 256 (one accumulator of 256 columns) or TT_SMALL = 32 (two of 32); the
// A ring of the dequantised weight tiles follows the accumulators in TMEM.
__host__ __device__ constexpr int a_bytes(int tt) { return tt * BK * 2; }  // the fp16 x tile
__host__ __device__ constexpr uint32_t tmem_cols(int tt) { return tt == BM ? 512u : 256u; }
__host__ __device__ constexpr int num_acc(int tt) { return tt == BM ? 1 : 2; }
__host__ __device__ constexpr uint32_t ta_acol0(int tt) { return (uint32_t)(num_acc(tt) * tt); }
constexpr uint32_t TA_ACOLS = BK / 2;   // an A stage: 64 fp16 per row = 32 columns

// Stages of the ring: as many as fit, up to six (TT = 256: six A stages of 32 columns fit beside the
// 256-column accumulator).  int4 adds the metadata ring [MSLOTS][META_SLOT_BYTES] and its barriers.
constexpr int NUM_BARS_PER_STAGE = 3;  // tma_full, b_full, empty
constexpr int NUM_BARS_FIXED = 5;      // acc_full[2], acc_empty[2], final
__host__ __device__ constexpr int stage_bytes(int fmt, int bits, int tt) {
  return a_bytes(tt) + p_bytes(fmt, bits);
}
__host__ __device__ constexpr int meta_bytes(int fmt) { return fmt == FMT_INT4 ? MSLOTS * META_SLOT_BYTES : 0; }
__host__ __device__ constexpr int meta_bars(int fmt) { return fmt == FMT_INT4 ? 2 * MSLOTS : 0; }
// each epilogue warp's copy of the tile's token scale exponents, one signed byte per token
__host__ __device__ constexpr int xe_bytes(int tt) { return 4 * tt; }
__host__ __device__ constexpr int smem_need(int fmt, int bits, int tt, int st) {
  return st * stage_bytes(fmt, bits, tt) + meta_bytes(fmt) + xe_bytes(tt) +
         (NUM_BARS_PER_STAGE * st + NUM_BARS_FIXED + meta_bars(fmt)) * 8 + 16 + 1024;
}
__host__ __device__ constexpr int stages(int fmt, int bits, int tt) {
  return smem_need(fmt, bits, tt, 6) <= SMEM_LIMIT ? 6
       : smem_need(fmt, bits, tt, 5) <= SMEM_LIMIT ? 5
       : smem_need(fmt, bits, tt, 4) <= SMEM_LIMIT ? 4 : 3;
}

// byte offsets inside the dynamic shared memory (base aligned to 1024)
__host__ __device__ constexpr int off_a(int tt, int s) { return s * a_bytes(tt); }
__host__ __device__ constexpr int off_p(int fmt, int bits, int tt, int s) {
  return stages(fmt, bits, tt) * a_bytes(tt) + s * p_bytes(fmt, bits);
}
__host__ __device__ constexpr int off_meta(int fmt, int bits, int tt, int s) {
  return stages(fmt, bits, tt) * stage_bytes(fmt, bits, tt) + s * META_SLOT_BYTES;
}
__host__ __device__ constexpr int off_xe(int fmt, int bits, int tt) {
  return stages(fmt, bits, tt) * stage_bytes(fmt, bits, tt) + meta_bytes(fmt);
}
__host__ __device__ constexpr int off_bar(int fmt, int bits, int tt) { return off_xe(fmt, bits, tt) + xe_bytes(tt); }
// barriers: tma_full[S], b_full[S], empty[S], acc_full[2], acc_empty[2], final, (int4) meta_full[MS],
// meta_empty[MS]; then the tmem base and the abort flag
__host__ __device__ constexpr int smem_bytes(int fmt, int bits, int tt) {
  return smem_need(fmt, bits, tt, stages(fmt, bits, tt));
}

struct Params {
  int64_t M, N, K;
  int G;
  const __nv_bfloat16 *bias;  // [N] or NULL: added in fp32 before the rounding to bf16
  const uint8_t *gmeta;
  const uint8_t *steps;
  __nv_bfloat16 *y;
  GemmWorkspace ws;
  // the gated form only (y is then h [M][N / 2])
  int act;
  int share_tiles;      // TT = 256: the dequantisers help to finish every tile, not the last alone
                        // (in the padding beside act: with eight bytes more of parameters the plain affine
                        // GEMM took 8 % longer, 80.3 -> 87.9 us at M = 512)
  int8_t *saved;        // codes [M][2][save8_cols(N / 2)] of (g, u), or NULL
  uint8_t *saved_exps;  // [M][2][save8_cols(N / 2) / 16]
  float4 *scratch;      // TT = 256: [CTA][TT / 4][BN]
};

// The gated form: the layer's rows are F = N / 2 gate rows, then F up rows, and a tile is 64 features:
// their 64 gate rows and 64 up rows (one code box of 2 x 64 rows of the layer as [2][F] rows).  Which of the tile's rows goes to which
// TMEM lane is the dequantisers' choice, and they give each lane quarter 16 features, gate rows in its
// lanes 0-15 and up rows in lanes 16-31: g and u of a feature then meet in one epilogue warp by a
// shuffle, without shared memory.  Box row (and metadata slot row) of lane r of the tile:
constexpr int GATED_F = BN / 2;  // features a tile
template <bool GATED>
QL_DEVI int box_row(int r) {
  return GATED ? ((r & 16) ? GATED_F : 0) + 16 * (r >> 5) + (r & 15) : r;
}
// Layer row of box row br.  A tile's last features may be past F: their codes are zeros, their metadata that of
// other rows (or, past N, zeros), and their results are not stored.
template <bool GATED>
QL_DEVI int64_t layer_row(int64_t n_tile, int br, int64_t N) {
  return GATED ? (br < GATED_F ? n_tile * GATED_F + br : N / 2 + n_tile * GATED_F + br - GATED_F) : n_tile * BN + br;
}

// Metadata of one 32-weight chunk (see formats.cuh): int4 (gm, st); int6
// (two scale codes, st); affine (gm, unused).
template <int FMT>
QL_DEVI void load_meta(const Params &p, int64_t n, int64_t c, uint32_t &gm, uint32_t &st) {
  if (n >= p.N) {
    gm = 0;
    st = 0;
    return;
  }
  if constexpr (FMT == FMT_INT4) {
    gm = __ldg(reinterpret_cast<const uint16_t *>(p.gmeta) + n * (p.K / 32) + c);
    st = __ldg(reinterpret_cast<const uint32_t *>(p.steps) + n * (p.K / 256) + (c >> 3));
  } else if constexpr (FMT == FMT_INT6 || FMT == FMT_INT6P) {
    gm = __ldg(reinterpret_cast<const uint16_t *>(p.gmeta + n * (p.K / 16)) + c);
    st = __ldg(reinterpret_cast<const uint16_t *>(p.steps) + n * (p.K / 256) + (c >> 3));
  } else {
    gm = __ldg(reinterpret_cast<const uint32_t *>(p.gmeta) + n * (p.K / p.G) + (32 * c) / p.G);
    st = 0;
  }
}

// Decode one chunk whose codes sit in shared memory at `src` (int6 planar: the chunk's 16 low-plane
// bytes at `src`, its 8 high-plane bytes at `src_hi`).
template <int FMT, int BITS>
QL_DEVI void smem_decode32(const uint8_t *src, const uint8_t *src_hi, uint32_t gm, uint32_t st, float (&w)[32]) {
  if constexpr (FMT == FMT_INT6P) {
    const uint4 l = *reinterpret_cast<const uint4 *>(src);
    const uint2 h = *reinterpret_cast<const uint2 *>(src_hi);
    const uint32_t lo[4] = {l.x, l.y, l.z, l.w}, hi[2] = {h.x, h.y};
    int6p_decode32(lo, hi, gm, st, w);
  } else if constexpr (FMT == FMT_INT4) {
    const uint4 v = *reinterpret_cast<const uint4 *>(src);
    const uint32_t c[4] = {v.x, v.y, v.z, v.w};
    int4_decode32(c, gm, st, w);
  } else if constexpr (FMT == FMT_INT6) {
    const uint2 *s2 = reinterpret_cast<const uint2 *>(src);
    const uint2 a = s2[0], b = s2[1], d = s2[2];
    const uint32_t c[6] = {a.x, a.y, b.x, b.y, d.x, d.y};
    int6_decode32(c, gm, st, w);
  } else {
    uint32_t c[BITS];
    if constexpr (BITS == 2) {
      const uint2 v = *reinterpret_cast<const uint2 *>(src);
      c[0] = v.x;
      c[1] = v.y;
    } else {
#pragma unroll
      for (int t = 0; t < BITS / 4; ++t) {
        const uint4 v = reinterpret_cast<const uint4 *>(src)[t];
        c[4 * t] = v.x; c[4 * t + 1] = v.y; c[4 * t + 2] = v.z; c[4 * t + 3] = v.w;
      }
    }
    affine_decode32<BITS>(c, gm, w);
  }
}

// Words of one 32-weight chunk's codes, read from shared memory (int4, affine): code_bits words.
template <int FMT, int BITS>
QL_DEVI void load_code_words(const uint8_t *src, uint32_t (&cw)[code_bits(FMT, BITS)]) {
  if constexpr (code_bits(FMT, BITS) == 2) {
    const uint2 v = *reinterpret_cast<const uint2 *>(src);
    cw[0] = v.x;
    cw[1] = v.y;
  } else {
#pragma unroll
    for (int t = 0; t < code_bits(FMT, BITS) / 4; ++t) {
      const uint4 v = reinterpret_cast<const uint4 *>(src)[t];
      cw[4 * t] = v.x; cw[4 * t + 1] = v.y; cw[4 * t + 2] = v.z; cw[4 * t + 3] = v.w;
    }
  }
}

// One 32-weight chunk of a tile row -> 16 words of fp16 pairs, each weight times 2^b_n (sc is the
// row's 2^b_n).  Word 4 q + e holds weights (8 q + e, 8 q + e + 4): the k order of the x tile, whose
// 16-byte chunks hold k = 0,4,1,5,2,6,3,7 of their 8 values.  int4 and affine take the chunk's code
// words `cw`; int6 (and int6 planar, with its high-plane bytes at `src_hi`) decode from `src`.
template <int FMT, int BITS>
QL_DEVI void chunk_to_f16(const uint32_t (&cw)[code_bits(FMT, BITS)], const uint8_t *src, const uint8_t *src_hi,
                          uint32_t gm, uint32_t st, float sc, uint32_t (&o)[16]) {
  if constexpr (FMT == FMT_INT4) {
    // packed-half arithmetic: q as 1024+q / 64+q from one bit operation, then
    // w * 2^b_n = q * S' - Z * S' in fp16 with S' = S * 2^b_n; the codes sc, zc become floats
    // by placing the byte in the mantissa of 2^23 and subtracting 2^23 (exact)
    const float scf = __uint_as_float(0x4B000000u | (gm & 0xffu)) - 8388608.f;
    const float zcf = __uint_as_float(0x4B000000u | ((gm >> 8) & 0xffu)) - 8388608.f;
    const float S = __fmul_rn(scf, f16_bits_to_f32(st)) * sc;
    const float ZS = __fmul_rn(zcf, f16_bits_to_f32(st >> 16)) * S;
    const __half2 s2 = __float2half2_rn(S), nz2 = __float2half2_rn(-ZS);
    const __half2 m1024 = __float2half2_rn(1024.f), m64 = __float2half2_rn(64.f);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t wd = cw[q], w8 = wd >> 8;
      uint32_t pr[4];
      pr[0] = (wd & 0x000F000Fu) | 0x64006400u;  // (1024 + n0, 1024 + n4)
      pr[1] = (wd & 0x00F000F0u) | 0x54005400u;  // (64 + n1, 64 + n5)
      pr[2] = (w8 & 0x000F000Fu) | 0x64006400u;  // (1024 + n2, 1024 + n6)
      pr[3] = (w8 & 0x00F000F0u) | 0x54005400u;  // (64 + n3, 64 + n7)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __half2 qv = __hsub2(*reinterpret_cast<const __half2 *>(&pr[e]), (e & 1) ? m64 : m1024);
        const __half2 wv = __hfma2(qv, s2, nz2);
        o[4 * q + e] = *reinterpret_cast<const uint32_t *>(&wv);
      }
    }
  } else if constexpr (FMT == FMT_AFFINE) {
    // packed-half arithmetic: the codes become 1024 + q halves by bit operations (q exact after
    // one subtraction), then w * 2^b_n = q * s' + b' in one fused multiply-add with s' = s * 2^b_n
    // and b' = b * 2^b_n, which are exact in fp16 (bf16 values scaled into fp16's range), so each
    // weight is rounded once
    const __half2 s2 = __float2half2_rn(bf16_bits_to_f32(gm) * sc);
    const __half2 b2 = __float2half2_rn(bf16_bits_to_f32(gm >> 16) * sc);
    const __half2 m1024 = __float2half2_rn(1024.f);
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // output words 4q..: weights 8q .. 8q+7 of the chunk, as (k, k+4) pairs
      uint32_t pr[4];
      if constexpr (BITS == 4) {
        const uint32_t wd = cw[q], w8 = wd >> 8;
        pr[0] = (wd & 0x000F000Fu) | 0x64006400u;  // (1024 + n0, 1024 + n4)
        pr[1] = ((wd >> 4) & 0x000F000Fu) | 0x64006400u;
        pr[2] = (w8 & 0x000F000Fu) | 0x64006400u;
        pr[3] = ((w8 >> 4) & 0x000F000Fu) | 0x64006400u;
      } else if constexpr (BITS == 8) {
        const uint32_t w0 = cw[2 * q], w1 = cw[2 * q + 1];  // k 0..3, k 4..7
        const uint32_t t0 = __byte_perm(w0, w1, 0x5140), t1 = __byte_perm(w0, w1, 0x7362);  // (0 4 1 5) (2 6 3 7)
        pr[0] = __byte_perm(t0, 0x64646464u, 0x4140);
        pr[1] = __byte_perm(t0, 0x64646464u, 0x4342);
        pr[2] = __byte_perm(t1, 0x64646464u, 0x4140);
        pr[3] = __byte_perm(t1, 0x64646464u, 0x4342);
      } else {  // 2-bit: codes 8q .. 8q+7 are bits 16 (q & 1) .. of word q / 2
        const uint32_t wd = cw[q >> 1] >> (16 * (q & 1));
        const uint32_t u = __byte_perm(wd, 0u, 0x4140);  // codes 0-3 in byte 0, codes 4-7 in byte 2
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[e] = ((u >> (2 * e)) & 0x00030003u) | 0x64006400u;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __half2 qv = __hsub2(*reinterpret_cast<const __half2 *>(&pr[e]), m1024);
        const __half2 wv = __hfma2(qv, s2, b2);
        o[4 * q + e] = *reinterpret_cast<const uint32_t *>(&wv);
      }
    }
  } else {
    float w[32];
    smem_decode32<FMT, BITS>(src, src_hi, gm, st, w);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[4 * q + e] = pack_f16x2(w[8 * q + e] * sc, w[8 * q + e + 4] * sc);
  }
}

// Epilogue of the gated form for 16 tokens (m0 ..) of one feature f: lanes 0-15 of the warp hold the 16
// tokens' g in r, lanes 16-31 the same features' u.  Each lane sends half of its tokens to its partner
// (lane ^ 16) and receives the other projection of the half it keeps: lanes 0-15 finish tokens 0-7, lanes
// 16-31 tokens 8-15, 16 contiguous features of each.  These warps run beside the dequantisers, whose issue
// slots they take, so this is written for few instructions: values travel and are stored in pairs (h) and
// fours (codes) after a transposition among neighbouring lanes, and a group's scale is reduced once, not in
// every lane.

// What a lane needs of its row of a gated tile: its feature, its scale exponent, the tile's tokens, where its outputs
// go, and whether every exponent sum of the warp's rows and these tokens is that of a normal float (then D * 2^e is
// one multiplication by 2^e built from its bits, the same single rounding as mul_pow2).  A lane finishes 8 of a
// chunk's 16 tokens (first: 0 or 8).
struct GatedRow {
  int64_t f, F, m0;
  int we, chunks;  // chunks of 16 tokens that hold any
  int left, left_saved;  // tokens of the tile from `first` on whose h, whose codes this lane stores
  bool one_mul;
  __nv_bfloat16 *h;  // of its first store
  int8_t *codes;
  uint8_t *exps;
  QL_DEVI GatedRow(const Params &p, int64_t n_tile, int64_t m_tile, int tt, int e, int lane, int down) {
    const int64_t n = layer_row<true>(n_tile, box_row<true>(32 * e + lane), p.N);
    we = (n < p.N ? p.ws.wexp[n] : 0) + down;  // the weights sit 2^-down below the row scales
    f = n_tile * GATED_F + 16 * e + (lane & 15);
    F = p.N / 2;
    m0 = m_tile * tt;
    const int64_t rest = p.M - m0;
    const int tokens = (int)(rest < tt ? rest : tt);
    chunks = (tokens + 15) / 16;
    int lo = 1 << 20, hi = -(1 << 20);
    for (int t = lane; t < tokens; t += 32) {
      const int xe = __ldg(p.ws.xexp + m0 + t);
      lo = min(lo, xe);
      hi = max(hi, xe);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    one_mul = __all_sync(0xffffffffu, lo + we >= -126 && hi + we <= 127);
    const int first = lane < 16 ? 0 : 8, l = lane & 15;
    const int64_t fp = save8_cols(F), m = m0 + first;
    left = f < F ? tokens - first : 0;
    left_saved = f < fp ? tokens - first : 0;
    h = F % 2 == 0 ? p.y + (m + (lane & 1)) * F + (f & ~(int64_t)1) : p.y + m * F + f;
    codes = p.saved + 2 * (m + (lane & 3)) * fp + (f & ~(int64_t)3);
    exps = p.saved_exps + ((m + 2 * ((l >> 1) & 3) + (l & 1)) * 2 + (l >> 3)) * (fp / 16) + (f >> 4);
  }
};

// h of 8 tokens of chunk c.  Words of two tokens become words of two features: the even lane of a pair keeps the
// first token, the odd lane the second.
QL_DEVI void gated_store_h(const GatedRow &row, const float (&h)[8], int c, int lane) {
  const int left = row.left - 16 * c;
  __nv_bfloat16 *dst = row.h + (int64_t)(16 * c) * row.F;
  if (row.F % 2 == 0) {
    const int odd = lane & 1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t own = pack_bf16x2(h[2 * j], h[2 * j + 1]), other = __shfl_xor_sync(0xffffffffu, own, 1);
      const uint32_t w = __byte_perm(own, other, odd ? 0x3276 : 0x5410);
      if (2 * j + odd < left) *reinterpret_cast<uint32_t *>(dst) = w;
      dst += 2 * row.F;
    }
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t < left) *dst = __float2bfloat16_rn(h[t]);
      dst += row.F;
    }
  }
}

// The checkpoint of 8 tokens' g and u.  The 16 lanes' features are one group of each token and projection.
// A value's upper 16 bits plus one, without the sign, order like save8_key and hold it in their upper bits
// (the sum is the key's carry); two values share a word.  Words 0-3 are the tokens' g, 4-7 their u.
QL_DEVI void gated_save(const GatedRow &row, const float (&g)[8], const float (&u)[8], int ch, int lane) {
  const int l = lane & 15;
  uint32_t k[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float v0 = j < 4 ? g[2 * j] : u[2 * j - 8], v1 = j < 4 ? g[2 * j + 1] : u[2 * j - 7];
    k[j] = (__byte_perm(__float_as_uint(v0), __float_as_uint(v1), 0x7632) & 0x7FFF7FFFu) + 0x00010001u;
  }
  // halve the words and the lanes in turn: bit 3 of l picks g or u, bits 2 and 1 the word; then the last bit's
  // lanes meet
  uint32_t a4[4], a2[2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, (l & 8) ? k[j] : k[j + 4], 8);
    a4[j] = __vmaxu2((l & 8) ? k[j + 4] : k[j], got);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, (l & 4) ? a4[j] : a4[j + 2], 4);
    a2[j] = __vmaxu2((l & 4) ? a4[j + 2] : a4[j], got);
  }
  uint32_t w = __vmaxu2((l & 2) ? a2[1] : a2[0], __shfl_xor_sync(0xffffffffu, (l & 2) ? a2[0] : a2[1], 2));
  w = __vmaxu2(w, __shfl_xor_sync(0xffffffffu, w, 1));
  // lane l now has the two keys of word l >> 1; exponents, and the inverse scales' upper 16 bits
  const uint32_t e0 = save8_exponent(min((w & 0xFFFFu) >> 7, 255u)), e1 = save8_exponent(min(w >> 23, 255u));
  const uint32_t inv = ((254u - min(e0, 254u)) << 7) | ((254u - min(e1, 254u)) << 23);  // 0 for E = 255
  const int64_t fp = save8_cols(row.F);
  const int left = row.left_saved - 16 * ch;
  // this lane stores its key's exponent of token 2 ((l >> 1) & 3) + (l & 1): g's in lanes 0-7, u's in 8-15
  if (2 * ((l >> 1) & 3) + (l & 1) < left) row.exps[2 * ch * fp] = (uint8_t)((l & 1) ? e1 : e0);
  // codes: v 2^(127 - E) + 1.5 2^23 holds rint(v 2^(127 - E)) in its low byte
  uint32_t c[4];  // bytes of tokens 0-3, 4-7 of g, then of u
  const bool finite = !__any_sync(0xffffffffu, e0 == 255u || e1 == 255u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t iw = __shfl_sync(0xffffffffu, inv, (lane & 16) + 4 * i + 2 * j);
      const float i0 = __uint_as_float(iw << 16), i1 = __uint_as_float(iw & 0xFFFF0000u);
      const int t = 4 * (i & 1) + 2 * j;
      b[2 * j] = __float_as_uint(fmaf(i < 2 ? g[t] : u[t], i0, 12582912.f));
      b[2 * j + 1] = __float_as_uint(fmaf(i < 2 ? g[t + 1] : u[t + 1], i1, 12582912.f));
      if (!finite) {  // codes of groups that are not are 0
        if (i0 == 0.f) b[2 * j] = 0u;
        if (i1 == 0.f) b[2 * j + 1] = 0u;
      }
    }
    c[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
  // 4 x 4 bytes turn among four lanes: lane q of a quad gets token q (or 4 + q) of the quad's features
  const int q = lane & 3;
  const uint32_t turn1 = (q & 1) ? 0x3715u : 0x6240u, turn2 = (q & 2) ? 0x3276u : 0x5410u;
  int8_t *dst = row.codes + 32 * ch * fp;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v = c[i];
    v = __byte_perm(v, __shfl_xor_sync(0xffffffffu, v, 1), turn1);  // bytes (t, t of the neighbour) x 2 tokens
    v = __byte_perm(v, __shfl_xor_sync(0xffffffffu, v, 2), turn2);
    if (4 * (i & 1) + q < left) *reinterpret_cast<uint32_t *>(dst + (i >> 1) * fp + 8 * (i & 1) * fp) = v;
  }
}

QL_DEVI void gated_store(const Params &p, const GatedRow &row, const uint32_t (&r)[16], int c, int lane) {
  const bool up = lane >= 16;
  float g[8], u[8], h[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const float other = __uint_as_float(__shfl_xor_sync(0xffffffffu, up ? r[t] : r[8 + t], 16));
    g[t] = up ? other : __uint_as_float(r[t]);
    u[t] = up ? __uint_as_float(r[8 + t]) : other;
  }
  if (row.f >= row.F) {  // features past the last: zeros in the checkpoint's padding
#pragma unroll
    for (int t = 0; t < 8; ++t) g[t] = u[t] = 0.f;
  }
  if (p.act == ACT_SILU) {
#pragma unroll
    for (int t = 0; t < 8; ++t) h[t] = act_value(ACT_SILU, g[t]) * u[t];
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t) h[t] = act_value(p.act, g[t]) * u[t];
  }
  gated_store_h(row, h, c, lane);
  if (p.saved) gated_save(row, g, u, c, lane);
}

// chunk_to_f16 of the gated form, whose epilogue shares the issue slots.  int4 and affine codes are shifted to the top of
// a half's ten mantissa bits, where alone they are the fp16 subnormal q 2^-18 (2-bit: 2^-16, 8-bit: 2^-22); the inverse
// power goes into the scale, and a pair of weights is a shift, a mask and one fused multiply-add.  For that scale to be
// an fp16 number (the prep pass leaves S <= 2^15 / 7.5 and s <= 2^16 / (2^bits - 1)) a row's weights lie below 1, 2^-15
// of where the plain GEMM has them.  fp16 keeps 11 bits down to 2^-14: a group whose largest weight is 2^-13 of the row's
// or more has its weights to 2^-11 of that largest one, a smaller group one bit less a power of two.  (Codes left at the
// bottom of the half, q 2^-24, are a shift less and reach 2^-7, 2-bit ones 2^-4: too little for a layer whose columns
// differ, and 0 to 5 % faster.)  The plain GEMM's way, 1024 + q and a subtraction, reaches 2^-28, but the half-precision
// pipe then sets the pace: M = 2048, K = 5120, N = 27648: int4 600 us against 542; K = 4096, N = 14336: 4-bit 306 against
// 284, 2-bit 306 against 278, 8-bit 302 against 306; M = 20, N = 27648: int4 60 against 54, 8-bit 73 against 64.
// int6 does subtract, and multiplies by its scale as an fp16 number (two roundings, 2^-12 of the weight each): 596 us
// where the plain GEMM's product in fp32 takes 690.
template <int FMT, int BITS>
__host__ __device__ constexpr int gated_down() { return FMT == FMT_INT6 || FMT == FMT_INT6P ? 0 : 15; }

template <int FMT, int BITS>
QL_DEVI void gated_chunk_to_f16(const uint32_t (&cw)[code_bits(FMT, BITS)], const uint8_t *src, const uint8_t *src_hi,
                                uint32_t gm, uint32_t st, float sc, uint32_t (&o)[16]) {
  auto half2_of = [](uint32_t u) { return *reinterpret_cast<const __half2 *>(&u); };
  auto word_of = [](__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); };
  if constexpr (FMT == FMT_INT4 || FMT == FMT_AFFINE) {
    // 2^(24 - TOP) undoes the code's place (its lowest bit is mantissa bit TOP), 2^-DOWN lowers the row
    constexpr int TOP = 10 - (FMT == FMT_INT4 ? 4 : BITS);
    constexpr float DOWN = 1.f / (float)(1 << gated_down<FMT, BITS>()), UP = (float)(1 << (24 - TOP)) * DOWN;
    constexpr uint32_t MASK = 0x00010001u * (uint32_t)(1024 - (1 << TOP));
    float S, z;
    if constexpr (FMT == FMT_INT4) {
      const float scf = __uint_as_float(0x4B000000u | (gm & 0xffu)) - 8388608.f;
      const float zcf = __uint_as_float(0x4B000000u | ((gm >> 8) & 0xffu)) - 8388608.f;
      S = scf * f16_bits_to_f32(st) * sc;
      z = -(zcf * f16_bits_to_f32(st >> 16)) * S * DOWN;
    } else {
      S = bf16_bits_to_f32(gm) * sc;
      z = bf16_bits_to_f32(gm >> 16) * sc * DOWN;
    }
    const __half2 s2 = __float2half2_rn(S * UP), z2 = __float2half2_rn(z);
    auto weight = [&](uint32_t q) { return word_of(__hfma2(half2_of(BITS == 8 ? q : q & MASK), s2, z2)); };
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (FMT == FMT_INT4 || BITS == 4) {
        o[4 * q] = weight(cw[q] << 6);
        o[4 * q + 1] = weight(cw[q] << 2);
        o[4 * q + 2] = weight(cw[q] >> 2);
        o[4 * q + 3] = weight(cw[q] >> 6);
      } else if constexpr (BITS == 8) {
        const uint32_t w0 = cw[2 * q], w1 = cw[2 * q + 1];
        const uint32_t t0 = __byte_perm(w0, w1, 0x5140), t1 = __byte_perm(w0, w1, 0x7362);  // (0 4 1 5) (2 6 3 7)
        o[4 * q] = weight(__byte_perm(t0, 0u, 0x4140) << TOP);
        o[4 * q + 1] = weight(__byte_perm(t0, 0u, 0x4342) << TOP);
        o[4 * q + 2] = weight(__byte_perm(t1, 0u, 0x4140) << TOP);
        o[4 * q + 3] = weight(__byte_perm(t1, 0u, 0x4342) << TOP);
      } else {
        const uint32_t u = __byte_perm(cw[q >> 1] >> (16 * (q & 1)), 0u, 0x4140);  // codes 0-3 in byte 0, 4-7 in byte 2
#pragma unroll
        for (int e = 0; e < 4; ++e) o[4 * q + e] = weight(u << (TOP - 2 * e));
      }
    }
  } else {  // int6: fields f = q + 32 (the code's sign bit flipped) as 1024 + f; two 16-weight groups
    const float step = f16_bits_to_f32(st) * sc;
    const __half2 s[2] = {__float2half2_rn((float)(int8_t)gm * step), __float2half2_rn((float)(int8_t)(gm >> 8) * step)};
    const __half2 m1056 = __float2half2_rn(1056.f);
    auto weight = [&](uint32_t f, __half2 sq) { return word_of(__hmul2(__hsub2(half2_of(f ^ 0x64206420u), m1056), sq)); };
    if constexpr (FMT == FMT_INT6P) {
      const uint4 l = *reinterpret_cast<const uint4 *>(src);
      const uint2 h = *reinterpret_cast<const uint2 *>(src_hi);
      const uint32_t c[4] = {l.x, l.y, l.z, l.w}, hi[4] = {h.x, h.x >> 16, h.y, h.y >> 16};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t u = __byte_perm(hi[q], 0u, 0x4140);
        o[4 * q] = weight((c[q] & 0x000F000Fu) | ((u << 4) & 0x00300030u), s[q >> 1]);
        o[4 * q + 1] = weight(((c[q] >> 4) & 0x000F000Fu) | ((u << 2) & 0x00300030u), s[q >> 1]);
        o[4 * q + 2] = weight(((c[q] >> 8) & 0x000F000Fu) | (u & 0x00300030u), s[q >> 1]);
        o[4 * q + 3] = weight(((c[q] >> 12) & 0x000F000Fu) | ((u >> 2) & 0x00300030u), s[q >> 1]);
      }
    } else {  // eight 24-bit units of four codes
      const uint2 *s2 = reinterpret_cast<const uint2 *>(src);
      const uint2 x = s2[0], y = s2[1], w = s2[2];
      const uint32_t u[8] = {x.x, __funnelshift_r(x.x, x.y, 24), __funnelshift_r(x.y, y.x, 16), y.x >> 8,
                             y.y, __funnelshift_r(y.y, w.x, 24), __funnelshift_r(w.x, w.y, 16), w.y >> 8};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t a = __byte_perm(u[2 * q], u[2 * q + 1], 0x5410);
        const uint32_t b = __byte_perm(u[2 * q] >> 12, u[2 * q + 1] >> 12, 0x5410);
        o[4 * q] = weight(a & 0x003F003Fu, s[q >> 1]);
        o[4 * q + 1] = weight((a >> 6) & 0x003F003Fu, s[q >> 1]);
        o[4 * q + 2] = weight(b & 0x003F003Fu, s[q >> 1]);
        o[4 * q + 3] = weight((b >> 6) & 0x003F003Fu, s[q >> 1]);
      }
    }
  }
}

// The token exponents of chunk c (those of tokens past M are read, their section of the workspace being
// padded, and not used).
struct ChunkExp {
  int4 v[4];
  QL_DEVI void load(const Params &p, const GatedRow &row, int c) {
    const int4 *src = reinterpret_cast<const int4 *>(p.ws.xexp + row.m0 + 16 * c);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __ldg(src + j);
  }
  QL_DEVI int operator[](int t) const { return (t & 3) == 0 ? v[t >> 2].x : (t & 3) == 1 ? v[t >> 2].y : (t & 3) == 2 ? v[t >> 2].z : v[t >> 2].w; }
};

// Chunk c of a row's accumulator: undo the power-of-two scales (exponents added first, see mul_pow2),
// then the gated epilogue.
QL_DEVI void gated_chunk(const Params &p, const GatedRow &row, uint32_t (&r)[16], const ChunkExp &xe, int c, int lane) {
  if (row.one_mul) {
    const int w_bits = row.we * (1 << 23) + 0x3F800000;
#pragma unroll
    for (int t = 0; t < 16; ++t)
      r[t] = __float_as_uint(__fmul_rn(__uint_as_float(r[t]), __int_as_float(xe[t] * (1 << 23) + w_bits)));
  } else {
#pragma unroll
    for (int t = 0; t < 16; ++t) r[t] = __float_as_uint(mul_pow2(__uint_as_float(r[t]), xe[t] + row.we));
  }
  gated_store(p, row, r, c, lane);
}

template <int FMT, int BITS, int TT, int CPS = 1, bool GATED = false>
__global__ void __launch_bounds__(num_threads(TT, CPS), CPS)
    gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_codes,
                Params p) {
  constexpr int NACC = num_acc(TT);  // accumulators in TMEM
  constexpr uint32_t A_COL0 = ta_acol0(TT);
  constexpr bool SHARES = GATED && NACC == 1;  // the dequantisers help to finish tiles
  // dequantising warps per stage: TT = 256 alternates stages between two groups of four
  static_assert(CPS == 1 || (CPS == 2 && TT != BM), "two CTAs an SM: the 32-token form only");
  constexpr int DEQ_WARPS = deq_warps(TT, CPS), NG = DEQ_WARPS / 4;  // dequantiser groups
  constexpr int DEQ_PER_STAGE = 4;                                   // one group fills a stage
  static_assert(NG >= 1 && 4 % NG == 0, "groups take whole turns within a super-block");

  constexpr int PROW = p_row_bytes(FMT, BITS);
  constexpr int STAGES = stages(FMT, BITS, TT);
  constexpr uint32_t STAGE_TX = a_bytes(TT) + p_bytes(FMT, BITS);
  constexpr uint32_t TMEM_COLS = tmem_cols(TT);
  static_assert(NG < STAGES, "a group's step through the ring crosses its end at most once");
  static_assert(A_COL0 + STAGES * TA_ACOLS <= TMEM_COLS, "A ring beside the accumulators");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + off_bar(FMT, BITS, TT));
  uint32_t *tmem_holder =
      reinterpret_cast<uint32_t *>(bars + NUM_BARS_PER_STAGE * STAGES + NUM_BARS_FIXED + meta_bars(FMT));
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  auto bar_tma_full = [&](int s) { return smem_u32(bars + s); };
  auto bar_b_full = [&](int s) { return smem_u32(bars + STAGES + s); };
  auto bar_empty = [&](int s) { return smem_u32(bars + 2 * STAGES + s); };
  auto bar_acc_full = [&](int a) { return smem_u32(bars + 3 * STAGES + a); };
  auto bar_acc_empty = [&](int a) { return smem_u32(bars + 3 * STAGES + 2 + a); };
  const uint32_t bar_final = smem_u32(bars + 3 * STAGES + 4);
  auto bar_meta_full = [&](int s) { return smem_u32(bars + 3 * STAGES + 5 + s); };
  auto bar_meta_empty = [&](int s) { return smem_u32(bars + 3 * STAGES + 5 + MSLOTS + s); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t m_tiles = (p.M + TT - 1) / TT, n_tiles = GATED ? (p.N / 2 + GATED_F - 1) / GATED_F : (p.N + BN - 1) / BN;
  const int64_t num_tiles = m_tiles * n_tiles;
  const int num_kb = (int)(p.K / BK);
  const int64_t my_tiles = (num_tiles - blockIdx.x + gridDim.x - 1) / gridDim.x;
  const int64_t total_it = my_tiles * num_kb;  // k-stages this CTA runs, in order

  // (k-step, tile) of a stage, advanced one stage at a time
  struct Cursor {
    int kb;
    int64_t tile, n_tile, m_tile;
  };
  auto cursor0 = [&]() {
    Cursor c;
    c.kb = 0;
    c.tile = blockIdx.x;
    c.n_tile = c.tile / m_tiles;
    c.m_tile = c.tile - c.n_tile * m_tiles;
    return c;
  };
  auto advance = [&](Cursor &c) {
    if (++c.kb == num_kb) {
      c.kb = 0;
      c.tile += gridDim.x;
      c.n_tile = c.tile / m_tiles;
      c.m_tile = c.tile - c.n_tile * m_tiles;
    }
  };
  // slot and phase of a ring position, advanced one use at a time
  auto step_ring = [](int &slot, uint32_t &phase, int depth) {
    if (++slot == depth) {
      slot = 0;
      phase ^= 1u;
    }
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_tma_full(s), 1);
      mbar_init(bar_b_full(s), DEQ_PER_STAGE);
      mbar_init(bar_empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar_acc_full(a), 1);
      mbar_init(bar_acc_empty(a), SHARES && p.share_tiles ? 4 + DEQ_WARPS : 4);
    }
    mbar_init(bar_final, 1);
    if constexpr (FMT == FMT_INT4) {
      for (int s = 0; s < MSLOTS; ++s) {
        mbar_init(bar_meta_full(s), NUM_META_WARPS * 32);  // one cp.async arrival per copying thread
        mbar_init(bar_meta_empty(s), DEQ_WARPS);            // every dequantising warp, once a super-block
      }
    }
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
  // launched as a programmatic dependent of the weight-scale pass (which waits for the x pass): the
  // set-up above overlapped them; the workspace they write is read only from here on
  pdl_wait();

  if (warp == WARP_TMA) {
    if (lane == 0) {
      tma_prefetch_desc(&map_x);
      tma_prefetch_desc(&map_codes);
    }
    __syncwarp();
    int64_t it = 0;
    int s = 0;
    uint32_t ph = 0;
    Cursor cur = cursor0();
    bool ok = true;
    const int64_t n_it = copies_withheld() ? 0 : total_it;  // steps whose copies are started
    for (; it < n_it; ++it) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar_empty(s), ph ^ 1u, abort_flag))) {
        ok = false;
        break;
      }
      const uint32_t bar = bar_tma_full(s);
      mbar_expect_tx_elected(bar, STAGE_TX);
      // the tile's code rows: one box (gated: 64 gate rows and the 64 up rows of the same features)
      auto load_codes = [&](int off, int32_t x) {
        const uint32_t dst = sbase + off_p(FMT, BITS, TT, s) + off;
        if constexpr (GATED) tma_load_3d_elected(dst, &map_codes, bar, x, (int32_t)(cur.n_tile * GATED_F), 0);
        else tma_load_2d_elected(dst, &map_codes, bar, x, (int32_t)(cur.n_tile * BN));
      };
      if constexpr (FMT == FMT_INT6P) {  // k-step kb: low-plane bytes 32 (kb % 4) .. and high-plane
                                         // bytes 128 + 16 (kb % 4) .. of super-block kb / 4, by 16-byte boxes
        const int32_t x0 = 192 * (cur.kb >> 2) + 32 * (cur.kb & 3), xh = 192 * (cur.kb >> 2) + 128 + 16 * (cur.kb & 3);
        load_codes(0, x0);
        load_codes(16 * BN, x0 + 16);
        load_codes(32 * BN, xh);
      } else {
        load_codes(0, cur.kb * PROW);
      }
      tma_load_2d_elected(sbase + off_a(TT, s), &map_x, bar, cur.kb * BK, (int32_t)(cur.m_tile * TT));
      step_ring(s, ph, STAGES);
      advance(cur);
    }
    if (!ok) {  // let copies already issued land before the CTA can exit
      for (int64_t j = it - 1; j >= 0 && j >= it - STAGES; --j) {
        const long long t0 = clock64();
        while (!mbar_try_wait(bar_tma_full((int)(j % STAGES)), (uint32_t)((j / STAGES) & 1)) &&
               clock64() - t0 < QL_WAIT_LIMIT_CYCLES) {
        }
      }
    }
  } else if (warp == WARP_MMA) {
    // D[weight row][token] += W tile (A, M = 128) x x tile (B, N = TT).  This warp sets the kernel's pace, so
    // its loop is unrolled over the ring's slots (slot j's x-tile descriptor and A columns are compile-time
    // offsets from slot 0's, and the phase flips once a ring cycle), and all of it runs the loop, one elected
    // lane issuing (see umma_stage_tmem_a).
    constexpr uint32_t idesc = umma_idesc_f16_f32(BN, TT);
    constexpr uint32_t XDESC_STEP = (uint32_t)(a_bytes(TT) >> 4);  // descriptor address units
    const uint64_t xdesc0 = umma_desc_k_sw128(sbase + off_a(TT, 0));
    const uint32_t a_tmem0 = tmem_base + A_COL0;
    int64_t tcount = 0, tile = blockIdx.x;
    int kb = 0;  // stage within the current tile
    uint32_t ph = 0, d_tmem = tmem_base;
    bool ok = true, issued = false;
    // start a tile: its accumulator must have been drained (bounded wait)
    auto begin_tile = [&]() {
      const int a = (int)(tcount % NACC);
      const uint32_t ause = (uint32_t)(tcount / NACC);
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar_acc_empty(a), (ause & 1) ^ 1, abort_flag))) return false;
      tc_fence_after();
      d_tmem = tmem_base + (uint32_t)(a * TT);  // accumulator a: columns a * TT ..
      return true;
    };
    if (tile < num_tiles) ok = begin_tile();
    while (ok && tile < num_tiles) {
#pragma unroll
      for (int j = 0; j < STAGES; ++j) {
        if (!ok || tile >= num_tiles) break;
        // b_full alone: its arrivals come from dequantisers that waited for this stage's tma_full,
        // so the x tile has landed before the MMAs read it (and a copy that never lands ends their
        // wait, and so this one, by the abort flag)
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar_b_full(j), ph, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        umma_stage_tmem_a(d_tmem, a_tmem0 + (uint32_t)(j * TA_ACOLS), xdesc0 + (uint64_t)(j * XDESC_STEP), idesc,
                          kb != 0, bar_empty(j));
        issued = true;
        if (++kb == num_kb) {  // the tile's last stage
          kb = 0;
          umma_commit_elected(bar_acc_full((int)(tcount % NACC)));
          tile += gridDim.x;
          ++tcount;
          if (tile < num_tiles) ok = begin_tile();
        }
      }
      ph ^= 1u;
    }
    if (issued) {  // all MMAs retired before teardown
      umma_commit_elected(bar_final);
      const long long t0 = clock64();
      while (!mbar_try_wait(bar_final, 0) && clock64() - t0 < QL_WAIT_LIMIT_CYCLES) {
      }
    }
  } else if (warp >= WARP_META0 && warp < WARP_META0 + NUM_META_WARPS) {
    if constexpr (FMT == FMT_INT4) {
      // for every super-block, each tile row's 16 bytes of group words and its step word, up to
      // MSLOTS super-blocks ahead of the dequantisers
      const int t = threadIdx.x - WARP_META0 * 32;  // 0..63: rows t and t + 64
      int ms = 0;
      uint32_t phm = 0;
      Cursor cur = cursor0();
      for (int64_t it = 0; it < total_it; it += 4) {
        if (!mbar_wait_bounded(bar_meta_empty(ms), phm ^ 1u, abort_flag)) break;
        const uint32_t dst = sbase + off_meta(FMT, BITS, TT, ms);
#pragma unroll
        for (int i = 0; i < BN / 64; ++i) {
          const int r = t + 64 * i;
          const int64_t n = layer_row<GATED>(cur.n_tile, r, p.N);
          const bool valid = n < p.N;
          const int64_t nn = valid ? n : p.N - 1;
          cp_async16(dst + r * 16, p.gmeta + nn * (p.K / 16) + 16 * (cur.kb >> 2), valid);
          cp_async4(dst + BN * 16 + r * 4, p.steps + 4 * (nn * (p.K / 256) + (cur.kb >> 2)), valid);
        }
        cp_async_arrive_noinc(bar_meta_full(ms));
        step_ring(ms, phm, MSLOTS);
        for (int j = 0; j < 4; ++j) advance(cur);
      }
      cp_async_wait_all();  // no copy may land after the CTA is gone
    }
  } else if (warp >= WARP_EPI0 && warp < WARP_EPI0 + 4) {
    // lane = weight row n of the tile (TMEM lane 32 e + lane); its TT columns = the tile's tokens
    const int e = warp - WARP_EPI0;  // TMEM lane quarter
    int64_t tcount = 0;
    if constexpr (GATED) {
      // Two accumulators (TT = 32): the next tile's MMAs run beside the epilogue.  One (TT = 256): they can
      // only start once it has been read, and act and the rounding to 8 bits take longer than the reading,
      // so a tile is first moved as it is to this CTA's scratch (in L2) and finished from there beside the
      // next tile's MMAs; each thread reads back what it wrote itself.  Nothing follows the last tile, so it is
      // finished from tensor memory, by the dequantisers too; and so is every tile while K is short (share_tiles:
      // the next tile's stages then take less time than the two thirds of this one's elements that they take over).
      float4 *scratch = p.scratch + (int64_t)blockIdx.x * (BN * TT / 4) + 32 * e + lane;
      for (int64_t tile = blockIdx.x; tile < num_tiles; tile += gridDim.x, ++tcount) {
        const int64_t n_tile = tile / m_tiles, m_tile = tile - n_tile * m_tiles;
        const int a = (int)(tcount % NACC);
        const bool moved = NACC == 1 && !p.share_tiles && tile + gridDim.x < num_tiles;
        const bool shared_out = NACC == 1 && !moved;
        const GatedRow row(p, n_tile, m_tile, TT, e, lane, gated_down<FMT, BITS>());
        if (!mbar_wait_suspend(bar_acc_full(a), (uint32_t)(tcount / NACC) & 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t t_acc = tmem_base + ((uint32_t)(32 * e) << 16) + (uint32_t)(a * TT);
        if (moved) {
#pragma unroll 1
          for (int c = 0; c < row.chunks; c += 4) {  // (columns past the tokens are moved too, within the tile)
            uint32_t r[2][32];
            tmem_ld_32x32b_x32(t_acc + 16 * c, r[0]);
            tmem_ld_32x32b_x32(t_acc + 16 * c + 32, r[1]);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint32_t *v = r[j >> 3] + 4 * (j & 7);
              scratch[(4 * c + j) * BN] = make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]),
                                                      __uint_as_float(v[2]), __uint_as_float(v[3]));
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_acc_empty(a));
          float4 next[4];  // the chunk after, on its way
          ChunkExp xe;
          xe.load(p, row, 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) next[j] = scratch[j * BN];
#pragma unroll 1
          for (int c = 0; c < row.chunks; ++c) {
            uint32_t r[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              r[4 * j] = __float_as_uint(next[j].x);
              r[4 * j + 1] = __float_as_uint(next[j].y);
              r[4 * j + 2] = __float_as_uint(next[j].z);
              r[4 * j + 3] = __float_as_uint(next[j].w);
            }
            const ChunkExp cur = xe;
            if (c + 1 < row.chunks) {
              xe.load(p, row, c + 1);
#pragma unroll
              for (int j = 0; j < 4; ++j) next[j] = scratch[(4 * (c + 1) + j) * BN];
            }
            gated_chunk(p, row, r, cur, c, lane);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < row.chunks; c += shared_out ? 1 + NG : 1) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(t_acc + 16 * c, r);
            ChunkExp xe;
            xe.load(p, row, c);
            tmem_ld_wait();
            gated_chunk(p, row, r, xe, c, lane);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_acc_empty(a));
        }
      }
    }
    for (int64_t tile = GATED ? num_tiles : blockIdx.x; tile < num_tiles; tile += gridDim.x, ++tcount) {
      const int64_t n_tile = tile / m_tiles, m_tile = tile - n_tile * m_tiles;
      const int a = (int)(tcount % NACC);
      const uint32_t ause = (uint32_t)(tcount / NACC);
      // the tile's scale exponents and bias, loaded while its MMAs run: lane l holds the exponents of
      // tokens l, l + 32, .. (a load per column chunk would put an L2 round trip between the chunks)
      const int64_t n = n_tile * BN + 32 * e + lane;
      const int we = n < p.N ? p.ws.wexp[n] : 0;
      const float bn = (p.bias && n < p.N) ? __bfloat162float(p.bias[n]) : 0.f;
      // (each exponent lies in [-126, 126], so one signed byte holds it: a chunk's 16 are one broadcast
      // 16-byte load from this warp's own copy, which no other warp touches)
      int8_t *xe_s = reinterpret_cast<int8_t *>(smem + off_xe(FMT, BITS, TT)) + TT * e;
      int xe_lo = 1 << 20, xe_hi = -(1 << 20);
      __syncwarp();  // every lane is done with the previous tile's copy
#pragma unroll
      for (int j = 0; j < TT / 32; ++j) {
        const int64_t m = m_tile * TT + 32 * j + lane;
        const int xe = m < p.M ? p.ws.xexp[m] : 0;
        xe_s[32 * j + lane] = (int8_t)xe;
        xe_lo = min(xe_lo, xe);
        xe_hi = max(xe_hi, xe);
      }
      __syncwarp();
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        xe_lo = min(xe_lo, __shfl_xor_sync(0xffffffffu, xe_lo, o));
        xe_hi = max(xe_hi, __shfl_xor_sync(0xffffffffu, xe_hi, o));
      }
      // every exponent sum of the warp's rows and the tile's tokens is that of a normal float: then
      // D * 2^e is one multiplication by 2^e built from its bits, the same single rounding as mul_pow2
      const bool one_mul = __all_sync(0xffffffffu, xe_lo + we >= -126 && xe_hi + we <= 127);
      const int w_bits = we * (1 << 23) + 0x3F800000;  // bits of 2^(xe + we) = xe * 2^23 + w_bits
      if (!mbar_wait_bounded(bar_acc_full(a), ause & 1, abort_flag)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < TT / 16; ++c) {  // 16 tokens at a time
        uint32_t r[16];
        tmem_ld_32x32b_x16(tmem_base + ((uint32_t)(32 * e) << 16) + (uint32_t)(a * TT + 16 * c), r);
        tmem_ld_wait();
        if (c == TT / 16 - 1) {  // the accumulator is in registers: the next tile's MMAs may start
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_acc_empty(a));
        }
        const int64_t m0 = m_tile * TT + 16 * c;
        const uint4 xv = *reinterpret_cast<const uint4 *>(xe_s + 16 * c);  // tokens 16c .. 16c + 15
        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
        // y = D * 2^-(a_m + b_n) (exponents added first), + bias, one rounding
        if (one_mul) {
#pragma unroll
          for (int t = 0; t < 16; ++t) {
            const int xe = (int)(int8_t)(xw[t >> 2] >> (8 * (t & 3)));
            r[t] = __float_as_uint(__fmul_rn(__uint_as_float(r[t]), __int_as_float(xe * (1 << 23) + w_bits)) + bn);
          }
        } else {
#pragma unroll
          for (int t = 0; t < 16; ++t) {
            const int xe = (int)(int8_t)(xw[t >> 2] >> (8 * (t & 3)));
            r[t] = __float_as_uint(mul_pow2(__uint_as_float(r[t]), xe + we) + bn);
          }
        }
        if (n < p.N) {  // token t of row n: the warp's 32 rows are 64 contiguous bytes of y's row m0 + t
          __nv_bfloat16 *dst = p.y + m0 * p.N + n;
          const int64_t rows_left = p.M - m0;
#pragma unroll
          for (int t = 0; t < 16; ++t) {
            if (t < rows_left) *dst = __float2bfloat16_rn(__uint_as_float(r[t]));
            dst += p.N;
          }
        }
      }
    }
  } else if (warp >= WARP_DEQ0) {
    auto row_scale = [&](int64_t n) { return n < p.N ? p.ws.wsc[n] : 0.f; };
    // Stages go round the NG groups of four warps (warps 8-11 take stages 0, NG, 2 NG, ..., warps
    // 12-15 stages 1, NG + 1, ...).  A thread fills one whole tile row (64 weights, both 32-weight
    // chunks) of its stage into TMEM lane r = its warp's lane quarter + lane, columns A_COL0 + 32 s ..:
    // the A operand of that stage's MMAs.
    const int wd = warp - WARP_DEQ0;     // 0 .. DEQ_WARPS - 1
    const int g = wd >> 2;               // stages it = g, g + NG, ...
    const int r = 32 * (wd & 3) + lane;  // lane of the tile
    const int br = box_row<GATED>(r);    // its row in the code box and the metadata slots
    auto row_of = [&](int64_t n_tile) { return layer_row<GATED>(n_tile, br, p.N); };
    const uint32_t t_row = tmem_base + ((uint32_t)(32 * (wd & 3)) << 16) + A_COL0;
    auto step_ng = [](int &slot, uint32_t &phase, int depth) {
      slot += NG;
      if (slot >= depth) {
        slot -= depth;
        phase ^= 1u;
      }
    };
    Cursor cur = cursor0();
    for (int j = 0; j < g; ++j) advance(cur);
    int s = g, ms = 0;  // every group visits every super-block's slot
    uint32_t ph = 0, phm = 0;
    uint32_t gm[2] = {0, 0}, st[2] = {0, 0};
    float sc = 0.f;
    if (g < total_it) {
      if constexpr (FMT != FMT_INT4) {
        load_meta<FMT>(p, row_of(cur.n_tile), (int64_t)cur.kb * 2, gm[0], st[0]);
        load_meta<FMT>(p, row_of(cur.n_tile), (int64_t)cur.kb * 2 + 1, gm[1], st[1]);
      }
      sc = row_scale(row_of(cur.n_tile));
    }
    // SHARES: once it is done with a tile's stages, a group finishes its chunks (1 + g, 2 + NG + g, ..) of the tile; the
    // turn behind the last stage is for the last tile.
    int64_t done = 0, tile_end = num_kb;  // tiles whose stages this group is done with; the end of the next
    const int64_t end_it = SHARES ? total_it + NG : total_it;
    for (int64_t it = g; it < end_it; it += NG) {
      if constexpr (SHARES) {
        bool ok = true;
        for (; ok && done < my_tiles && it >= tile_end; ++done, tile_end += num_kb) {
          if (!p.share_tiles && done + 1 < my_tiles) continue;
          const int64_t tile = blockIdx.x + done * gridDim.x, n_tile = tile / m_tiles;
          const GatedRow row(p, n_tile, tile - n_tile * m_tiles, TT, wd & 3, lane, gated_down<FMT, BITS>());
          ok = __all_sync(0xffffffffu, mbar_wait_suspend(bar_acc_full(0), (uint32_t)done & 1, abort_flag));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 1 + g; c < row.chunks; c += 1 + NG) {
            uint32_t r16[16];
            tmem_ld_32x32b_x16(tmem_base + ((uint32_t)(32 * (wd & 3)) << 16) + 16 * c, r16);
            ChunkExp xe;
            xe.load(p, row, c);
            tmem_ld_wait();
            gated_chunk(p, row, r16, xe, c, lane);
          }
          tc_fence_before();
          __syncwarp();
          if (p.share_tiles && lane == 0) mbar_arrive(bar_acc_empty(0));
        }
        if (!ok || it >= total_it) break;
      }
      Cursor nx = cur;  // this group's next stage
      for (int j = 0; j < NG; ++j) advance(nx);
      uint32_t ngm[2] = {0, 0}, nst[2] = {0, 0};
      float nsc = sc;
      if (it + NG < total_it) {  // its metadata (int6, affine) and row scale, loaded ahead
        const int64_t n = row_of(nx.n_tile);
        if constexpr (FMT != FMT_INT4) {
          load_meta<FMT>(p, n, (int64_t)nx.kb * 2, ngm[0], nst[0]);
          load_meta<FMT>(p, n, (int64_t)nx.kb * 2 + 1, ngm[1], nst[1]);
        }
        if (nx.n_tile != cur.n_tile) nsc = row_scale(n);
      }
      if constexpr (FMT == FMT_INT4) {  // this stage's group and step words, from the metadata ring
        const int q = (int)(it & 3);  // stage of the super-block: this group sees q = g, g + NG, ..
        if (q == g && !__all_sync(0xffffffffu, mbar_wait_bounded(bar_meta_full(ms), phm, abort_flag))) break;
        const uint8_t *slot = smem + off_meta(FMT, BITS, TT, ms);
        const uint32_t w = *reinterpret_cast<const uint32_t *>(slot + br * 16 + 4 * q);
        gm[0] = w & 0xffffu;
        gm[1] = w >> 16;
        st[0] = st[1] = *reinterpret_cast<const uint32_t *>(slot + BN * 16 + br * 4);
        if (q == g + 4 - NG) {  // this group's last stage of the super-block: release the slot
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_meta_empty(ms));
          step_ring(ms, phm, MSLOTS);
        }
      }
      // the codes have landed, and the MMAs that last read this A stage have completed (they
      // released the stage before TMA refilled it).  Where the ring is not a whole number of group turns, the
      // stage's previous use was another group's: this group did not see it land, copies may land out of turn,
      // and a wait by parity is only right once that phase is over, so the release is tested first (both
      // tests are on their way together: one after the other cost 1-5 % of the kernel).
      bool landed;
      if constexpr (STAGES % NG != 0) {
        const bool released = mbar_try_wait(bar_empty(s), ph ^ 1u);
        landed = mbar_try_wait(bar_tma_full(s), ph);
        if (!(released && landed))
          landed = mbar_wait_bounded(bar_empty(s), ph ^ 1u, abort_flag) && mbar_wait_bounded(bar_tma_full(s), ph, abort_flag);
      } else {
        landed = mbar_wait_bounded(bar_tma_full(s), ph, abort_flag);
      }
      if (!__all_sync(0xffffffffu, landed)) break;
      tc_fence_after();
      const uint8_t *prow = smem + off_p(FMT, BITS, TT, s) + br * PROW;
      uint32_t o[32];
      auto to_f16 = [&](const uint32_t(&cw)[code_bits(FMT, BITS)], const uint8_t *src, const uint8_t *src_hi,
                        uint32_t g1, uint32_t s1, uint32_t(&out)[16]) {
        if constexpr (GATED) gated_chunk_to_f16<FMT, BITS>(cw, src, src_hi, g1, s1, sc, out);
        else chunk_to_f16<FMT, BITS>(cw, src, src_hi, g1, s1, sc, out);
      };
      if constexpr (PROW == 32 && (FMT == FMT_INT4 || FMT == FMT_AFFINE)) {
        // the row's two 16-byte chunks, read in the order (h ^ bit 2 of the row) so that the 32 lanes'
        // first reads cover all 32 banks in four wavefronts (rows are 32 bytes apart)
        const int sw = (br >> 2) & 1;
        const uint4 va = reinterpret_cast<const uint4 *>(prow)[sw];
        const uint4 vb = reinterpret_cast<const uint4 *>(prow)[sw ^ 1];
        const uint4 c0 = sw ? vb : va, c1 = sw ? va : vb;
        const uint32_t cw0[4] = {c0.x, c0.y, c0.z, c0.w}, cw1[4] = {c1.x, c1.y, c1.z, c1.w};
        uint32_t o0[16], o1[16];
        to_f16(cw0, nullptr, nullptr, gm[0], st[0], o0);
        to_f16(cw1, nullptr, nullptr, gm[1], st[1], o1);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          o[i] = o0[i];
          o[16 + i] = o1[i];
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t *src = prow + h * (PROW / 2);
          const uint8_t *src_hi = nullptr;
          if constexpr (FMT == FMT_INT6P) {
            src = smem + off_p(FMT, BITS, TT, s) + h * 16 * BN + br * 16;
            src_hi = smem + off_p(FMT, BITS, TT, s) + 32 * BN + br * 16 + 8 * h;
          }
          uint32_t cw[code_bits(FMT, BITS)];
          if constexpr (FMT == FMT_INT4 || FMT == FMT_AFFINE) load_code_words<FMT, BITS>(src, cw);
          uint32_t oh[16];
          to_f16(cw, src, src_hi, gm[h], st[h], oh);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[16 * h + i] = oh[i];
        }
      }
      tmem_st_32x32b_x32(t_row + (uint32_t)s * TA_ACOLS, o);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_b_full(s));
      step_ng(s, ph, STAGES);
      cur = nx;
      sc = nsc;
      gm[0] = ngm[0];
      gm[1] = ngm[1];
      st[0] = nst[0];
      st[1] = nst[1];
    }
  }

  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

}  // namespace gemm
}  // namespace ql
