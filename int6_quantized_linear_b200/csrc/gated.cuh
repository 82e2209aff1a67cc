// gated.cuh -- the elementwise parts of a gated feed-forward block, and activations held in 8 bits.
//
//   forward    h = act(g) u
//   backward   dg = dh u act'(g),  du = dh act(g)
//
// 8-bit form of an activation row (qlinear_save8): groups of 16 values along the row share one
// power-of-two scale.  With top the group's largest magnitude, the scale 2^(E - 127) is the smallest
// power of two for which rint(top / scale) <= 127, so
//     key = (bits(top) + 2^16) >> 23      (the exponent, bumped when top rounds to 128 steps)
//     E = max(key - 6, 1),  code = rint(v 2^(127 - E)),  value = code 2^(E - 127).
// A power of two (rather than top / 127) makes the scaling exact, the exponent the only thing to
// reduce over a group, and every restored value exact in bf16 (seven significant bits); the up to
// one bit that it gives away is repaid by groups of 16, whose largest value is nearer the others than
// that of a longer group.  A group of values that are not all finite, or with one of at least
// 255/256 * 2^128 (bf16's largest, which would round to 2^128), gets E = 255 and is restored as NaN.
#pragma once
#include "formats.cuh"

namespace ql {

enum : int { ACT_SILU = 0, ACT_GELU_TANH = 1, ACT_GELU = 2 };

constexpr float GELU_C = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float GELU_B = 0.044715f;

// act(g) and act'(g).  exp and the reciprocal are the fast forms (a few 2^-23 off, the exponential |z| / 2^23 more
// for an argument z; a sigmoid below 2^-126 is 0); the results are rounded to bf16 or to an fp16 operand.
QL_DEVI float sigmoid_fast(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

QL_DEVI float act_value(int act, float g) {
  if (act == ACT_SILU) return g * sigmoid_fast(g);
  if (act == ACT_GELU_TANH) return g * sigmoid_fast(2.f * GELU_C * fmaf(GELU_B * g * g, g, g));  // (1 + tanh z) / 2
  return g * (0.5f * erfcf(g * -0.7071067811865476f));
}

QL_DEVI void act_grad(int act, float g, float &a, float &d) {
  if (act == ACT_SILU) {
    const float p = sigmoid_fast(g);
    a = g * p;
    d = p * fmaf(g, 1.f - p, 1.f);
  } else if (act == ACT_GELU_TANH) {
    const float g2 = g * g, p = sigmoid_fast(2.f * GELU_C * fmaf(GELU_B * g2, g, g));
    a = g * p;
    const float q = 2.f * p * (1.f - p);  // 0 where g^3 has left the range: the slope's other factor is not finite there
    d = q > 0.f ? fmaf(g * q, GELU_C * fmaf(3.f * GELU_B, g2, 1.f), p) : p;
  } else {
    const float p = 0.5f * erfcf(g * -0.7071067811865476f);
    a = g * p;
    d = fmaf(g * __expf(-0.5f * g * g), 0.3989422804014327f, p);  // 1 / sqrt(2 pi)
  }
}

// ---- 8-bit form ----------------------------------------------------------------------------------
constexpr int SAVE8_GROUP = 16;
__host__ __device__ constexpr int64_t save8_cols(int64_t cols) { return (cols + 15) / 16 * 16; }  // codes a row

QL_DEVI uint32_t save8_key(float v) {  // monotonic in |v|; 255: not finite
  return min((__float_as_uint(fabsf(v)) + 0x10000u) >> 23, 255u);
}
QL_DEVI uint32_t save8_exponent(uint32_t key) { return key == 255u ? 255u : max(key, 7u) - 6u; }
// 2^(127 - E) for E = 1 .. 249; 0 for E = 255 (the codes of such a group are 0)
QL_DEVI float save8_inverse(uint32_t E) { return E == 255u ? 0.f : __uint_as_float((254u - E) << 23); }
QL_DEVI int save8_code(float v, float inv) { return inv == 0.f ? 0 : __float2int_rn(v * inv); }
QL_DEVI float save8_scale(uint32_t E) { return E == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(E << 23); }

// Rows of whole groups (cols % 16 == 0): the rows follow each other without gaps, so group i of the
// matrix is values 16 i .. of x, codes 16 i .. and exponent i.  One thread a group: 32 bytes in, 17 out.
// The instructions a value are what bounds it (70 % of the issue slots with a conversion a value), so magnitudes
// are compared two at a time as their bf16 bits, and a code is the low byte of v / scale + 1.5 2^23 (which rounds).
__global__ void __launch_bounds__(256) save8_kernel(const __nv_bfloat16 *x, int64_t groups, int8_t *codes,
                                                    uint8_t *exps) {
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (i >= groups) return;
  const uint4 *src = reinterpret_cast<const uint4 *>(x) + 2 * i;
  const uint4 a = __ldcs(src), b = __ldcs(src + 1);  // read once: what L2 should keep is the codes
  const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t top = 0u;  // magnitudes order like their bits
#pragma unroll
  for (int j = 0; j < 8; ++j) top = __vmaxu2(top, u[j] & 0x7FFF7FFFu);
  top = max(top & 0xFFFFu, top >> 16);
  const uint32_t E = save8_exponent(save8_key(__uint_as_float(top << 16)));
  const float inv = save8_inverse(E);
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t c[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const uint32_t w = u[2 * j + (h >> 1)];
      c[h] = __float_as_uint(fmaf(__uint_as_float((h & 1) ? w & 0xffff0000u : w << 16), inv, 12582912.f));
    }
    o[j] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    if (E == 255u) o[j] = 0u;  // not finite
  }
  reinterpret_cast<uint4 *>(codes)[i] = make_uint4(o[0], o[1], o[2], o[3]);
  exps[i] = (uint8_t)E;
}

__global__ void __launch_bounds__(256) restore8_kernel(const int8_t *codes, const uint8_t *exps, int64_t groups,
                                                       __nv_bfloat16 *out) {
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (i >= groups) return;
  const uint4 c = __ldg(reinterpret_cast<const uint4 *>(codes) + i);
  const float s = save8_scale(__ldg(exps + i));
  const uint32_t u[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    o[2 * j] = pack_bf16x2((float)(int8_t)u[j] * s, (float)(int8_t)(u[j] >> 8) * s);
    o[2 * j + 1] = pack_bf16x2((float)(int8_t)(u[j] >> 16) * s, (float)(int8_t)(u[j] >> 24) * s);
  }
  uint4 *dst = reinterpret_cast<uint4 *>(out) + 2 * i;
  __stcs(dst, make_uint4(o[0], o[1], o[2], o[3]));
  __stcs(dst + 1, make_uint4(o[4], o[5], o[6], o[7]));
}

// Rows of any length: their values start at any 2-byte boundary, so 16 lanes take a group, one value
// each (every lane stays for the shuffles).
__global__ void __launch_bounds__(256) save8_ragged_kernel(const __nv_bfloat16 *x, int64_t rows, int64_t cols,
                                                           int8_t *codes, uint8_t *exps) {
  const int64_t t = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;  // padded element
  const int64_t cp = save8_cols(cols), row = t / cp, c = t - row * cp;
  const bool live = row < rows;
  const float v = live && c < cols ? __bfloat162float(x[row * cols + c]) : 0.f;
  uint32_t key = save8_key(v);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
  if (!live) return;
  const uint32_t E = save8_exponent(key);
  codes[t] = (int8_t)save8_code(v, save8_inverse(E));
  if ((t & 15) == 0) exps[t >> 4] = (uint8_t)E;
}

__global__ void __launch_bounds__(256) restore8_ragged_kernel(const int8_t *codes, const uint8_t *exps, int64_t rows,
                                                              int64_t cols, __nv_bfloat16 *out) {
  const int64_t t = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  const int64_t cp = save8_cols(cols), row = t / cp, c = t - row * cp;
  if (row >= rows || c >= cols) return;
  out[row * cols + c] = __float2bfloat16_rn((float)codes[t] * save8_scale(exps[t >> 4]));
}

}  // namespace ql
