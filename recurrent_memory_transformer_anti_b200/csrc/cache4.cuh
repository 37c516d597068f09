// The 4-bit key/value cache: page layout, and the arithmetic of its numbers.
//
// A page holds 64 tokens of every kv head. Per (page, kv head) there is one contiguous block of
// 72 dh bytes -- key codes [64][dh/2], key scales [64][dh/16], value codes, value scales -- so
// that one bulk copy brings all that attention needs of 64 tokens (2304, 4608 or 9216 bytes for
// dh of 32, 64 or 128).
//
// 16 consecutive channels x of a row share one scale s:
//   s = the u5.3 number nearest to max|x| / 7 (ties to even), at most 9216;
//   q = x / s rounded to the nearest integer (ties to even), clamped to -7..7;
// and the row stands for q * s. A u5.3 byte b (5 exponent bits, 3 mantissa bits, no sign) is the
// f16 with bits b << 7, so a scale becomes an MMA operand by one shift, with f16's range. q * s
// has at most 3 + 4 significant bits: exact in f16 and in bf16. Codes are held as q + 8.
// +-inf saturates to +-64512 (and takes its block's resolution); NaN is stored as 0.
#pragma once

#include "common.cuh"

namespace rmt {
namespace cache4 {

constexpr int kPage = 64;      // tokens per page
constexpr int kBlock = 16;     // channels per scale
constexpr float kAmax = 64512.f;  // 7 * 9216: the largest magnitude a block holds

template <int DH>
struct Layout {
  static constexpr int CODE_ROW = DH / 2, SCALE_ROW = DH / kBlock;
  static constexpr int CODES = kPage * CODE_ROW, SCALES = kPage * SCALE_ROW;
  static constexpr int V_OFF = CODES + SCALES;  // the value half has the key half's layout
  static constexpr int BLOCK = 2 * V_OFF;       // bytes of one (page, kv head)
};

// Everything a kernel needs to find a token: see rmt_cache in rmt.h.
struct CacheArgs {
  unsigned char* pages;
  const int* table;  // [n_seqs, max_pages]
  const int* lens;   // [n_seqs]
  int n_pages, n_seqs, max_pages, Hkv;
  int* err;
};

// Page of token `pos` of sequence b as the table has it, -1 for a position that does not fit it.
__device__ __forceinline__ int table_entry(const CacheArgs& c, int b, int pos) {
  const int slot = pos / kPage;
  return pos >= 0 && slot < c.max_pages ? __ldg(c.table + static_cast<size_t>(b) * c.max_pages + slot) : -1;
}
// Whether that is a page of the cache; if not, kErrPage goes to the error word, and the caller makes no access.
__device__ __forceinline__ bool page_ok(const CacheArgs& c, int page) {
  if (page >= 0 && page < c.n_pages) return true;
  if (c.err) atomicOr(c.err, kErrPage);
  return false;
}

template <int DH>
__device__ __forceinline__ size_t block_offset(const CacheArgs& c, int page, int head) {
  return (static_cast<size_t>(page) * c.Hkv + head) * Layout<DH>::BLOCK;
}

// Scale byte of a block whose largest finite magnitude is amax (>= 0; +inf allowed).
__device__ __forceinline__ uint32_t encode_scale(float amax) {
  amax = fminf(amax, kAmax);
  // amax / 7 rounded to odd: truncated, its last bit set when anything was cut off. Rounding that
  // to 4 bits gives the correctly rounded result (24 bits hold 4 + 2), with no false ties.
  float t = __fdiv_rz(amax, 7.f);
  if (fmaf(-t, 7.f, amax) != 0.f) t = __uint_as_float(__float_as_uint(t) | 1u);
  if (t < 6.103515625e-05f)  // below 2^-14: steps of 2^-17 (adding 1.5 * 2^6 leaves that step)
    return __float_as_uint(t + 96.f) - __float_as_uint(96.f);
  uint32_t u = __float_as_uint(t);
  u = (u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20;  // to 3 mantissa bits, ties to even
  return u - (112u << 3);                       // exponent bias 127 -> 15
}

__device__ __forceinline__ float decode_scale(uint32_t b) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(b << 7)));
}

// q + 8 for the value x (finite or infinite, not NaN) under scale s > 0, rs about 1 / s. The
// product x * rs may be an ulp off the quotient, which matters next to a tie only: the remainder
// x - q s is exact (q s has 7 significant bits), and settles it.
__device__ __forceinline__ uint32_t encode_value(float x, float s, float rs) {
  const float y = fminf(fmaxf(x * rs, -8.f), 8.f);
  float q = (y + 12582912.f) - 12582912.f;  // nearest integer (1.5 * 2^23)
  const float r = fmaf(-q, s, x), r2 = fabsf(r + r);
  const bool odd = static_cast<int>(q) & 1;
  if (r2 > s || (r2 == s && odd)) q += copysignf(1.f, r);
  q = fminf(fmaxf(q, -7.f), 7.f);
  return static_cast<uint32_t>(static_cast<int>(q) + 8);
}

// encode_scale for amax a bf16 in [7 * 2^-14, kAmax]. It has 8 significant bits, so amax / 7 is halfway
// between two scales or at least 2^-9 of its value off: the product with 1 / 7, two steps of 2^-23 off
// at most, rounded to 15 mantissa bits, is halfway when the quotient is.
__device__ __forceinline__ uint32_t encode_scale_short(float amax) {
  const uint32_t v = (__float_as_uint(amax * (1.f / 7.f)) + 0x80u) >> 8;
  return ((v + 0x7FFu + ((v >> 12) & 1u)) >> 12) - (112u << 3);
}

// encode_value for two bf16 x and a scale whose quotients stay below 7.5 in magnitude: q + 8 in the low byte.
// x and s have 8 and 4 significant bits, so x / s is a tie or at least 2^-12 off one: rounding
// x * rs, which is within 2^-18 of it (rs within 2^-22 of 1 / s), to steps of 2^-14 puts the ties back
// where they belong, and the second sum rounds to the nearest integer. Its constant is 1.5 * 2^23 + 8
// less the first's 1.5 * 2^9.
__device__ __forceinline__ void encode_short(uint32_t& x0, uint32_t& x1, float rs) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 z, {%4, %4};\n\tadd.rn.f32x2 x, x, z;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+r"(x0), "+r"(x1)
      : "f"(rs), "f"(768.f), "f"(12582152.f));
}

}  // namespace cache4

struct CacheRowsArgs {
  cache4::CacheArgs c;
  void* k;  // [n_seqs, M] rows of Hkv * dh values, rows ld elements apart
  void* v;
  long long ld;
  int M;
  const int* n_new;  // [n_seqs] or null (M)
};
cudaError_t launch_cache_write(const CacheRowsArgs& a, int dh, bool bf16, cudaStream_t st);
cudaError_t launch_cache_read(const CacheRowsArgs& a, int dh, bool bf16, cudaStream_t st);

struct CacheAttnArgs {
  cache4::CacheArgs c;
  const void* q;  // [n_seqs, n_q] rows of H * dh values, rows ldq elements apart
  long long ldq;
  void* out;      // [n_seqs, n_q, H * dh]
  int n_q, H, window, sinks;
  void* ws;
};
size_t cache_attention_workspace(int n_seqs, int max_pages, int n_q, int H, int Hkv, int dh, int window, int sinks);
cudaError_t launch_cache_attention(const CacheAttnArgs& a, int dh, bool bf16, cudaStream_t st);

struct WindowAttnArgs {
  const void* qkv;
  void* out;
  int G, M, H, Hkv;
  int window, sinks;  // window as an effective length >= 1
  const int* lens;    // [G] or null (M)
  int* err;
};
cudaError_t launch_window_attention(const WindowAttnArgs& a, int dh, bool bf16, cudaStream_t st);
cudaError_t launch_window_attention_tc(const WindowAttnArgs& a, int dh, cudaStream_t st);  // bf16, dh 64 or 128

}  // namespace rmt
