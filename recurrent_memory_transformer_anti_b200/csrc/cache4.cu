// Writing rows into the 4-bit key/value cache, and reading them back (layout and arithmetic:
// cache4.cuh). Both stream. Writing, a thread holds the 16 channels of one scale, so a block's maximum
// needs no other lane and a scale is worked out once (8 channels a thread and an exchange between two: 45 us
// for the write and read of the 153 MB below instead of 37); reading, it holds 8 channels, 16 bytes
// of bf16, so that each store of a warp fills whole sectors (16 channels: 33.0 us instead of 26.5 for 136 MB).
// A warp takes four neighbouring heads of its tokens where there are warps enough: their loads in flight
// together, their tokens' pages looked up once, and one address for all, the rest being constants.
//
// Bound by HBM if the arithmetic stays at about 5 instructions a channel: a bf16 channel is rounded in
// half a packed operation twice (encode_short), read in one and a half (decode8), and places are found
// without a division. Blocks with a NaN, a saturating value or a scale below 2^-14, and fp32, take the
// general way (encode_value). bf16 rows of 8 heads: 67 MB into 19 MB of codes and scales take 15.8 us
// (5.4 TB/s), 30 MB into 106 MB 25.4 us (5.4 TB/s). What is left is the chain of three loads (length, page,
// codes) at the head of each wave of CTAs. fp32 rows, 134 MB and 19 MB of codes and scales: written in 50 us
// (3.1 TB/s: every block the general way, and 16 bytes a lane at a stride of 64), read in 39 us (3.9 TB/s: a
// lane's 32 bytes are two stores at a stride of 32, so that each of a warp's stores fills half sectors).
#include "cache4.cuh"
#include "launch.h"

namespace rmt {
namespace {

using cache4::kPage;

constexpr uint32_t kWarps = 8;  // of a CTA

// n / d of numbers below 2^31: (n * m) >> s, m = 2^s / d rounded up and below 2^32 + 1, so that what
// rounding adds, n / 2^s at most, does not reach the next integer.
struct Divider {
  uint32_t m;
  int s;
  explicit Divider(uint32_t d) : s(31) {
    while ((uint64_t(1) << (s - 31)) < d) ++s;
    m = static_cast<uint32_t>(((uint64_t(1) << s) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> s);
  }
};

// What a launch adds to its arguments: a warp's columns are COLS neighbouring heads of keys or of values,
// `cols` such ranges for both, and `warps` of them in all.
struct Deal {
  uint32_t cols, warps;
  Divider by_cols, by_m;
};

// Where this thread's token is: its row of k and v, and the table's page for it.
struct Spot {
  bool on;
  size_t row;
  int page, in_page;
};

// CH: channels of a thread
template <int DH, int CH>
__device__ __forceinline__ Spot find_spot(const CacheRowsArgs& a, const Deal& d, uint32_t group) {
  constexpr uint32_t LANES = DH / CH, TOK = 32 / LANES;
  Spot s{};
  const uint32_t row = group * TOK + (threadIdx.x & 31u) / LANES;
  if (row >= static_cast<uint32_t>(a.c.n_seqs) * a.M) return s;
  const uint32_t b = d.by_m(row), i = row - b * a.M;
  const int n = a.n_new ? min(__ldg(a.n_new + b), a.M) : a.M;
  const int pos = __ldg(a.c.lens + b) - n + static_cast<int>(i);
  if (static_cast<int>(i) >= n || pos < 0) return s;  // past the sequence's new rows, or of an empty slot
  s.on = true;
  s.row = row;
  s.page = cache4::table_entry(a.c, b, pos);
  s.in_page = pos % kPage;
  return s;
}

// 16 consecutive values of a row, as loaded
template <typename T>
struct Raw {
  uint4 v[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Raw<T> load16(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) r.v[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  return r;
}

// Their scale byte and codes
__device__ __forceinline__ uint32_t encode_general(float (&x)[16], uint32_t& lo, uint32_t& hi) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    x[i] = x[i] == x[i] ? x[i] : 0.f;
    amax = fmaxf(amax, fabsf(x[i]));
  }
  const uint32_t sb = cache4::encode_scale(amax);
  lo = hi = 0x88888888u;  // a block of zeros
  if (sb) {
    const float sc = cache4::decode_scale(sb), rs = 1.f / sc;
    lo = hi = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo |= cache4::encode_value(x[i], sc, rs) << (4 * i);
      hi |= cache4::encode_value(x[8 + i], sc, rs) << (4 * i);
    }
  }
  return sb;
}
__device__ __forceinline__ uint32_t encode16(const Raw<float>& r, uint32_t& lo, uint32_t& hi) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[4 * i] = __uint_as_float(r.v[i].x), x[4 * i + 1] = __uint_as_float(r.v[i].y);
    x[4 * i + 2] = __uint_as_float(r.v[i].z), x[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
  return encode_general(x, lo, hi);
}
__device__ __forceinline__ uint32_t encode16(const Raw<__nv_bfloat16>& r, uint32_t& lo, uint32_t& hi) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
  __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]));
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
  const float amax = __bfloat162float(__hmax_nan(m.x, m.y));
  uint32_t u[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    u[2 * i] = w[i] << 16;
    u[2 * i + 1] = w[i] & 0xFFFF0000u;
  }
  // short way: scales from 2^-14 on (within 1/16 of max / 7, so quotients stay below 7.5), no
  // saturation, no NaN
  if (!(amax >= 7.f * 6.103515625e-05f && amax <= cache4::kAmax)) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(u[i]);
    return encode_general(x, lo, hi);
  }
  const uint32_t sb = cache4::encode_scale_short(amax);
  float rs;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(cache4::decode_scale(sb)));  // off by one step at most
#pragma unroll
  for (int i = 0; i < 16; i += 2) cache4::encode_short(u[i], u[i + 1], rs);
  // low bytes: even channels, then odd ones in the high nibbles
  auto bytes = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  };
  lo = bytes(u[0], u[2], u[4], u[6]) + 16u * bytes(u[1], u[3], u[5], u[7]);
  hi = bytes(u[8], u[10], u[12], u[14]) + 16u * bytes(u[9], u[11], u[13], u[15]);
  return sb;
}

template <int DH, typename T, int COLS>
__global__ void __launch_bounds__(32 * kWarps) cache_write_kernel(const CacheRowsArgs a, const Deal d) {
  pdl_trigger();
  pdl_wait();
  using L = cache4::Layout<DH>;
  const uint32_t warp = blockIdx.x * kWarps + (threadIdx.x >> 5);  // the threads' numbers may pass 32 bits
  if (warp >= d.warps) return;
  const uint32_t group = d.by_cols(warp);
  uint32_t head = (warp - group * d.cols) * COLS;
  const bool value = head >= static_cast<uint32_t>(a.c.Hkv);
  if (value) head -= a.c.Hkv;
  const int blk = (threadIdx.x & 31) % (DH / cache4::kBlock);
  const Spot s = find_spot<DH, 16>(a, d, group);
  if (!s.on) return;
  // the rows' loads go out before the page's number is looked at
  const T* const src = static_cast<const T*>(value ? a.v : a.k) + s.row * a.ld + head * DH + blk * cache4::kBlock;
  Raw<T> raw[COLS];
#pragma unroll
  for (int c = 0; c < COLS; ++c) raw[c] = load16(src + c * DH);
  if (!cache4::page_ok(a.c, s.page)) return;
  unsigned char* const half =
      a.c.pages + cache4::block_offset<DH>(a.c, s.page, head) + (value ? L::V_OFF : 0);
  unsigned char* const codes = half + s.in_page * L::CODE_ROW + blk * 8;
  unsigned char* const scale = half + L::CODES + s.in_page * L::SCALE_ROW + blk;
#pragma unroll
  for (int c = 0; c < COLS; ++c) {
    uint32_t lo, hi;
    const uint32_t sb = encode16(raw[c], lo, hi);
    *reinterpret_cast<uint2*>(codes + c * L::BLOCK) = make_uint2(lo, hi);
    scale[c * L::BLOCK] = static_cast<unsigned char>(sb);
  }
}

// 8 channels from their codes and scale byte. A nibble or-ed into the pattern of a power of two is that
// plus q + 8; less that and 8, times the scale: exact.
__device__ __forceinline__ void decode8(float* dst, uint32_t w, uint32_t sb) {
  const float sc = cache4::decode_scale(sb), less = -8388616.f * sc;  // exact: (2^20 + 1) * 15 < 2^24
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf(__uint_as_float(((w >> (4 * i)) & 15u) | 0x4B000000u), sc, less);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    __stcs(reinterpret_cast<float4*>(dst) + i, make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
}
// In bf16: the bits 0..15 of a nibble are l * 2^-133, which times 2^120 less 8 * 2^-13 is q * 2^-13; the
// scale's byte, four bits up, is 2^-112 of the scale, which times 2^125 is 2^13 of it. All exact.
__device__ __forceinline__ void decode8(__nv_bfloat16* dst, uint32_t w, uint32_t sb) {
  auto pair = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
  const __nv_bfloat162 sc = __hmul2(pair(sb * 0x00100010u), pair(0x7E007E00u));  // 2^125
  const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  uint32_t v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // channels 2 j and 2 j + 1: byte j of each, in the low byte of a half
    uint32_t n;  // selectors with their top bit set fill a byte with the named byte's sign, here 0
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(n) : "r"(even), "r"(odd), "r"(0xC480u + 0x1111u * j));
    const __nv_bfloat162 q = __hmul2(__hfma2(pair(n), pair(0x7B807B80u), pair(0xBA80BA80u)), sc);
    v[j] = *reinterpret_cast<const uint32_t*>(&q);
  }
  __stcs(reinterpret_cast<uint4*>(dst), make_uint4(v[0], v[1], v[2], v[3]));
}

template <int DH, typename T, int COLS>
__global__ void __launch_bounds__(32 * kWarps) cache_read_kernel(const CacheRowsArgs a, const Deal d) {
  pdl_trigger();
  pdl_wait();
  using L = cache4::Layout<DH>;
  const uint32_t warp = blockIdx.x * kWarps + (threadIdx.x >> 5);  // the threads' numbers may pass 32 bits
  if (warp >= d.warps) return;
  const uint32_t group = d.by_cols(warp);
  uint32_t head = (warp - group * d.cols) * COLS;
  const bool value = head >= static_cast<uint32_t>(a.c.Hkv);
  if (value) head -= a.c.Hkv;
  const int part = (threadIdx.x & 31) % (DH / 8);
  const Spot s = find_spot<DH, 8>(a, d, group);
  if (!s.on || !cache4::page_ok(a.c, s.page)) return;
  const unsigned char* const half =
      a.c.pages + cache4::block_offset<DH>(a.c, s.page, head) + (value ? L::V_OFF : 0);
  const unsigned char* const codes = half + s.in_page * L::CODE_ROW + part * 4;
  const unsigned char* const scale = half + L::CODES + s.in_page * L::SCALE_ROW + part / 2;
  uint32_t w[COLS], sb[COLS];
#pragma unroll
  for (int c = 0; c < COLS; ++c) {
    w[c] = *reinterpret_cast<const uint32_t*>(codes + c * L::BLOCK);
    sb[c] = scale[c * L::BLOCK];
  }
  T* const dst = static_cast<T*>(value ? a.v : a.k) + s.row * a.ld + head * DH + part * 8;
#pragma unroll
  for (int c = 0; c < COLS; ++c) decode8(dst + c * DH, w[c], sb[c]);
}

template <int DH, typename T, int COLS>
cudaError_t launch_cols(const CacheRowsArgs& a, bool write, long long groups, cudaStream_t st) {
  const uint32_t cols = 2u * a.c.Hkv / COLS;
  const long long warps = groups * cols;
  if (warps > 0x7fffffffLL) return cudaErrorInvalidValue;  // Divider's range; the C entries let 2^30 through
  const long long blocks = (warps + kWarps - 1) / kWarps;
  const Deal d{cols, static_cast<uint32_t>(warps), Divider(cols), Divider(a.M)};
  const cudaError_t e = launch_pdl(write ? cache_write_kernel<DH, T, COLS> : cache_read_kernel<DH, T, COLS>,
                                   dim3(static_cast<unsigned>(blocks)), dim3(32 * kWarps), 0, st, a, d);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int DH, typename T>
cudaError_t launch_rows(const CacheRowsArgs& a, bool write, cudaStream_t st) {
  const int TOK = 32 / (DH / (write ? 16 : 8));  // tokens of a warp
  const long long groups = (static_cast<long long>(a.c.n_seqs) * a.M + TOK - 1) / TOK;
  // Four (or two) heads a warp once that leaves every SM 16 warps. With 8 heads of 64 in bf16, of
  // four heads and of one: a write of 4096 tokens (14 warps an SM with four) takes 4.1 and 3.7 us, of 8192 4.7 and
  // 5.5; a read of 512 (4 warps) 2.25 and 2.05, of 4096 (28 warps) 3.7 and 4.1, of 65,536 27 and 43.
  const long long enough = 148 * 16;
  if (a.c.Hkv % 4 == 0 && groups * 2 * a.c.Hkv / 4 >= enough) return launch_cols<DH, T, 4>(a, write, groups, st);
  if (a.c.Hkv % 2 == 0 && groups * 2 * a.c.Hkv / 2 >= enough) return launch_cols<DH, T, 2>(a, write, groups, st);
  return launch_cols<DH, T, 1>(a, write, groups, st);
}

cudaError_t launch_any(const CacheRowsArgs& a, int dh, bool bf16, bool write, cudaStream_t st) {
  switch (dh) {
    case 32: return bf16 ? launch_rows<32, __nv_bfloat16>(a, write, st) : launch_rows<32, float>(a, write, st);
    case 64: return bf16 ? launch_rows<64, __nv_bfloat16>(a, write, st) : launch_rows<64, float>(a, write, st);
    case 128: return bf16 ? launch_rows<128, __nv_bfloat16>(a, write, st) : launch_rows<128, float>(a, write, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_cache_write(const CacheRowsArgs& a, int dh, bool bf16, cudaStream_t st) {
  return launch_any(a, dh, bf16, true, st);
}
cudaError_t launch_cache_read(const CacheRowsArgs& a, int dh, bool bf16, cudaStream_t st) {
  return launch_any(a, dh, bf16, false, st);
}

}  // namespace rmt
