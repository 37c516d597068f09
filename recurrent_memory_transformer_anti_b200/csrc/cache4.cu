// Writing rows into the 4-bit key/value cache, and reading them back (layout and arithmetic:
// cache4.cuh). Both stream. Writing, a thread holds the 16 channels of one scale, so a block's maximum
// needs no other lane and a scale is worked out once (8 channels a thread and an exchange: 26 us instead
// of 22 for 67 MB of bf16); reading, it holds 8 channels, 16 bytes of bf16, so that each
// store of a warp fills whole sectors (16 channels a thread: 22 us instead of 15). A warp takes
// four (keys or values, head) columns of its tokens where there are warps enough, with their loads in
// flight together and the tokens' pages looked up once.
//
// Bound by HBM if the arithmetic stays at about 5 instructions a channel: a bf16 channel is
// rounded in two (encode_short); blocks with a NaN, a saturating value or a scale below 2^-14, and fp32,
// take the general way (encode_value).
#include "cache4.cuh"
#include "launch.h"

namespace rmt {
namespace {

using cache4::kPage;

// Where this thread's token is: its row of k and v, and its page.
struct Spot {
  bool on;
  size_t row;
  unsigned char* page;
  int in_page;
};

// CH: channels of a thread
template <int DH, int CH>
__device__ __forceinline__ Spot find_spot(const CacheRowsArgs& a, unsigned group) {
  constexpr unsigned LANES = DH / CH, TOK = 32 / LANES;
  Spot s{};
  const unsigned row = group * TOK + (threadIdx.x & 31u) / LANES;
  if (row >= static_cast<unsigned>(a.c.n_seqs) * a.M) return s;
  const unsigned b = row / static_cast<unsigned>(a.M), i = row - b * a.M;
  const int n = a.n_new ? min(__ldg(a.n_new + b), a.M) : a.M;
  const int pos = __ldg(a.c.lens + b) - n + static_cast<int>(i);
  if (static_cast<int>(i) >= n || pos < 0) return s;  // past the sequence's new rows, or of an empty slot
  const int page = cache4::page_of(a.c, b, pos);
  if (page < 0) return s;
  s.on = true;
  s.row = row;
  s.page = a.c.pages + cache4::block_offset<DH>(a.c, page, 0);
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
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  const uint32_t sb = cache4::encode_scale(amax);
  // short way: scales from 2^-14 on (within 1/16 of max / 7, so quotients stay below 7.5), no
  // saturation, no NaN
  if (!(amax <= cache4::kAmax) || sb < 8) return encode_general(x, lo, hi);
  const float rs = 1.f / cache4::decode_scale(sb);
  uint32_t u[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) u[i] = cache4::encode_short(x[i], rs);
  // low bytes: even channels, then odd ones in the high nibbles
  auto bytes = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  };
  lo = bytes(u[0], u[2], u[4], u[6]) + 16u * bytes(u[1], u[3], u[5], u[7]);
  hi = bytes(u[8], u[10], u[12], u[14]) + 16u * bytes(u[9], u[11], u[13], u[15]);
  return sb;
}

// Columns col .. col + COLS - 1 of a token group: keys of heads 0 .. Hkv - 1, then values.
template <int DH, typename T, int COLS>
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheRowsArgs a, unsigned cols, unsigned warps) {
  pdl_trigger();
  pdl_wait();
  using L = cache4::Layout<DH>;
  const unsigned warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (warp >= warps) return;
  const unsigned group = warp / cols, col = (warp - group * cols) * COLS;
  const int blk = (threadIdx.x & 31) % (DH / cache4::kBlock);
  const Spot s = find_spot<DH, 16>(a, group);
  if (!s.on) return;
  Raw<T> raw[COLS];
#pragma unroll
  for (int c = 0; c < COLS; ++c) {
    const bool value = col + c >= static_cast<unsigned>(a.c.Hkv);
    const unsigned head = col + c - (value ? a.c.Hkv : 0);
    raw[c] = load16(static_cast<const T*>(value ? a.v : a.k) + s.row * a.ld + head * DH + blk * cache4::kBlock);
  }
#pragma unroll
  for (int c = 0; c < COLS; ++c) {
    const bool value = col + c >= static_cast<unsigned>(a.c.Hkv);
    const unsigned head = col + c - (value ? a.c.Hkv : 0);
    uint32_t lo, hi;
    const uint32_t sb = encode16(raw[c], lo, hi);
    unsigned char* half = s.page + static_cast<size_t>(head) * L::BLOCK + (value ? L::V_OFF : 0);
    *reinterpret_cast<uint2*>(half + s.in_page * L::CODE_ROW + blk * 8) = make_uint2(lo, hi);
    half[L::CODES + s.in_page * L::SCALE_ROW + blk] = static_cast<unsigned char>(sb);
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
__device__ __forceinline__ void decode8(__nv_bfloat16* dst, uint32_t w, uint32_t sb) {
  const __nv_bfloat162 sc = __float2bfloat162_rn(cache4::decode_scale(sb));  // 4 significant bits
  const __nv_bfloat162 less = __float2bfloat162_rn(-136.f);                  // 128 + 8
  uint32_t v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // channels j and j + 4
    const uint32_t n = ((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 q = __hmul2(__hadd2(*reinterpret_cast<const __nv_bfloat162*>(&n), less), sc);
    v[j] = *reinterpret_cast<const uint32_t*>(&q);
  }
  __stcs(reinterpret_cast<uint4*>(dst),
         make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                    __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632)));
}

template <int DH, typename T, int COLS>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheRowsArgs a, unsigned cols, unsigned warps) {
  pdl_trigger();
  pdl_wait();
  using L = cache4::Layout<DH>;
  const unsigned warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (warp >= warps) return;
  const unsigned group = warp / cols, col = (warp - group * cols) * COLS;
  const int part = (threadIdx.x & 31) % (DH / 8);
  const Spot s = find_spot<DH, 8>(a, group);
  if (!s.on) return;
  uint32_t w[COLS], sb[COLS];
#pragma unroll
  for (int c = 0; c < COLS; ++c) {
    const bool value = col + c >= static_cast<unsigned>(a.c.Hkv);
    const unsigned head = col + c - (value ? a.c.Hkv : 0);
    const unsigned char* half = s.page + static_cast<size_t>(head) * L::BLOCK + (value ? L::V_OFF : 0);
    w[c] = *reinterpret_cast<const uint32_t*>(half + s.in_page * L::CODE_ROW + part * 4);
    sb[c] = half[L::CODES + s.in_page * L::SCALE_ROW + part / 2];
  }
#pragma unroll
  for (int c = 0; c < COLS; ++c) {
    const bool value = col + c >= static_cast<unsigned>(a.c.Hkv);
    const unsigned head = col + c - (value ? a.c.Hkv : 0);
    decode8(static_cast<T*>(value ? a.v : a.k) + s.row * a.ld + head * DH + part * 8, w[c], sb[c]);
  }
}

template <int DH, typename T, int COLS>
cudaError_t launch_cols(const CacheRowsArgs& a, bool write, long long groups, cudaStream_t st) {
  const unsigned cols = 2u * a.c.Hkv / COLS;
  const long long blocks = (groups * cols + 7) / 8;
  if (blocks > 0x07ffffffLL) return cudaErrorInvalidValue;  // the threads' numbers are 32 bits
  const cudaError_t e = launch_pdl(write ? cache_write_kernel<DH, T, COLS> : cache_read_kernel<DH, T, COLS>,
                                   dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, a, cols,
                                   static_cast<unsigned>(groups * cols));
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int DH, typename T>
cudaError_t launch_rows(const CacheRowsArgs& a, bool write, cudaStream_t st) {
  const int TOK = 32 / (DH / (write ? 16 : 8));  // tokens of a warp
  const long long groups = (static_cast<long long>(a.c.n_seqs) * a.M + TOK - 1) / TOK;
  // four columns a warp once that leaves every SM its 64 warps
  if (a.c.Hkv % 2 == 0 && groups * 2 * a.c.Hkv / 4 >= 148 * 64) return launch_cols<DH, T, 4>(a, write, groups, st);
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
