// Writing rows into the 4-bit key/value cache, and reading them back (layout and arithmetic:
// cache4.cuh). Both stream: one thread holds the 16 channels of one scale, so a block's maximum
// needs no other lane, and a warp covers 512 channels of one head's keys or values -- 16, 8 or 4
// tokens -- so that its codes and its scales each land in whole 32-byte sectors.
#include "cache4.cuh"
#include "launch.h"

namespace rmt {
namespace {

using cache4::kPage;

// 16 consecutive values of a row
__device__ __forceinline__ void load16(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = __ldcs(reinterpret_cast<const float4*>(p) + i);
    x[4 * i] = f.x, x[4 * i + 1] = f.y, x[4 * i + 2] = f.z, x[4 * i + 3] = f.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ void store16(float* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    __stcs(reinterpret_cast<float4*>(p) + i, make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    __stcs(reinterpret_cast<uint4*>(p) + i,
           make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                      pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7])));
}

// The 16 channels of this thread: which token, which of the head's blocks, where in the cache.
struct Spot {
  long long row;  // row of k, v; -1: nothing to do
  int head, blk;
  bool value;
  unsigned char* block;  // the (page, kv head) block
  int in_page;
};

template <int DH>
__device__ __forceinline__ Spot find_spot(const CacheRowsArgs& a) {
  constexpr int BLK = DH / cache4::kBlock, TOK = 32 / BLK;
  Spot s;
  const long long warp = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int cols = 2 * a.c.Hkv;  // (keys or values, head) of a group of tokens
  const long long group = warp / cols;
  const int col = static_cast<int>(warp - group * cols);
  s.value = col >= a.c.Hkv;
  s.head = col - (s.value ? a.c.Hkv : 0);
  s.blk = lane % BLK;
  s.row = group * TOK + lane / BLK;
  if (s.row >= static_cast<long long>(a.c.n_seqs) * a.M) {
    s.row = -1;
    return s;
  }
  const int b = static_cast<int>(s.row / a.M), i = static_cast<int>(s.row - static_cast<long long>(b) * a.M);
  const int n = a.n_new ? min(__ldg(a.n_new + b), a.M) : a.M;
  const int pos = __ldg(a.c.lens + b) - n + i;
  if (i >= n || pos < 0) {  // a row past the sequence's new ones, or of an empty slot
    s.row = -1;
    return s;
  }
  const int page = cache4::page_of(a.c, b, pos);
  if (page < 0) {
    s.row = -1;
    return s;
  }
  s.block = a.c.pages + cache4::block_offset<DH>(a.c, page, s.head);
  s.in_page = pos % kPage;
  return s;
}

template <int DH, typename T>
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheRowsArgs a) {
  pdl_trigger();
  pdl_wait();
  using L = cache4::Layout<DH>;
  const Spot s = find_spot<DH>(a);
  if (s.row < 0) return;
  const T* src = static_cast<const T*>(s.value ? a.v : a.k) + s.row * a.ld + s.head * DH + s.blk * cache4::kBlock;
  float x[16];
  load16(src, x);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    x[i] = x[i] == x[i] ? x[i] : 0.f;
    amax = fmaxf(amax, fabsf(x[i]));
  }
  const uint32_t sb = cache4::encode_scale(amax);
  uint32_t lo = 0x88888888u, hi = 0x88888888u;  // a block of zeros
  if (sb) {
    const float sc = cache4::decode_scale(sb), rs = 1.f / sc;
    lo = hi = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo |= cache4::encode_value(x[i], sc, rs) << (4 * i);
      hi |= cache4::encode_value(x[8 + i], sc, rs) << (4 * i);
    }
  }
  unsigned char* half = s.block + (s.value ? L::V_OFF : 0);
  *reinterpret_cast<uint2*>(half + s.in_page * L::CODE_ROW + s.blk * 8) = make_uint2(lo, hi);
  half[L::CODES + s.in_page * L::SCALE_ROW + s.blk] = static_cast<unsigned char>(sb);
}

template <int DH, typename T>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheRowsArgs a) {
  pdl_trigger();
  pdl_wait();
  using L = cache4::Layout<DH>;
  const Spot s = find_spot<DH>(a);
  if (s.row < 0) return;
  const unsigned char* half = s.block + (s.value ? L::V_OFF : 0);
  const uint2 w = *reinterpret_cast<const uint2*>(half + s.in_page * L::CODE_ROW + s.blk * 8);
  const float sc = cache4::decode_scale(half[L::CODES + s.in_page * L::SCALE_ROW + s.blk]);
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = static_cast<float>(static_cast<int>((w.x >> (4 * i)) & 15u) - 8) * sc;
    x[8 + i] = static_cast<float>(static_cast<int>((w.y >> (4 * i)) & 15u) - 8) * sc;
  }
  T* dst = static_cast<T*>(s.value ? a.v : a.k) + s.row * a.ld + s.head * DH + s.blk * cache4::kBlock;
  store16(dst, x);
}

template <int DH, typename T>
cudaError_t launch_rows(const CacheRowsArgs& a, bool write, cudaStream_t st) {
  constexpr int TOK = 32 / (DH / cache4::kBlock);
  const long long rows = static_cast<long long>(a.c.n_seqs) * a.M;
  const long long warps = (rows + TOK - 1) / TOK * (2 * a.c.Hkv);
  const long long blocks = (warps + 7) / 8;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  const cudaError_t e = launch_pdl(write ? cache_write_kernel<DH, T> : cache_read_kernel<DH, T>, grid, dim3(256), 0, st, a);
  return e != cudaSuccess ? e : cudaGetLastError();
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
