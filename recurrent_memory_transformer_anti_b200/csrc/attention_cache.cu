// Attention of a sequence's newest tokens over its pages of the 4-bit key/value cache.
#include "cache4.cuh"
#include "launch.h"

namespace rmt {
namespace {

using cache4::kPage;

// One CTA per (query row, query head): 64 threads, one key each, then the channels.
template <int DH, typename T>
__global__ void __launch_bounds__(64) cache_attn_simple_kernel(const CacheAttnArgs a) {
  using L = cache4::Layout<DH>;
  __shared__ float qs[DH], p[kPage], red[2];
  const int h = blockIdx.x, qi = blockIdx.y, b = blockIdx.z, t = threadIdx.x;
  const int head = h / (a.H / a.c.Hkv);
  const int len = a.c.lens[b], pos = len - a.n_q + qi;
  const T* q = static_cast<const T*>(a.q) + (static_cast<size_t>(b) * a.n_q + qi) * a.ldq + h * DH;
  bool odd = false;  // a query that is not finite
  for (int i = t; i < DH; i += 64) {
    qs[i] = to_f32(q[i]) * rsqrtf(static_cast<float>(DH));
    odd |= !isfinite(qs[i]);
  }
  odd = __syncthreads_or(odd);
  float o[DH / 32], m = -INFINITY, l = 0.f;
  for (int i = 0; i < DH / 32; ++i) o[i] = 0.f;
  int top = pos;
  if (pos >= a.c.max_pages * kPage) {  // a length past the cache
    if (t == 0 && a.c.err) atomicOr(a.c.err, kErrPage);
    top = -1;
  }
  for (int k0 = 0; k0 <= top; k0 += kPage) {
    if (k0 + kPage <= pos - a.window + 1 && k0 >= a.sinks) continue;
    const int page = cache4::page_of(a.c, b, k0);
    if (page < 0) continue;
    const unsigned char* blk = a.c.pages + cache4::block_offset<DH>(a.c, page, head);
    const int key = k0 + t;
    float s = -INFINITY;
    if (key <= top && (pos - key < a.window || key < a.sinks)) {
      s = 0.f;
      for (int i = 0; i < DH; ++i) {
        const int code = (blk[t * L::CODE_ROW + i / 2] >> (4 * (i & 1))) & 15;
        s += qs[i] * static_cast<float>(code - 8) * cache4::decode_scale(blk[L::CODES + t * L::SCALE_ROW + i / 16]);
      }
    }
    float mx = s;
    for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    __syncthreads();
    if ((t & 31) == 0) red[t >> 5] = mx;
    __syncthreads();
    mx = fmaxf(m, fmaxf(red[0], red[1]));
    if (mx == -INFINITY) continue;
    p[t] = s == -INFINITY ? 0.f : expf(s - mx);
    const float corr = m == -INFINITY ? 0.f : expf(m - mx);
    m = mx;
    __syncthreads();
    l *= corr;
    for (int i = 0; i < DH / 32; ++i) o[i] *= corr;
    for (int r = 0; r < kPage; ++r) {
      if (p[r] == 0.f) continue;
      l += p[r];
      for (int i = 0; i * 64 + t < DH; ++i) {
        const int c = i * 64 + t;
        const int code = (blk[L::V_OFF + r * L::CODE_ROW + c / 2] >> (4 * (c & 1))) & 15;
        o[i] += p[r] * static_cast<float>(code - 8) *
                cache4::decode_scale(blk[L::V_OFF + L::CODES + r * L::SCALE_ROW + c / 16]);
      }
    }
  }
  T* out = static_cast<T*>(a.out) + ((static_cast<size_t>(b) * a.n_q + qi) * a.H + h) * DH;
  for (int i = 0; i * 64 + t < DH; ++i) out[i * 64 + t] = from_f32<T>(odd && pos >= 0 ? NAN : l > 0.f ? o[i] / l : 0.f);
}

template <int DH, typename T>
cudaError_t launch_simple(const CacheAttnArgs& a, cudaStream_t st) {
  cache_attn_simple_kernel<DH, T><<<dim3(a.H, a.n_q, a.c.n_seqs), 64, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t cache_attention_workspace(int, int, int, int, int, int, int, int) { return 16; }

cudaError_t launch_cache_attention(const CacheAttnArgs& a, int dh, bool bf16, cudaStream_t st) {
  switch (dh) {
    case 32: return bf16 ? launch_simple<32, __nv_bfloat16>(a, st) : launch_simple<32, float>(a, st);
    case 64: return bf16 ? launch_simple<64, __nv_bfloat16>(a, st) : launch_simple<64, float>(a, st);
    case 128: return bf16 ? launch_simple<128, __nv_bfloat16>(a, st) : launch_simple<128, float>(a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace rmt
