// Attention over a sliding window and the first tokens (sinks), fp32 FMA: row i of a sequence sees
// the keys j <= i with i - j < window or j < sinks.
//
// A CTA of 128 threads holds 64 query rows of one head and passes over the keys they can see in
// tiles of 64: the tiles of the sinks, then those of the window, from the first row's oldest key
// to the last row's own. Each thread keeps 8 queries x 4 keys of the scores and 8 queries x dh/16
// channels of the output in registers; a row's maximum and sum run along (one pass over the keys).
// Key rows past the sequence's end are never read. A weight of zero adds nothing even when the
// value it belongs to is not finite, so what is masked cannot reach a row.
// Bound by the fp32 FMA pipe and the shared-memory reads that feed it. Serves fp32, and bf16 heads
// of 32 (bf16 heads of 64 and 128: attention_window_tc.cu).
#include "cache4.cuh"
#include "launch.h"

namespace rmt {
namespace {

template <int DH>
struct WinSimt {
  static constexpr int BQ = 64, BK = 64, PAD = 4;
  static constexpr int Q_OFF = 0;                        // [dh][BQ + PAD], scaled
  static constexpr int K_OFF = Q_OFF + DH * (BQ + PAD);  // [dh][BK + PAD]
  static constexpr int V_OFF = K_OFF + DH * (BK + PAD);  // [BK][dh]
  static constexpr int P_OFF = V_OFF + BK * DH;          // [BK][BQ + PAD]
  static constexpr int BYTES = (P_OFF + BK * (BQ + PAD)) * 4;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}

template <int DH, typename T>
__global__ void __launch_bounds__(128) window_simt_kernel(const WindowAttnArgs a) {
  pdl_trigger();
  pdl_wait();
  using S = WinSimt<DH>;
  constexpr int BQ = S::BQ, BK = S::BK, LQ = BQ + S::PAD, LK = BK + S::PAD, NC = DH / 16;
  extern __shared__ float sm[];
  float *Qs = sm + S::Q_OFF, *Ks = sm + S::K_OFF, *Vs = sm + S::V_OFF, *Ps = sm + S::P_OFF;
  const int h = blockIdx.y, g = blockIdx.z, t = threadIdx.x;
  const int len = a.lens ? min(a.lens[g], a.M) : a.M;
  const int q0 = static_cast<int>(gridDim.x - 1 - blockIdx.x) * BQ;  // long histories first
  if (q0 >= len) return;
  const int kvh = h / (a.H / a.Hkv);
  const size_t ld = static_cast<size_t>(a.H + 2 * a.Hkv) * DH;
  const T* base = static_cast<const T*>(a.qkv) + static_cast<size_t>(g) * a.M * ld;
  const int ty = t >> 4, tx = t & 15;  // queries 8 ty .., keys tx + 16 e, channels NC tx ..
  const float scale = rsqrtf(static_cast<float>(DH)) * 1.4426950408889634f;  // scores in powers of 2

  for (int e = t; e < BQ * (DH / 4); e += 128) {
    const int r = e % BQ, c = (e / BQ) * 4, row = q0 + r;
    const float4 v = row < len ? load4(base + row * ld + h * DH + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    Qs[c * LQ + r] = v.x * scale, Qs[(c + 1) * LQ + r] = v.y * scale;
    Qs[(c + 2) * LQ + r] = v.z * scale, Qs[(c + 3) * LQ + r] = v.w * scale;
  }
  float o[8][NC], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) o[i][c] = 0.f;
  }
  const int qlast = min(q0 + BQ, len) - 1;
  const int lo = max(0, q0 - a.window + 1);     // oldest key of the first row's window
  const int sink_end = min(a.sinks, lo);        // sinks not already in it
  const int n_sink = (sink_end + BK - 1) / BK;  // their tiles start at 0, the window's at lo
  const int n_win = (qlast - lo) / BK + 1;
  for (int tile = 0; tile < n_sink + n_win; ++tile) {
    const bool in_sink = tile < n_sink;
    const int k0 = in_sink ? tile * BK : lo + (tile - n_sink) * BK;
    const int kend = in_sink ? sink_end : qlast + 1;  // keys of this tile end here
    __syncthreads();
    for (int e = t; e < BK * (DH / 4); e += 128) {
      const int r = e % BK, c = (e / BK) * 4, row = k0 + r;
      const float4 v = row < kend ? load4(base + row * ld + (a.H + kvh) * DH + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      Ks[c * LK + r] = v.x, Ks[(c + 1) * LK + r] = v.y, Ks[(c + 2) * LK + r] = v.z, Ks[(c + 3) * LK + r] = v.w;
    }
    for (int e = t; e < BK * (DH / 4); e += 128) {
      const int c = (e % (DH / 4)) * 4, r = e / (DH / 4), row = k0 + r;
      const float4 v =
          row < kend ? load4(base + row * ld + (a.H + a.Hkv + kvh) * DH + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      *reinterpret_cast<float4*>(Vs + r * DH + c) = v;
    }
    __syncthreads();
    float s[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
#pragma unroll 8
    for (int d = 0; d < DH; ++d) {
      const float4 qa = *reinterpret_cast<const float4*>(Qs + d * LQ + 8 * ty);
      const float4 qb = *reinterpret_cast<const float4*>(Qs + d * LQ + 8 * ty + 4);
      const float qv[8] = {qa.x, qa.y, qa.z, qa.w, qb.x, qb.y, qb.z, qb.w};
      float kv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) kv[e] = Ks[d * LK + tx + 16 * e];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = fmaf(qv[i], kv[e], s[i][e]);
    }
    // every row of the tile sees every key of it?
    const bool whole = !in_sink && k0 + BK - 1 <= q0 && (qlast - k0 < a.window) && k0 + BK <= kend;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = q0 + 8 * ty + i;
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = k0 + tx + 16 * e;
        if (!whole && !(key < kend && key <= row && (row - key < a.window || key < a.sinks))) s[i][e] = -INFINITY;
        mx = fmaxf(mx, s[i][e]);
      }
#pragma unroll
      for (int w = 8; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: weights 2^-inf = 0
      const float corr = exp2f(m[i] - ref);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = exp2f(s[i][e] - ref);
        sum += p;
        Ps[(tx + 16 * e) * LQ + 8 * ty + i] = p;
      }
      l[i] = l[i] * corr + sum;  // this thread's keys; the sixteen threads of a row are added at the end
#pragma unroll
      for (int c = 0; c < NC; ++c) o[i][c] *= corr;
    }
    __syncwarp();  // a row's weights are written and read by the sixteen threads of one half warp
    auto add = [&](auto masked) {
#pragma unroll 4
      for (int k = 0; k < BK; ++k) {
        const float4 pa = *reinterpret_cast<const float4*>(Ps + k * LQ + 8 * ty);
        const float4 pb = *reinterpret_cast<const float4*>(Ps + k * LQ + 8 * ty + 4);
        const float pv[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
        float vv[NC];
        const float* vp = Vs + k * DH + NC * tx;
        if constexpr (NC == 2) {
          const float2 f = *reinterpret_cast<const float2*>(vp);
          vv[0] = f.x, vv[1] = f.y;
        } else {
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            const float4 f = *reinterpret_cast<const float4*>(vp + c);
            vv[c] = f.x, vv[c + 1] = f.y, vv[c + 2] = f.z, vv[c + 3] = f.w;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            if constexpr (decltype(masked)::value)
              o[i][c] = pv[i] != 0.f ? fmaf(pv[i], vv[c], o[i][c]) : o[i][c];
            else
              o[i][c] = fmaf(pv[i], vv[c], o[i][c]);
          }
      }
    };
    if (whole)
      add(std::false_type{});
    else
      add(std::true_type{});
  }
  T* out = static_cast<T*>(a.out) + static_cast<size_t>(g) * a.M * a.H * DH;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int w = 8; w; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    const int row = q0 + 8 * ty + i;
    if (row >= len) continue;
    const float inv = 1.f / l[i];  // a row sees itself: l > 0
    T* dst = out + (static_cast<size_t>(row) * a.H + h) * DH + NC * tx;
#pragma unroll
    for (int c = 0; c < NC; c += 2) {
      if constexpr (std::is_same_v<T, float>)
        *reinterpret_cast<float2*>(dst + c) = make_float2(o[i][c] * inv, o[i][c + 1] * inv);
      else
        *reinterpret_cast<uint32_t*>(dst + c) = pack2<T>(o[i][c] * inv, o[i][c + 1] * inv);
    }
  }
}

template <int DH, typename T>
cudaError_t launch_simt(const WindowAttnArgs& a, cudaStream_t st) {
  using S = WinSimt<DH>;
  static std::atomic<uint64_t> done;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(window_simt_kernel<DH, T>), S::BYTES, done);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.M + S::BQ - 1) / S::BQ, a.H, a.G);
  e = launch_pdl(window_simt_kernel<DH, T>, grid, dim3(128), S::BYTES, st, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_attention(const WindowAttnArgs& a, int dh, bool bf16, cudaStream_t st) {
  if (bf16 && dh >= 64) return launch_window_attention_tc(a, dh, st);
  switch (dh) {
    case 32: return bf16 ? launch_simt<32, __nv_bfloat16>(a, st) : launch_simt<32, float>(a, st);
    case 64: return launch_simt<64, float>(a, st);
    case 128: return launch_simt<128, float>(a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace rmt
