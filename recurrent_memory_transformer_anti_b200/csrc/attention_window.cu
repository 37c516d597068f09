// Attention over a sliding window and the first tokens (sinks), fp32 FMA: row i of a sequence sees
// the keys j <= i with i - j < window or j < sinks.
//
// A CTA of 128 threads holds 8 NQ query rows of one head (32, or 16 in calls of few rows) and passes
// over the keys they can see in tiles of 64: the sinks, then the window from the first row's oldest key
// to the last row's own, numbered u = 0, 1, .. without a gap. Each thread keeps NQ queries x 4 keys of the
// scores and NQ queries x dh/16 channels of the output in registers; a row's maximum and sum run along
// (one pass over the keys).
// Key rows past the sequence's end are never read. A masked key's weight is zero, and zero adds nothing even
// when the value it belongs to is not finite; a weight that is too small for fp32 is its smallest number.
// Bound by the fp32 FMA pipe and the shared-memory reads that feed it: 16 bytes at a time, 8 of them for
// 64 FMA. Two sequences of 1040 rows, 32 / 8 heads of 64, window 256, 16 sinks: 166 us, 24 TFLOP/s of
// what is visible; 16 sequences 1181 us, 27 TFLOP/s, a third of the pipe; 16 of bf16 heads of 32 755 us, 21 TFLOP/s;
// two of 208 rows with 4 / 2 heads, window 64, too few to fill the SMs: 9.0 us.
// Serves fp32, and bf16 heads of 32 (bf16 heads of 64 and 128: attention_window_tc.cu).
#include "cache4.cuh"
#include "launch.h"

namespace rmt {
namespace {

// Shared memory: rows padded by 16 bytes, so that eight rows' reads of 16 bytes at one column touch all banks.
template <int DH, int NQ>
struct WinSimt {
  static constexpr int BQ = 8 * NQ, BK = 64;
  static constexpr int LD = DH + 4, LP = BK + 4;
  static constexpr int Q_OFF = 0;                    // [BQ][LD], scaled
  static constexpr int K_OFF = Q_OFF + BQ * LD;      // [BK][LD]
  static constexpr int V_OFF = K_OFF + BK * LD;      // [BK][LD]
  static constexpr int P_OFF = V_OFF + BK * LD;      // [BQ][LP]
  static constexpr int BYTES = (P_OFF + BQ * LP) * 4;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}

// N consecutive floats
template <int N>
__device__ __forceinline__ void lds(const float* p, float (&v)[N]) {
  if constexpr (N == 2) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    v[0] = f.x, v[1] = f.y;
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + c);
      v[c] = f.x, v[c + 1] = f.y, v[c + 2] = f.z, v[c + 3] = f.w;
    }
  }
}

template <int DH, typename T, int NQ>
__global__ void __launch_bounds__(128) window_simt_kernel(const WindowAttnArgs a) {
  pdl_trigger();
  pdl_wait();
  using S = WinSimt<DH, NQ>;
  constexpr int BQ = S::BQ, BK = S::BK, LD = S::LD, LP = S::LP, NC = DH / 16;
  extern __shared__ float sm[];
  float *Qs = sm + S::Q_OFF, *Ks = sm + S::K_OFF, *Vs = sm + S::V_OFF, *Ps = sm + S::P_OFF;
  const int h = blockIdx.y, g = blockIdx.z, t = threadIdx.x;
  const int len = a.lens ? min(a.lens[g], a.M) : a.M;
  const int q0 = static_cast<int>(gridDim.x - 1 - blockIdx.x) * BQ;  // long histories first
  if (q0 >= len) return;
  const int kvh = h / (a.H / a.Hkv);
  const size_t ld = static_cast<size_t>(a.H + 2 * a.Hkv) * DH;
  const T* base = static_cast<const T*>(a.qkv) + static_cast<size_t>(g) * a.M * ld;
  const int ty = t >> 4, tx = t & 15;  // queries NQ ty .., keys tx + 16 e, channels NC tx ..
  const float scale = rsqrtf(static_cast<float>(DH)) * 1.4426950408889634f;  // scores in powers of 2

#pragma unroll
  for (int i = 0; i < BQ * (DH / 4) / 128; ++i) {
    const int e = t + 128 * i, r = e / (DH / 4), c = (e % (DH / 4)) * 4, row = q0 + r;
    const float4 v = row < len ? load4(base + row * ld + h * DH + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4*>(Qs + r * LD + c) = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
  }
  float o[NQ][NC], m[NQ], l[NQ];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) o[i][c] = 0.f;
  }
  const int qlast = min(q0 + BQ, len) - 1;
  const int lo = max(0, q0 - a.window + 1);     // oldest key of the first row's window
  const int sinks = min(a.sinks, lo);           // those not already in it
  const int keys = sinks + qlast - lo + 1;
  auto key_of = [&](int u) { return u < sinks ? u : lo + u - sinks; };
  for (int u0 = 0; u0 < keys; u0 += BK) {
    // a tile's loads in flight together
    constexpr int PER = BK * (DH / 4) / 128;
    float4 kr[PER], vr[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = t + 128 * i, u = u0 + e / (DH / 4), c = (e % (DH / 4)) * 4;
      kr[i] = vr[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (u < keys) {
        const T* const p = base + key_of(u) * ld + (a.H + kvh) * DH + c;
        kr[i] = load4(p);
        vr[i] = load4(p + a.Hkv * DH);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = t + 128 * i, at = e / (DH / 4) * LD + (e % (DH / 4)) * 4;
      *reinterpret_cast<float4*>(Ks + at) = kr[i];
      *reinterpret_cast<float4*>(Vs + at) = vr[i];
    }
    __syncthreads();
    float s[NQ][4];
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
#pragma unroll 4
    for (int d = 0; d < DH; d += 4) {
      float qv[NQ][4], kv[4][4];
#pragma unroll
      for (int i = 0; i < NQ; ++i) lds(Qs + (NQ * ty + i) * LD + d, qv[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) lds(Ks + (tx + 16 * e) * LD + d, kv[e]);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] = fmaf(qv[i][c], kv[e][c], s[i][e]);
    }
    // every row of the tile sees every key of it?
    const int k0 = lo + u0 - sinks;
    const bool whole = u0 >= sinks && k0 + BK - 1 <= q0 && qlast - k0 < a.window && u0 + BK <= keys;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int row = q0 + NQ * ty + i;
      float mx = -INFINITY;
      bool seen[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int u = u0 + tx + 16 * e, key = key_of(u);
        seen[e] = whole || (u < keys && key <= row && (row - key < a.window || key < a.sinks));
        if (!seen[e]) s[i][e] = -INFINITY;
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
        float p = exp2f(s[i][e] - ref);
        if (!whole && seen[e] && p == 0.f) p = 1.4e-45f;  // not 0, which stands for a masked key below
        sum += p;
        Ps[(NQ * ty + i) * LP + tx + 16 * e] = p;
      }
      l[i] = l[i] * corr + sum;  // this thread's keys; the sixteen threads of a row are added at the end
#pragma unroll
      for (int c = 0; c < NC; ++c) o[i][c] *= corr;
    }
    __syncwarp();  // a row's weights are written and read by the sixteen threads of one half warp
    auto add = [&](auto masked) {
#pragma unroll 2
      for (int k = 0; k < BK; k += 4) {
        float pv[NQ][4];
#pragma unroll
        for (int i = 0; i < NQ; ++i) lds(Ps + (NQ * ty + i) * LP + k, pv[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float vv[NC];
          lds(Vs + (k + j) * LD + NC * tx, vv);
#pragma unroll
          for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              if constexpr (decltype(masked)::value)
                o[i][c] = pv[i][j] != 0.f ? fmaf(pv[i][j], vv[c], o[i][c]) : o[i][c];
              else
                o[i][c] = fmaf(pv[i][j], vv[c], o[i][c]);
            }
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
  for (int i = 0; i < NQ; ++i) {
#pragma unroll
    for (int w = 8; w; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    const int row = q0 + NQ * ty + i;
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

template <int DH, typename T, int NQ>
cudaError_t launch_rows(const WindowAttnArgs& a, cudaStream_t st) {
  using S = WinSimt<DH, NQ>;
  static std::atomic<uint64_t> done;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(window_simt_kernel<DH, T, NQ>), S::BYTES, done);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.M + S::BQ - 1) / S::BQ, a.H, a.G);
  e = launch_pdl(window_simt_kernel<DH, T, NQ>, grid, dim3(128), S::BYTES, st, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int DH, typename T>
cudaError_t launch_simt(const WindowAttnArgs& a, cudaStream_t st) {
  // 16 rows a CTA where all those CTAs run at once. fp32, window 256, 16 sinks, of 16 rows and of 32: two
  // sequences of 1040 with 4 heads of 64 (520 CTAs of 16 rows, four an SM) 37 and 43 us, with 8 heads 68 and 48;
  // bf16 heads of 32 (eight an SM), 8 of them 37 and 38, 32 and four sequences 239 and 192. (64 rows a
  // CTA: 57, 76, 50 and 221.)
  using S = WinSimt<DH, 2>;
  constexpr int at_once = 148 * (227 * 1024 / (S::BYTES + 1024));
  const long long ctas = static_cast<long long>((a.M + S::BQ - 1) / S::BQ) * a.H * a.G;
  return ctas <= at_once ? launch_rows<DH, T, 2>(a, st) : launch_rows<DH, T, 4>(a, st);
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
