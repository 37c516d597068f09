// Attention over a sliding window and the first tokens (sinks) on 5th-generation tensor cores:
// bf16 in and out, fp32 accumulation and softmax, head_dim 64 or 128. Row i of a sequence sees the
// keys j <= i with i - j < window or j < sinks.
//
// Query tiles hold the heads of a key/value group together: 128 rows = TQ tokens x the group's
// heads (at most 16; TQ = 128 / heads, a multiple of 8), so a tile spans TQ tokens only and the
// keys that its rows see are window + TQ - 1 instead of window + 127: at 4 heads a group and a
// window of 256 that is 3 key tiles for 128 rows instead of 4. A work item is two such tiles, A
// and B, over neighbouring tokens; they share every key/value tile that both see.
//
// The keys of an item are numbered by what they cost, not by position: first the sinks (rounded
// up to 8 rows, the swizzle's row group), then the window from the first row's oldest key on.
// u < sp: key u; else key lo + u - sp. Tile t holds 128 consecutive u, brought by TMA boxes of
// 128, or 64, 32, 16 and 8 rows where the sinks end inside the tile: sinks cost their own rows,
// not a tile of their own.
//
// One persistent CTA per SM, 12 warps:
//   warp 0       one thread: TMA loads of the Q tiles and of the K and V rings;
//   warp 1       TMEM allocation; one thread issues S = Q K^T and O += P V for A and B in turn
//                (S of a tile's next keys before P V of its current ones, where P has columns of its
//                own: head_dim 64; at 128 P overwrites S, and the next S follows P V in the pipe);
//   warps 2-3    look through every V tile that some row sees only in part, before its P V: rows
//                behind the sequence's end, and rows that hold a value that is not finite, are
//                zeroed (0 * inf would reach rows that do not see them); the latter are noted
//                in a bit mask, and the rows that do see one give NaN;
//   warps 4-7    softmax of A, one query row a thread; warps 8-11 the same for B.
// The running maximum is only raised when it grows by more than 2^8 (weights stay <= 256, held as
// bf16: an operand pair has one type). Every wait is bounded; a timeout drains in-flight copies
// and MMAs, frees TMEM and sets the error word.
//
// Bound: at head_dim 64 the 16,384 exponentials of a 128 x 128 tile (1024 cycles of the special
// function unit, against 512 of MMA), at 128 MMA and exponentials alike.
#include <cuda.h>

#include "cache4.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace rmt {
namespace {

using bf16 = __nv_bfloat16;

template <int HD>
struct WtCfg {
  static constexpr int SUB = 128 * 64 * 2;  // one 128-row x 64-column swizzled block
  static constexpr int NSUB = HD / 64;
  static constexpr int TILE = NSUB * SUB;
  static constexpr bool OVERLAY = HD == 128;  // P in S's columns (512 TMEM columns hold no more)
  static constexpr int QST = HD == 64 ? 2 : 1, KST = HD == 64 ? 3 : 2;
  static constexpr int Q_OFF = 0;  // [x][QST]
  static constexpr int K_OFF = Q_OFF + 2 * QST * TILE;
  static constexpr int V_OFF = K_OFF + KST * TILE;
  static constexpr int BAR_OFF = V_OFF + KST * TILE;
  // barriers
  static constexpr int QFULL = 0, QEMPTY = QFULL + 2 * QST, KFULL = QEMPTY + 2 * QST, KEMPTY = KFULL + KST,
                       VFULL = KEMPTY + KST, VEMPTY = VFULL + KST, VSEEN = VEMPTY + KST, SFULL = VSEEN + KST,
                       SFREE = SFULL + 2, PREADY = SFREE + 2, OREADY = PREADY + 2, OFREE = OREADY + 2,
                       DRAIN = OFREE + 2, NBAR = DRAIN + 1;
  static constexpr int BAD_OFF = BAR_OFF + ((NBAR * 8 + 15) / 16) * 16;  // [KST][4] words: rows not finite
  static constexpr int SLOT_OFF = BAD_OFF + KST * 16;
  static constexpr int SMEM = 1024 + SLOT_OFF + 16;
  static constexpr int S_COL = 0, O_COL = 256, P_COL = OVERLAY ? 0 : 256 + 2 * HD;
  static constexpr int P_STEP = OVERLAY ? 128 : 64;
};

struct WtArgs {
  void* out;
  const int* lens;
  int* err;
  int G, M, H, Hkv;
  int group;   // query heads of a key/value head
  int heads;   // of a tile, at most 16
  int chunks;  // tiles' head ranges per group
  int tq;      // tokens of a tile
  int window, sinks;
  int blocks, items;
};

struct WtMaps {
  CUtensorMap q;      // box 64 columns x tq rows
  CUtensorMap kv[5];  // box 64 columns x 128 >> i rows
};

// A work item: two tiles of tq tokens from token a0 on (see the file comment for lo, sp and u).
struct Item {
  int g, kvh, h0, nh, a0, T, lo, sp, nt, last;
};

__device__ __forceinline__ Item item_of(const WtArgs& a, int it) {
  Item m;
  const int per = a.G * a.Hkv * a.chunks;
  const int r = it % per;
  m.a0 = (a.blocks - 1 - it / per) * 2 * a.tq;  // long histories first
  const int hc = r % (a.Hkv * a.chunks);
  m.g = r / (a.Hkv * a.chunks);
  m.kvh = hc / a.chunks;
  const int c = hc % a.chunks;
  m.h0 = m.kvh * a.group + c * a.heads;
  m.nh = min(a.heads, a.group - c * a.heads);
  m.T = a.lens ? min(__ldg(a.lens + m.g), a.M) : a.M;
  m.nt = m.lo = m.sp = m.last = 0;
  if (m.a0 >= m.T) return m;
  m.last = min(m.a0 + 2 * a.tq, m.T) - 1;
  m.lo = max(0, m.a0 - a.window + 1);
  if (a.sinks > 0) {
    const int s8 = (a.sinks + 7) & ~7;
    if (m.lo > s8)
      m.sp = s8;
    else
      m.lo = 0;
  }
  m.nt = (m.sp + m.last - m.lo + 128) / 128;
  return m;
}

// Tile x (0: A, 1: B) of an item: its tokens, and the u they see at least and at most.
struct Half {
  bool on;
  int b0, b1;         // first and last token
  int lo0, lo1, hi0, hi1;  // oldest window key and own key of the first and of the last token, as u
};
__device__ __forceinline__ Half half_of(const WtArgs& a, const Item& m, int x) {
  Half h;
  h.b0 = m.a0 + x * a.tq;
  h.on = h.b0 < m.T;
  h.b1 = min(h.b0 + a.tq, m.T) - 1;
  const int d = m.sp - m.lo;
  h.lo0 = max(h.b0 - a.window + 1, m.lo) + d;
  h.lo1 = max(h.b1 - a.window + 1, m.lo) + d;
  h.hi0 = h.b0 + d;
  h.hi1 = h.b1 + d;
  return h;
}
// Some row of the item sees only part of tile t.
__device__ __forceinline__ bool partial(const WtArgs& a, const Item& m, int t) {
  const int u0 = 128 * t, k0 = m.lo + u0 - m.sp;
  return u0 < m.sp || k0 + 127 > m.a0 || m.last - k0 >= a.window;
}

// The tiles of this CTA's items in order, from before the first; tau numbers them (ring stages).
struct Walk {
  int it, t, tau;
  Item m;
  __device__ __forceinline__ Walk() : it(static_cast<int>(blockIdx.x) - static_cast<int>(gridDim.x)), t(0), tau(-1) {
    m.nt = 0;
  }
  // to the next tile; false past the last
  __device__ __forceinline__ bool next(const WtArgs& a) {
    ++t;
    ++tau;
    if (t < m.nt) return true;
    t = 0;
    do {
      it += gridDim.x;
      if (it >= a.items) return false;
      m = item_of(a, it);
    } while (m.nt == 0);
    return true;
  }
};
// Tiles that a half needs: f .. l, and those of the sinks.
struct Need {
  int f, l;
};
__device__ __forceinline__ Need need_of(const WtArgs& a, const Item& m, int x) {
  const Half h = half_of(a, m, x);
  return {h.lo0 / 128, h.on ? h.hi1 / 128 : -1};
}
__device__ __forceinline__ bool needs(const WtArgs& a, const Need& n, int t) {
  return t <= n.l && (t >= n.f || 128 * t < a.sinks);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (a, b) = (a, b) * s + c, two at a time
__device__ __forceinline__ void fma_pair(uint32_t& a, uint32_t& b, float s, float c) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+r"(a), "+r"(b)
      : "r"(__float_as_uint(s)), "r"(__float_as_uint(c)));
}
__device__ __forceinline__ void add_pair(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ void sub_pair(uint32_t& a, uint32_t& b, float c) {
  float x = __uint_as_float(a), y = __uint_as_float(b);
  add_pair(x, y, -c, -c);
  a = __float_as_uint(x), b = __float_as_uint(y);
}
__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }

template <int HD>
__global__ void __launch_bounds__(384, 1)
    window_tc_kernel(const __grid_constant__ WtMaps maps, const __grid_constant__ WtArgs a) {
  using C = WtCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = sm100::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  auto bar = [&](int i) { return base + C::BAR_OFF + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SLOT_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* bad = reinterpret_cast<volatile uint32_t*>(smem + C::BAD_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i) {
      int n = 1;
      if (i >= C::VSEEN && i < C::VSEEN + C::KST) n = 64;
      if ((i >= C::SFREE && i < C::OREADY) || (i >= C::OFREE && i < C::DRAIN)) n = 128;
      sm100::mbar_init(bar(i), n);
    }
    *abort_flag = 0;
    sm100::fence_barrier_init();
    sm100::fence_proxy_async_smem();
    sm100::tma_prefetch_desc(&maps.q);
    sm100::tma_prefetch_desc(&maps.kv[0]);
  }
  if (warp == 1) sm100::tmem_alloc(sm100::smem_u32(tmem_slot), 512);
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  pdl_wait();  // qkv comes from earlier kernels of the stream

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int nq[2] = {0, 0}, nk = 0, nv = 0;  // loads issued: Q tiles of A and B, K tiles, V tiles
      Walk w;
      // rows u0 .. u0 + 127 of the item's keys (column col of the packed rows) into a ring tile
      auto load_tile = [&](uint32_t dst, uint32_t full, int col) {
        sm100::mbar_arrive_expect_tx(full, C::TILE);
        const int u0 = 128 * w.t;
        int r = 0;
        while (r < 128) {
          const int u = u0 + r;
          const bool sink = u < w.m.sp;
          int n = sink ? min(128 - r, w.m.sp - u) : 128 - r;
          const int key = sink ? u : w.m.lo + u - w.m.sp;
          int i = 0;
          while ((128 >> i) > n) ++i;  // the widest box that fits
          n = 128 >> i;
          for (int sb = 0; sb < C::NSUB; ++sb)
            sm100::tma_load_3d(dst + sb * C::SUB + r * 128, &maps.kv[i], col + 64 * sb, key, w.m.g, full);
          r += n;
        }
      };
      while (w.next(a)) {
        if (w.t == 0) {
          for (int x = 0; x < 2 && ok; ++x) {
            const int b0 = w.m.a0 + x * a.tq;
            if (b0 >= w.m.T) continue;
            const int qs = nq[x] % C::QST, id = x * C::QST + qs;
            ok = sm100::mbar_wait(bar(C::QEMPTY + id), ((nq[x] / C::QST) & 1) ^ 1u, abort_flag);
            if (!ok) break;
            sm100::mbar_arrive_expect_tx(bar(C::QFULL + id), C::NSUB * w.m.nh * a.tq * 128);
            for (int hh = 0; hh < w.m.nh; ++hh)
              for (int sb = 0; sb < C::NSUB; ++sb)
                sm100::tma_load_3d(base + C::Q_OFF + id * C::TILE + sb * C::SUB + hh * a.tq * 128, &maps.q,
                                   (w.m.h0 + hh) * HD + 64 * sb, b0, w.m.g, bar(C::QFULL + id));
            ++nq[x];
          }
          if (!ok) break;
        }
        const int st = w.tau % C::KST;
        const uint32_t ph = (w.tau / C::KST) & 1;
        ok = sm100::mbar_wait(bar(C::KEMPTY + st), ph ^ 1u, abort_flag);
        if (!ok) break;
        load_tile(base + C::K_OFF + st * C::TILE, bar(C::KFULL + st), (a.H + w.m.kvh) * HD);
        ++nk;
        ok = sm100::mbar_wait(bar(C::VEMPTY + st), ph ^ 1u, abort_flag);
        if (!ok) break;
        load_tile(base + C::V_OFF + st * C::TILE, bar(C::VFULL + st), (a.H + a.Hkv + w.m.kvh) * HD);
        ++nv;
      }
      if (!ok) {
        if (a.err) atomicOr(a.err, kErrTimeoutProducer);
        // let the copies already in flight land before the CTA's shared memory goes away
        for (int x = 0; x < 2; ++x)
          for (int n = max(0, nq[x] - C::QST); n < nq[x]; ++n)
            sm100::mbar_wait_drain(bar(C::QFULL + x * C::QST + n % C::QST), (n / C::QST) & 1);
        for (int n = max(0, nk - C::KST); n < nk; ++n)
          sm100::mbar_wait_drain(bar(C::KFULL + n % C::KST), (n / C::KST) & 1);
        for (int n = max(0, nv - C::KST); n < nv; ++n)
          sm100::mbar_wait_drain(bar(C::VFULL + n % C::KST), (n / C::KST) & 1);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idS = sm100::idesc_f32acc(128, 128, OpFormat<bf16>::value);
      constexpr uint32_t idO = sm100::idesc_f32acc_bmn(128, HD, OpFormat<bf16>::value);
      bool ok = true;
      int nq[2] = {-1, -1};                          // the Q tile in use, counted
      int ns[2] = {0, 0}, np[2] = {0, 0}, no[2] = {0, 0};  // S issued, P V issued, items begun
      bool fresh_q[2] = {true, true}, fresh_o[2] = {true, true};  // the next S / P V is an item's first
      auto wait = [&](int b, uint32_t parity) { return sm100::mbar_wait(bar(b), parity & 1u, abort_flag); };
      auto issue_s = [&](int x, int tau, bool last) -> bool {
        const int st = tau % C::KST;
        if (fresh_q[x]) ++nq[x];
        const int id = x * C::QST + nq[x] % C::QST;
        if (fresh_q[x] && !wait(C::QFULL + id, nq[x] / C::QST)) return false;
        fresh_q[x] = false;
        if (!wait(C::KFULL + st, tau / C::KST)) return false;
        if (!C::OVERLAY && ns[x] > 0 && !wait(C::SFREE + x, ns[x] - 1)) return false;
        sm100::tc_fence_after();
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const int sb = k >> 2, kk = k & 3;
          const uint64_t ad = sm100::smem_desc_k128(base + C::Q_OFF + id * C::TILE + sb * C::SUB) + 2ull * kk;
          const uint64_t bd = sm100::smem_desc_k128(base + C::K_OFF + st * C::TILE + sb * C::SUB) + 2ull * kk;
          sm100::mma_bf16(tmem + C::S_COL + 128 * x, ad, bd, idS, k > 0);
        }
        sm100::mma_commit(bar(C::SFULL + x));
        if (last) sm100::mma_commit(bar(C::QEMPTY + id));  // the item's last S of x has read its Q
        ++ns[x];
        return true;
      };
      auto issue_pv = [&](int x, int tau) -> bool {
        const int st = tau % C::KST;
        if (!wait(C::PREADY + x, np[x]) || !wait(C::VSEEN + st, tau / C::KST)) return false;
        // the first P V of an item overwrites O: the previous item's must have been read
        if (fresh_o[x] && no[x] > 0 && !wait(C::OFREE + x, no[x] - 1)) return false;
        sm100::tc_fence_after();
#pragma unroll
        for (int k = 0; k < 128 / 16; ++k) {  // P from TMEM: 16 keys per step = 8 columns of pairs
          const uint64_t bd = sm100::smem_desc_mn128(base + C::V_OFF + st * C::TILE + k * 2048, C::SUB);
          sm100::mma_f16_tmem_a(tmem + C::O_COL + HD * x, tmem + C::P_COL + C::P_STEP * x + 8 * k, bd, idO,
                                !fresh_o[x] || k > 0);
        }
        sm100::mma_commit(bar(C::OREADY + x));
        if (fresh_o[x]) ++no[x];
        fresh_o[x] = false;
        ++np[x];
        return true;
      };
      // S of the next tile and P V of the current one, for A and B in turn
      Walk nxt;
      int ct = 0, ctau = -1;
      Need cn[2] = {{0, -1}, {0, -1}}, nn[2] = {{0, -1}, {0, -1}};
      while (ok) {
        const bool more = nxt.next(a);
        if (more && nxt.t == 0) {
          for (int x = 0; x < 2; ++x) {
            nn[x] = need_of(a, nxt.m, x);
            fresh_q[x] = true;
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok) break;
          const bool s = more && needs(a, nn[x], nxt.t), p = ctau >= 0 && needs(a, cn[x], ct);
          if (ct == 0) fresh_o[x] = true;
          if (C::OVERLAY && p) ok = issue_pv(x, ctau);
          if (ok && s) ok = issue_s(x, nxt.tau, nxt.t == nn[x].l);
          if (ok && more && x == 1) sm100::mma_commit(bar(C::KEMPTY + nxt.tau % C::KST));
          if (!C::OVERLAY && ok && p) ok = issue_pv(x, ctau);
        }
        if (ok && ctau >= 0) sm100::mma_commit(bar(C::VEMPTY + ctau % C::KST));
        if (!more) break;
        ct = nxt.t;
        ctau = nxt.tau;
        cn[0] = nn[0];
        cn[1] = nn[1];
      }
      if (!ok) {
        if (a.err) atomicOr(a.err, kErrTimeoutMma);
        sm100::mma_commit(bar(C::DRAIN));
        sm100::mbar_wait_drain(bar(C::DRAIN), 0);
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    const int c = threadIdx.x - 64;
    bool ok = true;
    Walk w;
    while (w.next(a)) {
      const int st = w.tau % C::KST;
      ok = __all_sync(0xffffffffu, sm100::mbar_wait(bar(C::VFULL + st), (w.tau / C::KST) & 1, abort_flag));
      if (!ok) break;
      if (partial(a, w.m, w.t)) {
        // two rows a thread; 16 bytes at a time, each lane from another column of the row's
        // 128 bytes (the order within a row does not matter here)
#pragma unroll 1
        for (int rr = 0; rr < 2; ++rr) {
          const int row = c + 64 * rr, u = 128 * w.t + row;
          const bool behind = u >= w.m.sp && w.m.lo + u - w.m.sp >= w.m.T;
          uint4* const p = reinterpret_cast<uint4*>(smem + C::V_OFF + st * C::TILE + row * 128);
          __nv_bfloat162 acc = __float2bfloat162_rn(0.f);
          const __nv_bfloat162 zero = acc;
#pragma unroll
          for (int sb = 0; sb < C::NSUB; ++sb)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 v = p[sb * (C::SUB / 16) + ((i + lane) & 7)];
              acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.x), zero, acc);
              acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.y), zero, acc);
              acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.z), zero, acc);
              acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.w), zero, acc);
            }
          const bool fin = __hbeq2(acc, zero);  // 0 * x is NaN for infinities and NaN
          if (behind || !fin)
            for (int sb = 0; sb < C::NSUB; ++sb)
              for (int i = 0; i < 8; ++i) p[sb * (C::SUB / 16) + ((i + lane) & 7)] = make_uint4(0, 0, 0, 0);
          const uint32_t word = __ballot_sync(0xffffffffu, !fin && !behind);
          if (lane == 0) bad[4 * st + (row >> 5)] = word;
        }
        sm100::fence_async_smem();
      }
      sm100::mbar_arrive(bar(C::VSEEN + st));
    }
    if (!ok && lane == 0 && a.err) atomicOr(a.err, kErrTimeoutEpilogue);
  } else {
    const int x = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t loff = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + loff + C::S_COL + 128 * x, tO = tmem + loff + C::O_COL + HD * x,
                   tP = tmem + loff + C::P_COL + C::P_STEP * x;
    const float sl2 = rsqrtf(static_cast<float>(HD)) * 1.4426950408889634f;  // 1/sqrt(dh) * log2(e)
    const float raise = 8.f / sl2;  // the running maximum (of the raw scores) is only raised by that much
    const int hh = r / a.tq, tok = r - hh * a.tq;
    bool ok = true;
    int n = 0;    // tiles of x processed so far (barrier phases)
    int tau = 0;  // tiles of the CTA passed
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item m = item_of(a, it);
      const Half h = half_of(a, m, x);
      const Need need = need_of(a, m, x);
      const int tau0 = tau;
      tau += m.nt;
      if (m.nt == 0 || !h.on) continue;
      const bool idle = quarter * 32 >= m.nh * a.tq;  // warp-uniform: no row of this warp is used
      const int token = h.b0 + tok, d = m.sp - m.lo;
      const int uhi = token + d, ulo = max(token - a.window + 1, m.lo) + d, us = min(a.sinks, uhi + 1);
      float m_use = -3e38f, l = 0.f;
      bool poison = false, first = true;
      for (int t = 0; t < m.nt; ++t) {
        if (!needs(a, need, t)) continue;
        ok = __all_sync(0xffffffffu, sm100::mbar_wait(bar(C::SFULL + x), n & 1, abort_flag));
        if (!ok) break;
        if (idle) {  // the same waits and arrivals as the busy warps, in the same order
          sm100::mbar_arrive(bar(C::SFREE + x));
          if (n > 0) {
            ok = __all_sync(0xffffffffu, sm100::mbar_wait(bar(C::OREADY + x), (n - 1) & 1, abort_flag));
            if (!ok) break;
          }
          sm100::mbar_arrive(bar(C::PREADY + x));
          first = false;
          ++n;
          continue;
        }
        sm100::tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) sm100::tmem_ld32(tS + 32 * q4, s[q4]);
        sm100::tmem_wait_ld();
        sm100::tc_fence_before();
        if (!C::OVERLAY) sm100::mbar_arrive(bar(C::SFREE + x));
        const int u0 = 128 * t;
        if (u0 + 127 > h.hi0) {  // keys after some row's own
          const int vis = uhi - u0;
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * q4 + i > vis) s[q4][i] = __float_as_uint(-INFINITY);
        }
        if (u0 < h.lo1) {  // keys that left some row's window: from the sinks' end to its oldest
          const int from = max(us - u0, 0);
          const unsigned gone = static_cast<unsigned>(max(ulo - u0 - from, 0));
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (static_cast<unsigned>(32 * q4 + i - from) < gone) s[q4][i] = __float_as_uint(-INFINITY);
        }
        if (partial(a, m, t)) {
          const int st = (tau0 + t) % C::KST;
          ok = __all_sync(0xffffffffu,
                          sm100::mbar_wait(bar(C::VSEEN + st), ((tau0 + t) / C::KST) & 1, abort_flag));
          if (!ok) break;
          const uint32_t b0 = bad[4 * st], b1 = bad[4 * st + 1], b2 = bad[4 * st + 2], b3 = bad[4 * st + 3];
          if (b0 | b1 | b2 | b3) {  // rare
            for (int e = 0; e < 128; ++e) {
              const uint32_t wd = e < 64 ? (e < 32 ? b0 : b1) : (e < 96 ? b2 : b3);
              const int u = u0 + e;
              if (((wd >> (e & 31)) & 1u) && ((u >= ulo && u <= uhi) || u < us)) poison = true;
            }
          }
        }
        // row maximum over 4 independent partials (short dependency chains)
        float mxp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            mxp[(i >> 1) & 3] = max3(mxp[(i >> 1) & 3], u2f(s[q4][i]), u2f(s[q4][i + 1]));
        const float mx = fmaxf(fmaxf(mxp[0], mxp[1]), fmaxf(mxp[2], mxp[3]));
        float corr = 1.f;
        bool rescale = false;
        if (mx > m_use + raise) {  // a row that has seen nothing keeps -3e38: its weights are 2^-inf = 0
          corr = ex2((m_use - mx) * sl2);
          m_use = mx;
          rescale = !first;
        }
        // s * sl2 - m * sl2 in one rounding is off by up to 2^-24 of m * sl2: where scores are that
        // large the difference is taken first
        float less = m_use * sl2;
        const bool far = fabsf(m_use) > 4194304.f;
        if (__any_sync(0xffffffffu, far)) {
          const float by = far ? m_use : 0.f;  // the warp's other rows stay as they are
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
            for (int i = 0; i < 32; i += 2) sub_pair(s[q4][i], s[q4][i + 1], by);
          if (far) less = 0.f;
        }
        if (n > 0) {
          // P V of the tile before must be done before P and O change
          ok = __all_sync(0xffffffffu, sm100::mbar_wait(bar(C::OREADY + x), (n - 1) & 1, abort_flag));
          if (!ok) break;
          sm100::tc_fence_after();
          if (__any_sync(0xffffffffu, rescale)) {
            const float by = rescale ? corr : 1.f;
#pragma unroll 1
            for (int oc = 0; oc < HD / 16; ++oc) {
              uint32_t o[16];
              sm100::tmem_ld16(tO + 16 * oc, o);
              sm100::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(u2f(o[i]) * by);
              sm100::tmem_st16(tO + 16 * oc, o);
            }
          }
        }
        // weights, packed in place (keys 2c, 2c + 1 in column c) and sent 32 keys at a time
        float sp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            fma_pair(s[q4][i], s[q4][i + 1], sl2, -less);
            const float p0 = ex2(u2f(s[q4][i])), p1 = ex2(u2f(s[q4][i + 1]));
            add_pair(sp[i & 2], sp[(i & 2) + 1], p0, p1);
            s[q4][i >> 1] = pack2<bf16>(p0, p1);
          }
          sm100::tmem_st16(tP + 16 * q4, s[q4]);
        }
        l = l * corr + ((sp[0] + sp[1]) + (sp[2] + sp[3]));
        sm100::tmem_wait_st();
        sm100::tc_fence_before();
        sm100::mbar_arrive(bar(C::PREADY + x));
        first = false;
        ++n;
      }
      if (!ok) break;
      // end of the item: O after its last P V, normalised and stored; then O is free again
      ok = __all_sync(0xffffffffu, sm100::mbar_wait(bar(C::OREADY + x), (n - 1) & 1, abort_flag));
      if (!ok) break;
      sm100::tc_fence_after();
      const float inv = poison ? NAN : 1.f / l;
      const bool row_out = hh < m.nh && token < m.T;
      bf16* const dst = static_cast<bf16*>(a.out) +
                        ((static_cast<size_t>(m.g) * a.M + token) * a.H + m.h0 + hh) * HD;
#pragma unroll 1
      for (int oc = 0; oc < (idle ? 0 : HD / 32); ++oc) {
        uint32_t o[32];
        sm100::tmem_ld32(tO + 32 * oc, o);
        sm100::tmem_wait_ld();
        if (row_out) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = u2f(o[i]) * inv;
          store32_16(dst + 32 * oc, v);
        }
      }
      sm100::tc_fence_before();
      sm100::mbar_arrive_relaxed(bar(C::OFREE + x));
    }
    if (!ok && lane == 0 && a.err) atomicOr(a.err, kErrTimeoutEpilogue);
  }

  sm100::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc(tmem, 512);
  }
}

template <int HD>
cudaError_t launch_hd(const WindowAttnArgs& w, cudaStream_t st) {
  using C = WtCfg<HD>;
  WtArgs a{};
  a.out = w.out;
  a.lens = w.lens;
  a.err = w.err;
  a.G = w.G, a.M = w.M, a.H = w.H, a.Hkv = w.Hkv;
  a.group = w.H / w.Hkv;
  a.chunks = (a.group + 15) / 16;
  a.heads = (a.group + a.chunks - 1) / a.chunks;
  a.tq = 128 / a.heads / 8 * 8;
  a.window = w.window;
  a.sinks = w.sinks < w.M ? w.sinks : w.M;
  a.blocks = (w.M + 2 * a.tq - 1) / (2 * a.tq);
  const long long items = static_cast<long long>(a.blocks) * w.G * w.Hkv * a.chunks;
  if (items > 0x3fffffffLL) return cudaErrorInvalidValue;
  a.items = static_cast<int>(items);
  WtMaps maps;
  const uint64_t inner = static_cast<uint64_t>(w.H + 2 * w.Hkv) * HD;
  if (!make_tmap_bf16_3d(&maps.q, w.qkv, inner, w.M, w.G, a.tq)) return cudaErrorInvalidValue;
  for (int i = 0; i < 5; ++i)
    if (!make_tmap_bf16_3d(&maps.kv[i], w.qkv, inner, w.M, w.G, 128u >> i)) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(window_tc_kernel<HD>), C::SMEM, done);
  if (e != cudaSuccess) return e;
  const int grid = a.items < 148 ? a.items : 148;  // one CTA per SM
  e = launch_pdl(window_tc_kernel<HD>, dim3(grid), dim3(384), C::SMEM, st, maps, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_attention_tc(const WindowAttnArgs& a, int dh, cudaStream_t st) {
  if (dh == 64) return launch_hd<64>(a, st);
  if (dh == 128) return launch_hd<128>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace rmt
