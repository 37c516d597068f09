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
// One persistent CTA per SM, 20 warps:
//   warp 0       one thread: TMA loads of the Q tiles and of the K and V rings;
//   warps 1-     one thread each: TMEM allocation (warp 1), S = Q K^T and O += P V. At head_dim 64 each
//                query tile has an issuing thread, S of its next keys before P V of its current ones
//                (P has TMEM columns of its own); at 128, where P overwrites S and the next S follows
//                P V in the pipe, one thread issues for both in turn (two threads mix their
//                MMAs, which doubles each product's latency: 139 us for six prompts of up to 2063 rows,
//                window 777, against 111; 106 since, with no wait for P V: S behind it in the pipe says so);
//   up to 3      look through every V tile that some row sees only in part, before its P V: rows
//                behind the sequence's end, and rows that hold a value that is not finite, are
//                zeroed (0 * inf would reach rows that do not see them); the latter are noted
//                in a bit mask, and the rows that do see one give NaN;
//   warps 4-11   softmax of A, 12-19 of B: two threads a row, 64 columns each.
// A row's reference (what its scores are taken relative to) is the maximum of the first tile it sees;
// later tiles take their exponentials against it in one pass. Weights are held as bf16, whose relative
// precision is the same everywhere (an operand pair has one type), and summed in fp32, so a reference
// that turns out too low does no harm until a weight or an output leaves fp32's range. At head_dim 64 nothing is
// checked on the way: an item with a row whose weights add up to more than 2^60 (or, from 2^12 on, whose O is not
// finite) is noted, and after all items the CTA goes through the noted ones again, carefully: a tile whose
// weights add up to more than 2^12 is gone through again for its maximum, with O rescaled. At 128 that is
// done at once. (The careful way has both threads of a row meet at every tile, and a loop where the other has
// straight code: 1.20 ms instead of 1.01 for the long prompt below; at 128 102 us and 104.)
// Every wait is bounded; a timeout drains in-flight copies and MMAs, frees TMEM and sets the
// error word.
//
// Bound: the 32,768 exponentials of two 128 x 128 tiles take the special function unit 2048 cycles
// (the MMAs 1024, or 2048 at head_dim 128); the step takes 3,800 at head_dim 64: the instructions of the
// softmax warps and the latency of each one's own chain (barriers, TMEM accesses, one dependent
// instruction after another), which four such warps per scheduler hide only in part. A tile that some row sees
// in part costs about 1.4 times one that all see. Measured when the step took 4,500, and not better: one
// thread a row with 168 or 200 registers (4,840), four query tiles against 64-key tiles (4,750), one issuing
// thread that takes whatever is ready (4,800), three buffers of S in turn with P in their columns, so that
// S is always there before its softmax (4,850), longer waits between polls, a head start for A.
// 65,536 tokens, 32/8 heads of 64, window 1024, 4 sinks: 1.01 ms, 540 TFLOP/s.
#include <cuda.h>

#include "cache4.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace rmt {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kLostWords = 64;

template <int HD>
struct WtCfg {
  static constexpr int SUB = 128 * 64 * 2;  // one 128-row x 64-column swizzled block
  static constexpr int NSUB = HD / 64;
  static constexpr int TILE = NSUB * SUB;
  static constexpr bool OVERLAY = HD == 128;  // P in S's columns (512 TMEM columns hold no more)
  static constexpr bool TWICE = HD == 64;  // items in a first pass without, a second with raised references
  static constexpr int NX = OVERLAY ? 2 : 1;       // query tiles of an issuing thread (warps 1 .. 2 / NX)
  static constexpr int SEERS = 3 - 2 / NX;         // warps that look through V tiles (the rest up to warp 3)
  static constexpr int QST = HD == 64 ? 2 : 1, KST = HD == 64 ? 3 : 2;
  static constexpr int Q_OFF = 0;  // [x][QST]
  static constexpr int K_OFF = Q_OFF + 2 * QST * TILE;
  static constexpr int V_OFF = K_OFF + KST * TILE;
  static constexpr int BAR_OFF = V_OFF + KST * TILE;
  // barriers
  static constexpr int QFULL = 0, QEMPTY = QFULL + 2 * QST, KFULL = QEMPTY + 2 * QST, KEMPTY = KFULL + KST,
                       VFULL = KEMPTY + KST, VEMPTY = VFULL + KST, VSEEN = VEMPTY + KST, SFULL = VSEEN + KST,
                       SFREE = SFULL + 2, PREADY = SFREE + 2, OREADY = PREADY + 2, OFREE = OREADY + 2,
                       DRAIN = OFREE + 2, NBAR = DRAIN + 2;
  static constexpr int BAD_OFF = BAR_OFF + ((NBAR * 8 + 15) / 16) * 16;  // [KST][4] words: rows not finite
  static constexpr int MX_OFF = BAD_OFF + KST * 16;   // [2 tiles][2 halves][128 rows] fp32: maxima, then sums
  static constexpr int LOST_OFF = MX_OFF + 2 * 2 * 128 * 4;  // [kLostWords] items to go through again, a bit each
  static constexpr int STATE_OFF = LOST_OFF + kLostWords * 4;  // [20 warps][8] ints: where each role stopped
  static constexpr int SLOT_OFF = STATE_OFF + 20 * 8 * 4;
  static constexpr int SMEM = 1024 + SLOT_OFF + 16;
  static constexpr int S_COL = 0, O_COL = 256, P_COL = OVERLAY ? 0 : 256 + 2 * HD;
  static constexpr int P_STEP = OVERLAY ? 128 : 64, P_HALF = OVERLAY ? 64 : 32;  // each half where its own S was
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
  int step_hc, step_g, step_b;  // what grid-size items on adds to an item's head chunk, sequence and block
};

struct WtMaps {
  CUtensorMap q;      // box 64 columns x tq rows
  CUtensorMap kv[5];  // box 64 columns x 128 >> i rows
};

// Where in the items a CTA is: head chunk fastest, then sequence, then block of tokens (the last
// first: long histories first). Moved on without a division.
struct Place {
  int it, hc, g, blk, k;  // k: how many items of this CTA came before
  __device__ __forceinline__ explicit Place(const WtArgs& a) {
    k = 0;
    it = blockIdx.x;
    const int per = a.Hkv * a.chunks, r = it / per;
    hc = it - r * per;
    blk = r / a.G;
    g = r - blk * a.G;
  }
  __device__ __forceinline__ void next(const WtArgs& a) {
    ++k;
    it += gridDim.x;
    hc += a.step_hc;
    g += a.step_g;
    blk += a.step_b;
    if (hc >= a.Hkv * a.chunks) hc -= a.Hkv * a.chunks, ++g;
    if (g >= a.G) g -= a.G, ++blk;
  }
};

// The bit of an item among those to go through again (items 2048 apart share one).
__device__ __forceinline__ int lost_word(int k) { return (k >> 5) & (kLostWords - 1); }
__device__ __forceinline__ bool is_lost(const volatile uint32_t* lost, int k) {
  return (lost[lost_word(k)] >> (k & 31)) & 1u;
}

// A work item: two tiles of tq tokens from token a0 on (see the file comment for lo, sp and u).
struct Item {
  int g, kvh, h0, nh, a0, T, lo, sp, nt, last;
};

__device__ __forceinline__ Item item_of(const WtArgs& a, const Place& p) {
  Item m;
  m.a0 = (a.blocks - 1 - p.blk) * 2 * a.tq;
  m.g = p.g;
  m.kvh = p.hc;
  int c = 0;
  if (a.chunks > 1) {
    m.kvh = p.hc / a.chunks;
    c = p.hc - m.kvh * a.chunks;
  }
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
  m.nt = (m.sp + m.last - m.lo + 128) >> 7;
  return m;
}

// Query tile x (0: A, 1: B) of an item: its tokens, and the u they see at least and at most.
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

// The tiles of this CTA's items (of those in `lost`, if given) in order, from before the first; tau numbers
// them (ring stages).
struct Walk {
  int t, tau;
  bool begun;
  const volatile uint32_t* lost;
  Place p;
  Item m;
  __device__ __forceinline__ Walk(const WtArgs& a, const volatile uint32_t* lost_, int tau_)
      : t(0), tau(tau_), begun(false), lost(lost_), p(a) {
    m.nt = 0;
  }
  // to the next tile; false past the last
  __device__ __forceinline__ bool next(const WtArgs& a) {
    ++t;
    ++tau;
    if (t < m.nt) return true;
    t = 0;
    do {
      if (begun) p.next(a);
      begun = true;
      if (p.it >= a.items) return false;
      m.nt = 0;
      if (!lost || is_lost(lost, p.k)) m = item_of(a, p);
    } while (m.nt == 0);
    return true;
  }
};

// Key tiles that a query tile needs: f .. l, and those of the sinks (l = -1: none).
struct Need {
  int f, l;
};
__device__ __forceinline__ Need need_of(const WtArgs& a, const Item& m, int x) {
  const Half h = half_of(a, m, x);
  return {h.lo0 >> 7, h.on ? h.hi1 >> 7 : -1};
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
// v, as a value the compiler knows nothing of: what is computed from it is computed where it is used, and
// not kept in registers around a loop
__device__ __forceinline__ int fresh(int v) {
  int r;
  asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }

// What the warps of a CTA do, for all its items, or (AGAIN) for those noted in shared memory. CAREFUL: references
// are raised whenever a tile's weights add up to more than 2^12.
template <int HD, bool CAREFUL, bool AGAIN>
__device__ __forceinline__ void work(const WtMaps& maps, const WtArgs& a, uint8_t* const smem, const uint32_t base,
                                     const uint32_t tmem) {
  using C = WtCfg<HD>;
  auto bar = [&](int i) { return base + C::BAR_OFF + 8u * i; };
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + C::SLOT_OFF) + 1;
  volatile uint32_t* const bad = reinterpret_cast<volatile uint32_t*>(smem + C::BAD_OFF);
  volatile uint32_t* const lost_s = reinterpret_cast<volatile uint32_t*>(smem + C::LOST_OFF);
  const volatile uint32_t* const lost = AGAIN ? lost_s : nullptr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // where the first pass stopped, for the second to go on from (the first starts from constants: the compiler
  // makes better loops of those)
  volatile int* const mine = reinterpret_cast<volatile int*>(smem + C::STATE_OFF) + 8 * warp;
  constexpr bool KEEP = C::TWICE && !AGAIN;
  auto from = [&](int i) { return AGAIN ? mine[i] : 0; };
  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      // loads issued: Q tiles of A and B, K tiles, V tiles
      int nq[2] = {from(0), from(1)}, nk = from(2), nv = from(3);
      Walk w(a, lost, nk - 1);
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
      if (KEEP) mine[0] = nq[0], mine[1] = nq[1], mine[2] = nk, mine[3] = nv;
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
  } else if (warp <= 2 / C::NX) {
    if (lane == 0) {
      const int x0 = C::NX == 1 ? warp - 1 : 0;
      constexpr uint32_t idS = sm100::idesc_f32acc(128, 128, OpFormat<bf16>::value);
      constexpr uint32_t idO = sm100::idesc_f32acc_bmn(128, HD, OpFormat<bf16>::value);
      const uint64_t dq = sm100::smem_desc_k128(base + C::Q_OFF), dk = sm100::smem_desc_k128(base + C::K_OFF),
                     dv = sm100::smem_desc_mn128(base + C::V_OFF, C::SUB);
      bool ok = true;
      // per query tile: Q tile in use, S and P V issued, items begun; the next S / P V is an item's
      // first; the current key tile is needed
      int nq[C::NX], ns[C::NX], np[C::NX], no[C::NX];
      bool fresh_q[C::NX], fresh_o[C::NX], p[C::NX];
      Need nn[C::NX];
#pragma unroll
      for (int i = 0; i < C::NX; ++i) {
        nq[i] = from(3 * i) - 1, ns[i] = np[i] = from(3 * i + 1), no[i] = from(3 * i + 2);
        fresh_q[i] = fresh_o[i] = true;
        p[i] = false;
        nn[i] = {0, -1};
      }
      const int done = from(6);  // key tiles
      int st = done % C::KST, pst = 0;  // ring stages of the next key tile and of the current one
      uint32_t ph = (done / C::KST) & 1, pph = 0;
      auto wait = [&](int b, uint32_t parity) { return sm100::mbar_wait(bar(b), parity & 1u, abort_flag); };
      // S of the next key tile and P V of the current one, in turn
      Walk nxt(a, lost, done - 1);
      bool cur = false, cur_first = false;  // there is a current key tile; it is an item's first
      while (ok) {
        const bool more = nxt.next(a);
#pragma unroll
        for (int turn = 0; turn < 2 * C::NX; ++turn) {
          if (!ok) break;
          const int i = turn / 2, x = x0 + i;
          if (((turn & 1) == 0) != C::OVERLAY) {
            if (more && nxt.t == 0) {
              nn[i] = need_of(a, nxt.m, x);
              fresh_q[i] = true;
            }
            const bool s = more && needs(a, nn[i], nxt.t);
            if (s) {
              if (fresh_q[i]) ++nq[i];
              const int qs = nq[i] % C::QST;
              ok = (!fresh_q[i] || wait(C::QFULL + x * C::QST + qs, nq[i] / C::QST)) && wait(C::KFULL + st, ph) &&
                   (C::OVERLAY || ns[i] == 0 || wait(C::SFREE + x, ns[i] - 1));
              if (!ok) break;
              fresh_q[i] = false;
              ++ns[i];
              sm100::tc_fence_after();
              const uint64_t ad = dq + static_cast<uint32_t>((x * C::QST + qs) * (C::TILE >> 4));
              const uint64_t bd = dk + static_cast<uint32_t>(st * (C::TILE >> 4));
#pragma unroll
              for (int k = 0; k < HD / 16; ++k) {
                const uint32_t at = ((k >> 2) * C::SUB + (k & 3) * 32) >> 4;
                sm100::mma_bf16(tmem + C::S_COL + 128 * x, ad + at, bd + at, idS, k > 0);
              }
              sm100::mma_commit(bar(C::SFULL + x));
              sm100::mma_commit(bar(C::KEMPTY + st));
              if (nxt.t == nn[i].l) sm100::mma_commit(bar(C::QEMPTY + x * C::QST + qs));  // the item's last S
            } else if (more) {  // not before it has landed: two arrivals in one phase would pass for both tiles'
              ok = wait(C::KFULL + st, ph);
              if (!ok) break;
              sm100::mbar_arrive(bar(C::KEMPTY + st));
            }
            if (C::OVERLAY) p[i] = s;
          } else if (cur) {
            if (cur_first) fresh_o[i] = true;
            if (p[i]) {
              // the first P V of an item overwrites O: the previous item's must have been read
              ok = wait(C::PREADY + x, np[i]) && wait(C::VSEEN + pst, pph) &&
                   (!fresh_o[i] || no[i] == 0 || wait(C::OFREE + x, no[i] - 1));
              if (!ok) break;
              ++np[i];
              sm100::tc_fence_after();
              const uint64_t bd = dv + static_cast<uint32_t>(pst * (C::TILE >> 4));
#pragma unroll
              for (int k = 0; k < 128 / 16; ++k)  // P from TMEM: 16 keys per step = 8 columns of pairs
                sm100::mma_f16_tmem_a(tmem + C::O_COL + HD * x,
                                      tmem + C::P_COL + C::P_STEP * x + C::P_HALF * (k >> 2) + 8 * (k & 3), bd + static_cast<uint32_t>(k * 2048 >> 4), idO, !fresh_o[i] || k > 0);
              sm100::mma_commit(bar(C::OREADY + x));
              sm100::mma_commit(bar(C::VEMPTY + pst));
              if (fresh_o[i]) ++no[i];
              fresh_o[i] = false;
            } else {
              ok = wait(C::VSEEN + pst, pph);
              if (!ok) break;
              sm100::mbar_arrive(bar(C::VEMPTY + pst));
            }
          }
        }
        if (!ok || !more) break;
        if (!C::OVERLAY)
#pragma unroll
          for (int i = 0; i < C::NX; ++i) p[i] = needs(a, nn[i], nxt.t);
        cur = true;
        cur_first = nxt.t == 0;
        pst = st;
        pph = ph;
        if (++st == C::KST) {
          st = 0;
          ph ^= 1u;
        }
      }
      if (KEEP) {
#pragma unroll
        for (int i = 0; i < C::NX; ++i) mine[3 * i] = nq[i] + 1, mine[3 * i + 1] = np[i], mine[3 * i + 2] = no[i];
        mine[6] = nxt.tau;
      }
      if (!ok) {
        if (a.err) atomicOr(a.err, kErrTimeoutMma);
        sm100::mma_commit(bar(C::DRAIN + x0));
        sm100::mbar_wait_drain(bar(C::DRAIN + x0), 0);
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    bool ok = true;
    Walk w(a, lost, from(0) - 1);
    while (w.next(a)) {
      const int st = w.tau % C::KST;
      ok = __all_sync(0xffffffffu, sm100::mbar_wait(bar(C::VFULL + st), (w.tau / C::KST) & 1, abort_flag));
      if (!ok) break;
      if (partial(a, w.m, w.t)) {
        // some rows a thread; 16 bytes at a time, each lane from another column of the row's
        // 128 bytes (the order within a row does not matter here)
#pragma unroll 1
        for (int rr = 0; rr < 4 / C::SEERS; ++rr) {
          const int row = 32 * (C::SEERS * rr + 3 - warp) + lane, u = 128 * w.t + row;
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
    __syncwarp();
    if (KEEP && lane == 0) mine[0] = w.tau;
    if (!ok && lane == 0 && a.err) atomicOr(a.err, kErrTimeoutEpilogue);
  } else {
    // Two threads a row, 64 columns of S each: four softmax warps per scheduler, so that one's
    // barriers, loads and maxima run under another's exponentials.
    const int x = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t loff = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + loff + C::S_COL + 128 * x + 64 * half;
    const uint32_t tO = tmem + loff + C::O_COL + HD * x + HD / 2 * half;
    const uint32_t tP = tmem + loff + C::P_COL + C::P_STEP * x + C::P_HALF * half;
    float* const mx_own = reinterpret_cast<float*>(smem + C::MX_OFF) + (2 * x + half) * 128 + r;
    const float* const mx_other = reinterpret_cast<float*>(smem + C::MX_OFF) + (2 * x + 1 - half) * 128 + r;
    const int pair = 1 + 4 * x + quarter;  // named barrier of the two warps of these rows
    auto meet = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory"); };
    auto meet_any = [&](bool v) {  // and: does any of their threads say so
      uint32_t any;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
          "bar.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(any)
          : "r"(static_cast<uint32_t>(v)), "r"(pair)
          : "memory");
      return any != 0;
    };
    // A wait that gave up (or saw the abort flag) does not leave the loop: the other half's warp would
    // wait for this one for good. The rest is then gone through without waiting, its results not used.
    bool dead = false;
    auto await = [&](int b, int phase) {
      if (!__all_sync(0xffffffffu, sm100::mbar_wait(bar(b), phase & 1u, abort_flag))) dead = true;
    };
    const float sl2 = rsqrtf(static_cast<float>(HD)) * 1.4426950408889634f;  // 1/sqrt(dh) * log2(e)
    const int hh = r / a.tq, tok = r - hh * a.tq;
    int n = from(0);    // tiles of x processed so far (barrier phases)
    int tau = from(1);  // tiles of the CTA passed
    for (Place place(a); place.it < a.items; place.next(a)) {
      if (AGAIN && !is_lost(lost_s, place.k)) continue;
      int nt, token, uhi, ulo, us, begin_to, late_from, early_to, part_to, part_from;
      Need need;
      bool idle;
      {
        const Item m = item_of(a, place);
        const Half h = half_of(a, m, x);
        need = need_of(a, m, x);
        nt = m.nt;
        const int d = m.sp - m.lo;
        token = h.b0 + tok;
        uhi = token + d, ulo = max(token - a.window + 1, m.lo) + d, us = min(a.sinks, uhi + 1);
        begin_to = a.sinks > 0 ? 0 : h.lo1 >> 7;
        // the tiles in which some row of x sees only part (late: keys after it; early: keys that
        // left its window), and those in which some row of the item does: before part_to, from part_from
        late_from = h.hi0 - 126 <= 0 ? 0 : (h.hi0 - 126 + 127) >> 7;
        early_to = (h.lo1 + 127) >> 7;
        part_to = max((m.sp + 127) >> 7, m.last - a.window + 1 + d <= 0 ? 0 : (m.last - a.window + 1 + d + 127) >> 7);
        part_from = m.a0 + d - 126 <= 0 ? 0 : (m.a0 + d - 126 + 127) >> 7;
        idle = quarter * 32 >= m.nh * a.tq;  // warp-uniform: no row of this warp is used
      }
      const int tau0 = tau;
      tau += nt;
      if (need.l < 0 || nt == 0) continue;
      float m_use = -3e38f, l = 0.f;  // a row that has seen nothing keeps that: its weights are 2^-inf = 0
      bool poison = false;
      for (int t = 0; t <= need.l; ++t) {
        if (!needs(a, need, t)) continue;
        await(C::SFULL + x, n);
        if (idle) {  // the same waits and arrivals as the busy warps, in the same order
          if (!C::OVERLAY) sm100::mbar_arrive(bar(C::SFREE + x));
          if (!C::OVERLAY && n > 0) await(C::OREADY + x, n - 1);
          sm100::mbar_arrive(bar(C::PREADY + x));
          ++n;
          continue;
        }
        sm100::tc_fence_after();
        const bool late = t >= late_from, early = t < early_to;
        const int u0 = 128 * t + 64 * half;
        // 32 columns from q on, masked keys at -inf
        auto mask = [&](uint32_t (&s)[32], int q) {
          const int vis = fresh(uhi - u0) - q;
          if (late && __any_sync(0xffffffffu, vis < 31)) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i > vis) s[i] = __float_as_uint(-INFINITY);
          }
          const int from = max(fresh(us - u0) - q, 0);
          const int gone = fresh(ulo - u0) - q - from;
          if (early && __any_sync(0xffffffffu, gone > 0 && from < 32)) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (static_cast<unsigned>(i - from) < static_cast<unsigned>(max(gone, 0))) s[i] = __float_as_uint(-INFINITY);
          }
        };
        float corr = 1.f, sum;
        // a tile that is the first one some row sees: gone through for its maximum (CAREFUL: of every row)
        const bool begins = t <= begin_to;
        bool rescale = false, over = begins && (CAREFUL || t == (fresh(us) > 0 ? 0 : fresh(ulo) >> 7));
        uint32_t pk[32];
        for (int tries = begins ? 1 : 0;; ++tries) {
          if (tries > 0) {
            // the row maximum, over both halves
            float mxp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
            for (int q = 0; q < 64; q += 32) {
              uint32_t s[32];
              sm100::tmem_ld32(tS + q, s);
              sm100::tmem_wait_ld();
              mask(s, q);
#pragma unroll
              for (int i = 0; i < 32; i += 2)
                mxp[(i >> 1) & 3] = max3(mxp[(i >> 1) & 3], u2f(s[i]), u2f(s[i + 1]));
            }
            float mx = fmaxf(fmaxf(mxp[0], mxp[1]), fmaxf(mxp[2], mxp[3]));
            // rows whose weights stayed small say so by NaN: they keep their reference
            *mx_own = over ? mx : NAN;
            meet();
            const float other = *mx_other;
            meet();
            const bool raise = over || other == other;
            if (raise) {
              // a half that was not over says nothing of its maximum, which is then not above the reference
              // by more than its sum allows
              mx = fmaxf(over ? mx : m_use, other == other ? other : m_use);
              if (mx > m_use) {
                corr = ex2((m_use - mx) * sl2);
                rescale = m_use > -3e38f;  // else O is 0
                m_use = mx;
              }
            }
          }
          // s * sl2 - m * sl2 in one rounding is off by up to 2^-24 of m * sl2: where scores are that
          // large the difference is taken first
          const bool far = fabsf(m_use) > 4194304.f;
          const bool any_far = __any_sync(0xffffffffu, far);
          const float by = far ? m_use : 0.f, less = far ? 0.f : m_use * sl2;
          float sp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 64; q += 32) {
            uint32_t c[32];
            sm100::tmem_ld32(tS + q, c);
            sm100::tmem_wait_ld();
            if (late || early) mask(c, q);
            if (any_far) {
#pragma unroll
              for (int i = 0; i < 32; i += 2) sub_pair(c[i], c[i + 1], by);
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              fma_pair(c[i], c[i + 1], sl2, -less);
              const float p0 = ex2(u2f(c[i])), p1 = ex2(u2f(c[i + 1]));
              add_pair(sp[i & 2], sp[(i & 2) + 1], p0, p1);
              pk[(q + i) >> 1] = pack2<bf16>(p0, p1);
            }
          }
          sum = (sp[0] + sp[1]) + (sp[2] + sp[3]);
          if (!CAREFUL || tries > 0) break;
          over = !(sum <= 4096.f);  // NaN too: gone through once more, to no effect
          if (!meet_any(over)) break;
        }
        sm100::tc_fence_before();
        if (!C::OVERLAY) sm100::mbar_arrive(bar(C::SFREE + x));
        // P V of the tile before must be done before P and O change; in S's columns that is so, S came after it
        if (!C::OVERLAY && n > 0) {
          await(C::OREADY + x, n - 1);
          sm100::tc_fence_after();
        }
        if (__any_sync(0xffffffffu, rescale)) {
          const float f = rescale ? corr : 1.f;
#pragma unroll 1
          for (int oc = 0; oc < HD / 32; ++oc) {
            uint32_t o[16];
            sm100::tmem_ld16(tO + 16 * oc, o);
            sm100::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(u2f(o[i]) * f);
            sm100::tmem_st16(tO + 16 * oc, o);
          }
        }
        sm100::tmem_st16(tP, pk);  // keys 2c, 2c + 1 in column c
        sm100::tmem_st16(tP + 16, pk + 16);
        l = l * corr + sum;
        if (t < part_to || t >= part_from) {
          const int st = (tau0 + t) % C::KST;
          await(C::VSEEN + st, (tau0 + t) / C::KST);
          const uint32_t b0 = bad[4 * st], b1 = bad[4 * st + 1], b2 = bad[4 * st + 2], b3 = bad[4 * st + 3];
          if (b0 | b1 | b2 | b3) {  // rare
            for (int e = 0; e < 128; ++e) {
              const uint32_t wd = e < 64 ? (e < 32 ? b0 : b1) : (e < 96 ? b2 : b3);
              const int u = 128 * t + e;
              if (((wd >> (e & 31)) & 1u) && ((u >= ulo && u <= uhi) || u < us)) poison = true;
            }
          }
        }
        sm100::tmem_wait_st();
        sm100::tc_fence_before();
        sm100::mbar_arrive(bar(C::PREADY + x));
        ++n;
      }
      // end of the item: the row's sum over both halves, and O after its last P V, normalised and
      // stored; then O is free again
      if (!idle) {
        *mx_own = l;
        meet();
        l += *mx_other;  // the next item's first tile meets before it writes there again
        meet();
      }
      await(C::OREADY + x, n - 1);
      sm100::tc_fence_after();
      const bool lost_row = !CAREFUL && l > 1.152921504606847e18f;
      const float inv = poison || lost_row ? NAN : 1.f / l;
      {
        const Item m = item_of(a, place);  // again, rather than in registers through the tiles
        bool row_out = hh < m.nh && token < m.T;
        bf16* const dst = static_cast<bf16*>(a.out) +
                          ((static_cast<size_t>(m.g) * a.M + token) * a.H + m.h0 + hh) * HD + HD / 2 * half;
#pragma unroll 1
        for (int oc = 0; oc < (idle ? 0 : HD / 64); ++oc) {
          // the second time only rows that are not finite yet: the others' bits do not depend on their neighbours
          if (AGAIN && row_out) {
            bool open = false;
            for (int i = 0; i < 4; ++i) {
              const uint4 w = *reinterpret_cast<const uint4*>(dst + 32 * oc + 8 * i);
              const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int k = 0; k < 4; ++k)
                open |= (ws[k] & 0x7F80u) == 0x7F80u || (ws[k] & 0x7F800000u) == 0x7F800000u;
            }
            row_out = open;
          }
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
        // Weights and sums have fp32's range, so a reference that is too low does no harm until a weight or O
        // leaves it; the item is then gone through again.
        if (!CAREFUL && !idle && __any_sync(0xffffffffu, l > 4096.f)) {
          float z = 0.f;
#pragma unroll 1
          for (int oc = 0; oc < HD / 32; ++oc) {
            uint32_t o[16];
            sm100::tmem_ld16(tO + 16 * oc, o);
            sm100::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) z = fmaf(u2f(o[i]), 0.f, z);  // 0 * x is NaN for infinities and NaN
          }
          if (row_out && (lost_row || (l > 4096.f && z != 0.f)))
            atomicOr(const_cast<uint32_t*>(lost_s) + lost_word(place.k), 1u << (place.k & 31));
        }
      }
      sm100::tc_fence_before();
      sm100::mbar_arrive_relaxed(bar(C::OFREE + x));
    }
    __syncwarp();
    if (KEEP && lane == 0) mine[0] = n, mine[1] = tau;
    if (dead && lane == 0 && a.err) atomicOr(a.err, kErrTimeoutEpilogue);
  }
}
// Out of line, so that its registers are not the first pass's
template <int HD>
__device__ __noinline__ void work_again(const WtMaps& maps, const WtArgs& a, uint8_t* smem, uint32_t base, uint32_t tmem) {
  work<HD, true, true>(maps, a, smem, base, tmem);
}

template <int HD>
__global__ void __launch_bounds__(640, 1)
    window_tc_kernel(const __grid_constant__ WtMaps maps, const __grid_constant__ WtArgs a) {
  using C = WtCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = sm100::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  auto bar = [&](int i) { return base + C::BAR_OFF + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SLOT_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* lost_s = reinterpret_cast<volatile uint32_t*>(smem + C::LOST_OFF);
  volatile int* state = reinterpret_cast<volatile int*>(smem + C::STATE_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i) {
      int n = 1;
      if (i >= C::VSEEN && i < C::VSEEN + C::KST) n = 32 * C::SEERS;
      if ((i >= C::KEMPTY && i < C::VFULL) || (i >= C::VEMPTY && i < C::VSEEN)) n = 2;
      if ((i >= C::SFREE && i < C::OREADY) || (i >= C::OFREE && i < C::DRAIN)) n = 256;
      sm100::mbar_init(bar(i), n);
    }
    *abort_flag = 0;
    for (int i = 0; i < kLostWords; ++i) lost_s[i] = 0;
    for (int i = 0; i < 20 * 8; ++i) state[i] = 0;
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

  work<HD, !C::TWICE, false>(maps, a, smem, base, tmem);
  if constexpr (C::TWICE) {
    sm100::tc_fence_before();
    __syncthreads();
    uint32_t again = 0;
    for (int i = lane; i < kLostWords; i += 32) again |= lost_s[i];
    if (!*abort_flag && __any_sync(0xffffffffu, again != 0)) {  // the same for every warp
      sm100::tc_fence_after();
      work_again<HD>(maps, a, smem, base, tmem);
    }
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
  const int per = a.Hkv * a.chunks, over = grid / per;
  a.step_hc = grid - over * per;
  a.step_b = over / a.G;
  a.step_g = over - a.step_b * a.G;
  e = launch_pdl(window_tc_kernel<HD>, dim3(grid), dim3(640), C::SMEM, st, maps, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_attention_tc(const WindowAttnArgs& a, int dh, cudaStream_t st) {
  if (dh == 64) return launch_hd<64>(a, st);
  if (dh == 128) return launch_hd<128>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace rmt
