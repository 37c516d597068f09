// Attention of a sequence's newest tokens over its pages of the 4-bit key/value cache.
//
// One pass over the codes: 72 dh bytes per 64 tokens and kv head. A unit of
// work is 64 tokens of one kv head (32 at head_dim 128: 4608 bytes either way) for one tile of query
// rows; an item is what one (sequence, kv head, row tile) sees of the cache, without what lies between
// the sinks and the window. Two ways of dealing the units, by the most units an item can have:
//   short items (deal_whole): a team of warps takes whole items, each warp every so-manieth unit, and adds
//     their results in shared memory: one launch, nothing read before the item's own length. A
//     team has as many warps of a CTA as leave every item a team at once, at most one per unit.
//   more: the units of all items form one list (lengths are read on the device), and each warp
//     of the grid takes an equal, contiguous stretch of it, so that one long sequence and many short
//     ones are both spread over all SMs, and no warp waits for another. A stretch that holds a whole
//     item gives its result; parts go to the workspace, and a second kernel adds them in the
//     order of the keys: no atomics, equal bits.
// Each warp has its own ring of bulk copies.
//
// What it takes: 64 sequences of up to 8192 tokens (166 MB; 32 / 8 heads of 64, bf16) 50 us in a run of calls,
// 3.3 TB/s; alone under the profiler 46.7 us and 8.9 for the second kernel. No unit is full: the schedulers
// issue in 51% of all cycles, the integer pipe is at 41%, the half2 pipe at 39%, HBM at 45%, the tensor pipe at 23%.
// Four warps a scheduler do not cover one another's waits, per issued instruction 1.4 for results of fixed
// latency, 0.9 for a pipe that issues every other cycle, 0.7 for memory. Fewer instructions a code would bring it
// nearer to HBM. One sequence of 131,072 tokens 31 us in all, of which 3 go to the chain of length, page number and
// codes before the first product.
//
// Arithmetic. Query rows are the MMA's N (8 or 16 rows: the heads of a group, times the tokens),
// keys or channels its M, so that few rows waste nothing: S^T = K Q^T, O^T = V^T P^T
// (mma.sync m16n8k16, f16 operands, fp32 sums: the codes turn into operands in registers, and tcgen05
// would have them pass through shared memory again, four times their bytes). A code's nibble
// or-ed into the f16 pattern of 64 is 64 + (q + 8); times the scale minus 72 scales is q * scale,
// exact, in one fused operation for two codes (dequant). Scales are taken at 2^-7 of their value; the
// factor comes back with the row's scale and at the end. A lane takes 16
// (or 8, or 32) consecutive channels of a key, since the order of a dot product's terms is free as long as
// Q has the same one, and for V eight neighbouring lanes' keys are chosen so that the reads of a warp are
// whole lines of shared memory. P^T turns from accumulator to operand layout by
// movmatrix. Queries are scaled by a power of two per row into f16's normal range: exact for
// bf16; fp32 queries and weights are taken as two f16 terms (22 bits). Weights are held at 2^7 to 2^15
// of their value; f16's smallest step is 2^-24, so what it cuts off is at most 2^-32 of the largest.
#include "cache4.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace rmt {
namespace {

using cache4::CacheArgs;
using cache4::kPage;

constexpr int kMaxWarps = 148 * 16;  // that share a list of units: 16 per SM
constexpr float kCodeScale = 128.f;  // operands hold 2^-7 of a value
constexpr uint32_t kWideScale = 224;  // scale bytes from here on take the exact way (dequant)

template <int DH>
struct Unit {
  static constexpr int TOK = DH == 128 ? 32 : 64;
  static constexpr int CODES = TOK * DH / 2, SCALES = TOK * DH / 16;
  static constexpr int V_OFF = CODES + SCALES;
  static constexpr int BYTES = 2 * V_OFF;
};

// What of a sequence some row of it sees, in units: the first `sinks` of them, then from `lo` on.
struct Span {
  int n, sinks, lo;
};
struct SpanArgs {
  int cap;  // tokens a sequence may hold
  int n_q, window, sinks;
};
template <int TOK>
__device__ __forceinline__ Span span_of(const SpanArgs& a, int T) {
  Span s{0, 0, 0};
  if (T <= 0 || T > a.cap) return s;
  s.lo = max(0, max(T - a.n_q, 0) - a.window + 1) / TOK;
  const int last = (T - 1) / TOK;
  s.sinks = min((min(a.sinks, T) + TOK - 1) / TOK, s.lo);
  s.n = s.sinks + last - s.lo + 1;
  return s;
}

struct DecodeArgs {
  CacheArgs c;
  SpanArgs span;
  const void* q;
  long long ldq;
  void* out;
  int n_q, H, group, rows, tiles;  // rows: n_q * group per kv head, in `tiles` tiles
  int team;       // warps that share an item (whole items)
  int* prefix;    // [n_seqs + 1] units before each sequence (workspace; for the second kernel)
  float* parts;   // two per warp: O [rows of a tile][dh], maxima, sums
};

// The list of units dealt to warps: equal stretches, the first `more` of them one unit longer.
struct Deal {
  int warps, units, each, more;
  __device__ __forceinline__ Deal(int units_, int grid_warps) {
    units = units_;
    warps = max(1, min(grid_warps, units));
    each = units / warps;
    more = units - each * warps;
  }
  __device__ __forceinline__ int begin(int w) const { return w * each + min(w, more); }
  __device__ __forceinline__ int warp_of(int u) const {
    const int cut = more * (each + 1);
    return u < cut ? u / (each + 1) : more + (u - cut) / each;
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// (x, y) = (x, y) * (a, b) + (c, d)
__device__ __forceinline__ void fma_pair(float& x, float& y, float a, float b, float c, float d) {
  asm("{\n\t.reg .b64 p, q, r;\n\t"
      "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmov.b64 r, {%4, %5};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b), "f"(c), "f"(d));
}
__device__ __forceinline__ uint32_t h2(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Two scales (f16 bits in the low and high half of b) as pairs: 2^-7 of the scales (x), and what
// takes the offset of a high nibble (y) and of a low one (z) away again.
struct Scale {
  __half2 x, y, z;
};
template <bool WIDE>
__device__ __forceinline__ Scale scale_pair(uint32_t b) {
  Scale s;
  const __half2 f = as_h2(b);
  s.x = __hmul2(f, __float2half2_rn(1.f / kCodeScale));
  s.y = __hmul2(f, __float2half2_rn(-72.f / kCodeScale));
  s.z = __hmul2(f, __float2half2_rn((WIDE ? -8.f : -1032.f) / kCodeScale));
  return s;
}
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// The codes j of the low and of the high half of w, j = 0..3, times their scales. A byte's high
// nibble h sits where it counts units of 64's f16 pattern: 64 + h, and its low one l where it
// counts those of 1024: 1024 + l. (64 + h) s - 72 s and (1024 + l) s - 1032 s are exact in one fused
// operation, since 72 and 1032 times a scale have at most 11 significant bits (1032 = 8 * 129, 129 * 15 <
// 2048) and at 2^-7 of the scale neither end of the format leaves f16's range -- but for the two
// largest scales, 8192 and 9216, whose 1032nd overflows. WIDE takes the low nibble as
// (1024 + l + 16 h) - 16 (64 + h) first, one operation more, for those.
// One shift per word: shifts and logic (the ALU pipe) and half2 operations (the heavy half of
// the FMA pipe) both issue every other cycle, and are the two fullest (41 and 39%).
template <bool WIDE>
__device__ __forceinline__ void dequant(uint32_t w, const Scale& s, uint32_t (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 h = as_h2(and_or(w, 0x00F000F0u, 0x54005400u));
    __half2 l = as_h2(and_or(w, WIDE ? 0x00FF00FFu : 0x000F000Fu, 0x64006400u));
    if (WIDE) l = __hfma2(h, __float2half2_rn(-16.f), l);
    v[2 * i] = h2(__hfma2(l, s.x, s.z));
    v[2 * i + 1] = h2(__hfma2(h, s.x, s.y));
    w >>= 8;
  }
}

template <int N>
__device__ __forceinline__ void lds_words(const unsigned char* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  }
}

struct Item {
  int b, head, tile, len;
  int begin;  // its first unit in the list
  Span s;
};

// Warps of a CTA, one CTA per SM: 16 of at most 128 registers, but fewer with more where they would spill too
// much. 64 sequences of 8192 tokens, bf16: two row tiles of 128 channels (16 heads to one) 8 warps 42 us, 12
// 48; two of 64 channels (32 heads to two, 16,384 tokens) 12 warps 65, 16 71; fp32 of 128 channels
// (32 / 8 heads) 12 warps 180, 16 193; one tile of bf16 of 128 channels 16 warps 143, 12 152. (Of
// two CTAs with 8 warps each the first on an SM is served first: it ended after 38 us of 64 sequences'
// 50, the other's four warps per scheduler then ran alone.)
template <int DH, typename T, int NT>
struct Shape {
  static constexpr bool F32 = std::is_same_v<T, float>;
  static constexpr int WARPS = DH == 128 && NT == 2 ? 8 : (DH == 64 && NT == 2) || (DH == 128 && F32) ? 12 : 16;
};

template <int DH, typename T, int NT, bool WHOLE>
struct DecodeSmem {
  static constexpr int kWarps = Shape<DH, T, NT>::WARPS;
  static constexpr int STAGES = WHOLE ? 2 : 3;  // of a warp's ring
  static constexpr int RING = 0;
  static constexpr int LD = DH + 4;
  static constexpr int MERGE = RING + kWarps * STAGES * Unit<DH>::BYTES;  // whole items: [warp][8][LD] fp32
  static constexpr int ML = MERGE + kWarps * 8 * LD * 4;                  // [2][warp][8 NT] fp32
  static constexpr int PRE = MERGE;  // dealt stretches: [threads + 1] units before each run of sequences
  static constexpr int SUM = PRE + (32 * kWarps + 4) * 4;  // [warps]
  static constexpr int LEN = SUM + 16 * 4;                 // [threads] lengths, when a run is one sequence
  static constexpr int BAR = WHOLE ? ML + 2 * kWarps * 8 * NT * 4 : LEN + 32 * kWarps * 4;
  static constexpr int BYTES = BAR + kWarps * STAGES * 8 + 16;
};

template <int DH, typename T, int NT, bool WHOLE>
__global__ void __launch_bounds__(32 * Shape<DH, T, NT>::WARPS, 1) cache_attn_kernel(const DecodeArgs a) {
  using U = Unit<DH>;
  using S = DecodeSmem<DH, T, NT, WHOLE>;
  constexpr int kStages = S::STAGES, kWarps = S::kWarps, kThreads = 32 * kWarps;
  constexpr bool SPLIT = std::is_same_v<T, float>;  // two f16 terms per query and weight
  constexpr int TERMS = SPLIT ? 2 : 1;
  constexpr int KS = DH / 16, WK = DH / 32;  // k16 steps of a key, 32-bit words of it per lane
  constexpr int MT = U::TOK / 16;            // 16-key tiles of a unit
  constexpr int MU = DH / 16;                // 16-channel tiles
  extern __shared__ __align__(128) unsigned char smem[];
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::BAR + kWarps * kStages * 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  unsigned char* const ring = smem + S::RING + warp * kStages * U::BYTES;
  const uint32_t ring_s = sm100::smem_u32(ring);
  const uint32_t bars = sm100::smem_u32(smem + S::BAR) + warp * kStages * 8;
  const int n = a.c.n_seqs, per_seq = a.c.Hkv * a.tiles;

  pdl_trigger();
  if (lane == 0)
    for (int i = 0; i < kStages; ++i) sm100::mbar_init(bars + 8 * i, 1);
  if (threadIdx.x == 0) *abort_flag = 0;
  sm100::fence_barrier_init();
  __syncthreads();
  pdl_wait();  // lengths, table, pages and q come from earlier kernels of the stream

  // ---- which units: r0 .. r1 of the list, or (WHOLE) items blockIdx.x, + gridDim.x, ..
  int r0 = 0, r1 = 0, wid = 0;
  const int run = (n + kThreads - 1) / kThreads;
  int* const pre = reinterpret_cast<int*>(smem + S::PRE);
  int* const sum_s = reinterpret_cast<int*>(smem + S::SUM);
  int* const len_s = reinterpret_cast<int*>(smem + S::LEN);
  if constexpr (!WHOLE) {
    // units before each sequence: every thread counts a run of sequences, then a scan over the threads
    int mine = 0;
    const int b0 = min(n, static_cast<int>(threadIdx.x) * run), b1 = min(n, b0 + run);
    for (int b = b0; b < b1; ++b) {
      const int len = __ldg(a.c.lens + b);
      mine += span_of<U::TOK>(a.span, len).n * per_seq;
      if (run == 1) len_s[b] = len;
      if (blockIdx.x == 0 && a.c.err && len > a.span.cap) atomicOr(a.c.err, kErrPage);
    }
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) sum_s[warp] = sum;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += sum_s[w];
    pre[threadIdx.x] = before + sum - mine;
    if (threadIdx.x == kThreads - 1) pre[kThreads] = before + sum;
    if (blockIdx.x == 0) {
      int at = before + sum - mine;
      for (int b = b0; b < b1; ++b) {
        a.prefix[b] = at;
        at += span_of<U::TOK>(a.span, __ldg(a.c.lens + b)).n * per_seq;
      }
      if (threadIdx.x == kThreads - 1) a.prefix[n] = before + sum;
    }
    __syncthreads();
    const Deal d(pre[kThreads], gridDim.x * kWarps);
    wid = warp * gridDim.x + blockIdx.x;  // a short list is spread over the SMs first
    if (wid >= d.warps) return;
    r0 = d.begin(wid);
    r1 = d.begin(wid + 1);
  }

  auto item_at = [&](int u) {
    Item x;
    if constexpr (WHOLE) {
      x.b = u / per_seq;
      const int i = u - x.b * per_seq;
      x.head = i / a.tiles;
      x.tile = i - x.head * a.tiles;
      x.len = __ldg(a.c.lens + x.b);
      x.begin = 0;
      x.s = span_of<U::TOK>(a.span, x.len);
    } else {
      int lo = 0, hi = (n - 1) / run;  // the last run of sequences that begins at or before u
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= u)
          lo = mid;
        else
          hi = mid - 1;
      }
      int b = lo * run, at = pre[lo];
      x.len = run == 1 ? len_s[b] : __ldg(a.c.lens + b);
      x.s = span_of<U::TOK>(a.span, x.len);
      while (at + x.s.n * per_seq <= u) {
        at += x.s.n * per_seq;
        x.len = __ldg(a.c.lens + ++b);
        x.s = span_of<U::TOK>(a.span, x.len);
      }
      const int i = (u - at) / x.s.n;
      x.b = b;
      x.head = i / a.tiles;
      x.tile = i - x.head * a.tiles;
      x.begin = at + i * x.s.n;
    }
    return x;
  };
  auto first_token = [&](const Item& x, int k) { return (k < x.s.sinks ? k : x.s.lo + k - x.s.sinks) * U::TOK; };

  bool dead = false;
  int st_in = 0, st_out = 0;  // ring stages of the next copy and of the next unit
  uint32_t ph_out = 0;
  unsigned bad = 0;          // bit per stage: no such page, the unit's keys are masked
  const int items = n * per_seq;
  const int team = WHOLE ? a.team : 1, my_team = warp / team, in_team = warp - my_team * team;
  for (int at = WHOLE ? static_cast<int>(blockIdx.x + gridDim.x * my_team) : r0; at < (WHOLE ? items : r1);) {
    const Item x = item_at(at);
    // this warp's units of the item: k0, k0 + step, .. (count of them)
    const int step = team;
    const int k0 = WHOLE ? in_team : at - x.begin;
    const int k1 = WHOLE ? x.s.n : min(x.s.n, r1 - x.begin);
    const int count = max(0, (k1 - k0 + step - 1) / step);
    if (WHOLE && x.head == 0 && x.tile == 0 && in_team == 0 && lane == 0 && a.c.err && x.len > a.span.cap)
      atomicOr(a.c.err, kErrPage);
    const unsigned char* const head_base = a.c.pages + static_cast<size_t>(x.head) * cache4::Layout<DH>::BLOCK;
    const int* const table = a.c.table + static_cast<size_t>(x.b) * a.c.max_pages;
    const unsigned page_bytes = static_cast<unsigned>(a.c.Hkv) * cache4::Layout<DH>::BLOCK;
    int pages = 0;  // of units 32 j .. 32 j + 31, one per lane
    auto copy = [&](int i) {
      if ((i & 31) == 0 && i + lane < count)
        pages = __ldg(table + first_token(x, k0 + (i + lane) * step) / kPage);
      int page = __shfl_sync(0xffffffffu, pages, i & 31);
      const int st = st_in;
      st_in = st_in + 1 == kStages ? 0 : st_in + 1;
      bad &= ~(1u << st);
      if (page < 0 || page >= a.c.n_pages) {
        if (lane == 0 && a.c.err) atomicOr(a.c.err, kErrPage);
        bad |= 1u << st;
        page = 0;
      }
      if (lane == 0) {
        const unsigned char* src = head_base + static_cast<unsigned long long>(page) * page_bytes;
        const uint32_t dst = ring_s + st * U::BYTES, bar = bars + 8 * st;
        sm100::mbar_arrive_expect_tx(bar, U::BYTES);
        if constexpr (U::TOK == kPage) {
          sm100::bulk_load(dst, src, U::BYTES, bar);
        } else {
          using L = cache4::Layout<DH>;
          const int r = first_token(x, k0 + i * step) % kPage;
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            sm100::bulk_load(dst + v * U::V_OFF, src + v * L::V_OFF + r * L::CODE_ROW, U::CODES, bar);
            sm100::bulk_load(dst + v * U::V_OFF + U::CODES, src + v * L::V_OFF + L::CODES + r * L::SCALE_ROW,
                             U::SCALES, bar);
          }
        }
      }
    };
    for (int i = 0; i < min(kStages, count); ++i) copy(i);
    const int len = x.len, first_pos = len - a.n_q;

    // ---- the tile's queries: row n of tile j, channels of this lane's share of a key
    uint32_t q[NT][TERMS][KS][2];
    float rs[NT][2];   // this lane's two accumulator columns (rows 2t, 2t + 1): score scale in powers of 2
    int pos[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int row = (x.tile * NT + j) * 8 + g;
      const bool on = row < a.rows;
      const int tok = on ? row / a.group : 0, hd = on ? row - tok * a.group : 0;
      const T* src = static_cast<const T*>(a.q) + (static_cast<size_t>(x.b) * a.n_q + tok) * a.ldq +
                     (x.head * a.group + hd) * DH + t * (DH / 4);
      float f[DH / 4];
      float amax = 0.f;
      bool fin = true;
#pragma unroll
      for (int i = 0; i < DH / 4; i += 16 / static_cast<int>(sizeof(T))) {  // 16 bytes at a time
        const uint4 v = on ? *reinterpret_cast<const uint4*>(src + i) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (SPLIT) {
            f[i + k] = __uint_as_float(w[k]);
          } else {
            f[i + 2 * k] = __uint_as_float(w[k] << 16);
            f[i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < DH / 4; ++i) {
        fin &= fabsf(f[i]) <= 3.4028235e38f;
        amax = fmaxf(amax, fabsf(f[i]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      fin = __shfl_xor_sync(0xffffffffu, fin, 1) && fin;
      fin = __shfl_xor_sync(0xffffffffu, fin, 2) && fin;
      // the row's largest magnitude to 2^10 .. 2^11
      const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -110), 127);
      const float up = amax > 0.f ? __uint_as_float(static_cast<uint32_t>(127 + 10 - e) << 23) : 1.f;
      const float down = amax > 0.f ? __uint_as_float(static_cast<uint32_t>(127 - 10 + e) << 23) : 1.f;
#pragma unroll
      for (int w = 0; w < WK; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v0 = f[8 * w + i] * up, v1 = f[8 * w + i + 4] * up;
          q[j][0][2 * w + (i >> 1)][i & 1] = pack2<__half>(v0, v1);
          if constexpr (SPLIT) q[j][1][2 * w + (i >> 1)][i & 1] = pack2<__half>(lo_term<__half>(v0), lo_term<__half>(v1));
        }
      fin |= first_pos + tok < 0;  // a row that sees nothing gives zeros whatever it holds
      // At most 2^96: a score before it is a multiple of 2^-48 (f16 subnormals both) below 2^28, so it stays in range,
      // and two scores that differ do so by 2^48, as one with all the weight and one with none.
      const float scale =
          fin ? fminf(down * (kCodeScale * rsqrtf(static_cast<float>(DH)) * 1.4426950408889634f), 7.9228163e28f) : NAN;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        rs[j][c] = __shfl_sync(0xffffffffu, scale, 4 * (2 * t + c));
        pos[j][c] = __shfl_sync(0xffffffffu, first_pos + tok, 4 * (2 * t + c));
      }
    }

    // reference and sum per row; what a score becomes a weight with (s - less) * rs + off
    float o[NT][MU][4], m[NT][2], mx[NT][2], l[NT][4], less[NT][2], off[NT][2];
    bool far = false;
    uint32_t top_scale = 0;  // the largest of the keys' scale bytes
    auto clear = [&]() {
      far = false;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        m[j][0] = m[j][1] = -INFINITY;
        less[j][0] = less[j][1] = 0.f;
        off[j][0] = off[j][1] = 7.f;
        l[j][0] = l[j][1] = l[j][2] = l[j][3] = 0.f;
#pragma unroll
        for (int i = 0; i < MU; ++i) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.f;
      }
    };
    auto pass = [&](auto wide) {
      constexpr bool WIDE = decltype(wide)::value;
      for (int i = 0; i < count; ++i) {
        const int st = st_out;
        const int key0 = first_token(x, k0 + i * step);
        const bool gone = (bad >> st) & 1u;
        const unsigned char* const kc = ring + st * U::BYTES;
        if (!sm100::mbar_wait(bars + 8 * st, ph_out, abort_flag)) dead = true;
        // mask: units that hold keys after some row's position, or before some row's window
        const bool edge = gone || key0 + U::TOK - 1 > first_pos ||
                          (len - 1 - key0 >= a.span.window && key0 + U::TOK > a.span.sinks);
        if (edge) {
          // Tokens behind the sequence's end, and those that no row of the call sees (after the sinks, before the first
          // row's window), need never have been written, and 0 * NaN would reach every row: their scales become 0.
          const int behind = len - key0, before = first_pos - a.span.window + 1 - key0, unseen = a.span.sinks - key0;
#pragma unroll
          for (int r = lane; r < U::TOK; r += 32)
            if (gone || r >= behind || (r < before && r >= unseen)) {
              using Row = std::conditional_t<DH == 128, uint2, std::conditional_t<DH == 64, uint32_t, unsigned short>>;
#pragma unroll
              for (int v = 0; v < 2; ++v) reinterpret_cast<Row*>(ring + st * U::BYTES + v * U::V_OFF + U::CODES)[r] = Row{};
            }
          sm100::fence_proxy_async_smem();  // the stage's next copy comes after these stores
          __syncwarp();
        }
        // S^T: keys g and g + 8 of each tile sit at rows (g >> 1) + 4 (g & 1) and 8 further
        const int rk = (g >> 1) + 4 * (g & 1);
        float s[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int j = 0; j < NT; ++j) s[mt][j][0] = s[mt][j][1] = s[mt][j][2] = s[mt][j][3] = 0.f;
          uint32_t w[2][WK];
          uint32_t sb[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = 16 * mt + rk + 8 * h;
            lds_words<WK>(kc + r * (DH / 2) + t * (DH / 8), w[h]);
            const unsigned char* sp = kc + U::CODES + r * (DH / 16);
            if constexpr (DH == 128)
              sb[h] = *reinterpret_cast<const unsigned short*>(sp + 2 * t);
            else
              sb[h] = sp[DH == 64 ? t : t >> 1];
          }
          if (!WIDE) top_scale = max(top_scale, DH == 128 ? max(max(sb[0] & 255u, sb[1] & 255u), max(sb[0], sb[1]) >> 8)
                                                          : max(sb[0], sb[1]));
          Scale sc[2];
#pragma unroll
          for (int i = 0; i < WK; ++i) {
            if (i == 0 || (DH == 128 && i == 2)) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t b = DH == 128 ? (i == 0 ? sb[h] & 255u : sb[h] >> 8) : sb[h];
                sc[h] = scale_pair<WIDE>(b * 0x800080u);
              }
            }
            uint32_t v0[4], v1[4];
            dequant<WIDE>(w[0][i], sc[0], v0);
            dequant<WIDE>(w[1][i], sc[1], v1);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < TERMS; ++e) {
                mma(s[mt][j], v0[0], v1[0], v0[1], v1[1], q[j][e][2 * i][0], q[j][e][2 * i][1]);
                mma(s[mt][j], v0[2], v1[2], v0[3], v1[3], q[j][e][2 * i + 1][0], q[j][e][2 * i + 1][1]);
              }
          }
        }
        if (edge) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = key0 + 16 * mt + rk + 8 * (i >> 1), p = pos[j][i & 1];
                if (gone || key > p || (p - key >= a.span.window && key >= a.span.sinks)) s[mt][j][i] = -INFINITY;
              }
        }
        // The rows' references are raised only when some score passes one by more than 2^8: most units
        // need no exchange between lanes and leave O as it is. Weights are 2^7 .. 2^15 at most.
        bool above = false;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            mx[j][c] = fmaxf(s[0][j][c], s[0][j][c + 2]);
#pragma unroll
            for (int mt = 1; mt < MT; ++mt) mx[j][c] = max3(mx[j][c], s[mt][j][c], s[mt][j][c + 2]);
            above |= (mx[j][c] - m[j][c]) * rs[j][c] > 8.f;  // -inf less -inf: no
          }
        if (__any_sync(0xffffffffu, above)) {
          far = false;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            float corr[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float top = mx[j][c];
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
              // this row's own: whether another row's is raised does not show in its bits
              if (!((top - m[j][c]) * rs[j][c] > 8.f)) top = m[j][c];
              const float ref = top == -INFINITY ? 0.f : top;  // nothing seen yet: weights 2^-inf = 0
              corr[c] = ex2((m[j][c] - ref) * rs[j][c]);
              m[j][c] = top;
              // s * rs - ref * rs in one rounding is off by 2^-24 of ref * rs: where that is large the
              // difference is taken first
              const bool big = fabsf(ref * rs[j][c]) > 1048576.f;
              far |= big;
              less[j][c] = big ? ref : 0.f;
              off[j][c] = big ? 7.f : 7.f - ref * rs[j][c];
            }
#pragma unroll
            for (int i = 0; i < MU; ++i) {
              o[j][i][0] *= corr[0], o[j][i][1] *= corr[1];
              o[j][i][2] *= corr[0], o[j][i][3] *= corr[1];
            }
            l[j][0] *= corr[0], l[j][1] *= corr[1];
          }
          far = __any_sync(0xffffffffu, far);
        }
        if (far) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[mt][j][i] -= less[j][i & 1];
        }
        uint32_t pb[MT][NT][TERMS][2];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              fma_pair(s[mt][j][2 * h], s[mt][j][2 * h + 1], rs[j][0], rs[j][1], off[j][0], off[j][1]);
              const float p0 = ex2(s[mt][j][2 * h]), p1 = ex2(s[mt][j][2 * h + 1]);
              pb[mt][j][0][h] = transpose8(pack2<__half>(p0, p1));
              if constexpr (SPLIT) pb[mt][j][1][h] = transpose8(pack2<__half>(lo_term<__half>(p0), lo_term<__half>(p1)));
            }
            // the rows' sums, of the weights as O takes them: a product with ones
#pragma unroll
            for (int e = 0; e < TERMS; ++e)
              mma(l[j], 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, pb[mt][j][e][0], pb[mt][j][e][1]);
          }
        // O^T += V^T P^T: keys 2t, 2t + 1, 2t + 8, 2t + 9 of a tile sit at rows t, t + 4, t + 8, t + 12
        const unsigned char* const vc = kc + U::V_OFF;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          constexpr int WV = DH == 128 ? 2 : 1;
          uint32_t w[4][WV], sb[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = 16 * mt + t + 4 * k;
            if constexpr (DH == 32)
              w[k][0] = *reinterpret_cast<const unsigned short*>(vc + r * (DH / 2) + 2 * g);
            else
              lds_words<WV>(vc + r * (DH / 2) + g * (DH / 16), w[k]);
            sb[k] = vc[U::CODES + r * (DH / 16) + (DH == 128 ? g : DH == 64 ? g >> 1 : g >> 2)];
          }
          const Scale sa = scale_pair<WIDE>((sb[0] + sb[1] * 0x10000u) * 128u),
                      sz = scale_pair<WIDE>((sb[2] + sb[3] * 0x10000u) * 128u);
#pragma unroll
          for (int i = 0; i < WV; ++i)
#pragma unroll
            for (int half = 0; half < (DH == 32 ? 1 : 2); ++half) {
              const uint32_t sel = half ? 0x7632u : 0x5410u;  // channels 4 half .. of both keys
              uint32_t v0[4], v1[4];
              dequant<WIDE>(__byte_perm(w[0][i], w[1][i], sel), sa, v0);
              dequant<WIDE>(__byte_perm(w[2][i], w[3][i], sel), sz, v1);
              const int mu = 4 * i + 2 * half;
#pragma unroll
              for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < TERMS; ++e) {
                  mma(o[j][mu], v0[0], v0[1], v1[0], v1[1], pb[mt][j][e][0], pb[mt][j][e][1]);
                  mma(o[j][mu + 1], v0[2], v0[3], v1[2], v1[3], pb[mt][j][e][0], pb[mt][j][e][1]);
                }
            }
        }
        __syncwarp();  // every lane has read the stage
        if (++st_out == kStages) {
          st_out = 0;
          ph_out ^= 1u;
        }
        if (i + kStages < count) copy(i + kStages);
      }
    };
    clear();
    pass(std::false_type{});
    // A scale that is too large for the short way: keys' are looked at, values' show in O. Once more
    // then, the long way (as for a query that is not finite, to no effect).
    bool again = top_scale >= kWideScale;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < MU; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) again |= !(fabsf(o[j][i][k]) <= 3.4028235e38f);
    if (__any_sync(0xffffffffu, again)) {
      clear();
      for (int i = 0; i < min(kStages, count); ++i) copy(i);
      pass(std::true_type{});
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) m[j][c] *= rs[j][c];  // in powers of 2
    auto out_row = [&](int rr) {
      const int tok = rr / a.group, hd = rr - tok * a.group;
      return static_cast<T*>(a.out) + ((static_cast<size_t>(x.b) * a.n_q + tok) * a.H + x.head * a.group + hd) * DH;
    };
    if constexpr (WHOLE) {
      // the warps' results of the item, added
      const int w0 = my_team * team;
      auto meet = [&]() {
        if (team == kWarps)
          __syncthreads();
        else if (team > 1)
          asm volatile("bar.sync %0, %1;" ::"r"(1 + my_team), "r"(32 * team) : "memory");
        else
          __syncwarp();
      };
      float* const merge = reinterpret_cast<float*>(smem + S::MERGE);
      float* const ml = reinterpret_cast<float*>(smem + S::ML);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (g == 0) {
            ml[warp * 8 * NT + 8 * j + 2 * t + c] = m[j][c];
            ml[(kWarps + warp) * 8 * NT + 8 * j + 2 * t + c] = l[j][c];
          }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        meet();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = -INFINITY;
          for (int w = w0; w < w0 + team; ++w) top = fmaxf(top, ml[w * 8 * NT + 8 * j + 2 * t + c]);
          const float by = top == -INFINITY && m[j][c] == top ? (l[j][c] == l[j][c] ? 0.f : NAN) : ex2(m[j][c] - top);
#pragma unroll
          for (int i = 0; i < MU; ++i)
            *reinterpret_cast<float2*>(merge + (warp * 8 + 2 * t + c) * S::LD + g * (DH / 8) + 2 * i) =
                make_float2(o[j][i][c] * by, o[j][i][c + 2] * by);
        }
        meet();
        for (int e = 32 * in_team + lane; e < 8 * DH / 4; e += 32 * team) {
          const int row = e / (DH / 4), ch = (e - row * (DH / 4)) * 4;
          const int rr = (x.tile * NT + j) * 8 + row;
          if (rr >= a.rows) continue;
          float top = -INFINITY, sum = 0.f;
          for (int w = w0; w < w0 + team; ++w) top = fmaxf(top, ml[w * 8 * NT + 8 * j + row]);
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int w = w0; w < w0 + team; ++w) {
            const float lw = ml[(kWarps + w) * 8 * NT + 8 * j + row], mw = ml[w * 8 * NT + 8 * j + row];
            sum += mw == -INFINITY ? lw * 0.f : lw * ex2(mw - top);  // 0, or NaN of a query that is not finite
            const float4 v = *reinterpret_cast<const float4*>(merge + (w * 8 + row) * S::LD + ch);
            acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
          }
          T* dst = out_row(rr) + ch;
          const float inv = sum == 0.f ? 0.f : kCodeScale / sum;
          if constexpr (SPLIT)
            *reinterpret_cast<float4*>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
          else
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
        }
      }
      meet();  // ml and merge may be written again
      at += gridDim.x * (kWarps / team);
    } else {
      const bool all = k0 == 0 && k1 == x.s.n;
      float* const part = a.parts + static_cast<size_t>(2 * wid + (at == r0 ? 0 : 1)) * (DH + 2) * 8 * NT;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int row = 8 * j + 2 * t + c, rr = x.tile * NT * 8 + row;
          if (!all && g == 0) {  // all rows: half a sector would have to be filled from memory when read
            part[8 * NT * DH + row] = m[j][c];
            part[8 * NT * (DH + 1) + row] = l[j][c];
          }
          if (rr >= a.rows) continue;
          const float by = !all ? 1.f : l[j][c] == 0.f ? 0.f : kCodeScale / l[j][c];
          float* const pd = part + row * DH + g * (DH / 8);
          T* const dst = out_row(rr) + g * (DH / 8);
#pragma unroll
          for (int i = 0; i < MU; i += 2) {
            const float v0 = o[j][i][c] * by, v1 = o[j][i][c + 2] * by;
            const float v2 = o[j][i + 1][c] * by, v3 = o[j][i + 1][c + 2] * by;
            if (!all)
              *reinterpret_cast<float4*>(pd + 2 * i) = make_float4(v0, v1, v2, v3);
            else if constexpr (SPLIT)
              *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(v0, v1, v2, v3);
            else
              *reinterpret_cast<uint2*>(dst + 2 * i) = make_uint2(pack2<T>(v0, v1), pack2<T>(v2, v3));
          }
        }
      at = x.begin + k1;
    }
  }
  if (dead) {
    if (lane == 0 && a.c.err) atomicOr(a.c.err, kErrTimeoutEpilogue);
    // let the copies in flight land before the CTA's shared memory goes away: stages from st_out on
    // are in phase ph_out, those before it in the next; waiting for both parities covers either
    for (int k = 0; k < 2 * kStages; ++k) sm100::mbar_wait_drain(bars + 8 * (k >> 1), k & 1);
  }
}

// Rows of items that several warps shared: their parts added in the order of the keys. Rows that
// see nothing: zeros. A CTA takes `per` rows of an item (gridDim.y slices): one thread per four
// channels of a row and per group of consecutive parts, so that the loads of many parts are in
// flight at once; then neighbouring groups are added, in a fixed tree.
template <int DH, typename T, int NT>
__global__ void __launch_bounds__(1024) cache_attn_join_kernel(const DecodeArgs a, int grid_warps, int per) {
  pdl_trigger();
  pdl_wait();
  __shared__ float top_s[1024], sum_s[1024];
  __shared__ float4 acc_s[1024];
  const int tile = blockIdx.x % a.tiles, bh = blockIdx.x / a.tiles;
  const int b = bh / a.c.Hkv, head = bh - b * a.c.Hkv;
  const int at = a.prefix[b], after = a.prefix[b + 1], units = a.prefix[a.c.n_seqs];
  const int n = (after - at) / (a.c.Hkv * a.tiles);
  const Deal d(units, grid_warps);
  const int begin = at + (head * a.tiles + tile) * n;
  int w0 = 0, w1 = -1;
  if (n > 0) {
    w0 = d.warp_of(begin);
    w1 = d.warp_of(begin + n - 1);
    if (w0 == w1) return;  // that warp wrote the result
  }
  constexpr int PART = (DH + 2) * 8 * NT, QUADS = DH / 4;
  const int lanes = per * QUADS, groups = blockDim.x / lanes;  // threads of a group of parts
  const int t = threadIdx.x, group = t / lanes, e = t - group * lanes;
  const int row = blockIdx.y * per + e / QUADS, ch = (e % QUADS) * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f, top = -INFINITY;
  if (group < groups) {
    const int each = (w1 - w0 + groups) / groups, from = w0 + group * each, to = min(from + each, w1 + 1);
    const bool second = begin > d.begin(w0);  // the first part is its warp's second stretch
    for (int w = from; w < to; w += 4) {
      float mw[4], lw[4];
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int x = min(w + k, to - 1);
        const float* p = a.parts + static_cast<size_t>(2 * x + (x == w0 && second ? 1 : 0)) * PART;
        mw[k] = p[8 * NT * DH + row];
        lw[k] = p[8 * NT * (DH + 1) + row];
        v[k] = *reinterpret_cast<const float4*>(p + row * DH + ch);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (w + k >= to) break;
        const float up = fmaxf(top, mw[k]);
        const float keep = top == -INFINITY ? 0.f : ex2(top - up), by = mw[k] == -INFINITY ? 0.f : ex2(mw[k] - up);
        top = up;
        sum = fmaf(lw[k], by, sum * keep);
        acc.x = fmaf(v[k].x, by, acc.x * keep), acc.y = fmaf(v[k].y, by, acc.y * keep);
        acc.z = fmaf(v[k].z, by, acc.z * keep), acc.w = fmaf(v[k].w, by, acc.w * keep);
      }
    }
  }
  top_s[t] = top;
  sum_s[t] = sum;
  acc_s[t] = acc;
  for (int s = 1; s < groups; s *= 2) {
    __syncthreads();
    const int o = t + s * lanes;
    if (group % (2 * s) == 0 && group + s < groups) {
      const float mo = top_s[o], up = fmaxf(top, mo);
      const float keep = top == -INFINITY ? 0.f : ex2(top - up), by = mo == -INFINITY ? 0.f : ex2(mo - up);
      const float4 v = acc_s[o];
      sum = fmaf(sum_s[o], by, sum * keep);
      acc.x = fmaf(v.x, by, acc.x * keep), acc.y = fmaf(v.y, by, acc.y * keep);
      acc.z = fmaf(v.z, by, acc.z * keep), acc.w = fmaf(v.w, by, acc.w * keep);
      top_s[t] = top = up;
      sum_s[t] = sum;
      acc_s[t] = acc;
    }
  }
  const int rr = tile * 8 * NT + row;
  if (group != 0 || row >= 8 * NT || rr >= a.rows) return;
  const int tok = rr / a.group, hd = rr - tok * a.group;
  T* dst = static_cast<T*>(a.out) + ((static_cast<size_t>(b) * a.n_q + tok) * a.H + head * a.group + hd) * DH + ch;
  const float inv = sum == 0.f ? 0.f : kCodeScale / sum;
  if constexpr (std::is_same_v<T, float>)
    *reinterpret_cast<float4*>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  else
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
}

int tile_rows(int rows, bool bf16) { return bf16 && rows > 8 ? 16 : 8; }

// Most units an item may have, and what follows from it
long long most_units(int max_pages, int n_q, int dh, int window, int sinks) {
  const int tok = dh == 128 ? 32 : 64;
  const long long all = static_cast<long long>(max_pages) * kPage / tok;
  // a window and the tokens before it cross at most one more unit than they fill
  const long long seen = (static_cast<long long>(window) + n_q + tok - 2) / tok + 1 + (sinks + tok - 1LL) / tok;
  return all < seen ? all : seen;
}
// Whether items are dealt whole. Whole, an item takes its warps' share of the longest one's units; dealt in
// stretches, the average, and a second kernel. bf16, 32 / 8 heads of 64, all lengths alike, whole and in
// stretches, for 2048, 4096 and 8192 tokens (32, 64 and 128 units): one sequence (8 items) 8.6 and 9.3, 13.0 and
// 9.9, 22.3 and 12.0 us; 8 sequences 10.4 and 13.8, 15.0 and 18.3, 24.1 and 23.2; 16 sequences 11.7 and 18.3,
// 16.8 and 23.4, 26.5 and 32.4; 64 sequences 25.8 and 32.3, 44.2 and 49.3, 78.7 and 78.5. Where lengths differ
// the shares of whole items do too, so beyond 32 units only items that have a CTA each and would fill most SMs.
// What decides is the table's width, since no launch knows the lengths: 64 sequences of 500 tokens take 11.6 us
// with a table that ends there and 17.1 with one for 131,072.
bool deal_whole(long long most, long long items) {
  return most <= 32 || (most <= 64 && items >= 64 && items <= 148);
}
struct Plan {
  bool whole;
  long long items, units;
  int ctas, warps;  // warps: of the grid, when they share a list of units
  int team;
};
Plan plan_of(int n_seqs, int max_pages, int n_q, int tiles, int Hkv, int dh, int window, int sinks,
             int cta_warps) {
  Plan p;
  const long long most = most_units(max_pages, n_q, dh, window, sinks);
  p.items = static_cast<long long>(n_seqs) * Hkv * tiles;
  p.units = p.items * most;
  p.whole = deal_whole(most, p.items);
  // the widest team that leaves every item one at once (148 SMs; 64 sequences of 1024 tokens, 512 items: teams
  // of 4 16.0 us, of 16 27.7; 32 sequences: 11.4 and 15.0)
  p.team = cta_warps;
  while (p.team > 1 && (cta_warps % p.team || p.team > most || p.items * p.team > 148LL * cta_warps)) --p.team;
  // a short list over all SMs, one unit a warp (one sequence of 4096 tokens 10.0 us, 11.9 with 16 warps a CTA at
  // work, 18.4 with stretches of at least four units)
  const long long share = p.whole ? cta_warps / p.team : 1;
  const long long want = ((p.whole ? p.items : p.units) + share - 1) / share;
  p.ctas = static_cast<int>(want < 148 ? want : 148);  // one per SM
  p.warps = p.ctas * cta_warps;
  return p;
}

template <int DH, typename T, int NT>
cudaError_t launch_decode(const CacheAttnArgs& c, cudaStream_t st) {
  constexpr int kWarps = Shape<DH, T, NT>::WARPS;
  DecodeArgs a{};
  a.c = c.c;
  a.span = {c.c.max_pages * kPage, c.n_q, c.window, c.sinks};
  a.q = c.q, a.ldq = c.ldq, a.out = c.out;
  a.n_q = c.n_q, a.H = c.H, a.group = c.H / c.c.Hkv;
  a.rows = c.n_q * a.group;
  a.tiles = (a.rows + 8 * NT - 1) / (8 * NT);
  const Plan p = plan_of(c.c.n_seqs, c.c.max_pages, c.n_q, a.tiles, c.c.Hkv, DH, c.window, c.sinks, kWarps);
  auto kernel = p.whole ? cache_attn_kernel<DH, T, NT, true> : cache_attn_kernel<DH, T, NT, false>;
  const int smem = p.whole ? DecodeSmem<DH, T, NT, true>::BYTES : DecodeSmem<DH, T, NT, false>::BYTES;
  static std::atomic<uint64_t> done[2];
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem, done[p.whole]);
  if (e != cudaSuccess) return e;
  a.team = p.team;
  if (!p.whole) {
    a.parts = static_cast<float*>(c.ws);
    a.prefix = reinterpret_cast<int*>(a.parts + static_cast<size_t>(2) * p.warps * (DH + 2) * 8 * NT);
  }
  e = launch_pdl(kernel, dim3(p.ctas), dim3(32 * kWarps), smem, st, a);
  if (e == cudaSuccess && !p.whole) {
    // threads for a group of about four parts each of an item's parts (were they alike): its rows
    // together, or fewer rows a CTA where that takes more than 1024
    const int rows = 8 * NT < a.rows ? 8 * NT : a.rows;
    const long long parts = p.units < p.warps ? p.units : p.warps;
    const int want = static_cast<int>((parts + 4 * p.items - 1) / (4 * p.items));
    int per = rows;
    while (per > 1 && per * (DH / 4) * want > 1024) per = (per + 1) / 2;
    const int threads = per * (DH / 4) * want < 1024 ? (per * (DH / 4) * want + 31) / 32 * 32 : 1024;
    e = launch_pdl(cache_attn_join_kernel<DH, T, NT>, dim3(static_cast<unsigned>(p.items), (rows + per - 1) / per),
                   dim3(threads), 0, st, a, p.warps, per);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int DH>
cudaError_t launch_dh(const CacheAttnArgs& a, bool bf16, cudaStream_t st) {
  if (!bf16) return launch_decode<DH, float, 1>(a, st);
  return tile_rows(a.n_q * (a.H / a.c.Hkv), true) == 16 ? launch_decode<DH, __nv_bfloat16, 2>(a, st)
                                                        : launch_decode<DH, __nv_bfloat16, 1>(a, st);
}

}  // namespace

size_t cache_attention_workspace(int n_seqs, int max_pages, int n_q, int H, int Hkv, int dh, int window, int sinks) {
  // the larger of what either type needs: its tiles decide how many parts there are, and their size
  size_t most = 0;
  const int rows = n_q * (H / Hkv);
  for (int bf16 = 0; bf16 < 2; ++bf16) {
    const int tr = tile_rows(rows, bf16), tiles = (rows + tr - 1) / tr;
    const Plan p = plan_of(n_seqs, max_pages, n_q, tiles, Hkv, dh, window, sinks, 16);
    if (p.units > 0x7fffffffLL) return 0;
    const size_t bytes = p.whole ? 0 : static_cast<size_t>(2) * kMaxWarps * (dh + 2) * tr * 4;
    most = bytes > most ? bytes : most;
  }
  return most + (static_cast<size_t>(n_seqs) + 1) * 4;
}

cudaError_t launch_cache_attention(const CacheAttnArgs& a, int dh, bool bf16, cudaStream_t st) {
  switch (dh) {
    case 32: return launch_dh<32>(a, bf16, st);
    case 64: return launch_dh<64>(a, bf16, st);
    case 128: return launch_dh<128>(a, bf16, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace rmt
