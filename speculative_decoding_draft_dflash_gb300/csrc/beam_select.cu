// The k best of beams x vocabulary by accumulated log-probability:
//
//   score(i, v) = s_i + ((x_iv - m_i) - log sum_u e^(x_iu - m_i)),  m_i = max_u x_iu,
// ordered by score, ties by the lowest i * vocab + v.
//
// Two kernels. The scan reads every logit once. A CTA takes a piece of one row, tile by tile: the
// sum of e^(x - ref) under a reference that hardly ever moves, and the piece's k largest logits. A row's
// own order needs no sum, and a candidate of the whole selection is among its row's k best.
// The merge, a CTA per sequence, joins the pieces' sums, ranks the candidates in 64 bits and writes.
//
// The k largest. Every lane keeps the maximum of what it has seen. The q-th largest of a warp's lanes, of
// the CTA's eight such values the s-th largest (q s >= k), is reached by at least k elements, so that
// nothing below it is a candidate. (s = 6: random logits reach it 1.8 k times; s = 8, the lowest value,
// 2.6 k times.) The first tile gives such a bound, more of them a better one (without waiting for
// one another: a warp's old value is only a lower one). A lane whose 64 bytes of a tile reach it notes their
// maximum and number, for itself; the elements of noted runs are looked at one by one at the end, against the
// bound of all tiles, of a few runs of a warp. A lane whose notes are full has the bound looked at again, and
// where that does not help (rows of equal or of ascending logits) the warp keeps the k runs of the largest
// maxima, of equal ones the first: each of the others has k elements before all of its own. From then on a run
// is noted only above the least of these, which themselves stay candidates. (Elements taken as they came, or a list of a
// warp's, cost more than the sums: what a warp does beside them waits for votes, shuffles and instructions
// that are not in the cache.)
//
// The sum. Which candidate of two beams is the better one is decided by the difference of two such
// sums, so their errors must stay far below the gaps between scores (about 10^-2 among the best of a
// vocabulary): d = x - ref (exact for bf16 within 16 binades), e^d = 2^(d log2 e). The product's rounding
// moves a term by up to 10^-6, but either way and by another amount for every value, so that 10^-8 is left
// of it in a sum of a vocabulary (measured: 2 10^-8 at most); the few large terms of a row, where
// it does not average out, are taken again by the merge. Terms in fp32, a thread's tiles added with their
// rounding errors kept, the rest in 64 bits. The order of the additions depends on the
// vocabulary alone, so equal rows have equal sums and their candidates tie as they should. (Terms that all err
// one way, as where a row repeats one value: d <= 12 is off by 12 2^-24, t = d log2 e by 12 2^-24 and 12 1.3 10^-8
// of e^d, 2^t by 2^-22, 1.9 10^-6 in all.)
//
// What bounds it. 256 rows of 131072 bf16 logits, 16 kept: 25.9 us in a replayed graph, where HBM would allow
// 9.9: the scan about 20 (12 instructions a logit; the issue slots are half used, as one SM has two rows and
// the next one), the merge the rest. 256 rows of 50001 f32 logits 22.4 (7.5), 1024 greedy rows of 131072 54.9
// (39.5), 2048 of 32000 50.5 (19.3). One row of 32000 9.8, 128 rows of 100 to 1000 9.6: launches and two short
// chains of barriers and code that is not in the cache yet. Rows whose notes fill up take longer: 256 of 131072
// clipped at 1.5 standard deviations 43.4, of zeros 34.2, with one token in 10^4 allowed 56.6.
#include <float.h>

#include "tree.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMergeCap = 1024;  // entries of the merge's list
constexpr float kFar = 12.f;   // how far above the reference a logit may lie

typedef unsigned long long u64;

// Largest first: the logit's bits in order (-0 as 0), then the lowest token. Never 0.
__device__ __forceinline__ u64 entry_of(float x, uint32_t token) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (u64)(b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u)) << 32 | (0xffffffffu - token);
}
__device__ __forceinline__ float logit_of(u64 e) {
  const uint32_t k = (uint32_t)(e >> 32);
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint32_t token_of(u64 e) { return 0xffffffffu - (uint32_t)e; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log2 e and ln 2 as a float and what it leaves.
constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f;
constexpr float kLn2 = 0.693147182f, kLn2Low = -1.90465421e-9f;

// The term of e^d: 0 for minus infinity.
__device__ __forceinline__ float2 exp_of(float2 d) {
  const float2 t = __fmul2_rn(d, make_float2(kLog2e, kLog2e));
  return make_float2(ex2(t.x), ex2(t.y));
}

// e^d to 2^-27 as hi + lo, -80 <= d <= 80: e^d = 2^n 2^(f + g), f = fl(d log2 e) - n and g what the
// product left, and 2^f = 1 + f ln 2 + f^2 P(f), the first product and sum with their rounding errors
// (P: the Taylor terms up to f^8, 10^-9 at |f| = 1/2).
__device__ __noinline__ float2 exp_pair(float d) {
  const float t = d * kLog2e, n = rintf(t), f = t - n;
  const float g = fmaf(d, kLog2eLow, fmaf(d, kLog2e, -t));
  float q = 1.32154868e-6f;
  q = fmaf(q, f, 1.52527338e-5f);
  q = fmaf(q, f, 1.54035304e-4f);
  q = fmaf(q, f, 1.33335581e-3f);
  q = fmaf(q, f, 9.61812911e-3f);
  q = fmaf(q, f, 5.55041087e-2f);
  q = fmaf(q, f, 0.240226507f);
  const float p = f * kLn2;
  const float pe = fmaf(f, kLn2, -p) + fmaf(f, kLn2Low, g * kLn2);
  const float s = 1.f + p, se = p - (s - 1.f);
  const float w = f * f * q, lo = se + (pe + (w + g * kLn2 * (p + w)));
  const float scale = __int_as_float(((int)n + 127) << 23);
  return make_float2(s * scale, lo * scale);
}
// log x to 10^-8 for a finite x > 0: x = 2^e m, log m = z + (m e^-z - 1), z = logf(m).
__device__ __forceinline__ double log_of(double x) {
  const long long b = __double_as_longlong(x);
  const int e = (int)(b >> 52) - 1023;
  const double m = __longlong_as_double((b & 0xfffffffffffffll) | 0x3ff0000000000000ll);
  const float mh = (float)m, ml = (float)(m - (double)mh), z = logf(mh);
  const float2 w = exp_pair(-z);
  const float p = mh * w.x, y = (p - 1.f) + (fmaf(mh, w.x, -p) + fmaf(mh, w.y, ml * w.x));
  return (double)e * 0.693147180559945309417 + ((double)z + (double)(y - 0.5f * y * y));
}

// 16 bytes of a row: eight bf16 logits or four f32.
struct Bytes16 {
  uint32_t w[4];
  // of the 32 bytes a, b those from byte `shift` on
  __device__ __forceinline__ void from(uint4 a, uint4 b, int shift) {
    uint32_t s[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (shift & 8) {
#pragma unroll
      for (int i = 0; i < 6; ++i) s[i] = s[i + 2];
    }
    if (shift & 4) {
#pragma unroll
      for (int i = 0; i < 5; ++i) s[i] = s[i + 1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(s[i], s[i + 1], (shift & 2) * 8);
  }
};
template <typename T> struct Vec;
template <> struct Vec<bf16> : Bytes16 {
  static constexpr int E = 8;
  static __device__ __forceinline__ float read(const bf16* x) { return __bfloat162float(*x); }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
  __device__ __forceinline__ void keep(int n) {  // all but the first n become -inf
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * i >= n) w[i] = (w[i] & 0xffff0000u) | 0xFF80u;
      if (2 * i + 1 >= n) w[i] = (w[i] & 0xffffu) | 0xFF800000u;
    }
  }
  // Largest elements, in as many lots as is cheap: two halves of a word (NaN only where all are)
  typedef uint32_t Most;
  static __device__ __forceinline__ Most larger(Most a, Most b) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  static __device__ __forceinline__ float value(Most a) {
    return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
  __device__ __forceinline__ Most most() const { return larger(larger(w[0], w[1]), larger(w[2], w[3])); }
  static constexpr Most kNone = 0xFF80FF80u;
};
template <> struct Vec<float> : Bytes16 {
  static constexpr int E = 4;
  static __device__ __forceinline__ float read(const float* x) { return *x; }
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(w[i]); }
  __device__ __forceinline__ void keep(int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i >= n) w[i] = 0xFF800000u;
  }
  typedef float Most;
  static __device__ __forceinline__ Most larger(Most a, Most b) { return fmaxf(a, b); }
  static __device__ __forceinline__ float value(Most a) { return a; }
  __device__ __forceinline__ Most most() const { return fmaxf(fmaxf(at(0), at(1)), fmaxf(at(2), at(3))); }
  static constexpr Most kNone = -INFINITY;
};

struct Piece {  // of a row: the reference and the sum under it
  double sum;   // NaN: a logit that is NaN or infinite
  float ref;    // -inf: no finite logit
  int pad;
};

struct Scan {
  const void* logits;
  long long ld_seq, ld_beam;
  u64* lists;     // [rows][splits][k], best first, 0 where there is none
  Piece* pieces;  // [rows][splits]
  int vocab, rows_per_seq, splits, chunk, k, pieces_n;
};

// (The code here is run once or twice a piece by warps that do different things. What does not fit the
// instruction cache is fetched again and again, so it is kept small: few instances, few loops unrolled.)

// An entry's place among those of a list, n of them padded with zeros to a multiple of four: how many
// are before it.
__device__ __forceinline__ int rank_of(const u64* e, int n, u64 mine) {
  int rank = 0;
#pragma unroll 1
  for (int j = 0; j < n; j += 4) {
    const ulonglong2 a = reinterpret_cast<const ulonglong2*>(e + j)[0], b = reinterpret_cast<const ulonglong2*>(e + j)[1];
    rank += (a.x > mine) + (a.y > mine) + (b.x > mine) + (b.y > mine);
  }
  return rank;
}

// A float's bits in order.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

constexpr int kSlots = 8;      // notes of a lane
constexpr int kEntries = 160;  // of a warp's list: kBeamMax and 32 at least

// Cuts a list of n entries in `slots` places (a multiple of 32; 0: none) to the k best, the others 0. Returns a
// value that these reach and the others do not: the k-th largest logit's bits one by one, of those in which the
// entries differ, then, among equal ones, the token's. FEW: with few registers, for calls out of the loop that reads
// the logits: what a call may use, its caller cannot keep over it (256 rows of 131072 25.9 us, and 28.1 with the
// halves of the entries in registers; 2 against 5 us a call). Counting those before each entry, and so sorting
// them, took 5 us a call.
static_assert(kEntries <= 32 * kSlots, "places of a list");
template <bool FEW>
__device__ __noinline__ u64 cut(u64* e, int slots, int n, int k) {
  constexpr int UNROLL = FEW ? 1 : kSlots;
  const int lane = threadIdx.x & 31;
  const uint32_t* half = reinterpret_cast<const uint32_t*>(e);  // of an entry: the token's, the logit's
  uint32_t limit[2] = {0, 1};
  if (n > k) {
#pragma unroll 1
    for (int word = 1; word >= 0; --word) {
      uint32_t kept[UNROLL];
      auto load = [&](int t) -> uint32_t {  // 0: not in question
        const int i = lane + 32 * t;
        const uint32_t hi = i < slots ? half[2 * i + 1] : 0;
        return hi != 0 && (word == 1 || hi == limit[1]) ? half[2 * i + word] : 0;
      };
      auto key = [&](int t) -> uint32_t { return FEW ? load(t) : kept[t % UNROLL]; };
      uint32_t any = 0, all = 0xffffffffu;
#pragma unroll UNROLL
      for (int t = 0; t < kSlots; ++t) {
        const uint32_t x = kept[t % UNROLL] = load(t);
        if (x != 0) any |= x, all &= x;
      }
      all = __reduce_and_sync(0xffffffffu, all);
      const uint32_t differ = __reduce_or_sync(0xffffffffu, any) & ~all;
      uint32_t least = 0;
#pragma unroll 1
      for (uint32_t left = differ; left != 0 && n != k;) {
        const uint32_t bit = 0x80000000u >> __clz(left), trial = least | bit;
        left ^= bit;
        int c = 0;
#pragma unroll UNROLL
        for (int t = 0; t < kSlots; ++t) c += (key(t) & differ) >= trial;
        c = __reduce_add_sync(0xffffffffu, c);
        if (c >= k) least = trial, n = c;
      }
      least |= all;
      (word == 1 ? limit[1] : limit[0]) = least;
      if (n == k) break;
      int sure = 0;  // (of the logits: what is above the k-th stays, and the rest are alike)
#pragma unroll UNROLL
      for (int t = 0; t < kSlots; ++t) sure += key(t) > least;
      sure = __reduce_add_sync(0xffffffffu, sure);
      n -= sure, k -= sure;
    }
  }
  const u64 last = (u64)limit[1] << 32 | limit[0];
  int at = 0;
#pragma unroll 1
  for (int i = lane; i < slots; i += 32) {
    const u64 v = e[i];
    const bool in = v >= last;
    const unsigned who = __ballot_sync(0xffffffffu, in);
    __syncwarp();
    if (in) e[at + __popc(who & ((1u << lane) - 1))] = v;
    at += __popc(who);
    __syncwarp();
  }
#pragma unroll 1
  for (int i = at + lane; i < slots; i += 32) e[i] = 0;
  __syncwarp();
  return last;
}

// A warp's notes, one lane's below one another: drops those below the bound and, if a lane is still full,
// all but the k best, which it spreads over the lanes. Returns a bound that these reach, the least that a later
// run has to have, which is above it (of equal maxima the first runs are kept, and later ones have k elements
// before all of theirs), and the lane's notes.
struct Cleared {
  float bound, later;
  int of_lane;
};
__device__ __noinline__ Cleared clear_notes(u64* notes, int n, int k, float bound) {
  const int lane = threadIdx.x & 31;
  const uint32_t reach = order_of(bound + 0.f);
  int kept = 0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const u64 note = notes[32 * i + lane];
    if ((uint32_t)(note >> 32) >= reach) notes[32 * kept++ + lane] = note;
  }
  if (!__any_sync(0xffffffffu, kept == kSlots)) return {bound, bound, kept};
#pragma unroll 1
  for (int i = kept; i < kSlots; ++i) notes[32 * i + lane] = 0;
  const int all = __reduce_add_sync(0xffffffffu, kept);
  __syncwarp();
  const int left = min(all, k);
  const u64 least = cut<true>(notes, 32 * kSlots, all, left);  // (spread over the lanes, even if all of them stay)
  const int of_lane = left > lane ? (left - lane + 31) / 32 : 0;
  if (all <= k) return {bound, bound, of_lane};
  const uint32_t reached = (uint32_t)(least >> 32);
  return {fmaxf(bound, float_of(reached)), fmaxf(bound, float_of(reached + 1)), of_lane};
}

// Enters the elements of a warp's noted runs (L each, numbered from element `begin` on) that reach the
// bound in its list, cut to the k best of them when it is full. Returns how many there are, at most k + 32, padded
// with zeros to a multiple of four.
template <typename T, int L>
__device__ __noinline__ int enter(const T* x, int begin, int end, u64* notes, int of_lane, u64* list, int k, float bound) {
  constexpr int PER = 32 / L, AHEAD = 4;  // runs at a time, and of them in flight
  const int lane = threadIdx.x & 31;
  const uint32_t reach = order_of(bound + 0.f);
  int kept = 0;  // notes that still reach the bound
  __syncwarp();
#pragma unroll 1
  for (int i = 0; __any_sync(0xffffffffu, i < of_lane); ++i) {
    const u64 note = i < of_lane ? notes[32 * i + lane] : 0;
    const bool is = note != 0 && (uint32_t)(note >> 32) >= reach;
    const unsigned who = __ballot_sync(0xffffffffu, is);
    if (is) notes[kept + __popc(who & ((1u << lane) - 1))] = note;
    kept += __popc(who);
    __syncwarp();
  }
  u64 least = 0;
  int count = 0;
#pragma unroll 1
  for (int g = 0; g < kept; g += PER * AHEAD) {
    float v[AHEAD];
    int at[AHEAD];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int i = g + a * PER + lane / L;
      at[a] = i < kept ? begin + (int)token_of(notes[i]) * L + lane % L : end;
      v[a] = at[a] < end ? Vec<T>::read(x + at[a]) : 0.f;
    }
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const u64 entry = entry_of(v[a], at[a]);
      unsigned who = __ballot_sync(0xffffffffu, at[a] < end && v[a] >= bound && entry > least);
      if (who == 0) continue;
      if (count + __popc(who) > kEntries) {
        for (int i = count + lane; i < kEntries; i += 32) list[i] = 0;
        __syncwarp();
        least = cut<false>(list, kEntries, count, k);
        count = k;
        who = __ballot_sync(0xffffffffu, (who >> lane & 1) != 0 && entry > least);
      }
      if (who >> lane & 1) list[count + __popc(who & ((1u << lane) - 1))] = entry;
      count += __popc(who);
      __syncwarp();
    }
  }
  if (count > k + 32) {  // (a few more are ranked with the rest: 128 rows of 100 to 1000 with k 1 to 11 10.4 -> 9.8 us)
    for (int i = count + lane; i < kEntries; i += 32) list[i] = 0;
    __syncwarp();
    cut<false>(list, kEntries, count, k);
    count = k;
  }
  if (lane < 3 && count + lane < kEntries) list[count + lane] = 0;
  return count;
}

// The lanes' values, largest in lane 0.
__device__ __forceinline__ float sort_lanes(float v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int step = size >> 1; step > 0; step >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, v, step);
      const bool down = (lane & size) == 0, low = (lane & step) == 0;
      v = down == low ? fmaxf(v, o) : fminf(v, o);
    }
  }
  return v;
}
// The q-th largest of the lanes' values.
__device__ __noinline__ float nth_lane(float v, int q) {
  if (q > 8) return q > 32 ? -INFINITY : __shfl_sync(0xffffffffu, sort_lanes(v), q - 1);
  const int lane = threadIdx.x & 31;
  uint32_t k = order_of(v), m = __reduce_max_sync(0xffffffffu, k);
#pragma unroll 1
  for (int i = 1; i < q; ++i) {
    if (lane == __ffs(__ballot_sync(0xffffffffu, k == m)) - 1) k = 0;
    m = __reduce_max_sync(0xffffffffu, k);
  }
  return m == 0 ? -INFINITY : float_of(m);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The nth largest of the first n <= 8 of the warps' values.
__device__ __noinline__ float nth_of(const volatile float* value, int n, int nth) {
  const int lane = threadIdx.x & 31;
  const float mine = lane < n ? value[lane] : -INFINITY;
  int before = lane < n ? 0 : 32;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float v = __shfl_sync(0xffffffffu, mine, w);
    before += v > mine || (v == mine && w < lane);
  }
  const unsigned who = __ballot_sync(0xffffffffu, before == nth - 1);
  return who ? __shfl_sync(0xffffffffu, mine, __ffs(who) - 1) : -INFINITY;
}

// Sums of (hi, lo) pairs, with the roundings of hi kept in lo.
__device__ __forceinline__ float2 add_pairs(float2 a, float2 b) {
  const float s = a.x + b.x, t = s - a.x;
  return make_float2(s, (a.y + b.y) + ((a.x - (s - t)) + (b.x - t)));
}
__device__ __forceinline__ float2 sum_lanes(float2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = add_pairs(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  return v;
}

constexpr int kStages = 3;   // tiles of a warp on their way or in use

// J: 16-byte blocks of a lane and tile.
template <int J>
struct ScanSmem {
  uint4 ring[kWarps][kStages][32 * J + 1];  // (one block more for rows that are not aligned)
  u64 notes[kWarps][32 * kSlots];
  u64 entries[kWarps][kEntries];
  float2 wsum[kWarps];
  float wbound[kWarps], wmax[kWarps], wref[kWarps];
  int wcount[kWarps];
};

// Persistent: CTA c takes the pieces c, c + CTAs, .., one after another. A tile is 4 J KB of the row, 512 J
// bytes a warp, 16 J bytes in order a lane. Each warp copies its own blocks ahead, into the next piece
// too, so that warps need not wait for one another within a piece and a piece's end hides behind the
// loads of the next. A lane reads its blocks, eight lanes at a time: with J = 4, blocks are exchanged
// within fours (by bits 3 and 4 of their number) to lie in different banks.
template <typename T, int J>
__global__ void __launch_bounds__(kThreads, 3) beam_scan_kernel(const Scan p) {
  constexpr int E = Vec<T>::E, L = J * E, TILE = kThreads * L, SPAN = 32 * J + 1;
  extern __shared__ __align__(16) unsigned char smem[];
  ScanSmem<J>& sh = *reinterpret_cast<ScanSmem<J>*>(smem);
  volatile float* wbound = sh.wbound;
  float* wmax = sh.wmax;
  grid_wait();
  grid_trigger();  // the merge may be scheduled
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // piece -> its row's first element; its elements [begin, end)
  auto row_of = [&](int piece, int& begin, int& end) -> const T* {
    const int row = piece / p.splits, split = piece - row * p.splits;
    const int seq = row / p.rows_per_seq, beam = row - seq * p.rows_per_seq;
    begin = split * p.chunk;
    end = min(p.vocab, begin + p.chunk);
    return (const T*)p.logits + seq * p.ld_seq + beam * p.ld_beam;
  };
  // ---- copies ahead
  constexpr int MIX = J == 4 ? 3 : 0;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sh.ring[warp]) + (lane ^ (lane >> 3 & MIX)) * 16;
  uint32_t to = ring;
  int next = blockIdx.x, tiles = 0, left = 0;  // the piece, tiles of it to copy, bytes from this lane's block on
  bool tail = false;                           // a block more: the row is not aligned
  const char* block = nullptr;
  auto copy = [&]() {
    if (tiles == 0 && next < p.pieces_n) {
      int begin, end;
      const T* x = row_of(next, begin, end);
      const int shift = (int)((uintptr_t)x & 15), skip = (warp * 32 * J + lane) * 16;
      tail = shift != 0 && lane == 0;
      block = (const char*)(x + begin) - shift + skip;
      left = shift + (end - begin) * (int)sizeof(T) - skip;
      tiles = (end - begin + TILE - 1) / TILE;
      next += gridDim.x;
    }
    if (tiles > 0) {
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (j * 512 < left) copy16(to + j * 512, block + j * 512);
      if (tail && J * 512 < left) copy16(to + J * 512, block + J * 512);
      block += TILE * sizeof(T);
      left -= TILE * (int)sizeof(T);
      to = to == ring + (kStages - 1) * SPAN * 16 ? ring : to + SPAN * 16;
      --tiles;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int s = 0; s < kStages - 1; ++s) copy();
  u64* notes = sh.notes[warp];
  int stage = 0;
#pragma unroll 1
  for (int piece = blockIdx.x; piece < p.pieces_n; piece += gridDim.x) {
    int begin, end;
    const T* x = row_of(piece, begin, end);
    const int shift = (int)((uintptr_t)x & 15);
    // Warps whose lanes all have an element in the first tile (or the first one) have a say in the bound: the
    // q-th largest of each one's lanes, and of these the s-th largest
    const int voters = min(kWarps, max(1, (end - begin + L - 1) / (32 * L))), some = max(1, (3 * voters) / 4);
    const int q = (p.k + some - 1) / some, nth = (p.k + q - 1) / q;
    int noted = 0;                               // by this lane
    int seen = 0, due = 2;                       // tiles
    typename Vec<T>::Most best = Vec<T>::kNone;  // this lane's largest so far
    float ref = -INFINITY, far = 0.f;            // far: beyond it the reference has to move
    float bound = 0.f;                           // what is below it is no candidate
    float noting = 0.f;                          // what a run has to reach to be noted: the bound, or above it
    float sum = 0.f, low = 0.f;                  // sum + low
    auto publish = [&]() {
      const float v = warp < voters ? nth_lane(Vec<T>::value(best), q) : -INFINITY;
      if (lane == 0) wbound[warp] = v;
    };
#pragma unroll 1
    for (int base = begin; base < end; base += TILE) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();
      Vec<T> now[J];
      const uint4* src = sh.ring[warp][stage] + lane * J;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint4 a = src[j ^ (lane >> 1 & MIX)];
        now[j].w[0] = a.x; now[j].w[1] = a.y; now[j].w[2] = a.z; now[j].w[3] = a.w;
      }
      if (shift != 0) {
        const uint4 behind = src[J + (lane == 31 ? 0 : (lane + 1) >> 1 & MIX)];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const Vec<T>& b = now[(j + 1) % J];
          now[j].from(make_uint4(now[j].w[0], now[j].w[1], now[j].w[2], now[j].w[3]),
                      j + 1 < J ? make_uint4(b.w[0], b.w[1], b.w[2], b.w[3]) : behind, shift);
        }
      }
      const int run = end - (base + (int)threadIdx.x * L);  // elements of this lane's run
      if (base + TILE > end) {
#pragma unroll
        for (int j = 0; j < J; ++j) now[j].keep(run - j * E);
      }
      __syncwarp();  // the stage before this one has been read
      copy();
      if (++stage == kStages) stage = 0;
      typename Vec<T>::Most lots = now[0].most();
#pragma unroll
      for (int j = 1; j < J; ++j) lots = Vec<T>::larger(lots, now[j].most());
      best = Vec<T>::larger(best, lots);
      const float most = Vec<T>::value(lots);
      if (base == begin) {
        publish();
        const float v = warp_max(most);
        if (lane == 0) wmax[warp] = v;
        __syncthreads();
        noting = bound = nth_of(wbound, voters, nth);
        ref = wmax[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) ref = fmaxf(ref, wmax[w]);
        far = ref + kFar;  // (minus infinity: no finite logit yet)
      }
      if (seen == due) {  // after 2, 6, 14, .. tiles: a better bound
        publish();
        __syncwarp();
        bound = fmaxf(bound, nth_of(wbound, voters, nth));
        noting = fmaxf(noting, bound);
        due = 2 * due + 2;
      }
      ++seen;
      if (most >= noting && run > 0) notes[32 * noted++ + lane] = entry_of(most, (base - begin) / L + threadIdx.x);
      if (__any_sync(0xffffffffu, noted == kSlots || most > far || most == INFINITY)) {
        if (__any_sync(0xffffffffu, noted == kSlots)) {
          publish();
          __syncwarp();
          const Cleared c = clear_notes(notes, noted, p.k, fmaxf(bound, nth_of(wbound, voters, nth)));
          bound = c.bound;
          noting = fmaxf(noting, c.later);
          noted = c.of_lane;
        }
        // ---- the reference
        if (__any_sync(0xffffffffu, most > far || most == INFINITY)) {
          const float top = warp_max(most);
          if (top == INFINITY) {
            sum = NAN;
          } else if (ref != -INFINITY) {
            const float k = expf(ref - top);
            sum *= k;
            low *= k;
          }
          ref = top;
          far = ref + kFar;
        }
      }
      // ---- the sum (no finite logit yet: of zeros)
      const float from = ref == -INFINITY ? 0.f : ref;
      const float2 minus = make_float2(-from, -from);
      float2 acc = make_float2(0.f, 0.f), acc2 = acc;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < E; i += 4) {
          acc = __fadd2_rn(acc, exp_of(__fadd2_rn(make_float2(now[j].at(i), now[j].at(i + 1)), minus)));
          acc2 = __fadd2_rn(acc2, exp_of(__fadd2_rn(make_float2(now[j].at(i + 2), now[j].at(i + 3)), minus)));
        }
      const float tile = (acc.x + acc.y) + (acc2.x + acc2.y);
      const float s = sum + tile, t = s - sum;  // and the rounding error of s
      low += (sum - (s - t)) + (tile - t);
      sum = s;
    }
    if (seen > 1) {  // (one tile: it is the bound of all)
      publish();
      __syncwarp();
      bound = fmaxf(bound, nth_of(wbound, voters, nth));
    }
    // ---- elements of the noted runs that reach the bound
    const int count = enter<T, L>(x, begin, end, notes, noted, sh.entries[warp], p.k, bound);
    const float2 part = sum_lanes(make_float2(sum, low));
    if (lane == 0) {
      sh.wsum[warp] = part;
      sh.wref[warp] = ref;
      sh.wcount[warp] = count;
    }
    __syncthreads();
    // ---- ranks among all warps' entries
    int n = 0, in = 0, of = 0;  // all; this thread's place in warp `of`'s list
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if ((int)threadIdx.x >= n) in = threadIdx.x - n, of = w;
      n += sh.wcount[w];
    }
    u64* out = p.lists + (size_t)piece * p.k;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      while (in >= sh.wcount[of]) in -= sh.wcount[of++];
      const u64 e = sh.entries[of][in];
      int r = 0;
#pragma unroll 1
      for (int w = 0; w < kWarps; ++w) r += rank_of(sh.entries[w], sh.wcount[w], e);
      if (r < p.k) out[r] = e;
      in += kThreads;
    }
    for (int i = n + threadIdx.x; i < p.k; i += kThreads) out[i] = 0;
    if (warp == kWarps - 1) {  // the warps' sums (the first ones are busy with ranks)
      const float mine = lane < kWarps ? sh.wref[lane] : -INFINITY, top = warp_max(mine);
      float2 v = lane < kWarps ? sh.wsum[lane] : make_float2(0.f, 0.f);
      if (mine != top && mine != -INFINITY) {
        const float2 w = exp_pair(fmaxf(mine - top, -80.f));
        const float q = v.x * w.x;
        // (0 times the sum, so that NaN stays the mark of its row)
        v = mine - top < -80.f ? make_float2(0.f * v.x, 0.f) : make_float2(q, fmaf(v.x, w.x, -q) + (v.x * w.y + v.y * w.x));
      }
      v = sum_lanes(v);
      if (lane == 0) p.pieces[piece] = {(double)v.x + (double)v.y, top, 0};
    }
  }
}

struct Merge {
  const u64* lists;
  const Piece* pieces;
  const float* scores;
  int32_t* tokens;
  int32_t* parents;
  float* scores_out;
  long long ld_out;
  int beams, rows_per_seq, splits, k, vocab, parent_base;
};

// A score's bits in order.
__device__ __forceinline__ u64 order_of(double s) {
  const u64 b = (u64)__double_as_longlong(s);
  return b ^ ((b >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double score_of(u64 k) {
  return __longlong_as_double((long long)(k ^ ((k >> 63) ? 1ull << 63 : ~0ull)));
}

// A sequence's ranked candidates: the score's order, then the beam, the logit's order and the token. (With the logit,
// as 64 bits do not tell all scores of a beam apart: logits of 10^-20, or next to a score of 10^30. The candidates of
// one piece would be its largest logits then, and those of several the first pieces'.)
struct Ranked {
  u64 score[kMergeCap];
  u64 place[kMergeCap];  // lowest first: beam, logit, largest first, token
  int count;
};
// A place: the token in `bits` bits, 32 of the logit above them. (Beams x vocabulary is below 2^31, so that a beam has
// 32 - bits.)
__device__ __forceinline__ u64 place_of(uint32_t beam, uint32_t order, uint32_t token, int bits) {
  return ((u64)beam << 32 | (0xffffffffu - order)) << bits | token;
}

constexpr int kMostRough = 16384;  // candidates of a sequence (kBeamMax beams of as many)
constexpr int kBins = 256, kFirstBin = 117 << 3;  // distances from 2^-10 to 2^22

// Entry i's place among n by `parts` neighbouring lanes (a power of two), all of which get it.
__device__ __forceinline__ int rank_of(const Ranked& l, int n, u64 score, u64 place, int parts) {
  int rank = 0;
#pragma unroll 4
  for (int j = threadIdx.x & (parts - 1); j < n; j += parts)
    rank += l.score[j] > score || (l.score[j] == score && l.place[j] < place);
  for (int o = parts >> 1; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
  return rank;
}

// Cuts the list to its k best, best first.
template <int THREADS>
__device__ __noinline__ void cut_ranked(Ranked& l, int k) {
  const int n = min(l.count, kMergeCap);
  u64 mine[kMergeCap / THREADS];
  u64 at[kMergeCap / THREADS];
  int rank[kMergeCap / THREADS];
#pragma unroll
  for (int t = 0; t < kMergeCap / THREADS; ++t) {
    const int i = threadIdx.x + t * THREADS;
    mine[t] = i < n ? l.score[i] : 0;
    at[t] = i < n ? l.place[i] : 0;
    rank[t] = rank_of(l, n, mine[t], at[t], 1);
    if (i >= n) rank[t] = k;
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < kMergeCap / THREADS; ++t)
    if (rank[t] < k) {
      l.score[rank[t]] = mine[t];
      l.place[rank[t]] = at[t];
    }
  if (threadIdx.x == 0) l.count = min(n, k);
  __syncthreads();
}

// A CTA per sequence. Few thousand candidates at most, so that latencies count: scores in 32 bits lie in
// shared memory, a histogram gives a threshold that between k and about 2 k of them reach, and these
// alone are scored in 64 bits and ranked, by counting those before each.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) beam_merge_kernel(const Merge p) {
  constexpr int WARPS = THREADS / 32;
  extern __shared__ float rough[];  // [beams * splits * k]
  __shared__ Ranked list;
  __shared__ double lse[kBeamMax], shift[kBeamMax];  // log of the row's sum under m; m
  __shared__ float4 beam_s[kBeamMax];                // score, log sum and m in 32 bits, or NaN
  __shared__ int spread_s;                           // largest |score| + |log sum| of a beam, as bits
  __shared__ int bins[kBins], bin_s;
  __shared__ float top_s[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.x;
  if (threadIdx.x == 0) {
    list.count = spread_s = 0;
    bin_s = kBins - 1;  // (no threshold)
  }
  for (int i = threadIdx.x; i < kBins; i += THREADS) bins[i] = 0;
  // the scan's lists. (The next call's scan waits for the end of this grid: let in earlier, its CTAs take the places
  // of this one's where there are many, 2048 greedy rows of 32000 51.0 -> 62.6 us.)
  grid_wait();
  const int per = p.splits * p.k;
  const u64* lists = p.lists + (size_t)b * p.rows_per_seq * per;
  const Piece* pieces = p.pieces + (size_t)b * p.rows_per_seq * p.splits;
  // ---- a row's sum, a warp per row. Terms above 1/16 of it among the pieces' first are taken again: the
  // scan's are off by up to 2^-22
  const int first = p.splits < 32 ? min(p.k, 32 / p.splits) : 1;  // looked at, of each piece
  for (int r = warp; r < p.rows_per_seq; r += WARPS) {
    const Piece* pc = pieces + r * p.splits;
    float m = -INFINITY;
    for (int s = lane; s < p.splits; s += 32) m = fmaxf(m, pc[s].ref);
    m = warp_max(m);
    double sum = 0.0;
    for (int i = lane; i < p.splits * first; i += 32) {
      const int s = i / first, j = i - s * first;
      const Piece c = pc[s];
      const float under = c.ref - m;
      const u64 e = lists[(size_t)r * per + s * p.k + j];
      double part = j == 0 ? c.sum : 0.0;
      if (e != 0) {
        const float d = logit_of(e) - c.ref;
        const float a = exp_of(make_float2(d, d)).x;
        if ((double)a * 16.0 > c.sum) {
          const float2 t = exp_pair(d);
          part += ((double)t.x - (double)a) + (double)t.y;
        }
      }
      if (c.ref != -INFINITY && under != 0.f) {
        const float2 w = exp_pair(fmaxf(under, -80.f));
        part *= under < -80.f ? 0.0 : (double)w.x + (double)w.y;
      }
      sum += part;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      const bool dead = !(sum > 0.0 && sum < INFINITY) || m == INFINITY || m == -INFINITY;
      lse[r] = dead ? NAN : log_of(sum);
      shift[r] = m;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.beams; i += THREADS) {
    const int r = p.rows_per_seq == 1 ? 0 : i;
    const float s = p.scores ? p.scores[(size_t)b * p.beams + i] : 0.f, z = (float)lse[r];
    const bool alive = isfinite(s) && !isnan(z);
    beam_s[i] = make_float4(alive ? s : NAN, z, (float)shift[r], 0.f);
    if (alive) atomicMax(&spread_s, __float_as_int(fabsf(s) + fabsf(z)));
  }
  __syncthreads();
  // ---- scores in 32 bits; NaN: no candidate. A beam without a probability has the lowest tokens, at
  // minus infinity. Candidate c is place c % per of its beam's lists
  const int total = p.beams * per;
  const float inv = 1.f / (float)per;
  auto beam_of = [&](int c) { return (int)(((float)c + 0.5f) * inv); };  // (c < 2^14: exact)
  float top = -INFINITY;
#pragma unroll 4
  for (int c = threadIdx.x; c < total; c += THREADS) {
    const int beam = beam_of(c), i = c - beam * per;
    const u64 x = lists[p.rows_per_seq == 1 ? i : c];
    const float4 of = beam_s[beam];
    float v = x == 0 ? NAN : of.x + ((logit_of(x) - of.z) - of.y);
    if (isnan(of.x)) v = i < min(p.k, p.vocab) ? -INFINITY : NAN;
    rough[c] = v;
    top = fmaxf(top, v);
  }
  top = warp_max(top);
  if (lane == 0) top_s[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w) top = fmaxf(top, top_s[w]);
  // ---- the threshold, from the numbers of candidates by their distance from the best, eight bins an
  // octave: the end of the bin that holds the k-th
  float bound = -INFINITY;
  if (top != -INFINITY) {
#pragma unroll 4
    for (int c = threadIdx.x; c < total; c += THREADS) {
      const float v = rough[c];
      if (v == v) atomicAdd(&bins[min(max((int)(__float_as_uint(top - v) >> 20) - kFirstBin, 0), kBins - 1)], 1);
    }
    __syncthreads();
    if (warp == 0) {
      int n[kBins / 32], mine = 0;
#pragma unroll
      for (int i = 0; i < kBins / 32; ++i) mine += n[i] = bins[lane * (kBins / 32) + i];
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
      }
      const int l = __ffs(__ballot_sync(0xffffffffu, upto >= p.k)) - 1;  // (none, were there fewer than k candidates)
      if (lane == l) {
        int have = upto - mine, i = 0;
        while (i < kBins / 32 - 1 && have + n[i] < p.k) have += n[i++];
        bin_s = lane * (kBins / 32) + i;
      }
    }
    __syncthreads();
    if (bin_s < kBins - 1) bound = top - __uint_as_float((uint32_t)(bin_s + 1 + kFirstBin) << 20);
  }
  // a rough score is off by eight roundings of |score|, |logit - m| and |log sum| at most
  const float slack = (2.f * __int_as_float(spread_s) + fabsf(bound) + fabsf(top)) * 9.6e-7f;
  if (bound != -INFINITY) bound -= slack;
  // ---- exact scores of what reaches it
  const int bits = 32 - __clz(p.vocab - 1);  // of a token
  u64 least = 0, least_place = ~0ull;
  for (int base = 0; base < total; base += THREADS) {
    const int c = base + threadIdx.x;
    bool todo = c < total && rough[c] >= bound;
    u64 key = 0, place = 0;
    if (todo) {
      const int beam = beam_of(c), i = c - beam * per, r = p.rows_per_seq == 1 ? 0 : beam;
      const float s = beam_s[beam].x;
      double score = -INFINITY;
      uint32_t token = i, order = 0;
      if (!isnan(s)) {
        const u64 e = lists[r == beam ? c : i];
        token = token_of(e);
        order = (uint32_t)(e >> 32);
        score = (double)s + (((double)logit_of(e) - shift[r]) - lse[r]);
      }
      key = order_of(score);
      place = place_of(beam, order, token, bits);
    }
    bool more;
    do {
      if (todo && (key < least || (key == least && place >= least_place))) todo = false;
      if (todo) {
        const int at = atomicAdd(&list.count, 1);
        if (at < kMergeCap) {
          list.score[at] = key;
          list.place[at] = place;
          todo = false;
        }
      }
      more = __syncthreads_or(todo);
      if (more) {
        cut_ranked<THREADS>(list, p.k);
        least = list.score[p.k - 1];  // (a full list has k entries)
        least_place = list.place[p.k - 1];
      }
    } while (more);
  }
  // ---- ranks
  const int n = min(list.count, kMergeCap);
  int parts = 1;
  while (2 * parts * n <= THREADS && parts < 8) parts *= 2;
  for (int i = threadIdx.x / parts; i < (n + 31) / 32 * 32; i += THREADS / parts) {
    const u64 score = i < n ? list.score[i] : 0;
    const u64 place = i < n ? list.place[i] : 0;
    const int r = rank_of(list, n, score, place, parts);
    if (i >= n || r >= p.k || (threadIdx.x & (parts - 1)) != 0) continue;
    const size_t at = (size_t)b * p.ld_out + r;
    p.tokens[at] = (int)(place & ((1ull << bits) - 1));
    if (p.parents) p.parents[at] = p.parent_base + (int)(place >> (32 + bits));
    if (p.scores_out) p.scores_out[at] = (float)score_of(score);
  }
  // The lists hold k candidates of a sequence; were there fewer, what the buffers held would still be no token
  for (int r = n + threadIdx.x; r < p.k; r += THREADS) {
    const size_t at = (size_t)b * p.ld_out + r;
    p.tokens[at] = 0;
    if (p.parents) p.parents[at] = p.parent_base;
    if (p.scores_out) p.scores_out[at] = -INFINITY;
  }
}

constexpr int kCtas = 3;  // of the scan, per SM

// How rows are cut. CTAs take pieces in turns; a piece costs the loads of its elements and about as much
// again as 54 K of them for its start and end (6 us), and more candidates for the merge, which holds kMostRough
// of a sequence. Measured, us (pieces a row):
//   256 rows of 131072, k 16       1: 26.9   2: 32.5   4: 37.8   8: 48.2
//   16 rows of 131072, k 16        1: 20.8   4: 15.3   8: 14.0  16: 15.2
//   4 rows of 131072, k 8          1: 19.4   4: 13.6  16: 12.1  32: 12.1
struct Cut {
  int splits, chunk;  // pieces of a row, and elements of a piece (whole runs of every thread)
};
Cut cut_of(int rows, int beams, int vocab, int k) {
  constexpr int UNIT = kThreads * 8;
  const int slots = kCtas * chunk_sms(), units = (vocab + UNIT - 1) / UNIT, fit = kMostRough / 2 / (beams * k);
  Cut best = {1, units * UNIT};
  double least = 1e300;
  // Every s that makes other pieces: the first of those that cut a row into pieces of `per` units (2 sqrt(units) of
  // them at most, as an s takes 10 ns of each call's host time; all s of 2^24 logits: 20 us)
  for (int s = 1; (s == 1 || s <= fit) && (long long)rows * (s - 1) < 8LL * slots;) {
    const int per = (units + s - 1) / s, n = (units + per - 1) / per;
    const long long turns = ((long long)rows * n + slots - 1) / slots;
    const double cost = (double)turns * (per + 27) + (double)beams * n * k / 128.;
    if (cost < least) {
      least = cost;
      best = {n, per * UNIT};
    }
    if (per == 1) break;
    s = (units + per - 2) / (per - 1);
  }
  return best;
}

template <typename T, int J>
cudaError_t scan_rows(const Scan& p, cudaStream_t s) {
  static SmemLimit limit;
  // all of the memory as shared, as the merge has it: an SM empties before that split changes, and the merge's CTAs,
  // which are let in early, would wait for that (256 rows of 100 to 1000: 10.3 us, and 16.4 with different splits)
  cudaError_t e = limit.raise(beam_scan_kernel<T, J>, (int)sizeof(ScanSmem<J>), false, true);
  if (e != cudaSuccess) return e;
  LaunchScope ls_(DFLASH_KERNEL_BEAM_SCAN, s);
  const int slots = kCtas * chunk_sms();
  return launch_overlapped(beam_scan_kernel<T, J>, dim3(p.pieces_n < slots ? p.pieces_n : slots), kThreads,
                           sizeof(ScanSmem<J>), s, p);
}

template <int THREADS>
cudaError_t merge_rows(const Merge& p, int batch, cudaStream_t s) {
  static SmemLimit limit;
  const cudaError_t e = limit.raise(beam_merge_kernel<THREADS>, (int)sizeof(float) * kMostRough, false, true);
  if (e != cudaSuccess) return e;
  LaunchScope ls_(DFLASH_KERNEL_BEAM_MERGE, s);
  return launch_overlapped(beam_merge_kernel<THREADS>, dim3(batch), THREADS, sizeof(float) * (size_t)p.beams * p.splits * p.k,
                           s, p);
}

// Both ways to cut a call's rows (one per beam, or one shared by them) and the workspace, which holds either.
struct Sizes {
  Cut each, shared;
  size_t pieces;
};
Sizes sizes_of(int batch, int beams, int vocab, int k) {
  Sizes z;
  z.each = z.shared = cut_of(batch * beams, beams, vocab, k);
  if (beams > 1) z.shared = cut_of(batch, beams, vocab, k);
  const size_t e = (size_t)batch * beams * z.each.splits, s = (size_t)batch * z.shared.splits;
  z.pieces = e > s ? e : s;
  return z;
}
struct Carved {
  u64* lists;
  Piece* pieces;
};
Carved carve(Carver& cv, const Sizes& z, int k) {
  Carved c;
  c.lists = cv.take<u64>(z.pieces * k);
  c.pieces = cv.take<Piece>(z.pieces);
  return c;
}

}  // namespace

size_t beam_workspace(int batch, int beams, int vocab, int k) {
  Carver cv(nullptr, ~size_t(0));
  carve(cv, sizes_of(batch, beams, vocab, k), k);
  return cv.off;
}

dflash_status beam_select(int dtype, const BeamParams& a, size_t ws_bytes, cudaStream_t s) {
  const Sizes sizes = sizes_of(a.batch, a.beams, a.vocab, a.k);
  Carver cv(a.workspace, ws_bytes);
  const Carved c = carve(cv, sizes, a.k);
  if (!cv.ok) return DFLASH_ERR_WORKSPACE;
  const int per_seq = a.ld_beam == 0 ? 1 : a.beams, rows = a.batch * per_seq;
  const Cut cut = per_seq == 1 ? sizes.shared : sizes.each;
  const int splits = cut.splits;
  const Scan scan = {a.logits, a.ld_seq, a.ld_beam, c.lists, c.pieces, a.vocab, per_seq, splits, cut.chunk, a.k, rows * splits};
  // short pieces: 16 bytes a lane and tile, so that more lanes have some
  const bool fine = cut.chunk <= kThreads * 16;
  cudaError_t e = dtype == DFLASH_F32 ? (fine ? scan_rows<float, 1>(scan, s) : scan_rows<float, 4>(scan, s))
                        : (fine ? scan_rows<bf16, 1>(scan, s) : scan_rows<bf16, 4>(scan, s));
  if (e != cudaSuccess) return cuda_status(e);
  const Merge merge = {c.lists, c.pieces, a.scores, a.tokens, a.parents, a.scores_out, a.ld_out,
                       a.beams, per_seq, splits, a.k, a.vocab, a.parent_base};
  // Four warps for few candidates of few rows: such sequences are many, and share an SM (2048 rows, greedy: 57 us
  // with 128 threads, 72 with 512, both before the scan's last steps; 64 sequences of 8 beams, k 8: 34 and 31)
  const bool small = per_seq * splits <= 4 && (long long)a.beams * splits * a.k <= 128;
  return cuda_status(small ? merge_rows<128>(merge, a.batch, s) : merge_rows<512>(merge, a.batch, s));
}

}  // namespace dflash
