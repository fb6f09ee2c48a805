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
// The k largest. Every lane keeps the maximum of what it has seen; the q-th largest of a warp's lanes,
// the lowest of the CTA's eight such values (8 q >= k), is reached by at least k elements, so that
// nothing below it is a candidate. Warps publish theirs when they meet candidates and need not wait for
// one another: an old value is only a lower one. A vector of eight logits that reaches the bound is
// noted, by its maximum and number; the noted vectors are read again at the end, against the last
// bound, and only then are elements looked at one by one (taken as they came, that cost twice the sum's
// instructions). Notes that do not fit (rows of equal or of ascending logits) are cut to the k vectors
// of the largest maxima: each of the others has k elements before all of its own.
//
// The sum. Which candidate of two beams is the better one is decided by the difference of two such
// sums, so their errors must stay far below the gaps between scores (about 10^-2 among the best of a
// vocabulary). d = x - ref is exact for bf16 within 16 binades; with t = fl(d log2 e) and
// r = d log2 e - t (a fused multiply-add and the constant's second word), e^d = 2^t (1 + r ln 2): the terms
// 2^t and 2^t r are added up apart. (t alone would be off by up to 10^-6.) Terms in fp32, a thread's
// tiles added with their rounding errors kept, the rest in 64 bits. The few large terms of a row, where
// 2^t's error of 2^-22 does not average out, are taken again by the merge. The order of the
// additions depends on the vocabulary alone, so equal rows have equal sums and their candidates tie as
// they should.
#include <float.h>

#include "tree.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kNotes = 192;    // noted vectors of a warp: kBeamMax and 32 at least
constexpr int kMergeCap = 1024;  // entries of the merge's list
constexpr float kFar = 40.f;   // how far above the reference a logit may lie

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

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log2 e and ln 2 as a float and what it leaves.
constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f;
constexpr float kLn2 = 0.693147182f, kLn2Low = -1.90465421e-9f;
constexpr float kDeep = -200.f;  // e^d is 0 from here on
constexpr float kLowest = -3.38953139e38f;  // of bf16: below it a reference has no floor

// The terms of e^d for kDeep <= d <= kFar: sum += 2^t, rest += 2^t r (twice).
__device__ __forceinline__ void add_exp(float2 d, float2& sum, float2& rest) {
  const float2 l = make_float2(kLog2e, kLog2e);
  const float2 t = __fmul2_rn(d, l);
  float2 r = __ffma2_rn(d, l, make_float2(-t.x, -t.y));
  r = __ffma2_rn(d, make_float2(kLog2eLow, kLog2eLow), r);
  const float2 e = make_float2(ex2(t.x), ex2(t.y));
  sum = __fadd2_rn(sum, e);
  rest = __ffma2_rn(e, r, rest);
}

// e^d to 2^-27 as hi + lo, -80 <= d <= 80: e^d = 2^n 2^(f + g), f = fl(d log2 e) - n and g what the
// product left, and 2^f = 1 + f ln 2 + f^2 P(f), the first product and sum with their rounding errors
// (P: the Taylor terms up to f^8, 10^-9 at |f| = 1/2).
__device__ __forceinline__ float2 exp_pair(float d) {
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
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
  // elements from e on, of which `end` exist; the others -inf
  __device__ __forceinline__ void load(const bf16* row, int e, int end) {
    const uint16_t* x = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (e + 2 * i < end ? x[e + 2 * i] : 0xFF80u) | (e + 2 * i + 1 < end ? x[e + 2 * i + 1] : 0xFF80u) << 16;
  }
  __device__ __forceinline__ void keep(int n) {  // all but the first n become -inf
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * i >= n) w[i] = (w[i] & 0xffff0000u) | 0xFF80u;
      if (2 * i + 1 >= n) w[i] = (w[i] & 0xffffu) | 0xFF800000u;
    }
  }
  __device__ __forceinline__ float most() const {  // (NaN only where all are)
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(w);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
  // x - ref of elements i and i + 1, where it matters: what is below the floor (a bf16 below
  // ref + kDeep, so its weight is 0) is taken for it, as a product with -inf would be NaN
  __device__ __forceinline__ float2 below(int i, float ref, uint32_t floor2) const {
    const __nv_bfloat162 m = __hmax2_nan(reinterpret_cast<const __nv_bfloat162*>(w)[i >> 1],
                                         *reinterpret_cast<const __nv_bfloat162*>(&floor2));
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
    return __fadd2_rn(make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)), make_float2(-ref, -ref));
  }
  static __device__ __forceinline__ uint32_t floor_of(float ref) {
    const bf16 f = __float2bfloat16_rd(ref + 2 * kDeep);
    uint32_t u = *reinterpret_cast<const uint16_t*>(&f);
    if (__uint_as_float(u << 16) >= ref) u = u & 0x8000u ? u + 1 : u - 1;  // |ref| so large that 400 is lost
    return u | u << 16;
  }
};
template <> struct Vec<float> : Bytes16 {
  static constexpr int E = 4;
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(w[i]); }
  __device__ __forceinline__ void load(const float* row, int e, int end) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = e + i < end ? __float_as_uint(row[e + i]) : 0xFF800000u;
  }
  __device__ __forceinline__ void keep(int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i >= n) w[i] = 0xFF800000u;
  }
  __device__ __forceinline__ float most() const { return fmaxf(fmaxf(at(0), at(1)), fmaxf(at(2), at(3))); }
  __device__ __forceinline__ float2 below(int i, float ref, uint32_t) const {
    return make_float2(max_nan(at(i) - ref, kDeep), max_nan(at(i + 1) - ref, kDeep));
  }
  static __device__ __forceinline__ uint32_t floor_of(float) { return 0; }
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
  int vocab, rows_per_seq, splits, chunk, k;
};

// Entry i's place among n: how many are before it.
__device__ __forceinline__ int rank_of(const u64* e, int n, u64 mine) {
  int rank = 0;
  int j = 0;
  for (; j + 2 <= n; j += 2) {
    const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(e + j);
    rank += (two.x > mine) + (two.y > mine);
  }
  if (j < n) rank += e[j] > mine;
  return rank;
}

// Cuts a warp's list of n entries, k <= n <= N, to its k best, best first.
template <int N>
__device__ __forceinline__ void cut_warp_list(u64* e, int n, int k) {
  const int lane = threadIdx.x & 31;
  u64 mine[N / 32];
  int rank[N / 32];
#pragma unroll
  for (int t = 0; t < N / 32; ++t) {
    const int i = lane + 32 * t;
    mine[t] = i < n ? e[i] : 0;
    rank[t] = i < n ? rank_of(e, n, mine[t]) : k;
  }
  __syncwarp();
#pragma unroll
  for (int t = 0; t < N / 32; ++t)
    if (rank[t] < k) e[rank[t]] = mine[t];
  __syncwarp();
}

// A float's bits in order.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// Reads a warp's noted vectors (numbers from element `begin` on) again and enters the elements that reach
// the bound in its list, at most kEntries of which the k best are kept. Returns how many there are, at most k
// or what was entered in a list that was never full.
constexpr int kEntries = 256;
template <typename T>
__device__ __noinline__ int enter(const T* x, int begin, int end, const u64* notes, int n, u64* list, int k, float bound) {
  constexpr int E = Vec<T>::E;
  const int lane = threadIdx.x & 31;
  const uint32_t reach = order_of(bound + 0.f);
  u64 least = 0;
  int count = 0;
  for (int g = 0; g < n; g += 32) {
    const u64 note = g + lane < n ? notes[g + lane] : 0;
    const bool is = note != 0 && (uint32_t)(note >> 32) >= reach;
    if (!__any_sync(0xffffffffu, is)) continue;
    const int e = is ? begin + (int)token_of(note) * E : end;
    Vec<T> v;
    v.load(x, e, end);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const u64 entry = entry_of(v.at(i), e + i);
      unsigned who = __ballot_sync(0xffffffffu, e + i < end && v.at(i) >= bound && entry > least);
      if (who == 0) continue;
      if (count + __popc(who) > kEntries) {
        cut_warp_list<kEntries>(list, count, k);
        count = k;
        least = list[k - 1];
        who = __ballot_sync(0xffffffffu, (who >> lane & 1) != 0 && entry > least);
      }
      if (who >> lane & 1) list[count + __popc(who & ((1u << lane) - 1))] = entry;
      count += __popc(who);
      __syncwarp();
    }
  }
  if (count > k) {
    cut_warp_list<kEntries>(list, count, k);
    count = k;
  }
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
__device__ __forceinline__ float nth_lane(float v, int q) {
  if (q > 8) return q > 32 ? -INFINITY : __shfl_sync(0xffffffffu, sort_lanes(v), q - 1);
  const int lane = threadIdx.x & 31;
  uint32_t k = order_of(v), m = __reduce_max_sync(0xffffffffu, k);
  for (int i = 1; i < q; ++i) {
    if (lane == __ffs(__ballot_sync(0xffffffffu, k == m)) - 1) k = 0;
    m = __reduce_max_sync(0xffffffffu, k);
  }
  return m == 0 ? -INFINITY : float_of(m);
}

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

constexpr int kVecs = 4;     // of a thread and tile
constexpr int kStages = 3;   // tiles of a warp on their way or in use
constexpr int kSpan = 33;    // 16-byte blocks of a warp's vectors of one number, one more for rows that are not aligned

struct ScanSmem {
  uint4 ring[kWarps][kStages][kVecs][kSpan];
  u64 notes[kWarps][kNotes];
  double wsum[kWarps];
  float wbound[kWarps], wmax[kWarps];
  int count;
};

// Vector j of a thread in the tile at `base`: elements base + (j * kThreads + thread) * E and on. Each warp
// copies its own vectors ahead, so that warps need not wait for one another.
template <typename T>
__global__ void __launch_bounds__(kThreads, 3) beam_scan_kernel(const Scan p) {
  constexpr int J = kVecs, E = Vec<T>::E, STEP = kThreads * E, TILE = STEP * J;
  extern __shared__ __align__(16) unsigned char smem[];
  ScanSmem& sh = *reinterpret_cast<ScanSmem*>(smem);
  volatile float* wbound = sh.wbound;
  float* wmax = sh.wmax;
  double* wsum = sh.wsum;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge may be scheduled
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seq = blockIdx.x, beam = blockIdx.y, split = blockIdx.z;
  const T* x = (const T*)p.logits + seq * p.ld_seq + beam * p.ld_beam;
  const int shift = (int)((uintptr_t)x & 15);
  const char* blocks = (const char*)x - shift;  // the row's 16-byte blocks
  const int begin = min(p.vocab, split * p.chunk), end = min(p.vocab, begin + p.chunk);
  const long long stop = shift + (long long)end * (int)sizeof(T);  // bytes of the blocks that matter
  u64* notes = sh.notes[warp];
  int noted = 0;
  // warps that have a vector per lane in the first tile have a say in the bound
  const int voters = min(kWarps, (end - begin) / (32 * E)), q = voters ? (p.k + voters - 1) / voters : 64;
  auto copy = [&](int base, int stage) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const long long at = (long long)(base + j * STEP + warp * 32 * E) * (int)sizeof(T);
      uint4* dst = sh.ring[warp][stage][j];
      if (at + 16 * lane < stop) copy16(dst + lane, blocks + at + 16 * lane);
      if (shift != 0 && lane == 0 && at + 512 < stop) copy16(dst + 32, blocks + at + 512);
    }
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (begin + s * TILE < end) copy(begin + s * TILE, s);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  float best = -INFINITY;                    // this lane's largest so far
  float ref = -INFINITY, far = 0.f;          // far: beyond it the reference has to move
  float bound = 0.f;                         // what is below it is no candidate
  uint32_t floor2 = 0;
  float sum = 0.f, low = 0.f;                // sum + low
  int stage = 0;
  for (int base = begin; base < end; base += TILE) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();
    Vec<T> now[J];
    const int vecs = min(J, (end - base + STEP - 1) / STEP);  // of the tile
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint4* src = sh.ring[warp][stage][j] + lane;
      const uint4 a = src[0];
      if (shift == 0) {
        now[j].w[0] = a.x; now[j].w[1] = a.y; now[j].w[2] = a.z; now[j].w[3] = a.w;
      } else {
        now[j].from(a, src[1], shift);
      }
    }
    if (base + TILE > end) {
#pragma unroll
      for (int j = 0; j < J; ++j) now[j].keep(end - (base + (j * kThreads + (int)threadIdx.x) * E));
    }
    __syncwarp();  // the stage before this one has been read
    if (base + (kStages - 1) * TILE < end) copy(base + (kStages - 1) * TILE, stage == 0 ? kStages - 1 : stage - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++stage == kStages) stage = 0;
    float vmax[J], most = -INFINITY;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      vmax[j] = now[j].most();
      most = fmaxf(most, vmax[j]);
    }
    best = fmaxf(best, most);
    auto publish = [&]() {  // the warp's share of the bound
      const float v = warp < voters ? nth_lane(best, q) : INFINITY;
      if (lane == 0) wbound[warp] = v;
    };
    auto read_bound = [&]() {
      float v = voters ? INFINITY : -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v = fminf(v, wbound[w]);
      return v;
    };
    if (base == begin) {
      publish();
      const float v = warp_max(best);
      if (lane == 0) wmax[warp] = v;
      __syncthreads();
      bound = read_bound();
      ref = wmax[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) ref = fmaxf(ref, wmax[w]);
      far = ref + kFar;  // (minus infinity: no finite logit yet)
      floor2 = Vec<T>::floor_of(ref);
    }
    if (__any_sync(0xffffffffu, most >= bound || most > far || most == INFINITY)) {
      if (base != begin && __popc(__ballot_sync(0xffffffffu, most >= bound)) >= 4) {
        publish();
        __syncwarp();
        bound = fmaxf(bound, read_bound());
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        unsigned who = __ballot_sync(0xffffffffu, j < vecs && vmax[j] >= bound);
        if (who == 0) continue;
        if (noted + __popc(who) > kNotes) {
          cut_warp_list<kNotes>(notes, noted, p.k);
          noted = p.k;
          // later vectors have to be above the last one kept
          bound = fmaxf(bound, float_of((uint32_t)(notes[p.k - 1] >> 32) + 1));
          who = __ballot_sync(0xffffffffu, j < vecs && vmax[j] >= bound);
        }
        if (who >> lane & 1)
          notes[noted + __popc(who & ((1u << lane) - 1))] =
              entry_of(vmax[j], (base - begin + j * STEP) / E + threadIdx.x);
        noted += __popc(who);
      }
      // ---- the reference
      if (__any_sync(0xffffffffu, most > far || most == INFINITY)) {
        const float top = warp_max(most);
        if (top == INFINITY) {
          sum = NAN;
        } else {
          const float k = ref == -INFINITY ? 1.f : expf(ref - top);
          sum *= k;
          low *= k;
          floor2 = Vec<T>::floor_of(top);
        }
        ref = top;
        far = ref + kFar;
      }
    }
    // ---- the sum
    float2 acc = make_float2(0.f, 0.f), acc2 = acc, rest = acc;
    if (ref > kLowest && ref != INFINITY) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (j >= vecs) continue;
#pragma unroll
        for (int i = 0; i < E; i += 4) {
          add_exp(now[j].below(i, ref, floor2), acc, rest);
          add_exp(now[j].below(i + 2, ref, floor2), acc2, rest);
        }
      }
    } else {  // nothing yet, or nothing but the lowest value (and a row with infinity has its NaN)
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float v = now[j].at(i);
          if (j < vecs) acc.x += v == ref && ref != -INFINITY ? 1.f : isnan(v) ? v : 0.f;
        }
    }
    const float tile = fmaf(rest.x + rest.y, kLn2, (acc.x + acc.y) + (acc2.x + acc2.y));
    const float s = sum + tile, t = s - sum;  // and the rounding error of s
    low += (sum - (s - t)) + (tile - t);
    sum = s;
  }
  // ---- elements of the noted vectors, against the last bound; the warps' lists become one
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (begin < end) {
    const float v = warp < voters ? nth_lane(best, q) : INFINITY;
    if (lane == 0) {
      wbound[warp] = v;
      wmax[warp] = ref;
    }
  } else if (lane == 0) {
    wbound[warp] = wmax[warp] = -INFINITY;
  }
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();  // (and the ring is free)
  float top = wmax[0], last = voters ? INFINITY : -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    top = fmaxf(top, wmax[w]);
    last = fminf(last, wbound[w]);
  }
  u64* mine = reinterpret_cast<u64*>(sh.ring[warp]);  // kEntries of them, then all warps' k each
  static_assert(sizeof(sh.ring[0]) >= kEntries * sizeof(u64) && sizeof(sh.ring) >= kWarps * kBeamMax * sizeof(u64), "ring");
  const int count = enter<T>(x, begin, end, notes, noted, mine, p.k, last);
  u64 held[kBeamMax / 32];
#pragma unroll
  for (int t = 0; t < kBeamMax / 32; ++t) held[t] = lane + 32 * t < count ? mine[lane + 32 * t] : 0;
  int place = 0;
  if (lane == 0 && count) place = atomicAdd(&sh.count, count);
  place = __shfl_sync(0xffffffffu, place, 0);
  __syncthreads();
  u64* list = reinterpret_cast<u64*>(sh.ring);
#pragma unroll
  for (int t = 0; t < kBeamMax / 32; ++t)
    if (lane + 32 * t < count) list[place + lane + 32 * t] = held[t];
  double d = (double)sum + (double)low;
  if (ref != top && ref != -INFINITY) d *= exp((double)ref - (double)top);  // (far apart: rare)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0) wsum[warp] = d;
  __syncthreads();
  const int n = sh.count;
  const size_t piece = ((size_t)seq * p.rows_per_seq + beam) * p.splits + split;
  u64* out = p.lists + piece * p.k;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const u64 e = list[i];
    const int r = rank_of(list, n, e);
    if (r < p.k) out[r] = e;
  }
  for (int i = n + threadIdx.x; i < p.k; i += kThreads) out[i] = 0;
  if (threadIdx.x == 0) {
    d = wsum[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) d += wsum[w];
    p.pieces[piece] = {d, top, 0};
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

// A sequence's ranked candidates: the score's order, then the lowest place.
struct Ranked {
  u64 score[kMergeCap];
  uint32_t place[kMergeCap];  // beam * vocab + token
  int count;
};

constexpr int kMergeThreads = 512;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kMostRough = 16384;  // candidates of a sequence (kBeamMax beams of as many)
constexpr int kCounts = 64;

// Entry i's place among n by `parts` neighbouring lanes (a power of two), all of which get it.
__device__ __forceinline__ int rank_of(const Ranked& l, int n, u64 score, uint32_t place, int parts) {
  int rank = 0;
#pragma unroll 4
  for (int j = threadIdx.x & (parts - 1); j < n; j += parts)
    rank += l.score[j] > score || (l.score[j] == score && l.place[j] < place);
  for (int o = parts >> 1; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
  return rank;
}

// Cuts the list to its k best, best first.
__device__ __noinline__ void cut_ranked(Ranked& l, int k) {
  const int n = min(l.count, kMergeCap);
  u64 mine[kMergeCap / kMergeThreads];
  uint32_t at[kMergeCap / kMergeThreads];
  int rank[kMergeCap / kMergeThreads];
#pragma unroll
  for (int t = 0; t < kMergeCap / kMergeThreads; ++t) {
    const int i = threadIdx.x + t * kMergeThreads;
    mine[t] = i < n ? l.score[i] : 0;
    at[t] = i < n ? l.place[i] : 0;
    rank[t] = rank_of(l, n, mine[t], at[t], 1);
    if (i >= n) rank[t] = k;
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < kMergeCap / kMergeThreads; ++t)
    if (rank[t] < k) {
      l.score[rank[t]] = mine[t];
      l.place[rank[t]] = at[t];
    }
  if (threadIdx.x == 0) l.count = min(n, k);
  __syncthreads();
}

// A CTA per sequence. Few thousand candidates at most, so that latencies count: scores in 32 bits lie in
// shared memory, a handful of counts finds a threshold that between k and about 2 k of them reach, and
// these alone are scored in 64 bits and ranked, by counting those before each.
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const Merge p) {
  extern __shared__ float rough[];  // [beams * splits * k]
  __shared__ Ranked list;
  __shared__ double lse[kBeamMax], shift[kBeamMax];  // log of the row's sum under m; m
  __shared__ float4 beam_s[kBeamMax];                // score, log sum and m in 32 bits, or NaN
  __shared__ int spread_s;                           // largest |score| + |log sum| of a beam, as bits
  __shared__ int counts[kCounts];
  __shared__ float top_s[kMergeWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.x;
  if (threadIdx.x == 0) list.count = spread_s = 0;
  if (threadIdx.x < kCounts) counts[threadIdx.x] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the scan's lists
  const int per = p.splits * p.k;
  const u64* lists = p.lists + (size_t)b * p.rows_per_seq * per;
  const Piece* pieces = p.pieces + (size_t)b * p.rows_per_seq * p.splits;
  // ---- a row's sum, a warp per row. Terms above 1/16 of it among the pieces' first are taken again: the
  // scan's are off by up to 2^-22
  const int first = p.splits < 32 ? min(p.k, 32 / p.splits) : 1;  // looked at, of each piece
  for (int r = warp; r < p.rows_per_seq; r += kMergeWarps) {
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
        float2 a = make_float2(0.f, 0.f), b2 = a;
        add_exp(make_float2(max_nan(d, kDeep), kDeep), a, b2);
        if ((double)a.x * 16.0 > c.sum) {
          const float2 t = exp_pair(d);
          part += ((double)t.x - (double)a.x) + (double)(t.y - b2.x * kLn2);
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
  for (int i = threadIdx.x; i < p.beams; i += kMergeThreads) {
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
  for (int c = threadIdx.x; c < total; c += kMergeThreads) {
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
  for (int w = 0; w < kMergeWarps; ++w) top = fmaxf(top, top_s[w]);
  // ---- the threshold
  int tries = 0;
  auto count = [&](float t) -> int {  // (at most kCounts times)
    int n = 0;
#pragma unroll 4
    for (int c = threadIdx.x; c < total; c += kMergeThreads) n += rough[c] >= t;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0 && n) atomicAdd(&counts[tries], n);
    __syncthreads();
    return counts[tries++];
  };
  float high = INFINITY, bound = -INFINITY;  // fewer than k reach `high`, k or more the bound
  if (top != -INFINITY) {
    float d = 0.5f;
    for (; d < 1e30f; d *= 4.f) {  // 51 counts at most, and 8
      const float t = top - d;
      const int n = count(t);
      if (n >= p.k) {
        bound = t;
        for (int i = 0, have = n; i < 8 && have > 2 * p.k + 16; ++i) {
          const float mid = high == INFINITY ? 0.5f * (top + bound) : 0.5f * (high + bound);
          const int c = count(mid);
          if (c >= p.k) {
            bound = mid;
            have = c;
          } else {
            high = mid;
          }
        }
        break;
      }
      high = t;
    }
  }
  // a rough score is off by eight roundings of |score|, |logit - m| and |log sum| at most
  const float slack = (2.f * __int_as_float(spread_s) + fabsf(bound) + fabsf(top)) * 9.6e-7f;
  if (bound != -INFINITY) bound -= slack;
  // ---- exact scores of what reaches it
  u64 least = 0;
  uint32_t least_place = 0xffffffffu;
  for (int base = 0; base < total; base += kMergeThreads) {
    const int c = base + threadIdx.x;
    bool todo = c < total && rough[c] >= bound;
    u64 key = 0;
    uint32_t place = 0;
    if (todo) {
      const int beam = beam_of(c), i = c - beam * per, r = p.rows_per_seq == 1 ? 0 : beam;
      const float s = beam_s[beam].x;
      double score = -INFINITY;
      uint32_t token = i;
      if (!isnan(s)) {
        const u64 e = lists[r == beam ? c : i];
        token = token_of(e);
        score = (double)s + (((double)logit_of(e) - shift[r]) - lse[r]);
      }
      key = order_of(score);
      place = (uint32_t)beam * (uint32_t)p.vocab + token;
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
        cut_ranked(list, p.k);
        least = list.score[p.k - 1];  // (a full list has k entries)
        least_place = list.place[p.k - 1];
      }
    } while (more);
  }
  // ---- ranks
  const int n = min(list.count, kMergeCap), parts = n <= 64 ? 8 : n <= 128 ? 4 : n <= 256 ? 2 : 1;
  for (int i = threadIdx.x / parts; i < (n + 31) / 32 * 32; i += kMergeThreads / parts) {
    const u64 score = i < n ? list.score[i] : 0;
    const uint32_t place = i < n ? list.place[i] : 0;
    const int r = rank_of(list, n, score, place, parts);
    if (i >= n || r >= p.k || (threadIdx.x & (parts - 1)) != 0) continue;
    const int beam = (int)(place / (uint32_t)p.vocab);
    const size_t at = (size_t)b * p.ld_out + r;
    p.tokens[at] = (int)(place - (uint32_t)beam * (uint32_t)p.vocab);
    if (p.parents) p.parents[at] = p.parent_base + beam;
    if (p.scores_out) p.scores_out[at] = (float)score_of(score);
  }
}

// Pieces of a row: enough CTAs to fill the GPU four times over, none below 2048 logits, and no more
// candidates of a sequence than the merge holds.
int splits_of(int rows, int beams, int vocab, int k) {
  const int most = (vocab + 2047) / 2048, fit = kMostRough / 2 / (beams * k);
  const long long want = (4LL * chunk_sms() + rows - 1) / rows;
  const int s = (int)(want > most ? most : want), t = s > fit ? fit : s;
  return t < 1 ? 1 : t;
}

// Whole vectors of every thread (of either type), where the row has that many.
int chunk_of(int splits, int vocab) {
  const int per = (vocab + splits - 1) / splits;
  return (per + kThreads * 8 - 1) / (kThreads * 8) * (kThreads * 8);
}

template <typename T>
cudaError_t scan_rows(const Scan& p, dim3 grid, cudaStream_t s) {
  static SmemLimit limit;
  cudaError_t e = limit.raise(beam_scan_kernel<T>, (int)sizeof(ScanSmem));
  if (e != cudaSuccess) return e;
  beam_scan_kernel<T><<<grid, kThreads, sizeof(ScanSmem), s>>>(p);
  return cudaGetLastError();
}

struct Carved {
  u64* lists;
  Piece* pieces;
};
// (rows: of the call with a row per beam, which needs the most)
Carved carve(Carver& cv, int batch, int beams, int vocab, int k) {
  size_t pieces = 0;
  for (int rows : {batch, batch * beams}) {  // a shared row per sequence, or one per beam
    const size_t n = (size_t)rows * splits_of(rows, beams, vocab, k);
    pieces = n > pieces ? n : pieces;
  }
  Carved c;
  c.lists = cv.take<u64>(pieces * k);
  c.pieces = cv.take<Piece>(pieces);
  return c;
}

}  // namespace

size_t beam_workspace(int batch, int beams, int vocab, int k) {
  Carver cv(nullptr, ~size_t(0));
  carve(cv, batch, beams, vocab, k);
  return cv.off;
}

cudaError_t beam_select(int dtype, const BeamParams& a, cudaStream_t s) {
  Carver cv(a.workspace, ~size_t(0));
  const Carved c = carve(cv, a.batch, a.beams, a.vocab, a.k);
  const int per_seq = a.ld_beam == 0 ? 1 : a.beams, rows = a.batch * per_seq;
  const int splits = splits_of(rows, a.beams, a.vocab, a.k);
  const Scan scan = {a.logits, a.ld_seq, a.ld_beam, c.lists, c.pieces, a.vocab, per_seq, splits, chunk_of(splits, a.vocab), a.k};
  {
    LaunchScope ls_(DFLASH_KERNEL_BEAM_SCAN, s);
    const dim3 grid(a.batch, per_seq, splits);
    cudaError_t e;
    if (dtype == DFLASH_F32)
      e = scan_rows<float>(scan, grid, s);
    else
      e = scan_rows<bf16>(scan, grid, s);
    if (e != cudaSuccess) return e;
  }
  LaunchScope ls_(DFLASH_KERNEL_BEAM_MERGE, s);
  const Merge merge = {c.lists, c.pieces, a.scores, a.tokens, a.parents, a.scores_out, a.ld_out,
                       a.beams, per_seq, splits, a.k, a.vocab, a.parent_base};
  static SmemLimit limit;
  cudaError_t e = limit.raise(beam_merge_kernel, (int)sizeof(float) * kMostRough);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.batch);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = sizeof(float) * (size_t)a.beams * splits * a.k;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // scheduled as SMs fall free
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_merge_kernel, merge);
}

}  // namespace dflash
