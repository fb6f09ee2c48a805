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
// The k largest. The first tile's per-thread maxima give a bound that at least k elements reach (the
// lowest of the warps' q-th largest, 8 q >= k); what reaches it goes to a list in shared memory, which is
// cut to its k best whenever it has grown to a few times that, and then its last entry is the
// bound. Of a long row only a handful of elements per tile are looked at twice.
//
// The sum. Which candidate of two beams is the better one is decided by the difference of two such
// sums, so their errors must stay far below the gaps between scores (about 10^-2 among the best of a
// vocabulary): d = x - ref (exact for bf16 within 16 binades), n = round(d log2 e),
// f = d log2 e - n in two terms, e^d = 2^f 2^n. Without the split the rounding of d log2 e alone
// would be 10^-6. Terms in fp32, a thread's tiles added with their rounding errors kept, the rest in
// 64 bits. A piece's few large terms, where an error does not average out, are taken again in 64 bits by
// the merge. The order of the additions depends on the vocabulary alone, so equal rows have equal sums
// and their candidates tie as they should.
#include <float.h>

#include "tree.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCap = 1024;     // entries of the list
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

// log2 e as a float and what it leaves.
constexpr float kL = 1.44269502f, kLlo = 1.92596303e-8f;
constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number, held in the low bits

// acc + (e^d0, e^d1) for d up to kFar; 0 below e^-88, NaN for NaN.
__device__ __forceinline__ float2 exp2_add(float2 d, float2 acc) {
  float2 t = __fmul2_rn(d, make_float2(kL, kL));
  t.x = max_nan(t.x, -127.f);
  t.y = max_nan(t.y, -127.f);
  const float2 r = __fadd2_rn(t, make_float2(kRound, kRound));
  const float2 n = __fadd2_rn(r, make_float2(-kRound, -kRound));
  float2 f = __ffma2_rn(d, make_float2(kL, kL), make_float2(-n.x, -n.y));
  f = __ffma2_rn(d, make_float2(kLlo, kLlo), f);
  const float2 p = make_float2(__uint_as_float((__float_as_uint(r.x) << 23) + (127u << 23)),
                               __uint_as_float((__float_as_uint(r.y) << 23) + (127u << 23)));
  return __ffma2_rn(make_float2(ex2(f.x), ex2(f.y)), p, acc);
}

// Eight logits from element e of a row (of which `end` exist; the others -inf).
template <typename T> struct Eight;
template <> struct Eight<bf16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const bf16* row, int e, int end, int shift) {
    if (e + 8 <= end) {
      if (shift == 0) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(row + e));
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
      } else {  // the two aligned 16-byte blocks that hold them, shifted by `shift` bytes
        const uint4* at = reinterpret_cast<const uint4*>((uintptr_t)(row + e) & ~(uintptr_t)15);
        const uint4 a = __ldg(at), b = __ldg(at + 1);
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
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = e + 2 * i < end ? reinterpret_cast<const uint16_t*>(row)[e + 2 * i] : 0xFF80u;
        const uint32_t hi = e + 2 * i + 1 < end ? reinterpret_cast<const uint16_t*>(row)[e + 2 * i + 1] : 0xFF80u;
        w[i] = lo | hi << 16;
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
};
template <> struct Eight<float> {
  float x[8];
  __device__ __forceinline__ void load(const float* row, int e, int end, int shift) {
    if (shift == 0 && e + 8 <= end) {
      const float4 a = __ldcs(reinterpret_cast<const float4*>(row + e)), b = __ldcs(reinterpret_cast<const float4*>(row + e + 4));
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = e + i < end ? __ldg(row + e + i) : -INFINITY;
    }
  }
  __device__ __forceinline__ float at(int i) const { return x[i]; }
};
template <typename T> constexpr int kVecs = sizeof(T) == 2 ? 4 : 2;  // vectors of a thread and tile

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

struct List {
  u64 e[kCap];
  int count;
};

// Cuts the list to its k best, best first; all threads. Returns how many there are.
__device__ __forceinline__ int keep_best(List& l, int k) {
  const int n = min(l.count, kCap);
  u64 mine[kCap / kThreads];
  int rank[kCap / kThreads] = {};
#pragma unroll
  for (int t = 0; t < kCap / kThreads; ++t) {
    const int i = threadIdx.x + t * kThreads;
    mine[t] = i < n ? l.e[i] : 0;
    if (t * kThreads < n) {
#pragma unroll 4
      for (int j = 0; j < n; ++j) rank[t] += l.e[j] > mine[t];
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < kCap / kThreads; ++t)
    if (threadIdx.x + t * kThreads < n && rank[t] < k) l.e[rank[t]] = mine[t];
  if (threadIdx.x == 0) l.count = min(n, k);
  __syncthreads();
  return min(n, k);
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

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_scan_kernel(const Scan p) {
  constexpr int J = kVecs<T>, TILE = kThreads * 8 * J;
  __shared__ List list;
  __shared__ float wmax[kWarps], wth[kWarps];
  __shared__ double wsum[kWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge may be scheduled
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x / p.splits, split = blockIdx.x - row * p.splits;
  const int seq = row / p.rows_per_seq, beam = row - seq * p.rows_per_seq;
  const T* x = (const T*)p.logits + seq * p.ld_seq + beam * p.ld_beam;
  const int shift = (int)((uintptr_t)x & 15);
  const int begin = min(p.vocab, split * p.chunk), end = min(p.vocab, begin + p.chunk);
  if (threadIdx.x == 0) list.count = 0;
  Eight<T> now[J], nxt[J];
#pragma unroll
  for (int j = 0; j < J; ++j) now[j].load(x, begin + (j * kThreads + (int)threadIdx.x) * 8, end, shift);
  float ref = -INFINITY, far = -INFINITY;  // far: beyond it the reference has to move
  float bound = -INFINITY;                 // the logit of what has to be beaten
  u64 least = 0;                           // what has to be beaten
  float sum = 0.f, low = 0.f;              // sum + low
  bool first = true;
  const int full = max(2 * p.k, 64);       // entries that are cut to k
  for (int base = begin; base < end; base += TILE) {
    if (base + TILE < end) {
#pragma unroll
      for (int j = 0; j < J; ++j) nxt[j].load(x, base + TILE + (j * kThreads + (int)threadIdx.x) * 8, end, shift);
    }
    float most = -INFINITY;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) most = fmaxf(most, now[j].at(i));
    if (first) {
      const float v = sort_lanes(most);
      const float q = __shfl_sync(0xffffffffu, v, (p.k + kWarps - 1) / kWarps - 1);
      if (lane == 0) {
        wmax[warp] = v;
        wth[warp] = q;
      }
      __syncthreads();
      bound = wth[0];
      float top = wmax[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        bound = fminf(bound, wth[w]);
        top = fmaxf(top, wmax[w]);
      }
      least = entry_of(bound, 0xffffffffu) - 1;  // the bound itself beats it
      ref = top;
      far = ref + kFar;  // (infinity stays; a row without a finite logit so far: -inf)
      first = false;
    }
    const bool jump = most > far || most == INFINITY;
    uint32_t todo = 0;  // elements to be entered
    if (most >= bound) {
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = base + (j * kThreads + (int)threadIdx.x) * 8 + i;
          const float v = now[j].at(i);
          if (v >= bound && e < end && entry_of(v, e) > least) todo |= 1u << (8 * j + i);
        }
    }
    if (__syncthreads_or(todo != 0 || jump)) {
      // ---- the list
      bool more;
      do {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if ((todo >> (8 * j + i) & 1) == 0) continue;
            const u64 v = entry_of(now[j].at(i), base + (j * kThreads + (int)threadIdx.x) * 8 + i);
            const int at = v > least ? atomicAdd(&list.count, 1) : 0;
            if (v > least && at >= kCap) continue;  // full: once more, when it has been cut
            if (v > least) list.e[at] = v;
            todo &= ~(1u << (8 * j + i));
          }
        more = __syncthreads_or(todo != 0);
        if (more || list.count >= full) {
          if (keep_best(list, p.k) == p.k) {
            least = list.e[p.k - 1];
            bound = logit_of(least);
          }
        }
      } while (more);
      // ---- the reference
      if (__syncthreads_or(jump)) {
        float top = warp_max(most);
        if (lane == 0) wmax[warp] = top;
        __syncthreads();
        top = wmax[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, wmax[w]);
        if (top == INFINITY) {
          sum = NAN;  // (and far is infinite: it stays that)
        } else if (ref != -INFINITY) {
          const float k = expf(ref - top);
          sum *= k;
          low *= k;
        }
        ref = top;
        far = ref + kFar;
      }
    }
    // ---- the sum
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    if (ref != -INFINITY && ref != INFINITY) {
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          acc[(i >> 1) & 1] = exp2_add(__fadd2_rn(make_float2(now[j].at(i), now[j].at(i + 1)), make_float2(-ref, -ref)),
                                       acc[(i >> 1) & 1]);
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (isnan(now[j].at(i))) acc[0].x = NAN;
    }
    const float tile = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
    const float s = sum + tile, t = s - sum;  // and the rounding error of s
    low += (sum - (s - t)) + (tile - t);
    sum = s;
#pragma unroll
    for (int j = 0; j < J; ++j) now[j] = nxt[j];
  }
  __syncthreads();
  const int kept = keep_best(list, p.k);
  const size_t piece = (size_t)row * p.splits + split;
  for (int i = threadIdx.x; i < p.k; i += kThreads) p.lists[piece * p.k + i] = i < kept ? list.e[i] : 0;
  double d = (double)sum + (double)low;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0) wsum[warp] = d;
  __syncthreads();
  if (threadIdx.x == 0) {
    d = wsum[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) d += wsum[w];
    p.pieces[piece] = {d, ref, 0};
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

// Ranked candidates: the score's order, then the lowest place.
struct Ranked {
  u64 score[kCap];
  uint32_t place[kCap];  // beam * vocab + token
  int count;
};

template <int THREADS>
__device__ __forceinline__ void keep_best(Ranked& l, int k) {
  const int n = min(l.count, kCap);
  u64 mine[kCap / THREADS];
  uint32_t at[kCap / THREADS];
  int rank[kCap / THREADS] = {};
#pragma unroll
  for (int t = 0; t < kCap / THREADS; ++t) {
    const int i = threadIdx.x + t * THREADS;
    mine[t] = i < n ? l.score[i] : 0;
    at[t] = i < n ? l.place[i] : 0;
    if (t * THREADS < n) {
#pragma unroll 4
      for (int j = 0; j < n; ++j) rank[t] += l.score[j] > mine[t] || (l.score[j] == mine[t] && l.place[j] < at[t]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < kCap / THREADS; ++t)
    if (threadIdx.x + t * THREADS < n && rank[t] < k) {
      l.score[rank[t]] = mine[t];
      l.place[rank[t]] = at[t];
    }
  if (threadIdx.x == 0) l.count = min(n, k);
  __syncthreads();
}

// A CTA per sequence.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) beam_merge_kernel(const Merge p) {
  constexpr int WARPS = THREADS / 32;
  __shared__ Ranked list;
  __shared__ double lse[kBeamMax], shift[kBeamMax];  // log of the row's sum under m; m
  __shared__ float wth[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the scan's lists
  const u64* lists = p.lists + (size_t)b * p.rows_per_seq * p.splits * p.k;
  const Piece* pieces = p.pieces + (size_t)b * p.rows_per_seq * p.splits;
  if (threadIdx.x == 0) list.count = 0;
  // ---- a row's sum: a warp per row, a lane per piece. Terms above 1/16 of it are taken again in
  // 64 bits: the scan's differ from them by up to 2^-22
  for (int r = warp; r < p.rows_per_seq; r += WARPS) {
    float m = -INFINITY;
    for (int s = lane; s < p.splits; s += 32) m = fmaxf(m, pieces[r * p.splits + s].ref);
    m = warp_max(m);
    double sum = 0.0, fix = 0.0;
    for (int s = lane; s < p.splits; s += 32) {
      const Piece c = pieces[r * p.splits + s];
      if (c.ref == -INFINITY) {
        sum += c.sum;  // 0, or NaN
        continue;
      }
      const double w = c.ref == m ? 1.0 : exp((double)c.ref - (double)m);
      sum += c.sum * w;
      const u64* l = lists + (size_t)(r * p.splits + s) * p.k;
      for (int i = 0; i < p.k; ++i) {
        const u64 e = l[i];
        if (e == 0) break;
        const float d = logit_of(e) - c.ref, term = exp2_add(make_float2(d, -INFINITY), make_float2(0.f, 0.f)).x;
        if (!((double)term * 16.0 > c.sum)) break;
        fix += (exp((double)d) - (double)term) * w;
      }
    }
    sum += fix;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      const bool dead = !(sum > 0.0 && sum < INFINITY) || m == INFINITY || m == -INFINITY;
      lse[r] = dead ? NAN : log(sum);
      shift[r] = m;
    }
  }
  __syncthreads();
  // ---- candidates: c = (beam * splits + split) * k + place in the piece's list
  const int per = p.splits * p.k, total = p.beams * per;
  // score in 32 bits with a bound of its error, to leave most of them out
  auto rough = [&](int c, float* err) -> float {
    const int beam = c / per, i = c - beam * per, r = p.rows_per_seq == 1 ? 0 : beam;
    const float s = p.scores ? p.scores[(size_t)b * p.beams + beam] : 0.f;
    *err = 0.f;
    if (!isfinite(s) || isnan(lse[r])) return i < min(p.k, p.vocab) ? -INFINITY : NAN;
    const u64 e = lists[(size_t)r * per + i];
    if (e == 0) return NAN;
    const float d = logit_of(e) - (float)shift[r], z = (float)lse[r];
    *err = (fabsf(s) + fabsf(d) + fabsf(z)) * 4.8e-7f;  // 2^-21: eight roundings
    const float v = s + (d - z);
    if (v == -INFINITY) *err = 0.f;
    return v;
  };
  // the lowest of the warps' q-th largest: at least k candidates reach it
  const int active = min(WARPS, (total + 31) / 32), q = (p.k + active - 1) / active;
  float most = -INFINITY;
  for (int c = threadIdx.x; c < total; c += THREADS) {
    float err;
    const float v = rough(c, &err);
    if (v == v) most = fmaxf(most, v - err);
  }
  const float sorted = sort_lanes(most);
  if (lane == 0 && warp < active) wth[warp] = INFINITY;
  __syncwarp();
  if (warp < active && lane == min(q, 32) - 1) wth[warp] = q <= 32 ? sorted : -INFINITY;
  __syncthreads();
  float bound = wth[0];
  for (int w = 1; w < active; ++w) bound = fminf(bound, wth[w]);
  // ---- exact scores of what reaches it
  u64 least = 0;
  uint32_t least_place = 0xffffffffu;
  for (int base = 0; base < total; base += THREADS) {
    const int c = base + threadIdx.x;
    bool todo = false;
    u64 key = 0;
    uint32_t place = 0;
    if (c < total) {
      float err;
      const float v = rough(c, &err);
      if (v == v && v + err >= bound) {
        const int beam = c / per, i = c - beam * per, r = p.rows_per_seq == 1 ? 0 : beam;
        const float s = p.scores ? p.scores[(size_t)b * p.beams + beam] : 0.f;
        double score = -INFINITY;
        uint32_t token = i;
        if (isfinite(s) && !isnan(lse[r])) {
          const u64 e = lists[(size_t)r * per + i];
          token = token_of(e);
          score = (double)s + (((double)logit_of(e) - shift[r]) - lse[r]);
        }
        key = order_of(score);
        place = (uint32_t)beam * (uint32_t)p.vocab + token;
        todo = true;
      }
    }
    bool more;
    do {
      if (todo && (key < least || (key == least && place >= least_place))) todo = false;
      if (todo) {
        const int at = atomicAdd(&list.count, 1);
        if (at < kCap) {
          list.score[at] = key;
          list.place[at] = place;
          todo = false;
        }
      }
      more = __syncthreads_or(todo);
      if (more) {
        keep_best<THREADS>(list, p.k);
        least = list.score[p.k - 1];  // (a full list has k entries)
        least_place = list.place[p.k - 1];
      }
    } while (more);
  }
  __syncthreads();
  keep_best<THREADS>(list, p.k);
  for (int i = threadIdx.x; i < p.k; i += THREADS) {
    const uint32_t place = list.place[i];
    const int beam = (int)(place / (uint32_t)p.vocab);
    const size_t at = (size_t)b * p.ld_out + i;
    p.tokens[at] = (int)(place - (uint32_t)beam * (uint32_t)p.vocab);
    if (p.parents) p.parents[at] = p.parent_base + beam;
    if (p.scores_out) p.scores_out[at] = (float)score_of(list.score[i]);
  }
}

// Pieces of a row: enough CTAs to fill the GPU four times over, none below 2048 logits.
int splits_of(int rows, int vocab) {
  const int most = (vocab + 2047) / 2048;
  const long long want = (4LL * chunk_sms() + rows - 1) / rows;
  const int s = (int)(want < 1 ? 1 : want > most ? most : want);
  return s;
}

int chunk_of(int splits, int vocab) { return ((vocab + splits - 1) / splits + 7) / 8 * 8; }

struct Carved {
  u64* lists;
  Piece* pieces;
};
// (rows: of the call with a row per beam, which needs the most)
Carved carve(Carver& cv, int batch, int beams, int vocab, int k) {
  size_t pieces = 0;
  for (int rows : {batch, batch * beams}) {  // a shared row per sequence, or one per beam
    const size_t n = (size_t)rows * splits_of(rows, vocab);
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
  const int splits = splits_of(rows, a.vocab);
  const Scan scan = {a.logits, a.ld_seq, a.ld_beam, c.lists, c.pieces, a.vocab, per_seq, splits, chunk_of(splits, a.vocab), a.k};
  {
    LaunchScope ls_(DFLASH_KERNEL_BEAM_SCAN, s);
    if (dtype == DFLASH_F32)
      beam_scan_kernel<float><<<rows * splits, kThreads, 0, s>>>(scan);
    else
      beam_scan_kernel<bf16><<<rows * splits, kThreads, 0, s>>>(scan);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  LaunchScope ls_(DFLASH_KERNEL_BEAM_MERGE, s);
  const Merge merge = {c.lists, c.pieces, a.scores, a.tokens, a.parents, a.scores_out, a.ld_out,
                       a.beams, per_seq, splits, a.k, a.vocab, a.parent_base};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.batch);
  const bool wide = (long long)a.beams * splits * a.k > 1024;
  cfg.blockDim = dim3(wide ? 512 : 128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // scheduled as SMs fall free
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return wide ? cudaLaunchKernelEx(&cfg, beam_merge_kernel<512>, merge) : cudaLaunchKernelEx(&cfg, beam_merge_kernel<128>, merge);
}

}  // namespace dflash
