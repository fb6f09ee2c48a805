// Causal chunk attention on FFMA (f32): softmax(q K^T scaling) V with one pass over the keys, the
// running maximum m and sum l of each row rescaling its output as m grows:
//   m' = max(m, max_j s_j);  l = l e^(m - m') + sum_j e^(s_j - m');
//   o = o e^(m - m') + sum_j e^(s_j - m') v_j;  out = o / l.
// fp32 products keep all 24 bits (a TF32 tensor-core product would lose about 11).
//
// Bound by the FFMA pipe: 4 n k d_h operations per head and row pair, at 128 multiply-adds per SM
// and cycle, issued two at a time. The two operands of a pair are two query rows (scores; Q lies
// transposed in shared memory) or two output columns (values).
//
// Persistent CTAs walk their shares of the cost line (chunk.cuh). 256 threads hold a 128 x 64 score
// tile as 8 rows x 4 keys a thread, and 8 rows x d_h / 16 columns of the output: 64 shared words
// per 128 pairs, half of what a 64 x 64 tile reads. Items of at most 64 rows take 4 rows a thread,
// of at most 16 rows one (a decoded token would spend eight times the arithmetic on rows that are
// not there); a warp none of whose rows sees a tile skips its products. K and V have one buffer
// each: the next K tile is copied in while the PV product runs, the next V tile during the next
// scores. Two CTAs share an SM up to d_h 64, and one computes while the other waits at a barrier.
//
// Measured on 6 prompts of 65 to 600 rows over up to 900 held, 8 heads of 64: 131 us, where the
// multiply-adds of whole tiles alone are 47. On one prompt of 8192 rows, where neither ragged tiles
// nor uneven shares (up to a fifth apart at six tiles a CTA) count: 1.64 ms, 42 TFLOP/s, the pipe
// busy for half of the time. The same with 64-row items, one CTA per SM and single multiply-adds:
// 189 us; pairs alone 176, 128-row items 168, two CTAs 148, idle warps skipped 144, Q read a row
// per thread 133, no mask where every row sees every key 131.
#include <float.h>

#include "chunk.cuh"

namespace dflash {
namespace {

constexpr int TK = 64;   // keys per tile (2^6)
constexpr int kThreads = 256;
constexpr int LP = TK + 4;

// Stacked query rows of an item: what shared memory holds next to the K and V tiles.
constexpr int item_rows(int d) { return d <= 128 ? 128 : 64; }
constexpr int ctas_per_sm(int d) { return d <= 64 ? 2 : 1; }

__device__ __forceinline__ void copy_async(float* dst, const float* src, int bytes, bool in) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  const int n = in ? bytes : 0;  // the rest is filled with zeros
  if (bytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A tile of `rows` key rows (the others zero) of d elements, rows LD apart in shared memory.
// (d is even: 16 bytes at a time where d is a multiple of 4, else 8.)
template <int LD>
__device__ __forceinline__ void load_tile(float* dst, const float* src, int d, int rows) {
  const int step = d % 4 == 0 ? 4 : 2, per = d / step;
  int r = threadIdx.x / per, c = threadIdx.x - r * per;
  const int dr = kThreads / per, dc = kThreads - dr * per;
  while (r < TK) {
    const bool in = r < rows;
    copy_async(dst + r * LD + c * step, in ? src + (size_t)r * d + c * step : src, 4 * step, in);
    r += dr;
    c += dc;
    if (c >= per) {
      c -= per;
      ++r;
    }
  }
}

// One piece of work. RPT: query rows per thread (the item has at most 16 RPT).
template <int DP, int RPT, bool TREE>
__device__ __forceinline__ void piece(const ChunkAttnParams& p, const chunk::Piece<TREE>& w, int r0, int rows, float* Qs,
                                      float* Ks, float* Vs, float* Ps) {
  constexpr int LD = DP + 4, LQ = item_rows(DP) + 4;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, d = p.d_h;
  const size_t slab = ((size_t)w.b * p.n_kv + w.kvh) * p.capacity;
  const float* ck = (const float*)p.cache_k + slab * d;
  const float* cv = (const float*)p.cache_v + slab * d;
  auto keys = [&](int j) { return min(TK, w.kv - (w.k0 + j * TK)); };  // what lies past the length is never read
  auto at = [&](int j) { return (size_t)(w.k0 + j * TK) * d; };
  if (w.tile0 < w.tile1) load_tile<LD>(Ks, ck + at(w.tile0), d, keys(w.tile0));
  copy_commit();
  if (w.tile0 < w.tile1) load_tile<LD>(Vs, cv + at(w.tile0), d, keys(w.tile0));
  copy_commit();
  // A thread copies one row's columns 4 c .. 4 c + 3, or two at a time, and writes them transposed.
  for (int r = threadIdx.x & (16 * RPT - 1), c0 = threadIdx.x / (16 * RPT) * 4; c0 < DP; c0 += 4 * (kThreads / (16 * RPT))) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows && c0 < d) {
      const int token = (r0 + r) / p.G, g = r0 + r - token * p.G;
      const float* q = (const float*)p.q + (size_t)(w.row0 + token) * p.ld_q + (size_t)(w.kvh * p.G + g) * d + c0;
      x.x = q[0];
      x.y = q[1];
      if (c0 + 2 < d) {
        x.z = q[2];
        x.w = q[3];
      }
    }
    Qs[c0 * LQ + r] = x.x;  // (a thread's rows of the products lie side by side)
    Qs[(c0 + 1) * LQ + r] = x.y;
    Qs[(c0 + 2) * LQ + r] = x.z;
    Qs[(c0 + 3) * LQ + r] = x.w;
  }
  float m[RPT], l[RPT];
  [[maybe_unused]] unsigned seen = 0;  // TREE: rows that have seen a key, whatever its score
  float2 o[RPT][DP / 32];  // columns 4 tx + 64 c .. + 3 in pairs
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < DP / 32; ++e) o[i][e] = make_float2(0.f, 0.f);
  }
  const int first = w.kv - w.n + r0 / p.G, last = w.kv - w.n + (r0 + rows - 1) / p.G;
  // Keys of this warp's 2 RPT rows: a warp skips the products of a tile that none of them sees.
  const int wr = (ty & ~1) * RPT;
  const int wlast = wr < rows ? w.kv - w.n + (r0 + min(wr + 2 * RPT, rows) - 1) / p.G : -1;
  int wfirst = p.window > 0 ? w.kv - w.n + (r0 + wr) / p.G - p.window + 1 : 0;
  int closed = first + 1;  // the first key that not every row sees, but for the window
  if constexpr (TREE) {
    closed = w.ctx;
    if (p.window > 0) wfirst = w.ctx - p.window + 1;
  }
  for (int j = w.tile0; j < w.tile1; ++j) {
    const int k0 = w.k0 + j * TK;
    const bool sees = k0 <= wlast && k0 + TK > wfirst;
    const bool open = k0 + TK <= closed && (p.window <= 0 || last - k0 < p.window);  // every key by every row
    const bool more = j + 1 < w.tile1;
    if constexpr (TREE) {
      // A row's mask words by one thread, behind the row's weights. (Sixteen threads share a row; with each looking
      // for itself 32 trees of 107 to 207 nodes, 8 heads of 64, took 174 us instead of 144.)
      const int r = threadIdx.x;
      if (!open && r < rows) {
        const uint4 bits = chunk::tree_bits(p.tree, w.b, w.kv - w.n + (r0 + r) / p.G - w.ctx, w.ctx, k0, p.window);
        *reinterpret_cast<uint2*>(Ps + r * LP + TK) = make_uint2(bits.x, bits.y);  // (a tile is 64 keys here)
      }
    }
    copy_wait<1>();  // K_j (V_j may be on its way)
    __syncthreads();
    float s[RPT][4] = {};
    if (!sees) {
    } else if constexpr (RPT == 1) {
#pragma unroll 4
      for (int c = 0; c < DP; c += 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 b = *reinterpret_cast<const float4*>(Ks + (tx + 16 * k) * LD + c);
          s[0][k] = fmaf(Qs[c * LQ + ty], b.x, s[0][k]);
          s[0][k] = fmaf(Qs[(c + 1) * LQ + ty], b.y, s[0][k]);
          s[0][k] = fmaf(Qs[(c + 2) * LQ + ty], b.z, s[0][k]);
          s[0][k] = fmaf(Qs[(c + 3) * LQ + ty], b.w, s[0][k]);
        }
      }
    } else {
      float2 s2[RPT / 2][4] = {};  // two rows
#pragma unroll 2
      for (int c = 0; c < DP; c += 4) {
        float b[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<float4*>(b[k]) = *reinterpret_cast<const float4*>(Ks + (tx + 16 * k) * LD + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int i = 0; i < RPT / 4; ++i) {
            const float4 a = *reinterpret_cast<const float4*>(Qs + (c + e) * LQ + ty * RPT + 4 * i);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 bb = make_float2(b[k][e], b[k][e]);
              s2[2 * i][k] = __ffma2_rn(make_float2(a.x, a.y), bb, s2[2 * i][k]);
              s2[2 * i + 1][k] = __ffma2_rn(make_float2(a.z, a.w), bb, s2[2 * i + 1][k]);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[i][k] = i & 1 ? s2[i / 2][k].y : s2[i / 2][k].x;
    }
    __syncthreads();  // K_j has been read
    if (more) load_tile<LD>(Ks, ck + at(j + 1), d, keys(j + 1));
    copy_commit();
    if (sees) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      float mx = m[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) s[i][k] *= p.scaling;
      if (!open) {
        const int r = ty * RPT + i, pos = r < rows ? w.kv - w.n + (r0 + r) / p.G : -1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = k0 + tx + 16 * k;
          if (!TREE && (key > pos || (p.window > 0 && pos - key >= p.window))) s[i][k] = -INFINITY;
        }
        if constexpr (TREE) {
          const uint2 bits = r < rows ? *reinterpret_cast<const uint2*>(Ps + r * LP + TK) : make_uint2(0, 0);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (((k < 2 ? bits.x : bits.y) >> (tx + 16 * (k & 1)) & 1) == 0) s[i][k] = -INFINITY;
          if (bits.x | bits.y) seen |= 1u << i;
        }
      } else if constexpr (TREE) {
        seen |= 1u << i;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) mx = fmaxf(mx, s[i][k]);
#pragma unroll
      for (int of = 8; of > 0; of >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, of));
      const float ref = mx == -INFINITY ? 0.f : mx;
      const float alpha = expf(m[i] - ref);  // 0 while the row has seen no key
      m[i] = mx;
      l[i] *= alpha;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float e = expf(s[i][k] - ref);
        l[i] += e;
        Ps[(ty * RPT + i) * LP + tx + 16 * k] = e;
      }
#pragma unroll
      for (int e = 0; e < DP / 32; ++e) o[i][e] = __fmul2_rn(o[i][e], make_float2(alpha, alpha));
    }
    }
    copy_wait<1>();   // V_j (K_{j+1} may be on its way)
    __syncthreads();  // (and P)
    // A key that a row does not see has weight 0, and its value must not enter even as 0 * NaN:
    // where the mask cuts a tile that holds such values, zero weights are skipped.
    bool plain = open;
    if (!plain) {
      float zero = 0.f;
      for (int i = threadIdx.x; i < TK * DP / 4; i += kThreads) {
        const float4 v = *reinterpret_cast<const float4*>(Vs + i / (DP / 4) * LD + i % (DP / 4) * 4);
        zero += 0.f * v.x + 0.f * v.y + 0.f * v.z + 0.f * v.w;  // NaN if one is not finite
      }
      plain = !__syncthreads_or(zero != 0.f);
    }
    if (!sees) {
    } else if (plain) {
#pragma unroll 2
      for (int k = 0; k < TK; k += 4) {
        float4 pr[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) pr[i] = *reinterpret_cast<const float4*>(Ps + (ty * RPT + i) * LP + k);
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) {
          float4 v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const float4*>(Vs + (k + e) * LD + tx * 4 + 64 * c);
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            const float pk[4] = {pr[i].x, pr[i].y, pr[i].z, pr[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[i][2 * c] = __ffma2_rn(make_float2(pk[e], pk[e]), make_float2(v[e].x, v[e].y), o[i][2 * c]);
              o[i][2 * c + 1] = __ffma2_rn(make_float2(pk[e], pk[e]), make_float2(v[e].z, v[e].w), o[i][2 * c + 1]);
            }
          }
        }
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < TK; ++k) {
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(Vs + k * LD + tx * 4 + 64 * c);
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            const float pv = Ps[(ty * RPT + i) * LP + k];
            if (pv == 0.f) continue;
            o[i][2 * c] = __ffma2_rn(make_float2(pv, pv), make_float2(v.x, v.y), o[i][2 * c]);
            o[i][2 * c + 1] = __ffma2_rn(make_float2(pv, pv), make_float2(v.z, v.w), o[i][2 * c + 1]);
          }
        }
      }
    }
    __syncthreads();  // V_j and P have been read
    if (more) load_tile<LD>(Vs, cv + at(j + 1), d, keys(j + 1));
    copy_commit();
  }
  copy_wait<0>();
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    float sum = l[i];
#pragma unroll
    for (int of = 8; of > 0; of >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, of);
    const int r = ty * RPT + i;
    if (r >= rows) continue;
    const size_t part = (size_t)(2 * blockIdx.x + (w.slot > 0)) * item_rows(DP) + r;
    const int token = (r0 + r) / p.G, g = r0 + r - token * p.G;
    float* dst = w.slot < 0 ? (float*)p.out + ((size_t)(w.row0 + token) * p.n_h + w.kvh * p.G + g) * d : p.part + part * d;
    // no weight at all: 0 where no key is seen, else (every score minus infinity) NaN
    const bool sees_any = TREE ? (seen >> i & 1) != 0 : w.kv - w.n + token >= 0;
    const float inv = w.slot >= 0 ? 1.f : sum != 0.f ? 1.f / sum : sees_any ? NAN : 0.f;
#pragma unroll
    for (int e = 0; e < DP / 32; ++e) {
      const int c = tx * 4 + 64 * (e >> 1) + 2 * (e & 1);  // (d is even)
      if (c < d) *reinterpret_cast<float2*>(dst + c) = make_float2(o[i][e].x * inv, o[i][e].y * inv);
    }
    if (w.slot >= 0 && tx == 0)
      p.part_ml[part] = make_float2(sum == 0.f && sees_any ? -FLT_MAX : m[i], sum);
  }
}

template <int DP, bool TREE>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(DP)) chunk_attn_simt_kernel(const ChunkAttnParams p) {
  constexpr int LD = DP + 4, RI = item_rows(DP);
  extern __shared__ float4 smem4[];
  float* Qs = reinterpret_cast<float*>(smem4);
  float* Ks = Qs + DP * (RI + 4);
  float* Vs = Ks + TK * LD;
  float* Ps = Vs + TK * LD;
  __shared__ chunk::Start<TREE> start;
  // Cost units: an item 2, a tile 6, one of an item of few rows 3 (or 2). In a replayed graph, an item at 0,
  // 2, 4, 8: 6 prompts 135, 133, 132, 132 us, 32 blocks of 16 rows 227, 227, 228, 237. A tile of few rows
  // at 2, 3, 6 of 6: 14 tokens and 6 chunks 149, 145, 190, 6 prompts 146, 133, 140.
  const chunk::Split<false, TREE> split = {p.cu_rows, p.kv_lens, p.batch, p.rows, p.n_kv, p.G, p.capacity,
                              p.window, RI, 0, RI / (RI > 64 ? 2 : 4), 6, 2, 6, RI > 64 ? 3 : 2, p.tree.nodes, p.tree.max_nodes};
  grid_wait();
  grid_trigger();  // the merge may be scheduled
  if (p.batch > 32)
    chunk::locate(split, smem4, &start, p.status);
  else if (threadIdx.x < 32)
    chunk::locate_by_warp(split, &start, p.status);
  __syncthreads();
  chunk::Walker<false, TREE> walk(split, start);
  // columns beyond d_h stay zero
  for (int i = threadIdx.x; i < 2 * TK * LD; i += kThreads) Ks[i] = 0.f;
  chunk::Piece<TREE> w;
  while (walk.next(&w)) {
    const int r0 = w.t * RI, rows = min(RI, w.n * p.G - r0);
    __syncthreads();
    if (rows <= 16)
      piece<DP, 1, TREE>(p, w, r0, rows, Qs, Ks, Vs, Ps);
    else if (RI == 64 || rows <= 64)
      piece<DP, 4, TREE>(p, w, r0, rows, Qs, Ks, Vs, Ps);
    else
      piece<DP, RI / 16, TREE>(p, w, r0, rows, Qs, Ks, Vs, Ps);
  }
  if (threadIdx.x == 0) p.merge[blockIdx.x] = walk.merge;
}

template <int DP, bool TREE>
cudaError_t launch(const ChunkAttnParams& p, cudaStream_t s) {
  constexpr int RI = item_rows(DP);
  const int tiles = (int)sizeof(float) * (DP * (RI + 4) + 2 * TK * (DP + 4) + RI * LP);
  const int scratch = (int)(chunk::kLocateBytes<TREE> * p.batch);
  const int smem = tiles > scratch ? tiles : scratch;
  const int most = (int)(chunk::kLocateBytes<TREE> * (TREE ? kTreeMaxBatch : kChunkMaxBatch));
  static SmemLimit limit;
  cudaError_t e = limit.raise(chunk_attn_simt_kernel<DP, TREE>, tiles > most ? tiles : most);
  if (e != cudaSuccess) return e;
  LaunchScope ls_(DFLASH_KERNEL_CHUNK_ATTN, s);
  return launch_overlapped(chunk_attn_simt_kernel<DP, TREE>, dim3(chunk_attn_simt_ctas(p.d_h)), kThreads, smem, s, p);
}

}  // namespace

int chunk_attn_simt_item_rows(int d_h) { return item_rows(d_h); }
int chunk_attn_simt_ctas(int d_h) { return chunk_sms() * ctas_per_sm(d_h); }

cudaError_t chunk_attn_simt(const ChunkAttnParams& p, cudaStream_t s) {
  if (p.d_h <= 64) return launch<64, false>(p, s);
  if (p.d_h <= 128) return launch<128, false>(p, s);
  return launch<256, false>(p, s);
}

cudaError_t tree_attn_simt(const ChunkAttnParams& p, cudaStream_t s) {
  if (p.d_h <= 64) return launch<64, true>(p, s);
  if (p.d_h <= 128) return launch<128, true>(p, s);
  return launch<256, true>(p, s);
}

}  // namespace dflash
