// Causal chunk attention on FFMA: softmax(q K^T scaling) V with one pass over the keys, the
// running maximum m and sum l of each row rescaling its output as m grows:
//   m' = max(m, max_j s_j);  l = l e^(m - m') + sum_j e^(s_j - m');
//   o = o e^(m - m') + sum_j e^(s_j - m') v_j;  out = o / l.
// fp32 products keep all 24 bits (a TF32 tensor-core product would lose about 11).
//
// Persistent: one CTA per SM walks its share of the cost line (chunk.cuh). 256 threads hold a
// 64 x 64 score tile as 4 x 4 per thread, and 4 rows x d_h / 16 columns of the output.
#include "chunk.cuh"

namespace dflash {
namespace {

constexpr int RI = 64;   // stacked query rows of an item
constexpr int TK = 64;   // keys per tile (2^6)
constexpr int kThreads = 256;

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) chunk_attn_simt_kernel(const ChunkAttnParams p) {
  constexpr int LD = DP + 4, LP = TK + 4;
  extern __shared__ float4 smem4[];
  float* Qs = reinterpret_cast<float*>(smem4);
  float* Ks = Qs + RI * LD;
  float* Vs = Ks + TK * LD;
  float* Ps = Vs + TK * LD;
  __shared__ chunk::Start start;
  const chunk::Split<false> split = {p.cu_rows, p.kv_lens, p.batch, p.rows, p.n_kv, p.G, p.capacity,
                              p.window, RI, 0, RI, 6, 1, 1, 1};
  chunk::locate(split, smem4, &start, p.status);
  chunk::Walker<false> walk;
  walk.init(split, start);
  __syncthreads();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, d = p.d_h;
  const float* q = (const float*)p.q;
  const float* ck = (const float*)p.cache_k;
  const float* cv = (const float*)p.cache_v;
  chunk::Piece w;
  while (walk.next(&w)) {
    const long long r0 = (long long)w.t * RI;
    const int rows = (int)min((long long)RI, (long long)w.n * p.G - r0);
    __syncthreads();
    for (int i = threadIdx.x; i < RI * DP; i += kThreads) {
      const int r = i / DP, c = i - r * DP;
      float x = 0.f;
      if (r < rows && c < d) {
        const int token = (int)((r0 + r) / p.G), g = (int)(r0 + r - (long long)token * p.G);
        x = q[(size_t)(w.row0 + token) * p.ld_q + (size_t)(w.kvh * p.G + g) * d + c];
      }
      Qs[r * LD + c] = x;
    }
    int pos[4];
    float m[4], l[4], o[4][DP / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      pos[i] = r < rows ? w.kv - w.n + (int)((r0 + r) / p.G) : -1;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int e = 0; e < DP / 16; ++e) o[i][e] = 0.f;
    }
    for (int j = w.tile0; j < w.tile1; ++j) {
      const int k0 = w.k0 + j * TK;
      __syncthreads();
      // keys past the length are zero (what their slots hold is never read)
      const size_t row = ((size_t)w.b * p.n_kv + w.kvh) * p.capacity + k0;
      for (int i = threadIdx.x; i < TK * DP; i += kThreads) {
        const int r = i / DP, c = i - r * DP;
        const bool in = k0 + r < w.kv && c < d;
        Ks[r * LD + c] = in ? ck[(row + r) * d + c] : 0.f;
        Vs[r * LD + c] = in ? cv[(row + r) * d + c] : 0.f;
      }
      __syncthreads();
      float s[4][4] = {};
#pragma unroll 4
      for (int c = 0; c < DP; c += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = *reinterpret_cast<const float4*>(Qs + (ty * 4 + i) * LD + c);
          b[i] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * i) * LD + c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            s[i][k] += a[i].x * b[k].x + a[i].y * b[k].y + a[i].z * b[k].z + a[i].w * b[k].w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = m[i];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = k0 + tx + 16 * k;
          const bool sees = key <= pos[i] && (p.window <= 0 || pos[i] - key < p.window);
          s[i][k] = sees ? s[i][k] * p.scaling : -INFINITY;
          mx = fmaxf(mx, s[i][k]);
        }
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
          Ps[(ty * 4 + i) * LP + tx + 16 * k] = e;
        }
#pragma unroll
        for (int e = 0; e < DP / 16; ++e) o[i][e] *= alpha;
      }
      __syncwarp();  // a warp holds whole rows of P: rows 8 w .. 8 w + 7
      // A key that a row does not see has weight 0, and its value must not enter even as
      // 0 * NaN: where the tile is cut by the mask, zero weights are skipped.
      const int first = w.kv - w.n + (int)(r0 / p.G);
      const int last = w.kv - w.n + (int)((r0 + rows - 1) / p.G);
      const bool open = k0 + TK - 1 <= first && (p.window <= 0 || last - k0 < p.window);
#pragma unroll 2
      for (int k = 0; k < TK; ++k) {
        float pv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pv[i] = Ps[(ty * 4 + i) * LP + k];
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(Vs + k * LD + tx * 4 + 64 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (!open && pv[i] == 0.f) continue;
            o[i][4 * c + 0] += pv[i] * v.x;
            o[i][4 * c + 1] += pv[i] * v.y;
            o[i][4 * c + 2] += pv[i] * v.z;
            o[i][4 * c + 3] += pv[i] * v.w;
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float sum = l[i];
#pragma unroll
      for (int of = 8; of > 0; of >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, of);
      const int r = ty * 4 + i;
      if (r >= rows) continue;
      const size_t at = (size_t)(2 * blockIdx.x + (w.slot > 0)) * RI + r;
      if (w.slot < 0) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int token = (int)((r0 + r) / p.G), g = (int)(r0 + r - (long long)token * p.G);
        float* dst = (float*)p.out + ((size_t)(w.row0 + token) * p.n_h + w.kvh * p.G + g) * d;
#pragma unroll
        for (int e = 0; e < DP / 16; ++e) {
          const int c = tx * 4 + 64 * (e >> 2) + (e & 3);
          if (c < d) dst[c] = o[i][e] * inv;
        }
      } else {
#pragma unroll
        for (int e = 0; e < DP / 16; ++e) {
          const int c = tx * 4 + 64 * (e >> 2) + (e & 3);
          if (c < d) p.part[at * d + c] = o[i][e];
        }
        if (tx == 0) p.part_ml[at] = make_float2(m[i], sum);
      }
    }
  }
  if (threadIdx.x == 0) p.merge[blockIdx.x] = walk.merge;
}

template <int DP>
cudaError_t launch(const ChunkAttnParams& p, cudaStream_t s) {
  const int tiles = (int)sizeof(float) * ((RI + 2 * TK) * (DP + 4) + RI * (TK + 4));
  const int scratch = (int)(chunk::kLocateBytes * p.batch);
  const int smem = tiles > scratch ? tiles : scratch;
  const int most = (int)(chunk::kLocateBytes * kChunkMaxBatch);
  static SmemLimit limit;
  cudaError_t e = limit.raise(chunk_attn_simt_kernel<DP>, tiles > most ? tiles : most);
  if (e != cudaSuccess) return e;
  LaunchScope ls_(DFLASH_KERNEL_CHUNK_ATTN, s);
  chunk_attn_simt_kernel<DP><<<sm_count(), kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t chunk_attn_simt(const ChunkAttnParams& p, cudaStream_t s) {
  if (p.d_h <= 64) return launch<64>(p, s);
  if (p.d_h <= 128) return launch<128>(p, s);
  return launch<256>(p, s);
}

}  // namespace dflash
