// Causal chunk attention: workspace, choice of kernel, and the merge of cut items.
#include "chunk.cuh"

namespace dflash {
namespace {

// Stacked query rows of an item, at most.
int item_rows(int dtype, int d_h) { return dtype == DFLASH_F32 ? chunk_attn_simt_item_rows(d_h) : 256; }
int attn_ctas(int dtype, int d_h) { return dtype == DFLASH_F32 ? chunk_attn_simt_ctas(d_h) : chunk_sms(); }

// CTA c of the first grid axis merges the item that was cut at the end of attention CTA c's
// share, if one was. Piece 0 is CTA c's partial 1, piece i > 0 is partial 0 of CTA c + i.
// out = sum_i w_i o_i / sum_i w_i l_i, w_i = exp(max_i - max). (f32 keeps its maxima in the
// natural domain, bf16 in log2 units.) A row that sees keys, all of them at a score of minus
// infinity, has l_i = 0 and the lowest finite maximum: its sum is 0 like that of a row that sees
// no key, but the result is NaN. Bound by L2: a partial of 256 rows is 128 KB.
__device__ __forceinline__ float piece_weight(float mx, float M, bool natural) {
  return mx == -INFINITY ? 0.f : natural ? expf(mx - M) : exp2f(mx - M);
}

// f32: a warp per query row; partials row by row.
__global__ void __launch_bounds__(256) chunk_merge_f32_kernel(const ChunkAttnParams p, int rows_max) {
  grid_wait();  // the attention kernel's partials
  grid_trigger();
  const int4 m = p.merge[blockIdx.x];
  if (m.w == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int row0 = p.cu_rows[m.x], n = p.cu_rows[m.x + 1] - row0;
  const int r0 = m.z * rows_max, rows = min(rows_max, n * p.G - r0);
  const int d2 = p.d_h >> 1;
  for (int r = (int)blockIdx.y * nw + warp; r < rows; r += (int)gridDim.y * nw) {
    auto at = [&](int i) -> size_t {
      return (size_t)(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * rows_max + r;
    };
    float M = -INFINITY;
    for (int i = lane; i < m.w; i += 32) M = fmaxf(M, p.part_ml[at(i)].x);
    M = warp_max(M);
    float L = 0.f;
    for (int i = lane; i < m.w; i += 32) {
      const float2 ml = p.part_ml[at(i)];
      L += ml.y == 0.f ? 0.f : piece_weight(ml.x, M, true) * ml.y;
    }
    L = warp_sum(L);
    float2 acc[4] = {};
#pragma unroll 4
    for (int i = 0; i < m.w; ++i) {
      const size_t a = at(i);
      const float w = piece_weight(p.part_ml[a].x, M, true);
      if (w == 0.f) continue;  // a piece whose keys the row does not see
      const float2* o = reinterpret_cast<const float2*>(p.part + a * p.d_h);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = lane + 32 * k;
        if (e < d2) {
          const float2 v = o[e];
          acc[k].x += w * v.x;
          acc[k].y += w * v.y;
        }
      }
    }
    const float inv = L == 0.f ? (M == -INFINITY ? 0.f : NAN) : 1.f / L;
    const int token = (r0 + r) / p.G, g = r0 + r - token * p.G;
    float* dst = (float*)p.out + ((size_t)(row0 + token) * p.n_h + m.y * p.G + g) * p.d_h;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = lane + 32 * k;
      if (e < d2) *reinterpret_cast<float2*>(dst + 2 * e) = make_float2(acc[k].x * inv, acc[k].y * inv);
    }
  }
}

// bf16, d_h = 128: partials are [column / 8][row][8]. A warp takes 8 rows x 32 columns: lane
// = (row, group of 8 columns); eight lanes of a column group read 256 bytes in a row.
__global__ void __launch_bounds__(256) chunk_merge_bf16_kernel(const ChunkAttnParams p, int rows_max) {
  grid_wait();  // the attention kernel's partials
  grid_trigger();
  const int4 m = p.merge[blockIdx.x];
  if (m.w == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = p.cu_rows[m.x], n = p.cu_rows[m.x + 1] - row0;
  const int r0 = m.z * rows_max, rows = min(rows_max, n * p.G - r0);
  // warps 0-3: the four 32-column quarters of 8 rows, warps 4-7: of the next 8
  const int c8 = (warp & 3) * 4 + (lane >> 3);
  for (int base = ((int)blockIdx.y * 2 + (warp >> 2)) * 8; base < rows; base += (int)gridDim.y * 16) {
    const int r = base + (lane & 7);
    if (r >= rows) continue;
    auto slot = [&](int i) -> size_t {
      return (size_t)(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * rows_max;
    };
    float M = -INFINITY, L = 0.f;
    float acc[8] = {};
    // running reference: pieces in order, a few requested ahead
#pragma unroll 4
    for (int i = 0; i < m.w; ++i) {
      const size_t at = slot(i);
      const float2 ml = p.part_ml[at + r];
      const float4* o = reinterpret_cast<const float4*>(p.part + at * 128 + ((size_t)c8 * rows_max + r) * 8);
      const float4 a = __ldcs(o), b = __ldcs(o + 1);
      const float M1 = fmaxf(M, ml.x);
      const float keep = piece_weight(M, M1, false), w = piece_weight(ml.x, M1, false);
      M = M1;
      L = L * keep + (ml.y == 0.f ? 0.f : w * ml.y);
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = acc[e] * keep + (w == 0.f ? 0.f : w * v[e]);  // (0: keys unseen)
    }
    const float inv = L == 0.f ? (M == -INFINITY ? 0.f : NAN) : 1.f / L;
    const int token = (r0 + r) / p.G, g = r0 + r - token * p.G;
    bf16* dst = (bf16*)p.out + ((size_t)(row0 + token) * p.n_h + m.y * p.G + g) * 128 + c8 * 8;
    uint4 w;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    *reinterpret_cast<uint4*>(dst) = w;
  }
}

bool carve(int dtype, int d_h, ChunkAttnParams* p, Carver& cv) {
  const int ctas = attn_ctas(dtype, d_h);
  const size_t slots = 2 * (size_t)ctas * item_rows(dtype, d_h);
  float* part = cv.take<float>(slots * d_h);
  float2* ml = cv.take<float2>(slots);
  int4* merge = cv.take<int4>((size_t)ctas);
  if (p) {
    p->part = part;
    p->part_ml = ml;
    p->merge = merge;
  }
  return cv.ok;
}

}  // namespace

int chunk_sms() {
  static int count[128] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 148;
  int n = __atomic_load_n(&count[dev], __ATOMIC_RELAXED);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  __atomic_store_n(&count[dev], n, __ATOMIC_RELAXED);
  return n;
}

size_t chunk_attn_workspace(int dtype, int d_h) {
  Carver cv(nullptr, ~size_t(0));
  carve(dtype, d_h, nullptr, cv);
  return cv.off;
}

bool chunk_attn_carve(int dtype, int d_h, ChunkAttnParams& p, void* workspace, size_t bytes) {
  Carver cv(workspace, bytes);
  return carve(dtype, d_h, &p, cv);
}

cudaError_t chunk_attn(int dtype, const ChunkAttnParams& p, cudaStream_t s) {
  const bool f32 = dtype == DFLASH_F32;
  cudaError_t e = p.tree.nodes ? (f32 ? tree_attn_simt(p, s) : tree_attn_tc(p, s))
                               : (f32 ? chunk_attn_simt(p, s) : chunk_attn_tc(p, s));
  if (e != cudaSuccess) return e;
  LaunchScope ls_(DFLASH_KERNEL_CHUNK_MERGE, s);
  const dim3 grid(attn_ctas(dtype, p.d_h), 16);  // every row at once
  return f32 ? launch_overlapped(chunk_merge_f32_kernel, grid, 256, 0, s, p, chunk_attn_simt_item_rows(p.d_h))
             : launch_overlapped(chunk_merge_bf16_kernel, grid, 256, 0, s, p, chunk_attn_tc_item_rows(p.G));
}

}  // namespace dflash
