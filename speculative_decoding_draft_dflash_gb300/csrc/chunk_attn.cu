// Causal chunk attention: workspace, choice of kernel, and the merge of cut items.
#include "chunk.cuh"

namespace dflash {
namespace {

constexpr int kSimtRows = 64;   // stacked query rows of an item (chunk_attn_simt.cu)
constexpr int kTcRows = 256;    // at most (chunk_attn_tc.cu)

int item_rows(int dtype) { return dtype == DFLASH_F32 ? kSimtRows : kTcRows; }

template <typename T> __device__ __forceinline__ void store2(T* p, float a, float b);
template <> __device__ __forceinline__ void store2(float* p, float a, float b) {
  *reinterpret_cast<float2*>(p) = make_float2(a, b);
}
template <> __device__ __forceinline__ void store2(bf16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}

// CTA c of the first grid axis merges the item that was cut at the end of attention CTA c's
// share, if one was; a warp per query row. Piece 0 is CTA c's partial 1, piece i > 0 is
// partial 0 of CTA c + i. out = sum_i w_i o_i / sum_i w_i l_i, w_i = exp(max_i - max).
// (f32 keeps its maxima in the natural domain, bf16 in log2 units.)
template <typename T>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkAttnParams p, int rows_max) {
  constexpr bool kNatural = sizeof(T) == 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the attention kernel's partials
  const int4 m = p.merge[blockIdx.x];
  if (m.w == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int row0 = p.cu_rows[m.x], n = p.cu_rows[m.x + 1] - row0;
  const long long r0 = (long long)m.z * rows_max;
  const int rows = (int)min((long long)rows_max, (long long)n * p.G - r0);
  const int d2 = p.d_h >> 1;
  for (int r = (int)blockIdx.y * nw + warp; r < rows; r += (int)gridDim.y * nw) {
    auto at = [&](int i) -> size_t {
      return (size_t)(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * rows_max + r;
    };
    float M = -INFINITY;
    for (int i = lane; i < m.w; i += 32) M = fmaxf(M, p.part_ml[at(i)].x);
    M = warp_max(M);
    auto weight = [&](float mx) -> float {
      if (mx == -INFINITY) return 0.f;
      return kNatural ? expf(mx - M) : exp2f(mx - M);
    };
    float L = 0.f;
    for (int i = lane; i < m.w; i += 32) {
      const float2 ml = p.part_ml[at(i)];
      L += ml.y == 0.f ? 0.f : weight(ml.x) * ml.y;
    }
    L = warp_sum(L);
    float2 acc[4] = {};
#pragma unroll 4
    for (int i = 0; i < m.w; ++i) {
      const size_t a = at(i);
      const float w = weight(p.part_ml[a].x);
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
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const long long q = r0 + r;
    const int token = (int)(q / p.G), g = (int)(q - (long long)token * p.G);
    T* dst = (T*)p.out + ((size_t)(row0 + token) * p.n_h + m.y * p.G + g) * p.d_h;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = lane + 32 * k;
      if (e < d2) store2(dst + 2 * e, acc[k].x * inv, acc[k].y * inv);
    }
  }
}

bool carve(int dtype, int d_h, ChunkAttnParams* p, Carver& cv) {
  const size_t slots = 2 * (size_t)sm_count() * item_rows(dtype);
  float* part = cv.take<float>(slots * d_h);
  float2* ml = cv.take<float2>(slots);
  int4* merge = cv.take<int4>((size_t)sm_count());
  if (p) {
    p->part = part;
    p->part_ml = ml;
    p->merge = merge;
  }
  return cv.ok;
}

}  // namespace

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
  cudaError_t e = dtype == DFLASH_F32 ? chunk_attn_simt(p, s) : chunk_attn_tc(p, s);
  if (e != cudaSuccess) return e;
  LaunchScope ls_(DFLASH_KERNEL_CHUNK_MERGE, s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sm_count(), dtype == DFLASH_F32 ? 8 : 16);  // one or two rows per warp
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // scheduled as SMs fall free
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return dtype == DFLASH_F32
             ? cudaLaunchKernelEx(&cfg, chunk_merge_kernel<float>, p, kSimtRows)
             : cudaLaunchKernelEx(&cfg, chunk_merge_kernel<bf16>, p, chunk_attn_tc_item_rows(p.G));
}

}  // namespace dflash
