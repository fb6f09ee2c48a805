// A chunk step's rows into the cache: per-head RMSNorm of Q and K, RoPE at each row's
// position, K and V stored at each row's slot (DFlash KV Injection Walkthrough, Steps 4.1-4.3:
// QNorm / KNorm per head, V not normalised, rotation of the pairs (i, i + d_h / 2) at the
// absolute position).
//
//   x' = x rsqrt(mean(x^2) + eps) gamma;  y_i = x'_i cos - x'_{i+h} sin,
//   y_{i+h} = x'_{i+h} cos + x'_i sin,  h = d_h / 2
//
// Every value is read once and written once, in between 7 operations: bound by HBM (and by
// the launch for a few rows). Sums and rotations in fp32, one rounding at the store.
#include "chunk.cuh"

namespace dflash {
namespace {

// Base of the d_h elements of (slot, KV head) in units of [n_kv][unit_rows][d_h].
__device__ __forceinline__ size_t slot_elem(const ChunkAppendParams& p, int slot, int kvh) {
  const int unit = slot / p.unit_rows, r = slot - unit * p.unit_rows;
  return (((size_t)unit * p.n_kv + kvh) * p.unit_rows + r) * p.d_h;
}

// Whether row r is stored; flags what is out of range.
__device__ __forceinline__ bool row_live(const ChunkAppendParams& p, int r, int* slot, int* pos) {
  *slot = p.slots[r];
  *pos = p.positions[r];
  if (*slot == -1) return false;
  if (*slot < 0 || *slot >= p.n_slots) {
    atomicOr(p.status, DFLASH_DEV_PAGE);
    return false;
  }
  if (p.rope && (*pos < 0 || *pos >= p.table_len)) {
    atomicOr(p.status, DFLASH_DEV_ROPE);
    return false;
  }
  return true;
}

// The lengths after the step (nothing in this kernel reads them).
__device__ __forceinline__ void publish_lens(const ChunkAppendParams& p) {
  if (blockIdx.x != 0) return;
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x) {
    const int kv = p.kv_lens[b];
    if (kv > 0 && kv <= p.capacity && (!p.rope || kv <= p.table_len)) p.lens[b] = kv;
  }
}

// ---------------------------------------------------------------------------
// bf16, d_h = 128: half a warp per head, 16 bytes per lane, kUnroll heads in flight. Lane l
// holds elements 8l .. 8l + 7 of a head, its rotation partner is lane l ^ 8.
// ---------------------------------------------------------------------------
constexpr int kUnroll = 4;
constexpr int kHeadsPerUnit = 2 * kUnroll;  // heads of one row that a warp takes

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(h[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint4 w;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
  return w;
}

// A unit is `span` groups of 8 heads of one row: the slot, the position and the (cos, sin) pairs
// are fetched once per unit, and the next group's rows are in flight while one is worked on.
__global__ void __launch_bounds__(256) chunk_append_bf16_kernel(const ChunkAppendParams p, int span) {
  publish_lens(p);
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const int n_q = p.q ? p.n_h : 0, heads = n_q + 2 * p.n_kv;
  const int groups = (heads + kHeadsPerUnit - 1) / kHeadsPerUnit, units = (groups + span - 1) / span;
  const long long unit = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int r = (int)(unit / units);
  if (r >= p.rows) return;
  const int g0 = (int)(unit - (long long)r * units) * span, g1 = min(g0 + span, groups);
  auto fetch = [&](int g, uint4 (&w)[kUnroll]) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = g * kHeadsPerUnit + half + 2 * i;
      if (g >= g1 || h >= heads) continue;
      const bf16* src = h < n_q ? (const bf16*)p.q + (size_t)r * p.ld_q + h * 128
                      : h < n_q + p.n_kv ? (const bf16*)p.k + (size_t)r * p.ld_k + (h - n_q) * 128
                                         : (const bf16*)p.v + (size_t)r * p.ld_v + (h - n_q - p.n_kv) * 128;
      w[i] = __ldcs(reinterpret_cast<const uint4*>(src) + l);
    }
  };
  uint4 next[kUnroll];
  fetch(g0, next);  // before the slot is known: a skipped row is read in vain
  int slot, pos;
  if (!row_live(p, r, &slot, &pos)) return;
  // (cos, sin) of this lane's 8 pairs; the upper half-head adds where the lower subtracts
  float c[8], s[8];
  if (p.rope) {
    const float4* t = reinterpret_cast<const float4*>(p.rope + (size_t)pos * 64 + (l & 7) * 8);
    const float sign = l < 8 ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = __ldg(t + i);
      c[2 * i] = f.x;
      s[2 * i] = sign * f.y;
      c[2 * i + 1] = f.z;
      s[2 * i + 1] = sign * f.w;
    }
  }
  const int u = slot / p.unit_rows;
  const size_t cache0 = (size_t)u * p.n_kv * p.unit_rows + (slot - u * p.unit_rows);  // head 0's row
#pragma unroll 1
  for (int g = g0; g < g1; ++g) {
    uint4 w[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) w[i] = next[i];
    fetch(g + 1, next);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = g * kHeadsPerUnit + half + 2 * i;
      const bool is_q = h < n_q, is_v = h >= n_q + p.n_kv;
      if (h >= heads) continue;
      float x[8];
      unpack8(w[i], x);
      const void* gamma = is_q ? p.gamma_q : p.gamma_k;
      if (!is_v && gamma) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffu << (half * 16), ss, o);
        const float inv = rsqrtf(ss * (1.f / 128.f) + p.eps);
        float gm[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(gamma) + l), gm);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * gm[e];
      }
      if (!is_v && p.rope) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = __shfl_xor_sync(0xffffu << (half * 16), x[e], 8);
          x[e] = x[e] * c[e] + y * s[e];
        }
      }
      if (is_q) {
        reinterpret_cast<uint4*>((bf16*)p.q_out + (size_t)r * p.n_h * 128 + h * 128)[l] = pack8(x);
      } else {
        const size_t at = (cache0 + (size_t)(is_v ? h - n_q - p.n_kv : h - n_q) * p.unit_rows) * 128 + 8 * l;
        void* cache = is_v ? p.cache_v : p.cache_k;
        if (p.fp8) {
          const float inv = is_v ? p.v_inv : p.k_inv;
          uint2 code;
          code.x = e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
          code.y = e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
          *reinterpret_cast<uint2*>((uint8_t*)cache + at) = code;
        } else {
          *reinterpret_cast<uint4*>((bf16*)cache + at) = pack8(x);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// f32, any even d_h up to 256: a warp per (row, head), lane k of it the pairs k, k + 32, ..
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) chunk_append_f32_kernel(const ChunkAppendParams p) {
  publish_lens(p);
  const int lane = threadIdx.x & 31;
  const int n_q = p.q ? p.n_h : 0, heads = n_q + 2 * p.n_kv, hd = p.d_h >> 1;
  const long long unit = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int r = (int)(unit / heads), h = (int)(unit - (long long)r * heads);
  if (r >= p.rows) return;
  int slot, pos;
  if (!row_live(p, r, &slot, &pos)) return;
  const bool is_q = h < n_q, is_v = h >= n_q + p.n_kv;
  const float* src = is_q ? (const float*)p.q + (size_t)r * p.ld_q + (size_t)h * p.d_h
                   : is_v ? (const float*)p.v + (size_t)r * p.ld_v + (size_t)(h - n_q - p.n_kv) * p.d_h
                          : (const float*)p.k + (size_t)r * p.ld_k + (size_t)(h - n_q) * p.d_h;
  float a[4], b[4], ss = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = lane + 32 * k;
    a[k] = i < hd ? src[i] : 0.f;
    b[k] = i < hd ? src[i + hd] : 0.f;
    ss += a[k] * a[k] + b[k] * b[k];
  }
  const float* gamma = (const float*)(is_q ? p.gamma_q : p.gamma_k);
  if (!is_v && gamma) {
    const float inv = 1.f / sqrtf(warp_sum(ss) / (float)p.d_h + p.eps);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = lane + 32 * k;
      if (i < hd) {
        a[k] *= inv * gamma[i];
        b[k] *= inv * gamma[i + hd];
      }
    }
  }
  float* dst = is_q ? (float*)p.q_out + ((size_t)r * p.n_h + h) * p.d_h
                    : (float*)(is_v ? p.cache_v : p.cache_k) +
                          slot_elem(p, slot, is_v ? h - n_q - p.n_kv : h - n_q);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = lane + 32 * k;
    if (i >= hd) continue;
    float x = a[k], y = b[k];
    if (!is_v && p.rope) {
      const float2 t = __ldg(p.rope + (size_t)pos * hd + i);
      x = a[k] * t.x - b[k] * t.y;
      y = b[k] * t.x + a[k] * t.y;
    }
    dst[i] = x;
    dst[i + hd] = y;
  }
}

}  // namespace

cudaError_t chunk_append(int dtype, const ChunkAppendParams& p, cudaStream_t s) {
  const int heads = (p.q ? p.n_h : 0) + 2 * p.n_kv;
  // bf16: a warp per 8 heads while the rows alone do not fill the GPU, else up to 24 heads
  const int groups = (heads + kHeadsPerUnit - 1) / kHeadsPerUnit;
  const int span = (long long)p.rows * groups > 96ll * sm_count() ? 3 : 1;
  const int units = dtype == DFLASH_F32 ? heads : (groups + span - 1) / span;
  const long long grid = ((long long)p.rows * units + 7) / 8;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  LaunchScope ls_(DFLASH_KERNEL_CHUNK_APPEND, s);
  if (dtype == DFLASH_F32)
    chunk_append_f32_kernel<<<(unsigned)grid, 256, 0, s>>>(p);
  else
    chunk_append_bf16_kernel<<<(unsigned)grid, 256, 0, s>>>(p, span);
  return cudaGetLastError();
}

}  // namespace dflash
