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
// bf16, d_h = 128: half a warp per head; lane l holds elements 4l .. 4l + 3 of both halves, so
// that a rotation stays in its lane. Norm weight and rotation are one set of coefficients per
// row, y_lo = inv (a A - b B), y_hi = inv (b C + a D) with A = g_lo cos, B = g_hi sin,
// C = g_hi cos, D = g_lo sin; per head that leaves the sum of squares (4 shuffles) and 12
// packed multiply-adds. (One 16-byte load per lane and the partner's elements by 8 shuffles:
// 57 us for 9911 rows of 32 + 8 + 8 heads, bound by issue slots.)
// ---------------------------------------------------------------------------
constexpr int kWarps = 4;                     // per CTA

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 neg2(float2 v) { return make_float2(-v.x, -v.y); }

// A unit is `span` heads of one row, two at a time: the slot, the position and the coefficients
// are made once per unit (and kind of head), and the next 2 U heads are in flight while as many are
// worked on. Addresses advance by a step and are looked up again where a tensor ends; Q, K and V
// take the same way (V's products are not used), so the halves of a warp stay together.
// 9911 rows of 32 + 8 + 8 heads 46 us (5.3 TB/s; with addresses and branches per head 49.9), 512
// rows 4.2 us, five prompts on E4M3 20.7 us. No unit is at its limit (issue slots 53 %, E4M3 57 %, DRAM
// 53 and 32 %): an issued instruction waits 1.8 cycles on a load, on E4M3 3.4, where a lane's 8 bytes
// loaded and 4 stored make as many instructions of half the bytes. More warps instead of long
// units, and fewer registers with more CTAs, were slower (56 to 79 us).
// ROPE false: the pairs are not mixed at all (an infinity times a sine of 0 would be a NaN).
template <bool FP8, int U, bool ROPE>
__global__ void __launch_bounds__(32 * kWarps, U == 2 ? 7 : 5) chunk_append_bf16_kernel(const ChunkAppendParams p, int span) {
  publish_lens(p);
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const int n_q = p.q ? p.n_h : 0, n_k = n_q + p.n_kv, heads = n_k + p.n_kv;
  const int units = (heads + span - 1) / span;
  const unsigned unit = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int r = (int)(unit / (unsigned)units);
  if (r >= p.rows) return;
  const int h0 = (int)(unit - (unsigned)r * units) * span, h1 = min(h0 + span, heads);
  // Where this half warp reads: head lh, up to the end of its tensor.
  int lh = h0 + half, lend = 0;
  const uint2* src = nullptr;
  auto seek = [&]() {
    const bf16* t = lh < n_q ? (const bf16*)p.q + (size_t)r * p.ld_q + lh * 128
                  : lh < n_k ? (const bf16*)p.k + (size_t)r * p.ld_k + (lh - n_q) * 128
                             : (const bf16*)p.v + (size_t)r * p.ld_v + (lh - n_k) * 128;
    src = reinterpret_cast<const uint2*>(t) + l;
    lend = min(h1, lh < n_q ? n_q : lh < n_k ? n_k : heads);
  };
  // elements 4l .. and 64 + 4l .. of the next heads
  auto fetch = [&](uint2 (&w)[U][2]) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (lh >= lend && lh < h1) seek();
      if (lh < h1) {
        w[i][0] = __ldcs(src);
        w[i][1] = __ldcs(src + 16);
      }
      src += 64;
      lh += 2;
    }
  };
  uint2 next[U][2] = {};
  fetch(next);  // before the slot is known: a skipped row is read in vain
  int slot, pos;
  if (!row_live(p, r, &slot, &pos)) return;
  // (cos, sin) of this lane's four pairs
  float2 cs[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, sn[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  if (ROPE) {
    const float4* t = reinterpret_cast<const float4*>(p.rope + (size_t)pos * 64 + l * 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 f = __ldg(t + i);
      cs[i] = make_float2(f.x, f.z);
      sn[i] = make_float2(f.y, f.w);
    }
  }
  const int u = slot / p.unit_rows;
  const size_t cache0 = (size_t)u * p.n_kv * p.unit_rows + (slot - u * p.unit_rows);  // head 0's row
  // Where it writes: head h of kind 0 Q, 1 K, 2 V, the coefficients of that kind.
  int h = h0 + half, hend = h, kind = 0;
  char* dst = nullptr;
  long long step = 0;
  bool norm = false;
  float2 A[2], B[2], C[2], D[2];
  auto turn = [&]() {
    kind = h < n_q ? 0 : h < n_k ? 1 : 2;
    hend = min(h1, kind == 0 ? n_q : kind == 1 ? n_k : heads);
    const int kh = h - (kind == 0 ? 0 : kind == 1 ? n_q : n_k);
    const int bytes = FP8 && kind > 0 ? 128 : 256;
    const size_t row = kind == 0 ? (size_t)r * p.n_h + kh : cache0 + (size_t)kh * p.unit_rows;
    dst = (char*)(kind == 0 ? p.q_out : kind == 1 ? p.cache_k : p.cache_v) + row * bytes + l * (bytes >> 5);
    step = 2ll * bytes * (kind == 0 ? 1 : p.unit_rows);
    const bf16* gamma = (const bf16*)(kind == 0 ? p.gamma_q : p.gamma_k);
    norm = gamma != nullptr;
    uint2 lo = make_uint2(0x3F803F80u, 0x3F803F80u), hi = lo;  // 1
    if (norm) {
      lo = __ldg(reinterpret_cast<const uint2*>(gamma) + l);
      hi = __ldg(reinterpret_cast<const uint2*>(gamma) + 16 + l);
    }
    const float2 gl[2] = {bf2(lo.x), bf2(lo.y)}, gh[2] = {bf2(hi.x), bf2(hi.y)};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      A[e] = __fmul2_rn(gl[e], cs[e]);
      B[e] = neg2(__fmul2_rn(gh[e], sn[e]));
      C[e] = __fmul2_rn(gh[e], cs[e]);
      D[e] = __fmul2_rn(gl[e], sn[e]);
    }
  };
  const int pairs = (h1 - h0 + 1) >> 1;
#pragma unroll 1
  for (int s = 0; s < pairs; s += U) {
    uint2 w[U][2];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      w[i][0] = next[i][0];
      w[i][1] = next[i][1];
    }
    fetch(next);
#pragma unroll
    for (int i = 0; i < U; ++i) {  // (both halves of the warp stay together)
      if (h >= hend && h < h1) turn();
      const float2 a[2] = {bf2(w[i][0].x), bf2(w[i][0].y)}, b[2] = {bf2(w[i][1].x), bf2(w[i][1].y)};
      float2 q = __fmul2_rn(a[0], a[0]);
      q = __ffma2_rn(a[1], a[1], q);
      q = __ffma2_rn(b[0], b[0], q);
      q = __ffma2_rn(b[1], b[1], q);
      float ss = q.x + q.y;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = norm ? rsqrtf(ss * (1.f / 128.f) + p.eps) : 1.f;
      const float2 n2 = make_float2(inv, inv);
      float2 y[2], z[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        y[e] = __fmul2_rn(ROPE ? __ffma2_rn(a[e], A[e], __fmul2_rn(b[e], B[e])) : __fmul2_rn(a[e], A[e]), n2);
        z[e] = __fmul2_rn(ROPE ? __ffma2_rn(b[e], C[e], __fmul2_rn(a[e], D[e])) : __fmul2_rn(b[e], C[e]), n2);
      }
      if (h < h1) {
        if (FP8 && kind > 0) {
          const float f = kind == 1 ? p.k_inv : p.v_inv;
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // V is stored as it is
            y[e] = kind == 1 ? y[e] : a[e];
            z[e] = kind == 1 ? z[e] : b[e];
          }
          *reinterpret_cast<uint32_t*>(dst) = e4m3x4(y[0].x * f, y[0].y * f, y[1].x * f, y[1].y * f);
          *reinterpret_cast<uint32_t*>(dst + 64) = e4m3x4(z[0].x * f, z[0].y * f, z[1].x * f, z[1].y * f);
        } else {
          if (kind < 2) {
            w[i][0] = make_uint2(pack2(y[0]), pack2(y[1]));
            w[i][1] = make_uint2(pack2(z[0]), pack2(z[1]));
          }
          *reinterpret_cast<uint2*>(dst) = w[i][0];
          *reinterpret_cast<uint2*>(dst + 128) = w[i][1];
        }
      }
      dst += step;
      h += 2;
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

template <bool ROPE>
void launch_bf16(const ChunkAppendParams& p, unsigned grid, int span, bool four, cudaStream_t s) {
  constexpr int threads = 32 * kWarps;
  if (p.fp8)
    chunk_append_bf16_kernel<true, 2, ROPE><<<grid, threads, 0, s>>>(p, span);
  else if (four)
    chunk_append_bf16_kernel<false, 4, ROPE><<<grid, threads, 0, s>>>(p, span);
  else
    chunk_append_bf16_kernel<false, 2, ROPE><<<grid, threads, 0, s>>>(p, span);
}

}  // namespace

cudaError_t chunk_append(int dtype, const ChunkAppendParams& p, cudaStream_t s) {
  const int heads = (p.q ? p.n_h : 0) + 2 * p.n_kv;
  // bf16: a warp per 8 heads while the step is small. Once units of 48 heads keep 16 warps of an SM
  // busy (of the 20 that fit), a row is cut into as few units of at most 48 as it takes, even in
  // number of heads and alike in size. us with 8 heads and with long units, by heads of a row:
  //   rows x heads     48 (one unit)   72 (two of 36)   80 (two of 40)   130 (three of 44)
  //   25 000           4.5    8.4      4.5    7.4       4.5    7.7       4.5    7.8
  //   60 000           8.4    9.6      8.7    8.7       8.4    8.8       8.3    9.1
  //   120 000         17.0   14.0     17.3   17.6      17.3   13.8      16.8   13.9
  //   500 000         60.5   47.2     60.9   47.5      60.3   47.6      61.1   46.6
  // Units of 48 and a short rest instead of equal ones: 72 heads 48.5, 80 heads 48.9 us.
  // Long units have four heads of each half warp in flight instead of two (500 000: 24 heads 50.2
  // and 51.7 us, 48 heads 47.2 and 52.1), short ones do not gain by it (18 heads 60.3 and 58.0, 7
  // heads 97 and 78). Next to E4M3 rows two stay in flight (four: 31 us instead of 20.8).
  const bool many = (long long)p.rows * heads > 16ll * 48 * chunk_sms();
  const int per_row = (heads + 47) / 48;
  const int span = many ? ((heads + per_row - 1) / per_row + 1) & ~1 : 8;
  const bool four = span >= 24;
  const int units = dtype == DFLASH_F32 ? heads : (heads + span - 1) / span;
  const int warps = dtype == DFLASH_F32 ? 8 : kWarps;
  const long long grid = ((long long)p.rows * units + warps - 1) / warps;
  if (grid > 0x0fffffffll) return cudaErrorInvalidValue;
  LaunchScope ls_(DFLASH_KERNEL_CHUNK_APPEND, s);
  if (dtype == DFLASH_F32)
    chunk_append_f32_kernel<<<(unsigned)grid, 256, 0, s>>>(p);
  else if (p.rope)
    launch_bf16<true>(p, (unsigned)grid, span, four, s);
  else
    launch_bf16<false>(p, (unsigned)grid, span, four, s);
  return cudaGetLastError();
}

}  // namespace dflash
