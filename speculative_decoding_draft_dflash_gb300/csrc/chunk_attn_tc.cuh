// (Included by chunk_attn_tc.cu and, with trees in place of the causal mask, by tree_attn_tc.cu.)
//
// Causal chunk attention on tcgen05 tensor cores (bf16; bf16 or E4M3 cache, d_h = 128).
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(s_ij - m_i),  s_ij = q_i k_j scaling log2(e)
// over the keys j that row i sees, in one pass over 128-key tiles with the running reference
// m_i. m_i only moves when a tile's maximum exceeds it by more than 8 (p stays below 2^8), so
// the rescaling of the accumulator in tensor memory is rare.
//
// Query rows: the rows that share a KV head, stacked token by token (row = token * G + head),
// fill M = 128 tiles of TQ = 128 / G whole tokens. An item (chunk.cuh) is two such tiles, A and
// B. With more than one tile of rows each K / V tile serves A and B in turn, and the tensor
// cores work on one while the other's softmax runs. An item of one tile (a decoded token, a
// verified block) takes the keys of even tiles through A and odd ones through B, with the same
// queries, and merges the two halves at the end.
//
// One persistent CTA per SM. Warps: 0-3 softmax of A, 4-7 softmax of B (a thread per row, all
// 128 columns: no exchange between threads), 8 work list and TMA loads, 9 and 10 MMA issue for
// A and B, 11 (bf16) check of the V tiles that the mask cuts, (E4M3) Q to codes and V to f16.
// Tensor memory: S_A, S_B, O_A, O_B of 128 columns each; P (16 bits) overwrites the first half
// of its S and is the A operand of the PV product from there. P is rounded to bf16 next to a
// bf16 V: both operands of an MMA have one type, and f16 does not hold every bf16 value. Relative
// errors, root mean square against 64 bits: 0.0023, of which the output's own rounding to bf16 is
// 0.0017. (A second term of P for the remainder would add half of a tile's MMAs again.) Next to
// E4M3 values P is rounded to f16, which holds them exactly (0.0017 in all). f16 has few
// exponents: weights and sums there carry a factor 2^7 (p stays below 2^15 of f16's 65504), which
// every quotient divides out again. So a weight keeps 11 bits down to 2^-21 of the row's reference,
// and one below 2^-32 is lost from the product (without the factor 2^-14 and 2^-25: 8191 keys of
// weight 2^-25.5 behind one of weight 1 and value 0 lost half of their output).
//
// What bounds it. Many rows: the MMAs (1024 cycles a key tile and row tile with both products)
// and the exponentials (128 x 128 at 16 a cycle and SM: 1024 too), which A and B overlap: 2800
// to 3000 cycles per key tile of two row tiles, of which 2048 are MMAs. 8192 rows of 32 heads
// from position 0: 355 us in a short run, 1.55 PFLOP/s of the 1.91 of a large matrix product, and
// 378 us once calls follow one another for a second (the power limit lowers the clock; the matrix
// product then runs at 1.72). Few rows: HBM, as long as an item is long (294400 keys of 8 heads read
// by single tokens: 187 us, 6.4 of 6.8 TB/s); each further item costs about 3.7 us, in which the
// last tile's chain of S, softmax, PV and epilogue has nothing behind it, as both accumulators end
// together (32 blocks of 16 tokens over 256 to 4096 keys: 67 us, 5.1 TB/s).
// E4M3 with few rows: 1990 cycles a tile on long sequences (294400 keys: 127 us, 4.7 TB/s) where
// HBM would allow 1400, with the tensor pipe busy for 46 %. Not the chain of S, softmax and PV: with
// half the MMAs of S it would be 122 us, with half of PV's 124, with a quarter of V converted
// 120, with all three 116, and a softmax of 32 columns a thread is no faster (below). What fits is
// the loads in flight: of the six stages of 16 KB one K tile is being multiplied and one V tile
// converted, which leaves about 64 KB on their way, where bf16 has about 96 of 160 KB; at 4.7 and
// 6.4 TB/s over 152 SMs both come to 2.1 to 2.3 us a load. Deeper rings have not been tried.
//
// The start: about 4 us from the launch to the first load, of lengths, split and page look-up one after another,
// run by the loading warp alone where there are at most 32 sequences.
//
// Tried and slower. The softmax run once on nothing while the work is looked for, so that its code is in the
// instruction cache (16 rows behind 1023 13.7 -> 14.1 us: it takes the fetches from the loading warp). Tiles fetched into L2 one to ten ahead of their loads, into the next item too (64
// tokens 147 -> 167 us on E4M3; bf16, 32 blocks 69 -> 72 at one ahead, 100 at six): the loads pass the
// same queue twice. P as three E5M2 terms and V as stored, with no conversion (20 MMAs a tile
// for 16, and the terms cost the softmax 420 instructions: 64 tokens 150 -> 200 us). Keys x rows
// for few rows, a key per thread and P through shared memory (64 rows 70 -> 132 us: at 10
// cycles an instruction the four warps wait for tensor memory and for one another). Q repeated
// in its tile so that each 32 lanes take a quarter of the keys (64 tokens 150 -> 167 us).
//
// A masked key has weight exactly 0, and its V row must not enter even as 0 * NaN. In tiles
// that are not visible to every row of the item, the checking warps replace what is not finite
// by 0 and flag the item; the epilogue of a flagged item then adds the replaced values of the
// keys that its row does see.
#pragma once

#include <float.h>
#include <string.h>

#include "chunk.cuh"
#include "sm100_ptx.cuh"

namespace dflash {

// The 2-D maps of the cache (gemm_tc.cu).
bool encode_2d_bf16(CUtensorMap* m, const void* base, long long rows, int cols, int box_rows);
bool encode_2d_u8(CUtensorMap* m, const void* base, long long rows, int box_rows);

namespace {

constexpr int TK = 128;                   // keys of a tile (2^7)
constexpr uint32_t TILE = 128 * 128 * 2;  // a 16-bit tile
constexpr uint32_t HALF = TILE / 2;       // its 64-column box
constexpr int kRing = 4;                  // items in flight between the roles

constexpr float kShiftF16 = 7.f;          // log2 of the factor of weights rounded to f16

constexpr uint32_t TM_S = 0, TM_O = 256;  // tensor-memory columns of S_A; O_A (B: + 128)

// Shared memory: Q_A, Q_B, then 160 KB of K / V. bf16: one ring of five 32 KB stages, filled in
// the order the MMAs take the tiles. E4M3: three 16 KB stages for K (an operand as it is),
// three for V, and two of V converted to f16.
template <bool FP8>
struct Plan {
  static constexpr int THREADS = 384, W_CHECK = 11;
  static constexpr uint32_t LOAD = FP8 ? TK * 128 : TILE;  // a tile as loaded
  static constexpr int STAGES = FP8 ? 3 : 5;
  static constexpr int C_STAGES = 2;
  static constexpr uint32_t OFF_KV = 2 * TILE;
  static constexpr uint32_t OFF_C = OFF_KV + 6 * (TK * 128);  // E4M3: after K and V
  static constexpr uint32_t OFF_END = OFF_KV + 5 * TILE;
  // registers: the softmax warpgroups take what the others give back (setmaxnreg draws on the
  // launch's own: 384 x 168 = 256 x 200 + 128 x 104 = 256 x 208 + 128 x 88)
  static constexpr int REG_SOFT = FP8 ? 200 : 208, REG_REST = FP8 ? 104 : 88;
  // barriers of the stages (Tail::kf, ke): E4M3 V stages follow the K stages
  static constexpr int V_BAR = FP8 ? 3 : 0;
};

template <bool TREE>
struct Params {
  CUtensorMap q, k, v;
  chunk::Split<true, TREE> split;
  const int32_t* table;  // paged: [batch][pps] page ids, or null
  int pps, n_pages;
  int oob_row;           // a row beyond the K / V maps: reads as zeros
  const void* cache_v;   // this layer's V (the rare repair reads it)
  bf16* out;
  float* part;
  float2* part_ml;
  int4* merge;
  unsigned* status;
  int n_h, TQ, RT;       // tokens and rows of a tile
  float sl2, v_scale;    // scaling * log2(e) (fp8: * k_scale); scale of the V codes
  int out32;             // out is 32-byte aligned
  unsigned long long wait_ns;
  TreeRows tree;
};

template <bool TREE>
struct Item {
  chunk::Piece<TREE> w;
  int bad;  // a V tile held something not finite under the mask
};

// What follows the tiles in shared memory (nothing is declared statically, so that the tiles
// start at the 1024-byte boundary their swizzle needs and fill the CTA's 227 KB).
// Barriers of what both MMA warps read (K and V stages, Q_A, oe) count the two.
template <bool TREE>
struct Tail {
  uint64_t qf[2], qe[2];          // Q tile landed / read by its last S
  uint64_t kf[6], ke[6];          // K / V tile landed / stage free again
  uint64_t vc[5];                 // bf16: V tile checked; E4M3: V tile converted
  uint64_t aux[5];                // bf16: a V tile to check is on its way to the stage;
                                  // E4M3: 0-1 converted stage free again, 2-3 Q codes ready
  uint64_t s[2], p[2];            // S complete; P stored
  uint64_t o[2], oe;              // O complete: of one row tile; of both halves of the keys
  uint64_t of;                    // O read by all softmax warps
  uint64_t x[2];                  // (reference, sum) exchanged
  uint64_t turn[2];               // two row tiles: the other MMA warp has issued its block
  uint64_t itf[kRing], ite[kRing], chk[kRing];  // item listed / released / V checks done
  uint64_t fin[2];                // all MMAs of a warp complete
  Item<TREE> ring[kRing];
  chunk::Start<TREE> start;
  uint32_t tmem_slot;
  int abort_flag;
  int rows[4];                    // of the last key tiles (the loading thread's)
  float2 xml[2][128];             // (reference, sum) of the even / odd half
  signed char qexp[2][128];       // E4M3: Q rows are codes of q 2^-qexp
};

__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity, unsigned* status) {
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (ptx::globaltimer() - t0 > ptx::kWaitLimitNs) {
      atomicOr(status, DFLASH_DEV_TIMEOUT);
      return;
    }
  }
}

// Waits of a whole warp on a barrier phase, with the same answer in every lane: false when the
// CTA was told to stop or the limit ran out (which tells it). A phase that is already complete
// costs one test and one vote; a warp that waits longer is suspended by the test (polling warps
// take shared-memory slots from those that work).
__device__ __forceinline__ bool wait_more(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* status,
                                          uint64_t limit_ns) {
  const uint64_t t0 = ptx::globaltimer();
#pragma unroll 1
  while (!__all_sync(0xffffffffu, ptx::mbar_try_wait_sleep(bar, parity, (uint32_t)min((uint64_t)10000, limit_ns)))) {
    const bool late = ptx::globaltimer() - t0 > limit_ns;
    if (late) {
      *abort_flag = 1;
      atomicOr(status, DFLASH_DEV_TIMEOUT);
    }
    if (__any_sync(0xffffffffu, late || *abort_flag)) return false;
  }
  return true;
}
__device__ __noinline__ bool wait_one(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* status,
                                      uint64_t limit_ns) {
  return ptx::mbar_wait_idle(bar, parity, abort_flag, status, limit_ns);
}
__device__ __noinline__ bool wait_more_call(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* status,
                                            uint64_t limit_ns) {
  return wait_more(bar, parity, abort_flag, status, limit_ns);
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));  // a -> low half
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
// kind::f8f6f4, both operands E4M3 in shared memory, K = 32.
__device__ __forceinline__ void mma_f8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A from tensor memory, B from shared memory.
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// kind::f16 with f16 operands, and kind::f8f6f4 with E4M3 ones: type fields 0, f32 accumulator.
constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t idesc_e4m3_f32(int M, int N) { return idesc_f16_f32(M, N); }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(tmap), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// One lane of the (converged) warp, as the compiler can see: code under it keeps descriptors
// and addresses in uniform registers. Under `lane == 0` each MMA cost its thread about 110
// cycles of issue (the tile itself takes 64), and that bound the kernel.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// 32 lanes x 16 columns of tensor memory.
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// 32 bytes to global memory.
__device__ __forceinline__ void st8(void* p, const uint32_t* w) {
  const uint32_t v[8] = {w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]};
  ptx::st_global_v8(p, v);
}

template <int N> __device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Facts of an item that every role derives alike.
template <bool TREE>
struct Geometry {
  int T;          // key tiles of the piece
  int key0;       // first key of its first tile
  int first, last;  // positions of the item's first and last row (TREE: the keys that are theirs,
                    // which their positions do not exceed)
  int closed;       // the first key that not every row sees, but for the window
  bool dual;      // two tiles of query rows (else even / odd key tiles)
  __device__ __forceinline__ Geometry(const Params<TREE>& p, const chunk::Piece<TREE>& w) {
    const int tok0 = w.t * 2 * p.TQ, tok1 = min(tok0 + 2 * p.TQ, w.n);
    T = w.tile1 - w.tile0;
    key0 = w.k0 + w.tile0 * TK;
    first = w.kv - w.n + tok0;
    last = w.kv - w.n + tok1 - 1;
    dual = tok1 - tok0 > p.TQ;
    closed = first + 1;
    if constexpr (TREE) closed = w.ctx;
  }
  // whether some row of the item does not see some key of tile j
  __device__ __forceinline__ bool cut(const Params<TREE>& p, int j) const {
    const int k = key0 + j * TK;
    return k + TK > closed || (p.split.window > 0 && last - k >= p.split.window);
  }
  // E4M3: which warps turn the Q tile of accumulator X into codes. More than 32 rows: its softmax
  // warps, a thread per row. At most 32: the checking warp, which is free before the softmax is
  // through with the last item (64 decoded tokens: 150 us, by the softmax 160; 32 blocks of 64
  // rows: 68 us, by the softmax 64).
  __device__ __forceinline__ bool coded_by_softmax(const Params<TREE>& p, int X) const {
    return dual || (X == 0 && (last - first + 1) * p.split.G > 32);
  }
  // keys of tile j that some row may see, counted from its start
  __device__ __forceinline__ int valid(int j) const { return min(TK, last + 1 - (key0 + j * TK)); }
  // Where V_j stands among the item's 2 T operand tiles. Two row tiles: K0 V0 K1 V1 ..;
  // even / odd: K0 K1 V0 K2 V1 K3 .. V(T-2) V(T-1), each S two tiles ahead of its PV.
  __device__ __forceinline__ int v_at(int j) const {
    return dual ? 2 * j + 1 : j == T - 1 ? 2 * T - 1 : 2 * j + 2;
  }
};

// A place in a ring of N stages that are used in order.
template <int N>
struct Cursor {
  int stage = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == N) {
      stage = 0;
      phase ^= 1;
    }
  }
  __device__ __forceinline__ void skip(int n) {
    stage += n;
    phase ^= (stage / N) & 1;
    stage %= N;
  }
};

// A row of Q to E4M3: two terms of q 2^-e (e: the row's largest exponent - 7, so that nothing
// overflows), the code and the code of its remainder, in place of the bf16 row, each 128 bytes
// of the swizzled layout. The remainder of a bf16's 8 bits has at most 4, so the two hold it
// exactly down to 2^-9 of the row's largest power of two; below, a remainder under the smallest
// code is rounded, by at most 2^-17 of that power. So an outlier of 2^p among elements around 1
// moves scores by about 2^(p - 18) rms (random keys around 1, scaling 128^-1/2), where the cache's
// rounding of the keys has moved them by about 2^-5: noticed from p = 12 on. Returns e.
__device__ __noinline__ int q_codes(uint8_t* tile, int row) {
  uint8_t* at = tile + row * 128;
  const int sw = row & 7;
  uint4 w[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) w[c] = *reinterpret_cast<const uint4*>(at + (c >> 3) * HALF + (((c & 7) ^ sw) << 4));
  uint32_t top = 0;  // largest magnitude, as the bits of a bf16
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    const uint32_t in[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, max(in[e] & 0x7FFFu, (in[e] >> 16) & 0x7FFFu));
  }
  // tiny rows keep 2^-107; a row with infinity or NaN becomes NaN, as its scores would
  const int ex = min(max((int)(top >> 7), 20), 254) - 127 - 7;
  const float mul = top >= 0x7F80u ? NAN : __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
  for (int c = 0; c < 8; ++c) {  // 16 values per chunk of codes
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint4 v = w[2 * c + (e >> 1)];
      const uint32_t p0 = e & 1 ? v.z : v.x, p1 = e & 1 ? v.w : v.y;
      e4m3x4_split(__uint_as_float(p0 << 16) * mul, __uint_as_float(p0 & 0xFFFF0000u) * mul,
                   __uint_as_float(p1 << 16) * mul, __uint_as_float(p1 & 0xFFFF0000u) * mul, hi[e], lo[e]);
    }
    *reinterpret_cast<uint4*>(at + ((c ^ sw) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(at + HALF + ((c ^ sw) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  return ex;
}

// A V tile of E4M3 codes to f16, by one warp, a row per lane at a time: 16 codes (a 16-byte chunk
// of a row) to two chunks, both in the 128-byte swizzled layout (chunk c of row k at c ^ (k & 7)).
// Rows from `rows` on (that no query sees) are zeros. Shared memory answers slowly while MMAs
// read it at its full rate, so a row's chunks are requested at once (64 tokens over 8 x 4600
// keys: 168 us; chunk by chunk 317).
__device__ __forceinline__ void convert_v(const uint8_t* src, uint8_t* dst, int lane, int rows) {
#pragma unroll 1
  for (int row = lane; row < TK; row += 32) {
    const uint8_t* sr = src + row * 128;
    uint8_t* dr = dst + row * 128;
    const int sw = row & 7;
    const bool in = row < rows;
    uint4 x[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = in ? *reinterpret_cast<const uint4*>(sr + ((c ^ sw) << 4)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint8_t* d = dr + (c >> 2) * HALF;
      const int c2 = 2 * (c & 3);
      *reinterpret_cast<uint4*>(d + ((c2 ^ sw) << 4)) = make_uint4(
          e4m3x2_to_f16x2(x[c].x), e4m3x2_to_f16x2(x[c].x >> 16), e4m3x2_to_f16x2(x[c].y), e4m3x2_to_f16x2(x[c].y >> 16));
      *reinterpret_cast<uint4*>(d + (((c2 + 1) ^ sw) << 4)) = make_uint4(
          e4m3x2_to_f16x2(x[c].z), e4m3x2_to_f16x2(x[c].z >> 16), e4m3x2_to_f16x2(x[c].w), e4m3x2_to_f16x2(x[c].w >> 16));
    }
  }
}
// Takes NaN codes (bytes whose low seven bits are all ones) out of the rows of a tile that its
// lane converts. Returns whether there was one.
__device__ __noinline__ bool drop_nan(uint8_t* tile, int lane, int rows) {
  bool nan = false;
#pragma unroll 1
  for (int row = lane; row < rows; row += 32) {
    uint4* at = reinterpret_cast<uint4*>(tile + row * 128);
    uint4 x[8];
    uint32_t hit = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = at[c ^ (row & 7)];  // (the order spreads lanes over banks)
#pragma unroll
    for (int c = 0; c < 8; ++c)  // a byte of 0x7F carries into its top bit
      hit |= ((x[c].x & 0x7F7F7F7Fu) + 0x01010101u) | ((x[c].y & 0x7F7F7F7Fu) + 0x01010101u) |
             ((x[c].z & 0x7F7F7F7Fu) + 0x01010101u) | ((x[c].w & 0x7F7F7F7Fu) + 0x01010101u);
    if ((hit & 0x80808080u) == 0) continue;
    nan = true;
    uint32_t* w = reinterpret_cast<uint32_t*>(at);
#pragma unroll 1
    for (int i = 0; i < 32; ++i) w[i] &= ~__vcmpeq4(w[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  }
  return nan;
}

// Adds to 16 columns of an output row what the checking warps took out of the V tiles: the
// values that are not finite, of keys the row sees.
template <bool FP8, bool TREE>
__device__ __noinline__ void repair(const Params<TREE>& p, const Item<TREE>& it, int pos, int col, float* o) {  // 16 columns
  const Geometry<TREE> g(p, it.w);
  for (int j = 0; j < g.T; ++j) {
    if (!g.cut(p, j)) continue;
    const int k = g.key0 + j * TK;
    long long row;
    if (p.table) {
      const int page = p.table[(size_t)it.w.b * p.pps + (k >> 7)];
      if (page < 0 || page >= p.n_pages) continue;
      row = ((long long)page * p.split.n_kv + it.w.kvh) * TK;
    } else {
      row = ((long long)it.w.b * p.split.n_kv + it.w.kvh) * p.split.capacity + k;
    }
    [[maybe_unused]] uint4 m;  // TREE: keys that the row sees
    if constexpr (TREE) m = chunk::tree_bits(p.tree, it.w.b, pos - it.w.ctx, it.w.ctx, k, p.split.window);
#pragma unroll 1
    for (int e = 0; e < TK; ++e) {
      if constexpr (TREE) {
        if (((e < 32 ? m.x : e < 64 ? m.y : e < 96 ? m.z : m.w) >> (e & 31) & 1) == 0) continue;
      } else {
        if (k + e > pos || (p.split.window > 0 && pos - (k + e) >= p.split.window)) continue;
      }
#pragma unroll 1
      for (int c = 0; c < 16; ++c) {
        const size_t at = (size_t)(row + e) * 128 + col + c;
        const float x = FP8 ? e4m3x2_value(((const uint8_t*)p.cache_v)[at]).x
                            : __bfloat162float(((const bf16*)p.cache_v)[at]);
        if (!isfinite(x)) o[c] += x;
      }
    }
  }
}

template <bool FP8, bool TREE>
__global__ void __launch_bounds__(Plan<FP8>::THREADS, 1) chunk_attn_tc_kernel(const __grid_constant__ Params<TREE> p) {
  using PL = Plan<FP8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Tail<TREE>& sh = *reinterpret_cast<Tail<TREE>*>(smem + PL::OFF_END);
  Item<TREE>(&ring)[kRing] = sh.ring;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = ptx::smem_u32(smem);
  if (sbase & 1023) {  // the swizzled tiles would be misplaced
    grid_wait();
    if (threadIdx.x == 0) {
      atomicOr(p.status, DFLASH_DEV_TIMEOUT);
      p.merge[blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  auto bar = [](uint64_t* b) { return ptx::smem_u32(b); };
  auto wait = [&](uint64_t& b, int parity) {  // one thread
    const uint32_t at = ptx::smem_u32(&b), ph = (uint32_t)(parity & 1);
    return ptx::mbar_try_wait(at, ph) || wait_one(at, ph, &sh.abort_flag, p.status, p.wait_ns);
  };
  auto waits = [&](uint64_t& b, int parity) {  // softmax warps (a call would cost them registers)
    const uint32_t at = ptx::smem_u32(&b), ph = (uint32_t)(parity & 1);
    return __all_sync(0xffffffffu, ptx::mbar_try_wait(at, ph)) ||
           wait_more(at, ph, &sh.abort_flag, p.status, p.wait_ns);
  };
  auto waitw = [&](uint64_t& b, int parity) {  // the others
    const uint32_t at = ptx::smem_u32(&b), ph = (uint32_t)(parity & 1);
    return __all_sync(0xffffffffu, ptx::mbar_try_wait(at, ph)) ||
           wait_more_call(at, ph, &sh.abort_flag, p.status, p.wait_ns);
  };

  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(&sh.qf[i]), 1);
      ptx::mbar_init(bar(&sh.qe[i]), i == 0 ? 2 : 1);
      ptx::mbar_init(bar(&sh.s[i]), 1);
      ptx::mbar_init(bar(&sh.p[i]), 4);
      ptx::mbar_init(bar(&sh.o[i]), 1);
      ptx::mbar_init(bar(&sh.x[i]), 4);
      ptx::mbar_init(bar(&sh.turn[i]), 1);
    }
    ptx::mbar_init(bar(&sh.oe), 2);
    ptx::mbar_init(bar(&sh.of), 8);
    for (int i = 0; i < 6; ++i) {
      ptx::mbar_init(bar(&sh.kf[i]), 1);
      ptx::mbar_init(bar(&sh.ke[i]), FP8 && i >= PL::V_BAR ? 1 : 2);
    }
    for (int i = 0; i < 5; ++i) {
      ptx::mbar_init(bar(&sh.vc[i]), 1);
      ptx::mbar_init(bar(&sh.aux[i]), !FP8 ? 1 : i < 2 ? 2 : 4);
    }
    for (int i = 0; i < kRing; ++i) {
      ptx::mbar_init(bar(&sh.itf[i]), 1);
      ptx::mbar_init(bar(&sh.ite[i]), 2 + 8 + 1);
      ptx::mbar_init(bar(&sh.chk[i]), 1);
    }
    ptx::mbar_init(bar(&sh.fin[0]), 1);
    ptx::mbar_init(bar(&sh.fin[1]), 1);
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(ptx::smem_u32(&sh.tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    ptx::prefetch_tmap(&p.q);
    ptx::prefetch_tmap(&p.k);
    ptx::prefetch_tmap(&p.v);
  }
  grid_wait();     // nothing of the caller's has been read or written yet
  grid_trigger();  // the merge may be scheduled
  // the work split, in what becomes the K / V ring
  static_assert(5 * TILE >= chunk::kLocateBytes<TREE> * (TREE ? kTreeMaxBatch : kChunkMaxBatch), "scratch of the work split");
  const bool few = p.split.batch <= 32;  // sequences: the loading warp finds the share by itself
  if (!few) {
    chunk::locate(p.split, smem + PL::OFF_KV, &sh.start, p.status);
    ptx::fence_proxy_async_smem();  // TMA overwrites them
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh.tmem_slot;

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax
    reg_inc<PL::REG_SOFT>();
    const int X = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + TM_S + X * 128, tO = tmem + lanes + TM_O;
    const int G = p.split.G, rt = r / G, rg = r - rt * G;     // token and head of this row
    const int wt0 = ((warp & 3) * 32) / G;                    // tokens of the warp's first and last row
    const int wt1 = ((warp & 3) * 32 + 31) / G;
    int ns = 0, no = 0, nd = 0, nx = 0, nq = 0;  // tiles, items with keys; of two row tiles, of one
    for (int n = 0;; ++n) {
      const int slot = n % kRing;
      if (!waits(sh.itf[slot], n / kRing)) break;
      const Item<TREE>& it = ring[slot];
      if (it.w.b < 0) break;
      const Geometry<TREE> g(p, it.w);
      const int tok = (g.dual ? X * p.TQ : 0) + rt;           // token of the item
      const int left = it.w.n - it.w.t * 2 * p.TQ;            // tokens from the item's start on
      const bool valid = r < p.RT && tok < left;
      const int pos = g.first + tok;
      const int wfirst = g.first + tok - rt + wt0;
      const bool any = __any_sync(0xffffffffu, valid);
      const int wlast = min(g.first + tok - rt + wt1, g.last);
      float m_ref = -INFINITY, l = 0.f, sl2 = p.sl2;
      bool alive = true, seen = false;  // (TREE: seen: a key, whatever its score)
      const int step = g.dual ? 1 : 2;
      int done = 0;  // tiles of this accumulator
      if (FP8 && g.T > 0) {
        if (g.coded_by_softmax(p, X)) {
          if (!waits(sh.qf[X], nq)) break;
          if (valid) sh.qexp[X][r] = (signed char)q_codes(smem + X * TILE, r);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(&sh.aux[2 + X]));
        }
        nq += X == 0 || g.dual;
      }
      // Warps without rows skip the tiles; the warpgroup's first warp hands in P for them.
      const int rows = min(p.RT, (g.last - g.first + 1) * G - (g.dual ? X * p.RT : 0));
      const int hand_in = (warp & 3) == 0 ? 5 - ((rows + 31) >> 5) : 1;
      if (!any) ns += g.dual ? g.T : (g.T + 1 - X) >> 1;
      for (int j = !any ? g.T : g.dual ? 0 : X; j < g.T; j += step, ++done) {
        [[maybe_unused]] uint4 tm;  // TREE: keys that this row sees; looked up while S is computed
        if constexpr (TREE) {
          const int k = g.key0 + j * TK;
          if (k + TK > g.closed || (p.split.window > 0 && wlast - k >= p.split.window)) {
            tm = chunk::tree_bits(p.tree, it.w.b, valid ? pos - it.w.ctx : -1, it.w.ctx, k, p.split.window);
            seen = seen || (tm.x | tm.y | tm.z | tm.w) != 0;
          } else {
            seen = true;
          }
        }
        alive = waits(sh.s[X], ns++);
        if (!alive) break;
        {
          // never 0 (or infinity): masked scores of -infinity have to stay that when scaled, and
          // scores that small do not tell the keys apart
          if (FP8 && done == 0) sl2 = fminf(fmaxf(ldexpf(p.sl2, sh.qexp[g.dual ? X : 0][r]), FLT_MIN), FLT_MAX);
          ptx::tc_fence_after();
          uint32_t raw[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) ptx::tmem_ld_32x32b_x32(tS + 32 * c, raw[c]);
          ptx::tmem_ld_wait();
          float s[TK];
#pragma unroll
          for (int e = 0; e < TK; ++e) s[e] = __uint_as_float(raw[e >> 5][e & 31]);
          const int k = g.key0 + j * TK;
          const bool open = (TREE ? k + TK <= g.closed : k + TK - 1 <= wfirst) && (p.split.window <= 0 || wlast - k < p.split.window);
          if (!open) {
            // visible columns lo .. hi, as bits of four words
            const int hi = valid ? min(pos - k, TK - 1) : -1;
            const int lo = p.split.window > 0 ? max(pos - k - p.split.window + 1, 0) : 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int h = hi - 32 * c, l0 = lo - 32 * c;
              uint32_t m = h < 0 ? 0u : h >= 31 ? 0xffffffffu : (2u << h) - 1u;
              m &= l0 <= 0 ? 0xffffffffu : l0 > 31 ? 0u : 0xffffffffu << l0;
              if constexpr (TREE) m = c == 0 ? tm.x : c == 1 ? tm.y : c == 2 ? tm.z : tm.w;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                s[32 * c + e] = m & (1u << e) ? s[32 * c + e] : -INFINITY;
            }
          }
          float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int e = 4; e < TK - 4; e += 8) {
            m4[0] = fmax3(m4[0], s[e], s[e + 1]);
            m4[1] = fmax3(m4[1], s[e + 2], s[e + 3]);
            m4[2] = fmax3(m4[2], s[e + 4], s[e + 5]);
            m4[3] = fmax3(m4[3], s[e + 6], s[e + 7]);
          }
          m4[0] = fmax3(m4[0], s[TK - 4], s[TK - 3]);
          m4[1] = fmax3(m4[1], s[TK - 2], s[TK - 1]);
          const float mx = fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * sl2;
          float alpha = 1.f;
          bool resc = false;
          if (m_ref == -INFINITY) {
            m_ref = mx;
          } else if (mx > m_ref + 8.f) {
            alpha = ptx::ex2(m_ref - mx);
            m_ref = mx;
            resc = true;
          }
          if (__any_sync(0xffffffffu, resc) && done > 0) {
            // S_j is complete, so is the PV before it: O holds the tiles so far
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t v[32];
              ptx::tmem_ld_32x32b_x32(tO + X * 128 + 32 * c, v);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
              ptx::tmem_st_32x32b_x32(tO + X * 128 + 32 * c, v);
            }
          }
          const float mu = (m_ref == -INFINITY ? 0.f : m_ref) - (FP8 ? kShiftF16 : 0.f);
          const float2 sl2v = make_float2(sl2, sl2), nmu = make_float2(-mu, -mu);
          float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x = __ffma2_rn(make_float2(s[32 * h + e], s[32 * h + e + 1]), sl2v, nmu);
              const float2 y = make_float2(ptx::ex2(x.x), ptx::ex2(x.y));
              acc[(e >> 1) & 1] = __fadd2_rn(acc[(e >> 1) & 1], y);
              pk[e >> 1] = FP8 ? pack_f16(y.x, y.y) : pack_bf16(y.x, y.y);
            }
            tmem_st_x16(tS + 16 * h, pk);
          }
          l = l * alpha + ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y));
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
        }
        __syncwarp();
        if (lane < hand_in) ptx::mbar_arrive(bar(&sh.p[X]));
      }
      if (!alive) break;
      // ---- epilogue
      if constexpr (TREE) {  // keys, all at a score of minus infinity
        if (seen && m_ref == -INFINITY) m_ref = -FLT_MAX;
      }
      const int token = it.w.t * 2 * p.TQ + tok;
      bf16* orow = p.out + ((size_t)(it.w.row0 + token) * p.n_h + it.w.kvh * G + rg) * 128;
      if (g.T == 0) {  // no row sees a key
        if (valid && (g.dual || X == 0)) {
          const uint32_t z[8] = {};
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(orow + 16 * c) = make_uint4(z[0], z[1], z[2], z[3]),
            *reinterpret_cast<uint4*>(orow + 16 * c + 8) = make_uint4(z[4], z[5], z[6], z[7]);
        }
      } else {
        float wa = 1.f, wb = 0.f;  // weights of the two accumulators (one: its own)
        if (!g.dual) {
          // the other half has read what the last exchange left
          if (no > 0 && !waits(sh.of, no - 1)) break;
          sh.xml[X][r] = make_float2(m_ref, l);
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(&sh.x[X]));
          if (!waits(sh.x[X ^ 1], nx)) break;
          const float2 other = sh.xml[X ^ 1][r];
          const float ma = X == 0 ? m_ref : other.x, mb = X == 0 ? other.x : m_ref;
          const float la = X == 0 ? l : other.y, lb = X == 0 ? other.y : l;
          m_ref = fmaxf(ma, mb);
          wa = ma == -INFINITY ? 0.f : ptx::ex2(ma - m_ref);
          wb = mb == -INFINITY ? 0.f : ptx::ex2(mb - m_ref);
          l = (la == 0.f ? 0.f : la * wa) + (lb == 0.f ? 0.f : lb * wb);
        }
        if (!(g.dual ? waits(sh.o[X], nd++) : waits(sh.oe, nx++))) break;
        if (!waits(sh.chk[slot], n / kRing)) break;
        ++no;
        ptx::tc_fence_after();
        const bool bad = *reinterpret_cast<const volatile int*>(&it.bad) != 0;
        const float inv = it.w.slot < 0 ? (l == 0.f ? 0.f : (FP8 ? p.v_scale : 1.f) / l) : (FP8 ? p.v_scale : 1.f);
        const int irow = (g.dual ? X * p.RT : 0) + r;
        const size_t pslot = (size_t)(2 * blockIdx.x + (it.w.slot > 0)) * (2 * p.RT);
        // two row tiles: all columns of this one's; else half of the columns of both. An
        // accumulator without keys (or without a tile) is not read as a number.
        const int c0 = g.dual ? 0 : 4 * X, c1 = g.dual ? 8 : 4 * X + 4;  // 16 columns each
        const uint32_t t0 = tO + (g.dual ? X * 128 : 0);
        const float fa = wa * inv, fb = wb * inv;
        if (any) {
#pragma unroll 1
          for (int c = c0; c < c1; ++c) {
            uint32_t v[16], u[16];
            float o[16];
            tmem_ld_x16(t0 + 16 * c, v);
            if (!g.dual) tmem_ld_x16(tO + 128 + 16 * c, u);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = wa == 0.f ? 0.f : __uint_as_float(v[e]) * fa;
            if (wb != 0.f) {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] += __uint_as_float(u[e]) * fb;
            }
            if (!(l > 0.f)) {  // no key (or none in this piece), or a score that is not a number
              // no weight at all on keys that are seen: every score is minus infinity
              const float none = l == 0.f && it.w.slot < 0 && (TREE ? m_ref != -INFINITY : pos >= 0) ? NAN : l;
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = none;
            }
            if (bad && valid) {
              float fix[16];
#pragma unroll 1
              for (int e = 0; e < 16; ++e) fix[e] = 0.f;
              repair<FP8, TREE>(p, it, pos, 16 * c, fix);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] += fix[e];
            }
            if (valid) {
              uint32_t w[16];
              if (it.w.slot < 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = pack_bf16(o[2 * i], o[2 * i + 1]);
                bf16* dst = orow + 16 * c;
                if (p.out32) {  // a whole 32-byte sector
                  st8(dst, w);
                } else {
                  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                  *reinterpret_cast<uint4*>(dst + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                }
              } else {
                // [column / 8][row][8]: a warp's store is one run of 1 KB
                float* dst = p.part + pslot * 128 + ((size_t)(2 * c) * (2 * p.RT) + irow) * 8;
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i]);
                st8(dst, w);
                st8(dst + (size_t)8 * (2 * p.RT), w + 8);  // the workspace is 256-byte aligned
              }
            }
          }
          if (it.w.slot >= 0 && valid && (g.dual || X == 0))
            p.part_ml[pslot + irow] = make_float2(!TREE && l == 0.f && pos >= 0 ? -FLT_MAX : m_ref, l);
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(&sh.of));
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(&sh.ite[slot]));
    }
  } else {
    reg_dec<PL::REG_REST>();
    if (warp == 8) {
      // ------------------------------------------------------------------ work list, TMA
      if (few) chunk::locate_by_warp(p.split, &sh.start, p.status);
      if (lane == 0) {
        chunk::Walker<true, TREE> walk(p.split, sh.start);
        chunk::Piece<TREE> w;
        int count[2] = {0, 0}, nq[2] = {0, 0};  // tiles (bf16: of both kinds), Q tiles
        chunk::Piece<TREE> cur = {};  // (before the first: no tiles)
        bool more = true;
#pragma unroll 1
        for (int n = -1;; ++n) {  // item n + 1 is looked for once item n's first loads are on their way
          if (n >= 0) {
            const int slot = n % kRing;
            if (n >= kRing && !wait(sh.ite[slot], n / kRing - 1)) break;
            if (!more) w.b = -1;
            ring[slot].w = w;
            ring[slot].bad = 0;
            ptx::mbar_arrive(bar(&sh.itf[slot]));
            if (!more) break;
            cur = w;
          }
          const Geometry<TREE> g(p, cur);
          more = walk.next(&w);
          if (n < 0) continue;
          const int32_t* table = p.table ? p.table + (size_t)cur.b * p.pps + (g.key0 >> 7) : nullptr;
          bool stop = false;
          int page = table && g.T > 0 ? table[0] : 0;
#pragma unroll 1
          for (int i = 0, jk = 0, jv = 0; i <= 2 * g.T; ++i) {
            // after the first K tile: Q, unless nothing is left to load
            if (i == 1) {
#pragma unroll 1
              for (int X = 0; X < (g.dual ? 2 : 1); ++X) {
                if (nq[X] > 0 && !wait(sh.qe[X], nq[X] - 1)) {
                  stop = true;
                  break;
                }
                ++nq[X];
                ptx::mbar_arrive_expect_tx(bar(&sh.qf[X]), (uint32_t)p.RT * 256);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  tma_load_3d(sbase + X * TILE + h * HALF, &p.q, bar(&sh.qf[X]), 64 * h, cur.kvh * p.split.G,
                              cur.row0 + (2 * cur.t + X) * p.TQ);
              }
              if (stop) break;
            }
            if (i == 2 * g.T) break;
            const int which = jv < g.T && i == g.v_at(jv);  // 0: a K tile, 1: a V tile
            if (!which) {
              // the row of tile jk: of its page (looked up a tile ahead), or in the sequence's slab
              int row = (cur.b * p.split.n_kv + cur.kvh) * p.split.capacity + g.key0 + jk * TK;
              if (table) {
                row = (page * p.split.n_kv + cur.kvh) * TK;
                if (page < 0 || page >= p.n_pages) {
                  atomicOr(p.status, DFLASH_DEV_PAGE);
                  row = p.oob_row;
                }
                if (jk + 1 < g.T) page = table[jk + 1];
              }
              sh.rows[jk & 3] = row;
            }
            const int y = sh.rows[(which ? jv : jk) & 3];
            int& at = FP8 && which ? count[1] : count[0];
            const int s = at % PL::STAGES, u = at / PL::STAGES, bi = s + which * PL::V_BAR;
            if (u > 0 && !wait(sh.ke[bi], u - 1)) {
              stop = true;
              break;
            }
            const CUtensorMap* map = which ? &p.v : &p.k;
            const uint32_t dst = sbase + PL::OFF_KV + bi * PL::LOAD;
            ptx::mbar_arrive_expect_tx(bar(&sh.kf[bi]), PL::LOAD);
            ptx::tma_load_2d(dst, map, bar(&sh.kf[bi]), 0, y);
            if (!FP8) ptx::tma_load_2d(dst + HALF, map, bar(&sh.kf[bi]), 64, y);
            // the checking warp looks at some stages only, so it is told which phase of the
            // stage's barrier is its: the one running now
            if (!FP8 && which && g.cut(p, jv)) ptx::mbar_arrive(bar(&sh.aux[s]));
            ++at;
            if (which) ++jv; else ++jk;
          }
          if (stop) break;
        }
        p.merge[blockIdx.x] = walk.merge;
        // nothing of ours may still be landing in shared memory when the CTA exits
        for (int X = 0; X < 2; ++X)
          if (nq[X] > 0) drain(bar(&sh.qf[X]), (nq[X] - 1) & 1, p.status);
        for (int k = 0; k < (FP8 ? 2 : 1); ++k)
          for (int i = count[k] > PL::STAGES ? count[k] - PL::STAGES : 0; i < count[k]; ++i)
            drain(bar(&sh.kf[i % PL::STAGES + k * PL::V_BAR]), (i / PL::STAGES) & 1, p.status);
      }
    } else if (warp < PL::W_CHECK) {
      // ------------------------------------------------------------------ MMA issue
      // Warp 9 issues for A and warp 10 for B, so that what one does between its MMAs (waits,
      // descriptors) hides behind the other's. Both go through every operand tile in the order
      // of the ring; a tile that only the other needs is freed at once. Every lane takes the
      // same way, one issues.
      constexpr uint32_t idesc_s = FP8 ? idesc_e4m3_f32(128, TK) : ptx::idesc_bf16_f32(128, TK);
      constexpr uint32_t idesc_pv = (FP8 ? idesc_f16_f32(128, 128) : ptx::idesc_bf16_f32(128, 128)) | (1u << 16);
      const int me = warp - 9;
      int np = 0, nq[2] = {0, 0}, nof = 0, items = 0;  // P tiles, Q tiles, waits for sh.of, items
      int blocks = 0;                                  // issued in items of two row tiles
      Cursor<PL::STAGES> cur;                          // next operand tile (E4M3: K tile)
      Cursor<PL::C_STAGES> cv;                         // E4M3: next V tile
      uint32_t chk = 0;                                // bf16: phases of the stages' check barriers
      bool issued = false;
      const uint64_t dq[2] = {ptx::smem_desc_sw128(sbase), ptx::smem_desc_sw128(sbase + TILE)};
      const uint64_t dk0 = ptx::smem_desc_sw128(sbase + PL::OFF_KV);
      const uint64_t dv0 = ptx::smem_desc_sw128_mn(sbase + (FP8 ? PL::OFF_C : PL::OFF_KV), HALF);
      // the softmax has read O of every item before this one
      auto wait_of = [&]() -> bool {
        while (nof < items)
          if (!waitw(sh.of, nof++)) return false;
        return true;
      };
      // by the elected lane
      auto mma_s = [&](int X, uint64_t da, uint64_t db) {  // S_X = Q K^T
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
          if (FP8)  // the codes of Q, then those of their remainders, 32 dims per step
            mma_f8(tmem + TM_S + X * 128, da + off, db + (((kk & 3) * 32) >> 4), idesc_s, kk > 0 ? 1u : 0u);
          else
            ptx::mma_bf16(tmem + TM_S + X * 128, da + off, db + off, idesc_s, kk > 0 ? 1u : 0u);
        }
        ptx::mma_commit(bar(&sh.s[X]));
      };
      auto mma_pv = [&](int X, uint64_t db, int steps, bool first) {  // O_X += P V, 16 keys a step
        const uint32_t pa = tmem + TM_S + X * 128, o = tmem + TM_O + X * 128;
        if (steps == 8) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(o, pa + kk * 8, db + kk * (2048 >> 4), idesc_pv, (!first || kk > 0) ? 1u : 0u);
        } else {
#pragma unroll 1
          for (int kk = 0; kk < steps; ++kk)
            mma_ts(o, pa + kk * 8, db + kk * (2048 >> 4), idesc_pv, (!first || kk > 0) ? 1u : 0u);
        }
      };
      for (int n = 0;; ++n) {
        const int slot = n % kRing;
        if (!waitw(sh.itf[slot], n / kRing)) break;
        const chunk::Piece<TREE> w = ring[slot].w;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(&sh.ite[slot]));
        if (w.b < 0) break;
        const Geometry<TREE> g(p, w);
        if (g.T == 0) continue;
        // a tile of the operand rings, in order: its stage, once it has landed
        auto take_k = [&](int& st) -> bool {
          st = cur.stage;
          const bool ok = waitw(sh.kf[st], cur.phase);
          cur.next();
          return ok;
        };
        auto take_v = [&](int& st, int j, bool own) -> bool {
          if (FP8) {
            st = cv.stage;
            const bool ok = waitw(sh.vc[st], cv.phase);
            cv.next();
            return ok;
          }
          if (!take_k(st)) return false;
          if (!g.cut(p, j)) return true;
          const bool ok = !own || waitw(sh.vc[st], (chk >> st) & 1);  // it has been through the check
          chk ^= 1u << st;
          return ok;
        };
        auto free_v = [&](int st) { return FP8 ? bar(&sh.aux[st]) : bar(&sh.ke[st]); };
        // this warp's tiles: all of them, or every other one
        const int mine = g.dual ? g.T : (g.T + 1 - me) >> 1;
        const int X = g.dual ? me : 0;  // its Q tile
        const int ahead = g.dual ? 1 : 2;
        // Q_A is waited for and released by both warps in every item, so that neither is ever
        // more than a phase away from its barriers
        bool ok = FP8 ? waitw(sh.aux[2], nq[0]) : waitw(sh.qf[0], nq[0]);
        ++nq[0];
        if (X == 1) {
          ok = ok && (FP8 ? waitw(sh.aux[3], nq[1]) : waitw(sh.qf[1], nq[1]));
          ++nq[1];
        }
        issued = issued || mine > 0;
        int ks = 0, vs;
        // first S of each accumulator: of K_0, and of K_1 for the odd half
        for (int j = 0; j < min(ahead, g.T) && ok; ++j) {
          ok = take_k(ks);
          if (!ok) break;
          if (g.dual || j == me) {
            ptx::tc_fence_after();
            if (elect_one()) {
              mma_s(me, dq[X], dk0 + ks * (PL::LOAD >> 4));
              ptx::mma_commit(bar(&sh.ke[ks]));
            }
            __syncwarp();
          } else if (lane == 0) {
            ptx::mbar_arrive(bar(&sh.ke[ks]));
          }
        }
        int done = 0;
        for (int j = 0; j < g.T && ok; ++j) {
          // what the next PV and S read is waited for first, so that the MMAs follow P at once
          const bool own = g.dual || (j & 1) == me, more = j + ahead < g.T;
          const int steps = (g.valid(j) + 15) >> 4;
          ks = 0;
          ok = take_v(vs, j, own) && (!more || take_k(ks));
          if (!own) {
            if (ok && lane == 0) {
              ptx::mbar_arrive(free_v(vs));
              if (more) ptx::mbar_arrive(bar(&sh.ke[ks]));
            }
            continue;
          }
          ok = ok && (done > 0 || wait_of());
          // With two row tiles the blocks of A and B take strict turns. Without that they drift
          // into step: both softmax at once with the tensor cores idle, then both blocks at
          // once (3650 instead of 2800 cycles per key tile).
          if (ok && g.dual) {
            if (blocks >= 1 - me) ok = waitw(sh.turn[me], blocks - (1 - me));
            ++blocks;
          }
          ok = ok && waitw(sh.p[me], np++);
          if (!ok) break;
          ptx::tc_fence_after();
          if (elect_one()) {
            mma_pv(me, dv0 + vs * (TILE >> 4), steps, done == 0);
            if (more) mma_s(me, dq[X], dk0 + ks * (PL::LOAD >> 4));
            if (done + 1 == mine) ptx::mma_commit(bar(g.dual ? &sh.o[me] : &sh.oe));
            ptx::mma_commit(free_v(vs));
            if (more) ptx::mma_commit(bar(&sh.ke[ks]));
            // Q (and its exponents) is free with this warp's last S, but not before its softmax
            // warps have handed in a tile
            if (done == max(mine - 2, 0)) {
              ptx::mma_commit(bar(&sh.qe[0]));
              if (X == 1) ptx::mma_commit(bar(&sh.qe[1]));
            }
          }
          __syncwarp();
          if (g.dual && lane == 0) ptx::mbar_arrive(bar(&sh.turn[me ^ 1]));
          ++done;
        }
        if (!ok) break;
        if (mine == 0) {  // nothing in this item: it is still not complete without this warp
          if (!wait_of()) break;
          if (lane == 0) {
            ptx::mbar_arrive(bar(&sh.oe));
            ptx::mbar_arrive(bar(&sh.qe[0]));
          }
        }
        ++items;
      }
      // every MMA issued by this warp has finished before tensor memory is released
      if (issued) {
        if (elect_one()) ptx::mma_commit(bar(&sh.fin[me]));
        __syncwarp();
        drain(bar(&sh.fin[me]), 0, p.status);
      }
    } else if (warp >= PL::W_CHECK) {
      int base = 0, nq = 0;
      uint32_t told = 0;  // bf16: phases of aux
      for (int n = 0;; ++n) {
        const int slot = n % kRing;
        if (!waitw(sh.itf[slot], n / kRing)) break;
        const chunk::Piece<TREE> w = ring[slot].w;
        if (w.b < 0) break;
        const Geometry<TREE> g(p, w);
        bool alive = true;
        if constexpr (FP8) {
          // -------------------------------------------------------------- Q codes
          if (g.T > 0) alive = waitw(sh.qf[0], nq++);
          if (!alive) break;
          if (g.T > 0 && !g.coded_by_softmax(p, 0)) {
            const int rows = min(p.RT, (g.last - g.first + 1) * p.split.G);
            for (int row = lane; row < rows; row += 32) sh.qexp[0][row] = (signed char)q_codes(smem, row);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane < 4) ptx::mbar_arrive(bar(&sh.aux[2]));
          }
          // -------------------------------------------------------------- V to f16
          for (int j = 0; j < g.T && alive; ++j) {
            const int a = base + j, st = a % PL::STAGES, cs = a % PL::C_STAGES;
            alive = waitw(sh.kf[PL::V_BAR + st], a / PL::STAGES) &&
                    (a < PL::C_STAGES || waitw(sh.aux[cs], a / PL::C_STAGES - 1));
            if (!alive) break;
            uint8_t* codes = smem + PL::OFF_KV + (PL::V_BAR + st) * PL::LOAD;
            if (g.cut(p, j) && drop_nan(codes, lane, g.valid(j))) *reinterpret_cast<volatile int*>(&ring[slot].bad) = 1;
            convert_v(codes, smem + PL::OFF_C + cs * TILE, lane, g.valid(j));
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              ptx::mbar_arrive(bar(&sh.vc[cs]));
              ptx::mbar_arrive(bar(&sh.ke[PL::V_BAR + st]));
            }
          }
        } else {
          // -------------------------------------------------------------- check of V
          // Lanes over 16-byte chunks (which chunk of its row does not matter, so the
          // swizzle does not either): x * 0 is 0 but for infinities and NaN. Rows past the
          // last visible key become zeros up to the end of their K-step.
          for (int j = 0; j < g.T && alive; ++j) {
            if (!g.cut(p, j)) continue;
            const int a = 2 * base + g.v_at(j), s = a % PL::STAGES;
            alive = waitw(sh.aux[s], (told >> s) & 1) && waitw(sh.kf[s], a / PL::STAGES);
            if (!alive) break;
            told ^= 1u << s;
            uint4* v = reinterpret_cast<uint4*>(smem + PL::OFF_KV + s * PL::LOAD);
            const int rows = g.valid(j), end = (rows + 15) & ~15;
            __nv_bfloat162 acc = __floats2bfloat162_rn(0.f, 0.f);
            const __nv_bfloat162 zero = acc;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint4* vh = v + h * (HALF / 16);
#pragma unroll 8
              for (int i = lane; i < rows * 8; i += 32) {
                const uint4 x = vh[i];
                const __nv_bfloat162* e = reinterpret_cast<const __nv_bfloat162*>(&x);
                acc = __hfma2(e[0], zero, acc);
                acc = __hfma2(e[1], zero, acc);
                acc = __hfma2(e[2], zero, acc);
                acc = __hfma2(e[3], zero, acc);
              }
              for (int i = rows * 8 + lane; i < end * 8; i += 32) vh[i] = make_uint4(0, 0, 0, 0);
            }
            const bool nan = __hisnan(acc.x) || __hisnan(acc.y);
            if (nan) {  // in the chunks that this thread looked at
              for (int h = 0; h < 2; ++h)
                for (int i = lane; i < rows * 8; i += 32) {
                  uint4 x = v[h * (HALF / 16) + i];
                  uint32_t* word = &x.x;
#pragma unroll
                  for (int e = 0; e < 4; ++e)  // halves whose exponent is all ones
                    word[e] &= ~__vcmpeq2(word[e] & 0x7F807F80u, 0x7F807F80u);
                  v[h * (HALF / 16) + i] = x;
                }
            }
            if (nan) *reinterpret_cast<volatile int*>(&ring[slot].bad) = 1;
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(&sh.vc[s]));
          }
        }
        if (!alive) break;
        base += g.T;
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(bar(&sh.chk[slot]));
          ptx::mbar_arrive(bar(&sh.ite[slot]));
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <bool FP8, bool TREE>
cudaError_t launch(const Params<TREE>& p, cudaStream_t s) {
  constexpr size_t smem = Plan<FP8>::OFF_END + sizeof(Tail<TREE>);
  static_assert(smem <= 227 * 1024, "shared memory");
  static SmemLimit limit;
  cudaError_t e = limit.raise(chunk_attn_tc_kernel<FP8, TREE>, (int)smem);
  if (e != cudaSuccess) return e;
  LaunchScope ls_(DFLASH_KERNEL_CHUNK_ATTN, s);
  return launch_overlapped(chunk_attn_tc_kernel<FP8, TREE>, dim3(chunk_sms()), Plan<FP8>::THREADS, smem, s, p);
}

}  // namespace

namespace {

// [rows][heads][128] view of bf16 rows ld elements apart, box {64 columns, box_heads heads,
// box_rows rows}, 128-byte swizzle, zero fill.
bool encode_3d_bf16(CUtensorMap* m, const void* base, long long rows, int heads, long long ld,
                    int box_heads, int box_rows) {
  static const decltype(&cuTensorMapEncodeTiled) fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess && q == cudaDriverEntryPointSuccess;
    return (decltype(&cuTensorMapEncodeTiled))(ok ? f : nullptr);
  }();
  if (!fn) return false;
  cuuint64_t dims[3] = {128, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {256, (cuuint64_t)ld * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool TREE>
cudaError_t attn_tc(const ChunkAttnParams& a, cudaStream_t s) {
  if (a.d_h != 128 || a.G > 128) return cudaErrorInvalidValue;
  Params<TREE> p;
  memset(&p, 0, sizeof(p));
  p.TQ = 128 / a.G;
  p.RT = p.TQ * a.G;
  // Cost units of the work split: an item (its start, and its end with nothing behind it), a key tile
  // of two row tiles, and of one. Measured, us in a replayed graph, by the item's cost:
  //   bf16                          0     4     8    12    16    24
  //   32 blocks of 16 rows       72.9  70.1  70.3  70.2  71.1  72.1
  //   8192-row prompt             421   389   351   374   376   383
  //   12 chunks of 100 to 900     242   189   162   159   166   172
  //   24 x 5 to 40 rows, G = 8  104.3  79.4  77.6  77.9  77.9  80.3
  //   E4M3                          0     7    14    20    24    36
  //   64 tokens                 168.6 158.3 151.1 152.6 154.0 158.9
  //   32 blocks of 16 rows      100.2  69.7  64.8  64.4  64.3  66.2
  //   8192-row prompt             543   495   455   427   413   420
  //   12 chunks of 100 to 900     300   278   235   207   205   201
  // (E4M3 stays at what is best for single tokens.) A tile of one row tile at 3/4 or half of one
  // of two instead of at the same: 34 tokens and 6 chunks 110.9 (bf16, 3 : 4), 114.8 (2 : 4), 120.6
  // (4 : 4); E4M3 121.6 (3 : 6), 133.4 (2 : 6), 151.1 (6 : 6).
  p.split = {a.cu_rows, a.kv_lens, a.batch, a.rows, a.n_kv, a.G, a.capacity, a.window, 2 * p.RT, 2 * p.TQ, p.RT, 7,
             a.fp8 ? 14 : 8, a.fp8 ? 6 : 4, 3, a.tree.nodes, a.tree.max_nodes};
  const long long kv_rows = a.block_table ? (long long)a.n_pages * a.n_kv * TK
                                          : (long long)a.batch * a.n_kv * a.capacity;
  p.oob_row = (int)kv_rows;
  if (!encode_3d_bf16(&p.q, a.q, a.rows, a.n_h, a.ld_q, a.G, p.TQ)) return cudaErrorInvalidValue;
  const bool ok = a.fp8 ? encode_2d_u8(&p.k, a.cache_k, kv_rows, TK) && encode_2d_u8(&p.v, a.cache_v, kv_rows, TK)
                        : encode_2d_bf16(&p.k, a.cache_k, kv_rows, 128, TK) &&
                              encode_2d_bf16(&p.v, a.cache_v, kv_rows, 128, TK);
  if (!ok) return cudaErrorInvalidValue;
  p.table = a.block_table;
  p.pps = a.pages_per_seq;
  p.n_pages = a.n_pages;
  p.cache_v = a.cache_v;
  p.out = (bf16*)a.out;
  p.part = a.part;
  p.part_ml = a.part_ml;
  p.merge = a.merge;
  p.status = a.status;
  p.n_h = a.n_h;
  p.sl2 = a.scaling * 1.4426950408889634f * (a.fp8 ? a.k_scale : 1.f);
  p.v_scale = a.v_scale;
  p.out32 = ((uintptr_t)a.out & 31) == 0;
  p.wait_ns = wait_limit_ns();
  p.tree = a.tree;
  return a.fp8 ? launch<true, TREE>(p, s) : launch<false, TREE>(p, s);
}

}  // namespace
}  // namespace dflash
