// kv8_store.cu -- the 8-bit K/V cache: quantising K/V rows as they are written, and reading
// them back to bf16.
//
// A block of 64 tokens of one (layer, slot, K/V head) has one scale for K and one for V, the
// smallest power of two s >= 2^-60 with amax / s <= 448. A power of two costs E4M3 nothing
// (its step is relative) and makes x / s exact, so that storing is one rounding to nearest
// even. A write that begins inside a block keeps the block's earlier tokens: its scale can
// only grow, and the kept tokens move by an exact shift of exponents (only values that reach
// E4M3's subnormals round again).
//
// Bound by memory: three bytes a value in each direction (two of bf16, one of the cache). Whole
// blocks are 82 % (64 x 18 x 788 tokens of 256 written and read back, 522 us) and 97 % (32 ragged
// rows of up to 4096 tokens of 8 x 128, 4 layers, read in 376 us) of the copy rate. Writes alone
// take 268 us of the 522, 79 %: their 32 registers of data a thread leave 32 warps an SM (and 20 bytes
// spilled).
#include <algorithm>

#include "kernels.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace vla {

namespace {

// 16 bytes of global memory, or zeros (nothing is read), to shared memory.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool any) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(any ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait0() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Unit of work: one block of one (layer, row, K/V head). Units of a launch are numbered with
// the block innermost, so that neighbouring CTAs read neighbouring tokens.
struct Unit {
  int l, b, h, slot, blk;        // layer (absolute), row, head, slot, block of the slot
  int lo, hi;                    // tokens of the block that are written or read
  int first;                     // token of the row that stands at `lo`
  size_t idx;                    // block number in the cache
  int lrow;                      // layer of the bf16 side (from 0)
};

// Unit `id`, as a warp sees it. false: nothing to do (past the row's end, or a refused row).
template <bool kWrite>
__device__ __forceinline__ bool make_unit(const Kv8RowsParams& p, unsigned id, Unit& u) {
  const int j = id % p.nblk_row;
  id /= p.nblk_row;
  u.h = id % p.c.n_kv;
  id /= p.c.n_kv;
  u.b = id % p.batch;
  u.lrow = id / p.batch;
  u.l = p.layer0 + u.lrow;
  u.slot = p.slots ? p.slots[u.b] : u.b;
  const int pos = p.pos ? p.pos[u.b] : 0;
  const int cnt = p.count ? p.count[u.b] : p.n_tokens;
  bool bad = u.slot < 0 || u.slot >= p.c.n_slots || pos < 0 || cnt < 0 || cnt > p.n_tokens ||
             pos > p.c.capacity - cnt;
  if (kWrite && p.slots) {   // two rows of one write that name the same slot: the later is refused
    bool dup = false;
    // (rows of no tokens name none. Both loads always: behind a branch the second cost 2 % of a write.)
    const int* n = p.count ? p.count : p.slots;
    for (int i = threadIdx.x & 31; i < u.b; i += 32) dup |= (p.slots[i] == u.slot) & ((n[i] != 0) | !p.count);
    bad |= __any_sync(0xffffffffu, dup) != 0;
  }
  if (bad) {
    if ((threadIdx.x & 31) == 0 && cnt != 0) report(p.err, kKv8BadRow);   // (no tokens: padding)
    return false;
  }
  u.blk = pos / kKv8Block + j;
  const int t0 = u.blk * kKv8Block;
  u.lo = max(pos - t0, 0);
  u.hi = min(pos + cnt - t0, kKv8Block);
  u.first = t0 + u.lo - pos;
  u.idx = ((static_cast<size_t>(u.l) * p.c.n_slots + u.slot) * p.c.n_kv + u.h) * p.c.nblk + u.blk;
  return cnt > 0 && u.lo < u.hi;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d) {
  return static_cast<uint32_t>(f2_to_e4m3x2(a, b)) | (static_cast<uint32_t>(f2_to_e4m3x2(c, d)) << 16);
}

// Four stored values moved to a scale 2^-shift of the old one.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  const uint32_t h0 = e4m3x2_to_h2(static_cast<uint16_t>(w)), h1 = e4m3x2_to_h2(static_cast<uint16_t>(w >> 16));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
  return quant4(a.x * f, a.y * f, b.x * f, b.y * f);
}

// Word index of (dim d, word of its row) in the transposing tile: the 32 lanes of a store have
// dims 8 apart, which the exclusive or spreads over all banks.
__device__ __forceinline__ int vt_word(int d, int word) { return (d * 16 + word) ^ ((d >> 3) & 31); }
// Token quad tg (2t, 2t+1, 2t+8, 2t+9 of the 16-token group w = tg / 4, t = tg % 4) is word 4t + w.
__device__ __forceinline__ int quad_word(int tg) { return 4 * (tg & 3) + (tg >> 2); }

}  // namespace

// What the threads of a write need of a unit.
struct WriteUnit {
  long long src;                 // element of K_in and V_in at which token 0 of the block would stand
  size_t idx;
  int lo, hi;                    // lo >= hi: nothing to do
};
__device__ __forceinline__ WriteUnit write_unit(const Kv8RowsParams& p, unsigned id, int D) {
  Unit u;
  WriteUnit w;
  const bool any = make_unit<true>(p, id, u);
  w.lo = any ? u.lo : 0;
  w.hi = any ? u.hi : 0;
  w.idx = any ? u.idx : 0;
  w.src = u.lrow * p.st_layer + u.b * p.st_row + static_cast<long long>(u.h) * D;
  if (any) w.src += static_cast<long long>(u.first - u.lo) * p.st_tok;
  return w;
}
// Token of the block of a thread's piece i, from that of its first piece (16 (tg / 4) + 2 (tg % 4)).
__device__ __forceinline__ int piece_token(int tok0, int i) { return tok0 + 32 * (i >> 2) + 8 * ((i >> 1) & 1) + (i & 1); }
// Largest magnitudes of two bf16 pairs (NaN if there is one), products and E4M3 of four values.
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t v) {
  uint32_t r;
  asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %2;\n\tmax.NaN.bf16x2 %0, %1, a;\n\t}\n" : "=r"(r) : "r"(m), "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t max_int16(uint32_t m) { return max(m & 0x7fffu, (m >> 16) & 0x7fffu); }
__device__ __forceinline__ uint32_t mul_bf2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int D>
constexpr int kWriteCtas = 512 / D;      // CTAs an SM (64 registers a thread)
template <int D>
constexpr int kWriteSmem = 2 * D * 128;  // pieces in flight

// 2 D threads: the first half holds a block's K, the second its V. Thread (vec, tg) of a
// half keeps 8 dims of the tokens tg and tg + 8 of the sixteen token quads (2t, 2t+1, 2t+8,
// 2t+9 of a 16-token group) in 8 registers of 16 bytes: the data is read once, and the maximum
// and the rounding work on registers. A CTA takes every gridDim-th unit; while it works on one,
// each thread's pieces of the next are on their way to a place of its own in shared memory, so
// that loads are always in flight. 64 x 18 x 788 tokens of 256: 318 us with one unit a CTA, no loads
// ahead and 877 instructions a warp, 268 us so (560 instructions), 212 at the copy rate.
template <int D>
__global__ void __launch_bounds__(2 * D, kWriteCtas<D>) kv8_write_kernel(const Kv8RowsParams p, const unsigned units) {
  constexpr int kVec = D / 8;              // 16-byte pieces of a token
  constexpr int kDs = D < 64 ? 64 : D;
  extern __shared__ __align__(16) uint8_t next[];        // [8][2 D] pieces
  constexpr int kWarps = D / 32;           // of a half
  __shared__ uint32_t vt[D * 16];          // transposed V block
  __shared__ uint32_t red[2][2 * kWarps];  // largest magnitudes of the warps, K's, then V's
  __shared__ int broken[kKv8Block];        // token of the block with a value that is not finite
  __shared__ WriteUnit us[2];
  const int half = threadIdx.x / D, tid = threadIdx.x % D;
  const int vec = tid % kVec, tg0 = tid / kVec;          // tg0 < 8
  const int tok0 = 16 * (tg0 >> 2) + 2 * (tg0 & 3);
  const uint32_t mine = smem_u32(next) + threadIdx.x * 16;
  auto fetch = [&](const WriteUnit& u) {
    const int lo = u.lo, hi = u.hi;
    const __nv_bfloat16* src = (half ? p.v_in : p.k_in) + u.src + vec * 8;
    if (lo == 0 && hi == kKv8Block) {
      src += tok0 * p.st_tok;
#pragma unroll
      for (int i = 0; i < 8; ++i) {        // tokens 0, 1, 8, 9, 32, 33, 40, 41 from the first
        cp_async16(mine + i * 2 * D * 16, src, true);
        src += (i == 3 ? 23 : i & 1 ? 7 : 1) * p.st_tok;
      }
    } else
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {          // (not unrolled: its addresses would take the pieces' registers)
      const int tok = piece_token(tok0, i);
      cp_async16(mine + i * 2 * D * 16, src + (tok >= lo && tok < hi ? tok : lo) * p.st_tok, tok >= lo && tok < hi);
    }
    cp_async_commit();
  };
  unsigned id = blockIdx.x;
  if (threadIdx.x < 32) {
    const WriteUnit a = write_unit(p, id, D);
    if (threadIdx.x == 0) us[0] = a;
    if (id + gridDim.x < units) {
      const WriteUnit c = write_unit(p, id + gridDim.x, D);
      if (threadIdx.x == 0) us[1] = c;
    }
  }
  __syncthreads();
  fetch(us[0]);
  for (int n = 0; id < units; ++n, id += gridDim.x) {
    const int lo = us[n & 1].lo, hi = us[n & 1].hi;
    const size_t idx = us[n & 1].idx;
    const bool whole = lo == 0 && hi == kKv8Block;
    float* sc = reinterpret_cast<float*>(p.c.scale + idx) + half;
    int e_old = 0;
    if (lo > 0) e_old = exp_of(*sc);
    uint4* slot = reinterpret_cast<uint4*>(next) + threadIdx.x;
    uint4 x[8];
    uint32_t top, bad = 0;                 // bad: pieces of broken tokens
    cp_async_wait0();
#pragma unroll 1
    while (true) {
      // largest magnitude as an integer (bf16 bits order like their values), of each warp, then of each half
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = slot[i * 2 * D];
        m = max_abs2(max_abs2(max_abs2(max_abs2(m, x[i].x), x[i].y), x[i].z), x[i].w);
      }
      m = __reduce_max_sync(0xffffffffu, max_int16(m));
      if ((threadIdx.x & 31) == 0) red[n & 1][threadIdx.x >> 5] = m;
      __syncthreads();
      const int at = threadIdx.x & 31;
      m = at < 2 * kWarps ? red[n & 1][at] : 0u;
      top = __reduce_max_sync(0xffffffffu, at / kWarps == half ? m : 0u);
      if (__builtin_expect(!__any_sync(0xffffffffu, m >= 0x7f80u), 1)) break;
      // a token with a value that is not finite is broken in K and V and takes no part in either
      // scale: zeros in its place, and once more
      for (int i = threadIdx.x; i < kKv8Block; i += 2 * D) broken[i] = 0;
      __syncthreads();
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const uint4 y = slot[i * 2 * D];
        if (max_int16(max_abs2(max_abs2(max_abs2(max_abs2(0, y.x), y.y), y.z), y.w)) >= 0x7f80u)
          broken[piece_token(tok0, i)] = 1;
      }
      __syncthreads();
#pragma unroll 1
      for (int i = 0; i < 8; ++i)
        if (broken[piece_token(tok0, i)]) {
          bad |= 1u << i;
          slot[i * 2 * D] = make_uint4(0, 0, 0, 0);
        }
    }
    if (id + gridDim.x < units) fetch(us[(n + 1) & 1]);
    if (lo < hi) {
      const int e_need = kv8_exp(__uint_as_float(top << 16));
      if (lo == 0) e_old = e_need;
      const int e = max(e_need, e_old);
      const bool rescale = e > e_old;      // kept tokens move to the larger scale
      // x / s is exact in bf16 wherever E4M3 does not round it to zero
      const uint32_t inv = (__float_as_uint(exp2i(-e)) >> 16) * 0x10001u;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = make_uint4(mul_bf2(x[i].x, inv), mul_bf2(x[i].y, inv), mul_bf2(x[i].z, inv), mul_bf2(x[i].w, inv));
      uint8_t* blk = (half ? p.c.v : p.c.k) + idx * (static_cast<size_t>(kDs) * 64);
      if (half == 0) {
        // K: each 8-byte piece of a token goes to its panel (bits 1 and 2 of all the thread's tokens
        // are tg0's)
        uint8_t* dst = blk + (vec >> 3) * 4096 + kv8_chunk(tok0, (vec & 7) >> 1) + (vec & 1) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = piece_token(tok0, i);
          uint2 q;
          q.x = quant4(bf_lo(x[i].x), bf_hi(x[i].x), bf_lo(x[i].y), bf_hi(x[i].y));
          q.y = quant4(bf_lo(x[i].z), bf_hi(x[i].z), bf_lo(x[i].w), bf_hi(x[i].w));
          if (bad >> i & 1) q = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
          if (whole || (tok >= lo && tok < hi)) *reinterpret_cast<uint2*>(dst + piece_token(0, i) * 64) = q;
        }
        if (rescale)
          for (int i = tid; i < lo * kVec; i += D) {
            const int tok = i / kVec, v = i % kVec;
            uint2* a = reinterpret_cast<uint2*>(blk + (v >> 3) * 4096 + kv8_chunk(tok, (v & 7) >> 1) + (v & 1) * 8);
            const uint2 w = *a;
            *a = make_uint2(rescale4(w.x, exp2i(max(e_old - e, -126))), rescale4(w.y, exp2i(max(e_old - e, -126))));
          }
      } else {
        // V: four tokens x 8 dims to eight words of four tokens, through shared memory
        // (vt_word of dims 8 vec + k, taken apart)
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int d2 = 0; d2 < 4; ++d2) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 y = x[4 * g + i];
              w[i] = d2 == 0 ? y.x : d2 == 1 ? y.y : d2 == 2 ? y.z : y.w;
            }
            const int word = quad_word(tg0 + 8 * g);
            vt[vec * 128 + d2 * 32 + (word ^ vec)] = quant4(bf_lo(w[0]), bf_lo(w[1]), bf_lo(w[2]), bf_lo(w[3]));
            vt[vec * 128 + d2 * 32 + ((word + 16) ^ vec)] = quant4(bf_hi(w[0]), bf_hi(w[1]), bf_hi(w[2]), bf_hi(w[3]));
          }
        named_bar_sync(1, D);
        int from = tid;
        asm volatile("" : "+r"(from));     // (nor are the sixteen places of the words)
#pragma unroll
        for (int i = 0; i < 4; ++i) {      // 16-byte pieces (dim, t): tokens 16w + 8h + 2t + e
          const int d = (from >> 2) + i * (D / 4), t = from & 3;
          uint32_t y[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) y[w] = vt[vt_word(d, 4 * t + w)];
          uint4* a = reinterpret_cast<uint4*>(blk + kv8_chunk(d, t));
          if (!whole) {                    // a ragged block keeps its other tokens
            uint32_t m[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              m[w] = 0;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int tok = 16 * w + 8 * (c >> 1) + 2 * t + (c & 1);
                if (tok >= lo && tok < hi) m[w] |= 0xffu << (8 * c);
              }
            }
            if (!rescale && !(m[0] | m[1] | m[2] | m[3])) continue;
            const uint4 old4 = *a;
            const uint32_t old[4] = {old4.x, old4.y, old4.z, old4.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) y[w] = (y[w] & m[w]) | ((rescale ? rescale4(old[w], exp2i(max(e_old - e, -126))) : old[w]) & ~m[w]);
          }
          *a = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      if (tid == 0) *sc = exp2i(e);
    }
    // the unit after the next, which the threads fetch behind the next one's barrier (K's half
    // has less to do than V's)
    if (threadIdx.x < 32 && id + 2 * gridDim.x < units) {
      const WriteUnit c = write_unit(p, id + 2 * gridDim.x, D);
      if (threadIdx.x == 0) us[n & 1] = c;
    }
  }
}

// A write of a few tokens a row (decoding): a CTA per unit, a thread per dim of K and V, five CTAs of
// 256 an SM, so that of an ordinary append's units 740 are on the chip at once: one token of 64 x 18
// rows of 256 (1152 units) in 16 us, 29 us with the kernel above, whose blocks wait in four waves. The bytes go straight to their
// places; a block's other bytes are touched only when its scale has to grow. What is left is the
// latency of lengths, rows and scales one after the other.
constexpr int kFewTokens = 8;
template <int D>
__global__ void __launch_bounds__(D) kv8_write_few_kernel(const Kv8RowsParams p) {
  constexpr int kDs = D < 64 ? 64 : D;
  constexpr int kWarps = D / 32;
  __shared__ uint32_t red[kWarps][2][kFewTokens];
  __shared__ WriteUnit unit;
  const int d = threadIdx.x;
  if (d < 32) {
    const WriteUnit a = write_unit(p, blockIdx.x, D);
    if (d == 0) unit = a;
  }
  __syncthreads();
  const WriteUnit u = unit;
  if (u.lo >= u.hi) return;
  const int n = u.hi - u.lo;
  const long long at = u.src + u.lo * p.st_tok + d;
  uint32_t x[kFewTokens];                  // K, V << 16
#pragma unroll
  for (int i = 0; i < kFewTokens; ++i) {
    x[i] = 0;
    if (i < n)
      x[i] = reinterpret_cast<const uint16_t*>(p.k_in)[at + i * p.st_tok] |
             static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p.v_in)[at + i * p.st_tok]) << 16;
  }
  float4* sc = p.c.scale + u.idx;
  const float2 old_s = u.lo > 0 ? *reinterpret_cast<const float2*>(sc) : make_float2(0.0f, 0.0f);
  // each token's largest magnitudes as integers; not finite: broken in K and V, in neither scale
#pragma unroll
  for (int i = 0; i < kFewTokens; ++i)
    if (i < n)
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, x[i] >> (16 * kv) & 0x7fffu);
        if ((d & 31) == 0) red[d >> 5][kv][i] = m;
      }
  __syncthreads();
  uint32_t am[2] = {0, 0};
  unsigned broken = 0;
#pragma unroll
  for (int i = 0; i < kFewTokens; ++i)
    if (i < n) {
      uint32_t m[2] = {0, 0};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        m[0] = max(m[0], red[w][0][i]);
        m[1] = max(m[1], red[w][1][i]);
      }
      if (max(m[0], m[1]) >= 0x7f80u) {
        broken |= 1u << i;
      } else {
        am[0] = max(am[0], m[0]);
        am[1] = max(am[1], m[1]);
      }
    }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const int e_need = kv8_exp(__uint_as_float(am[kv] << 16));
    const int e_old = u.lo > 0 ? exp_of(kv ? old_s.y : old_s.x) : e_need;
    const int e = max(e_need, e_old);
    const float inv = exp2i(-e);
    uint8_t* blk = (kv ? p.c.v : p.c.k) + u.idx * (static_cast<size_t>(kDs) * 64);
    if (e > e_old) {                       // the kept tokens move to the larger scale
      const float fold = exp2i(max(e_old - e, -126));
      if (kv) {                            // (the thread's own dim, all 64 tokens)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          uint4* a = reinterpret_cast<uint4*>(blk + kv8_chunk(d, t));
          const uint4 w = *a;
          *a = make_uint4(rescale4(w.x, fold), rescale4(w.y, fold), rescale4(w.z, fold), rescale4(w.w, fold));
        }
      } else {
        for (int i = d; i < u.lo * (D / 8); i += D) {
          const int tok = i / (D / 8), v = i % (D / 8);
          uint2* a = reinterpret_cast<uint2*>(blk + (v >> 3) * 4096 + kv8_chunk(tok, (v & 7) >> 1) + (v & 1) * 8);
          const uint2 w = *a;
          *a = make_uint2(rescale4(w.x, fold), rescale4(w.y, fold));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kFewTokens; ++i)
      if (i < n) {
        const int tok = u.lo + i;
        uint8_t q = static_cast<uint8_t>(f2_to_e4m3x2((kv ? bf_hi(x[i]) : bf_lo(x[i])) * inv, 0.0f));
        if (broken >> i & 1) q = kv ? 0 : 0x7f;
        if (kv) {                          // token 16 w + 8 h + 2 t + e is byte 16 t + 4 w + 2 h + e of its dim
          blk[kv8_chunk(d, (tok >> 1) & 3) + 4 * (tok >> 4) + 2 * ((tok >> 3) & 1) + (tok & 1)] = q;
        } else {
          blk[(d >> 6) * 4096 + kv8_chunk(tok, (d & 63) >> 4) + (d & 15)] = q;
        }
      }
    if (d == 0) (kv ? sc->y : sc->x) = exp2i(e);
  }
}

// 2 D threads, halves and token quads as in the write, and 32 registers a thread, so that an SM is
// full (with 40: 397 us for the ragged rows above, 376 so). Values are exact in bf16 (E4M3 has
// four significant bits, the scale is a power of two).
template <int D>
__global__ void __launch_bounds__(2 * D, 1024 / D) kv8_read_kernel(const Kv8RowsParams p) {
  constexpr int kVec = D / 8;
  constexpr int kDs = D < 64 ? 64 : D;
  __shared__ uint32_t vt[D * 16];
  Unit u;
  if (!make_unit<false>(p, blockIdx.x, u)) return;
  const int half = threadIdx.x / D, tid = threadIdx.x % D;
  const int vec = tid % kVec, tg0 = tid / kVec;
  const float4 sc = p.c.scale[u.idx];
  const float s = half ? sc.y : sc.x;
  const uint8_t* blk = (half ? p.c.v : p.c.k) + u.idx * (static_cast<size_t>(kDs) * 64);
  uint2 q[8];                              // 8 dims of the tokens of quads tg0 and tg0 + 8
  if (half == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int tg = tg0 + 8 * (i >> 2), c = i & 3;
      const int tok = 16 * (tg >> 2) + 8 * (c >> 1) + 2 * (tg & 3) + (c & 1);
      q[i] = make_uint2(0, 0);
      if (tok >= u.lo && tok < u.hi)
        q[i] = *reinterpret_cast<const uint2*>(blk + (vec >> 3) * 4096 + kv8_chunk(tok, (vec & 7) >> 1) + (vec & 1) * 8);
    }
  } else {
    for (int i = tid; i < D * 4; i += D) {
      const int d = i >> 2, t = i & 3;
      const uint4 y = *reinterpret_cast<const uint4*>(blk + kv8_chunk(d, t));
      vt[vt_word(d, 4 * t)] = y.x;
      vt[vt_word(d, 4 * t + 1)] = y.y;
      vt[vt_word(d, 4 * t + 2)] = y.z;
      vt[vt_word(d, 4 * t + 3)] = y.w;
    }
    named_bar_sync(1, D);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t w[8];
#pragma unroll
      for (int d = 0; d < 8; ++d) w[d] = vt[vt_word(vec * 8 + d, quad_word(tg0 + 8 * g))];
#pragma unroll
      for (int c = 0; c < 4; ++c) {        // byte c of the eight words
        const uint32_t sel = 0x0040u + 0x0011u * c;
        const uint32_t a = __byte_perm(w[0], w[1], sel), b = __byte_perm(w[2], w[3], sel);
        const uint32_t e = __byte_perm(w[4], w[5], sel), f = __byte_perm(w[6], w[7], sel);
        q[4 * g + c] = make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(e, f, 0x5410));
      }
    }
  }
  __nv_bfloat16* dst = (half ? p.v_out : p.k_out) + u.lrow * p.st_layer + u.b * p.st_row +
                       static_cast<long long>(u.h) * D + vec * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int tg = tg0 + 8 * (i >> 2), c = i & 3;
    const int tok = 16 * (tg >> 2) + 8 * (c >> 1) + 2 * (tg & 3) + (c & 1);
    if (tok < u.lo || tok >= u.hi) continue;
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w = k < 2 ? q[i].x : q[i].y;
      const uint32_t h2 = e4m3x2_to_h2(static_cast<uint16_t>(w >> (16 * (k & 1))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * s, f.y * s);
      o[k] = *reinterpret_cast<const uint32_t*>(&r);
    }
    *reinterpret_cast<uint4*>(dst + (u.first + tok - u.lo) * p.st_tok) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

__global__ void kv8_init_kernel(float4* scale, size_t n) {
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<size_t>(gridDim.x) * blockDim.x)
    scale[i] = make_float4(exp2i(kKv8MinExp), exp2i(kKv8MinExp), 0.0f, 0.0f);
}

template <typename... Args>
static cudaError_t launch(void (*kernel)(Args...), unsigned grid, unsigned threads, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_kv8_init(const Kv8Cache& c, cudaStream_t s) {
  const size_t n = static_cast<size_t>(c.n_layers) * c.n_slots * c.n_kv * c.nblk;
  return launch(kv8_init_kernel, static_cast<unsigned>(n < 1024 * 256 ? (n + 255) / 256 : 1024), 256, s, c.scale, n);
}

static unsigned units_of(const Kv8RowsParams& p) {
  return static_cast<unsigned>(p.n_layers) * p.batch * p.c.n_kv * p.nblk_row;
}

template <int D>
static cudaError_t launch_write(const Kv8RowsParams& p, cudaStream_t s) {
  const unsigned units = units_of(p);
  if (p.n_tokens <= kFewTokens) return launch(kv8_write_few_kernel<D>, units, D, s, p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min(units, static_cast<unsigned>(p.sm_count) * kWriteCtas<D>));
  cfg.blockDim = dim3(2 * D);
  cfg.dynamicSmemBytes = kWriteSmem<D>;
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kv8_write_kernel<D>, p, units);
}

cudaError_t launch_kv8_write(const Kv8RowsParams& p, cudaStream_t s) {
  switch (p.c.D) {
    case 32: return launch_write<32>(p, s);
    case 64: return launch_write<64>(p, s);
    case 128: return launch_write<128>(p, s);
    default: return launch_write<256>(p, s);
  }
}

cudaError_t configure_kv8_store_kernels() {   // (the static 48 KB limit is passed at head_dim 256 alone)
  return cudaFuncSetAttribute(kv8_write_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize, kWriteSmem<256>);
}

cudaError_t launch_kv8_read(const Kv8RowsParams& p, cudaStream_t s) {
  switch (p.c.D) {
    case 32: return launch(kv8_read_kernel<32>, units_of(p), 64, s, p);
    case 64: return launch(kv8_read_kernel<64>, units_of(p), 128, s, p);
    case 128: return launch(kv8_read_kernel<128>, units_of(p), 256, s, p);
    default: return launch(kv8_read_kernel<256>, units_of(p), 512, s, p);
  }
}

}  // namespace vla
