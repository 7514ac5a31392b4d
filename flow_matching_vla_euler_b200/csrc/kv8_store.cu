// kv8_store.cu -- the 8-bit K/V cache: quantising K/V rows as they are written, and reading
// them back to bf16.
//
// A block of 64 tokens of one (layer, slot, K/V head) has one scale for K and one for V, the
// smallest power of two s >= 2^-60 with amax / s <= 448. A power of two costs E4M3 nothing
// (its step is relative) and makes x / s exact, so that storing is one rounding to nearest
// even. A write that begins inside a block keeps the block's earlier tokens: its scale can
// only grow, and the kept tokens move by an exact shift of exponents (only values that reach
// E4M3's subnormals round again).
#include "kernels.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace vla {

namespace {

// Unit of work: one block of one (layer, row, K/V head). Units of a launch are numbered with
// the block innermost, so that neighbouring CTAs read neighbouring tokens.
struct Unit {
  int l, b, h, slot, blk;        // layer (absolute), row, head, slot, block of the slot
  int lo, hi;                    // tokens of the block that are written or read
  int first;                     // token of the row that stands at `lo`
  size_t idx;                    // block number in the cache
  int lrow;                      // layer of the bf16 side (from 0)
};

// false: nothing to do (past the row's end, or a refused row).
template <bool kWrite>
__device__ __forceinline__ bool make_unit(const Kv8RowsParams& p, Unit& u) {
  unsigned id = blockIdx.x;
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
    int dup = 0;
    for (int i = threadIdx.x; i < u.b; i += blockDim.x) dup |= p.slots[i] == u.slot;
    bad |= __syncthreads_or(dup) != 0;
  }
  if (bad) {
    if (threadIdx.x == 0) report(p.err, kKv8BadRow);
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

// 2 D threads: the first half holds the block's K, the second its V. Thread (vec, tg) of a
// half keeps 8 dims of the tokens tg and tg + 8 of the sixteen token quads (2t, 2t+1, 2t+8,
// 2t+9 of a 16-token group): 8 loads of 16 bytes, all in flight before the first maximum,
// so the data is read once and the maximum and the rounding work on registers.
template <int D>
__global__ void __launch_bounds__(2 * D) kv8_write_kernel(const Kv8RowsParams p) {
  constexpr int kVec = D / 8;              // 16-byte pieces of a token
  constexpr int kDs = D < 64 ? 64 : D;
  __shared__ uint32_t vt[D * 16];          // transposed V block
  __shared__ float red[2][(2 * D + 31) / 32];
  __shared__ int broken[kKv8Block];        // token of the block with a value that is not finite
  Unit u;
  if (!make_unit<true>(p, u)) return;
  const int half = threadIdx.x / D, tid = threadIdx.x % D;
  const int vec = tid % kVec, tg0 = tid / kVec;          // tg0 < 8
  const __nv_bfloat16* src = (half ? p.v_in : p.k_in) + u.lrow * p.st_layer + u.b * p.st_row +
                             static_cast<long long>(u.h) * D + vec * 8;
  for (int i = threadIdx.x; i < kKv8Block; i += 2 * D) broken[i] = 0;
  uint4 x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int tg = tg0 + 8 * (i >> 2), c = i & 3;
    const int tok = 16 * (tg >> 2) + 8 * (c >> 1) + 2 * (tg & 3) + (c & 1);
    x[i] = make_uint4(0, 0, 0, 0);
    if (tok >= u.lo && tok < u.hi)
      x[i] = *reinterpret_cast<const uint4*>(src + (u.first + tok - u.lo) * p.st_tok);
  }
  float4* sc = p.c.scale + u.idx;
  const float old_s = u.lo > 0 ? (half ? sc->y : sc->x) : 0.0f;
  __syncthreads();
  // largest magnitude as an integer (bf16 bits order like their values); a token with a value
  // that is not finite is broken in K and V and takes no part in either scale
  uint32_t mx[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w[4] = {x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu, x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu};
    const uint32_t m2 = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
    mx[i] = max(m2 & 0xffffu, m2 >> 16);
    const int tg = tg0 + 8 * (i >> 2), c = i & 3;
    if (mx[i] >= 0x7f80u) broken[16 * (tg >> 2) + 8 * (c >> 1) + 2 * (tg & 3) + (c & 1)] = 1;
  }
  __syncthreads();
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int tg = tg0 + 8 * (i >> 2), c = i & 3;
    if (!broken[16 * (tg >> 2) + 8 * (c >> 1) + 2 * (tg & 3) + (c & 1)]) am = max(am, mx[i]);
  }
  am = __reduce_max_sync(0xffffffffu, am);
  if ((threadIdx.x & 31) == 0) red[half][(threadIdx.x % D) >> 5] = __uint_as_float(am << 16);
  __syncthreads();
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < (D + 31) / 32; ++i) amax = fmaxf(amax, red[half][i]);
  int e = kv8_exp(amax);
  const int e_old = u.lo > 0 ? exp_of(old_s) : e;
  const int e_need = e;
  e = max(e, e_old);
  const bool rescale = u.lo > 0 && e_need > e_old;       // kept tokens move to the larger scale
  const float inv = exp2i(-e), fold = exp2i(max(e_old - e, -126));
  uint8_t* blk = (half ? p.c.v : p.c.k) + u.idx * (static_cast<size_t>(kDs) * 64);
  if (half == 0) {
    // K: each 8-byte piece of a token goes to its panel
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int tg = tg0 + 8 * (i >> 2), c = i & 3;
      const int tok = 16 * (tg >> 2) + 8 * (c >> 1) + 2 * (tg & 3) + (c & 1);
      if (tok < u.lo || tok >= u.hi) continue;
      uint2 q;
      q.x = quant4(bf_lo(x[i].x) * inv, bf_hi(x[i].x) * inv, bf_lo(x[i].y) * inv, bf_hi(x[i].y) * inv);
      q.y = quant4(bf_lo(x[i].z) * inv, bf_hi(x[i].z) * inv, bf_lo(x[i].w) * inv, bf_hi(x[i].w) * inv);
      if (broken[tok]) q = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
      *reinterpret_cast<uint2*>(blk + (vec >> 3) * 4096 + kv8_chunk(tok, (vec & 7) >> 1) + (vec & 1) * 8) = q;
    }
    if (rescale)
      for (int i = tid; i < u.lo * kVec; i += D) {
        const int tok = i / kVec, v = i % kVec;
        uint2* a = reinterpret_cast<uint2*>(blk + (v >> 3) * 4096 + kv8_chunk(tok, (v & 7) >> 1) + (v & 1) * 8);
        const uint2 w = *a;
        *a = make_uint2(rescale4(w.x, fold), rescale4(w.y, fold));
      }
    if (tid == 0) sc->x = exp2i(e);
  } else {
    // V: four tokens x 8 dims to eight words of four tokens, through shared memory
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int tg = tg0 + 8 * g;
      const int t0 = 16 * (tg >> 2) + 2 * (tg & 3);
      const uint32_t keep = (broken[t0] ? 0u : 0xffu) | (broken[t0 + 1] ? 0u : 0xff00u) |
                            (broken[t0 + 8] ? 0u : 0xff0000u) | (broken[t0 + 9] ? 0u : 0xff000000u);
#pragma unroll
      for (int d2 = 0; d2 < 4; ++d2) {
        float a[4], c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 y = x[4 * g + i];
          const uint32_t w = d2 == 0 ? y.x : d2 == 1 ? y.y : d2 == 2 ? y.z : y.w;
          a[i] = bf_lo(w) * inv;
          c[i] = bf_hi(w) * inv;
        }
        const int d = vec * 8 + 2 * d2;
        vt[vt_word(d, quad_word(tg))] = quant4(a[0], a[1], a[2], a[3]) & keep;
        vt[vt_word(d + 1, quad_word(tg))] = quant4(c[0], c[1], c[2], c[3]) & keep;
      }
    }
    named_bar_sync(1, D);
    const bool whole = u.lo == 0 && u.hi == kKv8Block;
    for (int i = tid; i < D * 4; i += D) {               // 16-byte pieces (dim, t): tokens 16w + 8h + 2t + e
      const int d = i >> 2, t = i & 3;
      uint32_t y[4], m[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        y[w] = vt[vt_word(d, 4 * t + w)];
        m[w] = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int tok = 16 * w + 8 * (c >> 1) + 2 * t + (c & 1);
          if (tok >= u.lo && tok < u.hi) m[w] |= 0xffu << (8 * c);
        }
      }
      if (!whole && !rescale && !(m[0] | m[1] | m[2] | m[3])) continue;
      uint4* a = reinterpret_cast<uint4*>(blk + kv8_chunk(d, t));
      if (!whole) {                                      // a ragged block keeps its other tokens
        const uint4 old4 = *a;
        const uint32_t old[4] = {old4.x, old4.y, old4.z, old4.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) y[w] = (y[w] & m[w]) | ((rescale ? rescale4(old[w], fold) : old[w]) & ~m[w]);
      }
      *a = make_uint4(y[0], y[1], y[2], y[3]);
    }
    if (tid == 0) sc->y = exp2i(e);
  }
}

// 2 D threads, halves and token quads as in the write. Values are exact in bf16 (E4M3 has
// four significant bits, the scale is a power of two).
template <int D>
__global__ void __launch_bounds__(2 * D) kv8_read_kernel(const Kv8RowsParams p) {
  constexpr int kVec = D / 8;
  constexpr int kDs = D < 64 ? 64 : D;
  __shared__ uint32_t vt[D * 16];
  Unit u;
  if (!make_unit<false>(p, u)) return;
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

cudaError_t launch_kv8_write(const Kv8RowsParams& p, cudaStream_t s) {
  switch (p.c.D) {
    case 32: return launch(kv8_write_kernel<32>, units_of(p), 64, s, p);
    case 64: return launch(kv8_write_kernel<64>, units_of(p), 128, s, p);
    case 128: return launch(kv8_write_kernel<128>, units_of(p), 256, s, p);
    default: return launch(kv8_write_kernel<256>, units_of(p), 512, s, p);
  }
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
