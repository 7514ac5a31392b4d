// kv8_attend.cu -- attention over the 8-bit K/V cache for few query rows (a token's heads).
//
// For each row b, K/V head h and query token i, over the visible keys j:
//   o = sum_j softmax_j(scale * q . k_j) v_j,   k_j = s_K e4m3, v_j = s_V e4m3 (block scales)
// The query rows of one K/V head are its tokens times its group of heads; a tile has 8 or 16.
//
// Few rows leave the cache bytes as the bound, so the work is split over the tokens alone,
// equally over the CTAs (kv8.cuh). A CTA's warps take the blocks of 64 tokens in turn, each
// warp on its own: it copies a K block in as soon as the scores of the block that stood there
// are done and a V block after the output, with a softmax of its own (reference maximum, sum
// and outputs in registers). The warps' partial results meet in shared
// memory once per item. An item that lies in one CTA is finished there; parts of an item go to
// a workspace that a second kernel merges.
//
// The products are m16n8k16 on fp16, transposed, so that tokens and dims are the sixteen and the
// query rows the eight of an instruction: S^T = K Q^T, O^T += V^T P^T. (m16n8k32 takes E4M3
// operands, but on this architecture it is made of conversions of both operands and fp16
// products: at head_dim 128 a block took 1390 instructions, with the conversions of K and V
// written out 1070, transposed about 700. 64 ragged rows of up to 8192 tokens, 8 K/V heads of 128:
// 163 us the first way, 124 us so; one row of 200001 tokens 102 and 80 us, 79 and 78 % of the copy
// rate. The rest is the start of the kernel and the merge, some 10 us. At head_dim 256 the kernels
// have all 255 registers and spill 112 bytes a thread with 8 rows, 224 with 16.)
//   K, V widen to fp16 exactly.
//   Q: each row times the power of two that brings its largest magnitude to [128, 256): exact
//      for every bf16 value above 2^-24 of the largest.
//   P: relative to the maximum of its own 64 tokens, fp16(exp2(x - m)): off by at most 2^-11 of p
//      or 2^-25. The product of the 64 tokens is added to the output in fp32 times
//      exp2(m - M) s_V 2^-32 (M the row's reference, 2^-32 for sums of values near bf16's end).
#include <float.h>

#include "kernels.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace vla {

namespace {

// The reference is a block's largest score, rounded to an integer. It moves when passed by 2^32, or by
// less where V's scale 2^ev leaves no room for that (ev <= 120). Outputs are kept times 2^-kKv8Lift:
// sums of V's 448 * 2^ev over 2^29 keys, with a lag of 2^(kTop - ev), stay below 2^128.
constexpr int kMoveBy = 32, kTop = 121;

template <int D, int R>
struct RowsCfg {
  // Warps of a CTA, each with `slots` K and V blocks in shared memory (up to 192 KB): enough to
  // cover the latency of memory, and few enough warps that their products do not get in each
  // other's way (12 warps with a slot each: 5 % slower than 6 with two at head_dim 128).
  static constexpr int slots = D == 64 && R == 8 ? 3 : 2;
  static constexpr int warps = D == 256 ? 3 : D == 128 ? 6 : 8;
  static constexpr int block = D * 64;                            // bytes of a K or V block
  static constexpr int qfrag = D / 16 * 32 * R;                   // B fragments of Q: 8 bytes a lane, step and 8 rows
  static constexpr int cols = D < 64 ? D : 64;                    // columns of a round of the exchange
  static constexpr int q = warps * slots * 2 * block;
  static constexpr int xch = q + qfrag;                           // [warps][R rows][pitch] fp32
  static constexpr int pitch = cols + 4;                          // floats: 4 row pairs x 8 dims touch all banks
  static constexpr int ml = xch + warps * R * pitch * 4;          // [warps][R rows] (maximum, sum)
  static constexpr int rowf = ml + warps * R * 8;                 // row factors
  static constexpr int bar = rowf + 64;                           // [warps][slots] K, V
  static constexpr int total = bar + warps * slots * 16;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], const uint2& b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}
// The first of a sum.
__device__ __forceinline__ void mma_f16_0(float (&c)[4], const uint32_t (&a)[4], const uint2& b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(0.0f));
}
// An 8 x 8 matrix of halves, row g in the four lanes 4 g + t, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Four E4M3 bytes to two pairs of halves.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

}  // namespace

template <int D, int R>
__global__ void __launch_bounds__(RowsCfg<D, R>::warps * 32, 1) kv8_attend_rows_kernel(const Kv8AttendParams p) {
  using S = RowsCfg<D, R>;
  constexpr int kWarps = S::warps;
  constexpr int kN = R / 8;                     // eights of query rows
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sm = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* rowf = reinterpret_cast<float*>(smem + S::rowf);         // [R] score factors
  // slot s of this warp: its barriers for K and V, and its blocks
  auto kfull = [&](int s) { return sm + S::bar + (warp * S::slots + s) * 16; };
  auto kslot = [&](int s) { return sm + (warp * S::slots + s) * 2 * S::block; };

  if (lane == 0) {
    for (int s = 0; s < S::slots; ++s) {
      mbar_init(kfull(s), 1);
      mbar_init(kfull(s) + 8, 1);
    }
    fence_mbar_init();
  }
  if (threadIdx.x == 0) pdl_trigger();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.batch; b += blockDim.x)
      if (kv8_tile(p, b, 0).slot < 0) report(p.err, kKv8BadRow);
  __syncwarp();
  Kv8Walk w = kv8_walk(p);
  Kv8Segment g;
  bool more = kv8_next(p, w, g);

  // This warp's blocks: block `warp`, `warp` + kWarps, ... of each segment. The walk of the loads
  // runs ahead by the number of slots, over the segments' ends.
  auto item_of = [&](const Kv8Segment& x) {
    return ((static_cast<size_t>(p.layer) * p.c.n_slots + x.row.slot) * p.c.n_kv + x.head) * p.c.nblk + x.blk;
  };
  Kv8Walk wl = w;
  Kv8Segment gl = g;
  bool morel = more;
  int jl = warp;
  auto skip = [&]() {                           // to the segment of the next block to load
    while (morel && jl >= gl.n) {
      morel = kv8_next(p, wl, gl);
      jl = warp;
    }
  };
  auto load = [&](uint32_t slot, const uint8_t* from, uint32_t full) {
    if (lane == 0) {
      mbar_arrive_expect_tx(full, S::block);
      bulk_load_g2s(slot, from + (item_of(gl) + jl) * S::block, S::block, full);
    }
  };
  skip();
  for (int s = 0; s < S::slots && morel; ++s) {
    load(kslot(s), p.c.k, kfull(s));
    load(kslot(s) + S::block, p.c.v, kfull(s) + 8);
    jl += kWarps;
    skip();
  }

  // gq: row (token or dim) of an A fragment, query row of a B fragment; accumulators: rows gq and
  // gq + 8, query rows 2 t and 2 t + 1
  const int gq = lane >> 2, t = lane & 3;
  const uint32_t lane_at = gq * 64 + ((t ^ ((gq >> 1) & 3)) << 4);   // chunk t of row gq, swizzled
  int cur = 0;                                  // slot of the next block
  uint32_t phase = 0;
  bool ok = true;
  for (; more; more = kv8_next(p, w, g)) {
    // ---- Q rows to fp16, laid out as B fragments: word m of a lane's 16 dims of a panel (dims
    // 64 p + 16 t + 4 m ..) is step 4 p + m
    const int rows = min(R, g.row.cnt * p.group - g.tile * R);
    __syncthreads();                            // the last segment's readers of Q are done
    for (int r = warp; r < R; r += kWarps) {
      constexpr int kPl = D / 32;               // values a lane
      float x[kPl];
      float am = 0.0f;
      const int row = g.tile * R + r;
      const __nv_bfloat16* q = p.q + g.b * p.q_st[0] + p.by_group.div(row) * p.q_st[1] +
                               (g.head * p.group + p.by_group.mod(row)) * p.q_st[2];
#pragma unroll
      for (int i = 0; i < kPl; i += 2) {
        uint32_t v = 0;
        const int d = i * 32 + lane * 2;
        if (r < rows && d < p.c.D) v = *reinterpret_cast<const uint32_t*>(q + d);
        x[i] = __uint_as_float(v << 16);
        x[i + 1] = __uint_as_float(v & 0xffff0000u);
        if (fabsf(x[i]) < INFINITY) am = fmaxf(am, fabsf(x[i]));
        if (fabsf(x[i + 1]) < INFINITY) am = fmaxf(am, fabsf(x[i + 1]));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
      const int e = am > 0.0f ? min(max(exp_of(am) - 7, -118), 120) : 0;
      const float inv = exp2i(-e);
#pragma unroll
      for (int i = 0; i < kPl; i += 2) {
        const int d = i * 32 + lane * 2;
        const int m = (d >> 2) & 3, kk = 4 * (d >> 6) + m, tq = (d >> 4) & 3;
        const float y0 = x[i] * inv, y1 = x[i + 1] * inv;
        // an infinity becomes NaN: all its scores may be -infinity, which is no key seen
        *reinterpret_cast<uint32_t*>(smem + S::q + ((kk * kN + (r >> 3)) * 32 + (r & 7) * 4 + tq) * 8 + (d & 2) * 2) =
            pack_h2(fmaf(y0, 0.0f, y0), fmaf(y1, 0.0f, y1));
      }
      if (lane == 0) rowf[r] = exp2i(e) * p.scale_log2;
    }
    __syncthreads();

    // ---- the visible ranges of this lane's rows, and of the tile
    const int r0 = g.tile * R, last = r0 + max(rows, 1) - 1;
    int lo[kN][2], hi[kN][2], lo_first, hi_first, lo_last, hi_last;
    float f[kN][2], m[kN][2], l[kN][2];
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * n + 2 * t + c;
        kv8_seen(p, g.row, p.by_group.div(r0 + r), lo[n][c], hi[n][c]);
        f[n][c] = rowf[r];
        m[n][c] = -INFINITY;
        l[n][c] = 0.0f;
      }
    kv8_seen(p, g.row, p.by_group.div(r0), lo_first, hi_first);
    kv8_seen(p, g.row, p.by_group.div(last), lo_last, hi_last);
    // with 8 rows the fragments of Q stay in registers
    const uint2* qs = reinterpret_cast<const uint2*>(smem + S::q) + lane;
    uint2 qf[R == 8 ? D / 16 : 1];
    if (R == 8) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) qf[R == 8 ? kk : 0] = qs[kk * 32];
    }
    const float4* scales = p.c.scale + item_of(g);
    float4 next_sc = warp < g.n ? __ldg(scales + warp) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);

    float o[D / 16][kN][4];
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[j][n][c] = 0.0f;

    for (int j = warp; j < g.n; j += kWarps) {
      const int tok = (g.blk + j) * kKv8Block;
      const float4 sc = next_sc;
      if (j + kWarps < g.n) next_sc = __ldg(scales + j + kWarps);
      ok = __all_sync(0xffffffffu, ok && mbar_wait(kfull(cur), phase, p.err)) != 0;
      const uint32_t kb = kslot(cur), vb = kb + S::block;
      // ---- scores: x[h][n][c] of token tok + 16 h + gq + 8 (c >> 1), query row 8 n + 2 t + (c & 1)
      float x[4][kN][4];
#pragma unroll
      for (int pp = 0; pp < D / 64; ++pp)
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint4 k0 = lds128(kb + pp * 4096 + h * 1024 + lane_at);
          const uint4 k1 = lds128(kb + pp * 4096 + h * 1024 + 512 + lane_at);
          const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a[4];
            widen4(w0[i], a[0], a[2]);
            widen4(w1[i], a[1], a[3]);
#pragma unroll
            for (int n = 0; n < kN; ++n) {
              const uint2 b = R == 8 ? qf[R == 8 ? 4 * pp + i : 0] : qs[((4 * pp + i) * kN + n) * 32];
              if (pp == 0 && i == 0) mma_f16_0(x[h][n], a, b);
              else mma_f16(x[h][n], a, b);
            }
          }
        }
      __syncwarp();                             // the K slot is free: the next block's K
      if (morel) load(kb, p.c.k, kfull(cur));
      if (tok < lo_last || tok + kKv8Block > hi_first) {   // some row does not see all of the block
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int k = tok + 16 * h + gq + 8 * (c >> 1);
              if (k < lo[n][c & 1] || k >= hi[n][c & 1]) x[h][n][c] = -INFINITY;
            }
      }
      // ---- weights relative to the block's own maximum
      float fac[kN][2];
      uint2 pb[4][kN];                          // B fragments of the four 16-token groups
      const float lag = static_cast<float>(min(kMoveBy, kTop - exp_of(sc.y)));
      const float sv = sc.y * exp2i(-kKv8Lift);
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        float off[2], sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          // the scores in bits, rounded before the maximum is taken off: fused with that, a product of
          // 2^28 and more would miss its own rounded value by bits
          const float gk = fmaxf(f[n][c] * sc.x, FLT_MIN);  // (0 would turn a masked score into NaN)
          float ms = -INFINITY;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            x[h][n][c] = __fmul_rn(x[h][n][c], gk);
            x[h][n][c + 2] = __fmul_rn(x[h][n][c + 2], gk);
            ms = fmaxf(ms, fmaxf(x[h][n][c], x[h][n][c + 2]));
          }
#pragma unroll
          for (int i = 4; i < 32; i <<= 1) ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, i));
          const bool move = ms > m[n][c] + lag || (m[n][c] == -INFINITY && ms > m[n][c]);
          if (__any_sync(0xffffffffu, move)) {
            const float nm = move ? rintf(ms) : m[n][c];
            const float k = nm == m[n][c] ? 1.0f : exp2_approx(m[n][c] - nm);
            m[n][c] = nm;
            l[n][c] *= k;
#pragma unroll
            for (int jj = 0; jj < D / 16; ++jj) {
              o[jj][n][c] *= k;
              o[jj][n][c + 2] *= k;
            }
          }
          off[c] = ms == -INFINITY ? 0.0f : -ms;
          fac[n][c] = ms == -INFINITY ? 0.0f : exp2_approx(ms - m[n][c]);
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          float w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            w[c] = exp2_approx(x[h][n][c] + off[c & 1]);
            sum[c & 1] += w[c];
          }
          pb[h][n] = make_uint2(transpose8(pack_h2(w[0], w[1])), transpose8(pack_h2(w[2], w[3])));
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          l[n][c] = fmaf(sum[c], fac[n][c], l[n][c]);
          fac[n][c] *= sv;
        }
      }
      // ---- o += fac * P V
      ok = __all_sync(0xffffffffu, ok && mbar_wait(kfull(cur) + 8, phase, p.err)) != 0;
#pragma unroll
      for (int jj = 0; jj < D / 16; ++jj) {
        const uint4 v0 = lds128(vb + jj * 1024 + lane_at), v1 = lds128(vb + jj * 1024 + 512 + lane_at);
        const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
        float y[kN][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a[4];
          widen4(w0[i], a[0], a[2]);
          widen4(w1[i], a[1], a[3]);
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            if (i == 0) mma_f16_0(y[n], a, pb[i][n]);
            else mma_f16(y[n], a, pb[i][n]);
          }
        }
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[jj][n][c] = fmaf(y[n][c], fac[n][c & 1], o[jj][n][c]);
      }
      __syncwarp();                             // the V slot is free: the next block's V
      if (morel) {
        load(vb, p.c.v, kfull(cur) + 8);
        jl += kWarps;
        skip();
      }
      if (++cur == S::slots) {
        cur = 0;
        phase ^= 1;
      }
    }

    // ---- the warps' results
    float2* ml = reinterpret_cast<float2*>(smem + S::ml);
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], i);
        l[n][c] *= exp2i(-kKv8Lift);       // (as o: a partial result, kv8.cuh)
        if (gq == 0) ml[warp * R + 8 * n + 2 * t + c] = make_float2(m[n][c], l[n][c]);
      }
    __syncthreads();
    float fac[kN][2];
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float mm = -INFINITY;
        for (int i = 0; i < kWarps; ++i) mm = fmaxf(mm, ml[i * R + 8 * n + 2 * t + c].x);
        fac[n][c] = m[n][c] == -INFINITY ? 1.0f : exp2_approx(m[n][c] - mm);
      }
    const int slot = g.slot;
    float* xb = reinterpret_cast<float*>(smem + S::xch);
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += S::cols) {
#pragma unroll
      for (int jj = 0; jj < S::cols / 16; ++jj)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            xb[(warp * R + 8 * n + 2 * t + (c & 1)) * S::pitch + jj * 16 + gq + 8 * (c >> 1)] =
                o[c0 / 16 + jj][n][c] * fac[n][c & 1];
      __syncthreads();
      for (int i = threadIdx.x; i < rows * (S::cols / 2); i += kWarps * 32) {
        const int rr = i / (S::cols / 2), cc = (i % (S::cols / 2)) * 2, d = c0 + cc;
        float mm = -INFINITY, ll = 0.0f;
        for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, ml[k * R + rr].x);
        float2 v = make_float2(0.0f, 0.0f);
        for (int k = 0; k < kWarps; ++k) {
          const float2 y = *reinterpret_cast<const float2*>(xb + (k * R + rr) * S::pitch + cc);
          const float2 z = ml[k * R + rr];
          v.x += y.x;
          v.y += y.y;
          ll += z.y * (z.x == -INFINITY ? 1.0f : exp2_approx(z.x - mm));
        }
        const int row = r0 + rr, qi = p.by_group.div(row), qh = g.head * p.group + row - qi * p.group;
        if (!g.whole) {
          *reinterpret_cast<float2*>(p.ws + (static_cast<size_t>(slot) * R + rr) * D + d) = v;
          if (d == 0) p.ws_ml[slot * R + rr] = make_float2(mm, ll);
        } else if (d < p.c.D) {
          const float norm = ll == 0.0f ? 0.0f : 1.0f / ll;
          *reinterpret_cast<__nv_bfloat162*>(p.out + g.b * p.o_st[0] + qi * p.o_st[1] + qh * p.o_st[2] + d) =
              __floats2bfloat162_rn(v.x * norm, v.y * norm);
          if (d == 0 && p.lse) p.lse[(static_cast<size_t>(g.b) * p.n_q + qi) * p.n_heads + qh] = kv8_lse(mm, ll);
        }
      }
      __syncthreads();
    }
  }
}

// ---- merging the parts of the items that more than one CTA worked on

// An item with cuts inside.
struct Kv8Cut {
  int b, tile, head, rows;      // rows: query rows of the tile
  int c0, c1;                   // parts c0 .. c1 - 1 meet the item
};
// Of item `head` of entry e, which begins with unit u0 and has cuts from `cut` on inside if any.
__device__ __forceinline__ bool kv8_parts(const Kv8AttendParams& p, const Kv8Line& line, const Kv8Tile& row, int e,
                                          int head, int u0, int cut, Kv8Cut& r) {
  // cuts of [u0 + snap + 1, u1 - snap - 1] stay
  const int lo = u0 + line.snap, hi = u0 + row.units - line.snap;
  const int uc = kv8_begin(line, cut);
  if (cut >= p.grid || uc <= lo || uc >= hi || kv8_begin(line, cut - 1) > lo) return false;
  r.b = p.by_tiles.div(e);
  r.tile = e - r.b * p.tiles;
  r.head = head;
  r.rows = min(p.tile_rows, row.cnt * p.group - r.tile * p.tile_rows);
  r.c0 = cut - 1;
  // (parts that meet the item have units: the cuts inside an item differ)
  r.c1 = min(p.grid, cut + (line.per > 0 ? (hi - uc - 1) / line.per + 1 : hi - uc));
  while (r.c1 > cut && kv8_begin(line, r.c1 - 1) >= hi) --r.c1;
  return true;
}
// The merges' second grid axis: the items, or the cuts where these are fewer (an item belongs to
// the first cut that stays inside it).
__device__ __forceinline__ bool kv8_cut(const Kv8AttendParams& p, const Kv8Line& line, int y, Kv8Cut& r) {
  if (kv8_merge_by_items(p)) {
    const int e = y / p.c.n_kv, head = y - e * p.c.n_kv;
    const int b = p.by_tiles.div(e);
    const Kv8Tile row = kv8_tile(p, b, e - b * p.tiles);
    if (row.units == 0) return false;
    int before = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (32 * i + static_cast<int>(threadIdx.x & 31) < e) before += line.w[i];
    const int u0 = __reduce_add_sync(0xffffffffu, before) + head * row.units;
    int cut = max(1, (u0 + line.snap) / (line.per + 1));
    while (cut < p.grid && kv8_begin(line, cut) <= u0 + line.snap) ++cut;
    return kv8_parts(p, line, row, e, head, u0, cut, r);
  }
  const int cut = y + 1, uc = kv8_begin(line, cut);
  if (uc >= line.total) return false;
  int inside;
  const int e = kv8_find(p, line, uc, &inside);
  const Kv8Tile row = kv8_tile(p, p.by_tiles.div(e), p.by_tiles.mod(e));
  return kv8_parts(p, line, row, e, inside / row.units, uc - inside % row.units, cut, r);
}

constexpr int kMergeWarps = 8;

// Few rows, as a rule of many parts: a CTA per (row, cut). Each warp sums every eighth part, a
// lane D / 32 columns; the eight sums are joined in order in shared memory.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) kv8_merge_rows_kernel(const Kv8AttendParams p) {
  constexpr int W = kMergeWarps;
  constexpr int kPl = D / 32 >= 4 ? D / 32 : 4;          // columns a lane, in groups of 4
  constexpr int kLanes = D / kPl;
  constexpr int kG = kPl / 4;
  __shared__ float2 sml[W];
  __shared__ float4 so[W][kG][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.x;
  const Kv8Line line = kv8_line(p);
  Kv8Cut cut;
  const bool mine = kv8_cut(p, line, blockIdx.y, cut);
  pdl_wait();
  if (!mine || r >= cut.rows) return;
  float mm = -INFINITY, ll = 0.0f;
  float4 v[kG] = {};
  for (int c0 = cut.c0 + warp; c0 < cut.c1; c0 += 32 * W) {
    // 32 parts' maxima and sums at once, a lane each
    const int c = c0 + lane * W;
    float2 ml = make_float2(-INFINITY, 0.0f);
    int at = 0;
    if (c < cut.c1) {
      at = kv8_slot(c, c == cut.c0) * p.tile_rows + r;
      ml = p.ws_ml[at];
    }
    float nm = ml.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, o));
    nm = fmaxf(nm, mm);
    const float k = mm == -INFINITY ? 1.0f : exp2_approx(mm - nm);
    mm = nm;
    ll *= k;
#pragma unroll
    for (int i = 0; i < kG; ++i) v[i] = make_float4(v[i].x * k, v[i].y * k, v[i].z * k, v[i].w * k);
    const float f = ml.x == -INFINITY ? 1.0f : exp2_approx(ml.x - mm);
    const int n = min(32, (cut.c1 - c0 + W - 1) / W);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const int ai = __shfl_sync(0xffffffffu, at, i);
      const float fi = __shfl_sync(0xffffffffu, f, i);
      ll = fmaf(__shfl_sync(0xffffffffu, ml.y, i), fi, ll);
      if (lane < kLanes) {
        const float4* x = reinterpret_cast<const float4*>(p.ws + static_cast<size_t>(ai) * D) + lane;
#pragma unroll
        for (int j = 0; j < kG; ++j) {
          const float4 y = x[j * kLanes];
          v[j] = make_float4(fmaf(y.x, fi, v[j].x), fmaf(y.y, fi, v[j].y), fmaf(y.z, fi, v[j].z), fmaf(y.w, fi, v[j].w));
        }
      }
    }
  }
  if (lane == 0) sml[warp] = make_float2(mm, ll);
#pragma unroll
  for (int j = 0; j < kG; ++j) so[warp][j][lane] = v[j];
  __syncthreads();
  if (warp != 0) return;
  float m0 = mm;
  for (int i = 1; i < W; ++i) m0 = fmaxf(m0, sml[i].x);
  float k = mm == -INFINITY ? 1.0f : exp2_approx(mm - m0);
  ll *= k;
#pragma unroll
  for (int j = 0; j < kG; ++j) v[j] = make_float4(v[j].x * k, v[j].y * k, v[j].z * k, v[j].w * k);
  for (int i = 1; i < W; ++i) {
    const float2 y = sml[i];
    k = y.x == -INFINITY ? 1.0f : exp2_approx(y.x - m0);
    ll = fmaf(y.y, k, ll);
#pragma unroll
    for (int j = 0; j < kG; ++j) {
      const float4 z = so[i][j][lane];
      v[j] = make_float4(fmaf(z.x, k, v[j].x), fmaf(z.y, k, v[j].y), fmaf(z.z, k, v[j].z), fmaf(z.w, k, v[j].w));
    }
  }
  const int q = cut.tile * p.tile_rows + r;
  const int qi = p.by_group.div(q), qh = cut.head * p.group + p.by_group.mod(q);
  const float norm = ll == 0.0f ? 0.0f : 1.0f / ll;
  __nv_bfloat16* dst = p.out + cut.b * p.o_st[0] + qi * p.o_st[1] + qh * p.o_st[2];
  if (lane < kLanes)
#pragma unroll
    for (int j = 0; j < kG; ++j) {
      const int d = (j * kLanes + lane) * 4;
      if (d < p.c.D) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v[j].x * norm, v[j].y * norm);
        const __nv_bfloat162 y = __floats2bfloat162_rn(v[j].z * norm, v[j].w * norm);
        *reinterpret_cast<uint2*>(dst + d) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
      }
    }
  if (lane == 0 && p.lse)
    p.lse[(static_cast<size_t>(cut.b) * p.n_q + qi) * p.n_heads + qh] = kv8_lse(m0, ll);
}

// Many rows: a CTA per (32 rows, cut); a lane is a row, a warp takes D / 8 of its columns. Parts
// are laid out [D / 4][rows][4], so a warp's reads are in line.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) kv8_merge_tiles_kernel(const Kv8AttendParams p) {
  constexpr int kG = D / 4 / kMergeWarps;                // groups of four columns a thread
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.x * 32 + lane;
  const Kv8Line line = kv8_line(p);
  Kv8Cut cut;
  const bool mine = kv8_cut(p, line, blockIdx.y, cut);
  pdl_wait();
  if (!mine || r >= cut.rows) return;
  float mm = -INFINITY, ll = 0.0f;
  for (int c = cut.c0; c < cut.c1; ++c) mm = fmaxf(mm, p.ws_ml[kv8_slot(c, c == cut.c0) * p.tile_rows + r].x);
  float4 v[kG] = {};
  for (int c = cut.c0; c < cut.c1; ++c) {
    const int slot = kv8_slot(c, c == cut.c0);
    const float2 ml = p.ws_ml[slot * p.tile_rows + r];
    const float f = ml.x == -INFINITY ? 1.0f : exp2_approx(ml.x - mm);
    ll = fmaf(ml.y, f, ll);
    const float4* x = reinterpret_cast<const float4*>(p.ws + static_cast<size_t>(slot) * p.tile_rows * D) + r;
#pragma unroll
    for (int j = 0; j < kG; ++j) {
      const float4 y = x[(warp * kG + j) * p.tile_rows];
      v[j] = make_float4(fmaf(y.x, f, v[j].x), fmaf(y.y, f, v[j].y), fmaf(y.z, f, v[j].z), fmaf(y.w, f, v[j].w));
    }
  }
  const int q = cut.tile * p.tile_rows + r;
  const int qi = p.by_group.div(q), qh = cut.head * p.group + p.by_group.mod(q);
  const float norm = ll == 0.0f ? 0.0f : 1.0f / ll;
  __nv_bfloat16* dst = p.out + cut.b * p.o_st[0] + qi * p.o_st[1] + qh * p.o_st[2];
#pragma unroll
  for (int j = 0; j < kG; j += 2) {
    const int d = (warp * kG + j) * 4;
    if (d < p.c.D) {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v[j + i].x * norm, v[j + i].y * norm);
        const __nv_bfloat162 y = __floats2bfloat162_rn(v[j + i].z * norm, v[j + i].w * norm);
        o[2 * i] = *reinterpret_cast<const uint32_t*>(&x);
        o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&y);
      }
      *reinterpret_cast<uint4*>(dst + d) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  if (warp == 0 && p.lse)
    p.lse[(static_cast<size_t>(cut.b) * p.n_q + qi) * p.n_heads + qh] = kv8_lse(mm, ll);
}

// Many rows in many parts (few items, so that many CTAs share each): a CTA per (32 rows, item, 32
// columns); a lane is a row, a warp takes every eighth part, and the eight sums are joined in
// order in shared memory. (Row by row of parts, as above, 128 parts of 128 rows of 256 took 200 us.)
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) kv8_merge_parts_kernel(const Kv8AttendParams p) {
  constexpr int W = kMergeWarps;
  __shared__ float2 sml[W][32];
  __shared__ float4 so[W][8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.x * 32 + lane, g0 = blockIdx.z * 8;
  const Kv8Line line = kv8_line(p);
  Kv8Cut cut;
  const bool mine = kv8_cut(p, line, blockIdx.y, cut);
  pdl_wait();
  if (!mine || static_cast<int>(blockIdx.x) * 32 >= cut.rows) return;
  float mm = -INFINITY, ll = 0.0f;
  float4 v[8] = {};
  if (r < cut.rows)
#pragma unroll 2
    for (int c = cut.c0 + warp; c < cut.c1; c += W) {
      const int slot = kv8_slot(c, c == cut.c0);
      const float2 ml = p.ws_ml[slot * p.tile_rows + r];
      const float4* x = reinterpret_cast<const float4*>(p.ws + static_cast<size_t>(slot) * p.tile_rows * D) + r;
      const float nm = fmaxf(mm, ml.x);
      const float k = mm == -INFINITY ? 1.0f : exp2_approx(mm - nm), f = ml.x == -INFINITY ? 1.0f : exp2_approx(ml.x - nm);
      mm = nm;
      ll = fmaf(ml.y, f, ll * k);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 y = x[(g0 + j) * p.tile_rows];
        v[j] = make_float4(fmaf(y.x, f, v[j].x * k), fmaf(y.y, f, v[j].y * k), fmaf(y.z, f, v[j].z * k),
                           fmaf(y.w, f, v[j].w * k));
      }
    }
  sml[warp][lane] = make_float2(mm, ll);
#pragma unroll
  for (int j = 0; j < 8; ++j) so[warp][j][lane] = v[j];
  __syncthreads();
  if (r >= cut.rows) return;
  // this warp's four columns of the row
  mm = sml[0][lane].x;
#pragma unroll
  for (int i = 1; i < W; ++i) mm = fmaxf(mm, sml[i][lane].x);
  ll = 0.0f;
  float4 o = {};
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float2 y = sml[i][lane];
    const float k = y.x == -INFINITY ? 1.0f : exp2_approx(y.x - mm);
    const float4 z = so[i][warp][lane];
    ll = fmaf(y.y, k, ll);
    o = make_float4(fmaf(z.x, k, o.x), fmaf(z.y, k, o.y), fmaf(z.z, k, o.z), fmaf(z.w, k, o.w));
  }
  const int q = cut.tile * p.tile_rows + r;
  const int qi = p.by_group.div(q), qh = cut.head * p.group + p.by_group.mod(q);
  const float norm = ll == 0.0f ? 0.0f : 1.0f / ll;
  const int d = (g0 + warp) * 4;
  if (d < p.c.D) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * norm, o.y * norm);
    const __nv_bfloat162 y = __floats2bfloat162_rn(o.z * norm, o.w * norm);
    *reinterpret_cast<uint2*>(p.out + cut.b * p.o_st[0] + qi * p.o_st[1] + qh * p.o_st[2] + d) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
  if (d == 0 && p.lse)
    p.lse[(static_cast<size_t>(cut.b) * p.n_q + qi) * p.n_heads + qh] = kv8_lse(mm, ll);
}

template <int D>
static cudaError_t launch_merge(const Kv8AttendParams& p, cudaStream_t s) {
  if (p.grid < 2) return cudaSuccess;
  const bool few = p.tile_rows <= 16, by_items = kv8_merge_by_items(p);
  const int items = p.batch * p.tiles * p.c.n_kv;
  // more than eight CTAs to an item
  const bool parts = !few && by_items && items * 8 < p.grid;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(few ? p.tile_rows : p.tile_rows / 32, by_items ? items : p.grid - 1, parts ? D / 32 : 1);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few ? kv8_merge_rows_kernel<D> : parts ? kv8_merge_parts_kernel<D>
                                                                          : kv8_merge_tiles_kernel<D>, p);
}

cudaError_t launch_kv8_merge(const Kv8AttendParams& p, cudaStream_t s) {
  switch (p.c.Ds) {
    case 64: return launch_merge<64>(p, s);
    case 128: return launch_merge<128>(p, s);
    default: return launch_merge<256>(p, s);
  }
}

template <int D, int R>
static cudaError_t launch_rows(const Kv8AttendParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(RowsCfg<D, R>::warps * 32);
  cfg.dynamicSmemBytes = RowsCfg<D, R>::total;
  cfg.stream = s;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_attend_rows_kernel<D, R>, p);
  return e != cudaSuccess ? e : launch_kv8_merge(p, s);
}

cudaError_t launch_kv8_attend_rows(const Kv8AttendParams& p, cudaStream_t s) {
  const bool r8 = p.tile_rows == 8;
  if (p.c.Ds == 64) return r8 ? launch_rows<64, 8>(p, s) : launch_rows<64, 16>(p, s);
  if (p.c.Ds == 128) return r8 ? launch_rows<128, 8>(p, s) : launch_rows<128, 16>(p, s);
  return r8 ? launch_rows<256, 8>(p, s) : launch_rows<256, 16>(p, s);
}

template <int D, int R>
static cudaError_t configure_rows() {
  static_assert(RowsCfg<D, R>::total <= 232448, "shared memory of a CTA");
  return cudaFuncSetAttribute(kv8_attend_rows_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              RowsCfg<D, R>::total);
}

cudaError_t configure_kv8_kernels() {
  cudaError_t e;
  if ((e = configure_rows<64, 8>()) != cudaSuccess || (e = configure_rows<64, 16>()) != cudaSuccess) return e;
  if ((e = configure_rows<128, 8>()) != cudaSuccess || (e = configure_rows<128, 16>()) != cudaSuccess) return e;
  if ((e = configure_rows<256, 8>()) != cudaSuccess) return e;
  return configure_rows<256, 16>();
}

}  // namespace vla
