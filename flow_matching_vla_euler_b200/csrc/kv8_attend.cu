// kv8_attend.cu -- attention over the 8-bit K/V cache for few query rows (a token's heads).
//
// For each row b, K/V head h and query token i, over the visible keys j:
//   o = sum_j softmax_j(scale * q . k_j) v_j,   k_j = s_K e4m3, v_j = s_V e4m3 (block scales)
// The query rows of one K/V head are its tokens times its group of heads; a tile has 8 or 16.
//
// Few rows leave the cache bytes as the bound, so the work is split over the tokens alone,
// equally over the CTAs (kv8.cuh). One thread feeds a ring of 32 KB stages with TMA; eight
// warps each take 32 tokens of a stage at a time with a softmax of their own (reference
// maximum, sum and outputs in registers), and the eight partial results meet in shared memory
// once per item. An item that lies in one CTA is finished there; parts of an item go to a
// workspace that a second kernel merges.
//
// The products run on E4M3 as the cache holds it, without widening: m16n8k32 on E4M3 takes
// 3.8e3 multiply-adds a clock and SM here, m16n8k16 on fp16 1.0e3 plus two conversions for
// four values. What is not E4M3 goes in as two terms:
//   Q: each row times the power of two that brings its largest magnitude to [128, 256), then
//      hi = e4m3(q), lo = e4m3(16 (q - hi)), summed apart, s = S_hi + S_lo / 16: exact for
//      every bf16 value above 2^-14 of the largest, to 2^-21 of the largest below.
//   P: relative to the maximum of its own 32 tokens, p = 256 exp2(x - m), hi = e4m3(p),
//      lo = e4m3(16 (p - hi)): off by at most 2^-8 of p or 2^-22 of the largest of the 32. The
//      product of the 32 tokens is added to the output in fp32 times exp2(m - M) s_V.
// With 8 rows the two terms are the two halves of one 16-row instruction.
#include "kernels.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace vla {

namespace {

constexpr int kWarps = 8;                    // consumer warps; warp 8 feeds the ring
// Three warpgroups, the last one only for the ring's feeder. Registers: 168 a thread at
// launch; the feeder's group goes down to 40 and the two others up to 232
// (2 x 128 x 232 + 128 x 40 = 64512 = 384 x 168), which holds 16 x 256 outputs.
constexpr int kThreads = 384;
constexpr int kStageK = 16384;               // K bytes of a stage; V follows
constexpr int kStage = 2 * kStageK;
constexpr int kStages = 5;
constexpr float kMoveBy = 32.0f;             // the reference maximum moves when passed by 2^32

template <int D, int R>
struct RowsSmem {
  static constexpr int qfrag = D / 32 * 512 * (R / 8);            // A fragments of Q, 16 bytes a lane
  static constexpr int q = kStages * kStage;
  static constexpr int xch = q + qfrag;                           // [8 warps][R rows][columns] fp32
  static constexpr int cols = D < 1024 / R ? D : 1024 / R;         // columns of a round of the exchange
  static constexpr int ml = xch + kWarps * R * cols * 4;          // [8 warps][R rows] (maximum, sum)
  static constexpr int misc = ml + kWarps * R * 8;                // row factors, scan
  static constexpr int scale = misc + 64;                         // [stages][4 blocks] float4
  static constexpr int bar = scale + kStages * 4 * 16;
  static constexpr int total = bar + kStages * 16;
};

__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// x, y as hi + lo E4M3 pairs, lo from `up` times the rest.
__device__ __forceinline__ void split2(float x, float y, float up, uint32_t& hi, uint32_t& lo) {
  const uint16_t h = f2_to_e4m3x2(x, y);
  const uint32_t h2 = e4m3x2_to_h2(h);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
  hi = h;
  lo = f2_to_e4m3x2((x - f.x) * up, (y - f.y) * up);
}

}  // namespace

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_attend_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const Kv8AttendParams p) {
  using S = RowsSmem<D, R>;
  constexpr int kPer = 256 / D;                 // blocks of a stage
  constexpr int kSlices = 2 * kPer;             // 32-token slices of a stage
  constexpr int kRows = R / 8;                  // rows a lane holds: gq, and gq + 8 if R is 16
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sm = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* rowf = reinterpret_cast<float*>(smem + S::misc);         // [R] score factors
  const uint32_t full0 = sm + S::bar, empty0 = full0 + 8 * kStages;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, kWarps);
    }
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    pdl_trigger();
  }
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.batch; b += blockDim.x)
      if (kv8_tile(p, b, 0).slot < 0) report(p.err, kKv8BadRow);
  Kv8Walk w = kv8_walk(p);
  __syncthreads();

  Kv8Segment g;
  int it = 0;                                   // stages so far
  bool ok = true;
  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == kWarps && lane == 0) {
      const uint64_t pol = policy_evict_first();
      while (ok && kv8_next(p, w, g)) {
        const size_t item = ((static_cast<size_t>(p.layer) * p.c.n_slots + g.row.slot) * p.c.n_kv + g.head) * p.c.nblk;
        for (int j = 0; j < g.n; j += kPer, ++it) {
          const int s = it % kStages, n = min(kPer, g.n - j);
          if (it >= kStages && !mbar_wait(empty0 + 8 * s, (it / kStages - 1) & 1, p.err)) {
            ok = false;
            break;
          }
          const uint32_t full = full0 + 8 * s;
          mbar_arrive_expect_tx(full, n * (2 * D * 64 + 16));
          const size_t blk = item + g.blk + j;
          bulk_load_g2s(sm + S::scale + s * 64, p.c.scale + blk, n * 16, full);
          for (int i = 0; i < n; ++i) {
            tma_load_2d(sm + s * kStage + i * D * 64, &tm_k, full, 0, static_cast<int>((blk + i) * D), pol);
            tma_load_2d(sm + s * kStage + kStageK + i * D * 64, &tm_v, full, 0, static_cast<int>((blk + i) * D), pol);
          }
        }
      }
      // no copies left in flight: the last load of every stage has landed
      const int from = it > kStages ? it - kStages : 0;
      for (int i = from; i < it; ++i) mbar_wait(full0 + 8 * (i % kStages), (i / kStages) & 1, p.err);
    }
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");

  const int gq = lane >> 2, t = lane & 3;       // fragment row (and column of B), and quad lane
  const int swz = (gq >> 1) & 3;                // 64-byte swizzle of the rows this lane reads
  while (kv8_next(p, w, g)) {
    // ---- Q rows to E4M3 pairs, laid out as A fragments
    const int rows = min(R, g.row.cnt * p.group - g.tile * R);
    named_bar_sync(1, kWarps * 32);             // the last segment's readers of Q are done
    for (int r = warp; r < R; r += kWarps) {
      constexpr int kPl = D / 32;               // values a lane
      float x[kPl];
      float am = 0.0f;
      const int row = g.tile * R + r;
      const __nv_bfloat16* q = p.q + g.b * p.q_st[0] + (row / p.group) * p.q_st[1] +
                               (g.head * p.group + row % p.group) * p.q_st[2];
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
        const int d = i * 32 + lane * 2;        // kk: 32 dims; c: 16-byte chunk; quad lane, byte
        const int kk = d >> 5, c = (d >> 4) & 1, tq = (d >> 2) & 3, j = d & 3;
        uint32_t hi, lo;
        // an infinity has no E4M3 value: NaN, like the score it gives
        float u = x[i] * inv, v = x[i + 1] * inv;
        u = fmaf(u, 0.0f, u);
        v = fmaf(v, 0.0f, v);
        split2(u, v, 16.0f, hi, lo);
        const int at = ((r & 7) * 4 + tq) * 16 + c * 8 + j;
        if (R == 8) {
          uint8_t* a = smem + S::q + kk * 512 + at;
          *reinterpret_cast<uint16_t*>(a) = static_cast<uint16_t>(hi);
          *reinterpret_cast<uint16_t*>(a + 4) = static_cast<uint16_t>(lo);
        } else {
          uint8_t* a = smem + S::q + kk * 1024 + at + (r >> 3) * 4;
          *reinterpret_cast<uint16_t*>(a) = static_cast<uint16_t>(hi);
          *reinterpret_cast<uint16_t*>(a + 512) = static_cast<uint16_t>(lo);
        }
      }
      if (lane == 0) rowf[r] = exp2i(e) * p.scale_log2;
    }
    named_bar_sync(1, kWarps * 32);

    // ---- the visible ranges of this lane's rows, and of the tile
    const int r0 = g.tile * R, last = r0 + max(rows, 1) - 1;
    int lo[kRows], hi[kRows], lo_first, hi_first, lo_last, hi_last;
    float f[kRows], m[kRows], l[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      kv8_seen(p, g.row, (r0 + gq + 8 * r) / p.group, lo[r], hi[r]);
      f[r] = rowf[gq + 8 * r];
      m[r] = -INFINITY;
      l[r] = 0.0f;
    }
    kv8_seen(p, g.row, r0 / p.group, lo_first, hi_first);
    kv8_seen(p, g.row, last / p.group, lo_last, hi_last);
    uint4 qf[R == 8 ? D / 32 : 1];              // 8 rows: the fragments stay in registers
    const uint4* qs = reinterpret_cast<const uint4*>(smem + S::q) + lane;
    if (R == 8) {
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) qf[R == 8 ? kk : 0] = qs[kk * 32];
    }

    float o[D / 8][2 * kRows];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int c = 0; c < 2 * kRows; ++c) o[j][c] = 0.0f;

    for (int j = 0; j < g.n; j += kPer, ++it) {
      const int s = it % kStages;
      const int base = (j / kPer) * kSlices;    // the segment's slices go round the warps
      const int sl = (warp - base % kWarps + kWarps) % kWarps;
      // every warp waits for every stage and releases it, also one it has no slice of: a warp
      // that skipped a stage could take the slot's last phase for its next one
      ok = __all_sync(0xffffffffu, ok && mbar_wait(full0 + 8 * s, (it / kStages) & 1, p.err)) != 0;
      const int bi = sl >> 1, wsl = sl & 1;
      const int tok = (g.blk + j + bi) * kKv8Block + wsl * 32;
      if (ok && sl < kSlices && j + bi < g.n && tok < hi_last && tok + 32 > lo_first) {
        const uint32_t kb = sm + s * kStage + bi * D * 64 + (wsl * 32 + gq) * 64 + 4 * t;
        const uint32_t vb = sm + s * kStage + kStageK + bi * D * 64 + gq * 64 + 4 * t;
        const float4 sc = *reinterpret_cast<const float4*>(smem + S::scale + s * 64 + bi * 16);
        // ---- scores: x[h][c] of token tok + 8 h + 2 t + (c & 1), row gq + 8 (c >> 1)
        float x[4][2 * kRows];
        {
          float a[4][4] = {}, b[R == 8 ? 1 : 4][4] = {};
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {
            uint4 qa, qb;
            if (R == 8) {
              qa = qf[R == 8 ? kk : 0];
            } else {
              qa = qs[kk * 64];
              qb = qs[kk * 64 + 32];
            }
            const uint32_t k0 = (kk >> 1) * 4096 + (((2 * (kk & 1)) ^ swz) << 4);
            const uint32_t k1 = (kk >> 1) * 4096 + (((2 * (kk & 1) + 1) ^ swz) << 4);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const uint32_t b0 = lds32(kb + k0 + h * 512), b1 = lds32(kb + k1 + h * 512);
              mma_e4m3(a[h], qa, b0, b1);
              if (R != 8) mma_e4m3(b[R == 8 ? 0 : h], qb, b0, b1);
            }
          }
#pragma unroll
          for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int c = 0; c < 2 * kRows; ++c)
              x[h][c] = R == 8 ? fmaf(a[h][c + 2], 0.0625f, a[h][c])
                               : fmaf(b[R == 8 ? 0 : h][c], 0.0625f, a[h][c]);
        }
        if (tok < lo_last || tok + 32 > hi_first) {      // some row does not see all of the slice
#pragma unroll
          for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int c = 0; c < 2 * kRows; ++c) {
              const int k = tok + 8 * h + 2 * t + (c & 1), r = c >> 1;
              if (k < lo[r] || k >= hi[r]) x[h][c] = -INFINITY;
            }
        }
        // ---- weights relative to the slice's own maximum
        float fac[kRows];
        uint4 ph, pl;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          float mx = -INFINITY;
#pragma unroll
          for (int h = 0; h < 4; ++h) mx = fmaxf(mx, fmaxf(x[h][2 * r], x[h][2 * r + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float gk = f[r] * sc.x, ms = mx * gk;
          const bool move = ms > m[r] + kMoveBy || (m[r] == -INFINITY && ms > m[r]);
          if (__any_sync(0xffffffffu, move)) {
            const float nm = move ? ms : m[r];
            const float k = nm == m[r] ? 1.0f : exp2_approx(m[r] - nm);
            m[r] = nm;
            l[r] *= k;
#pragma unroll
            for (int jj = 0; jj < D / 8; ++jj) {
              o[jj][2 * r] *= k;
              o[jj][2 * r + 1] *= k;
            }
          }
          const float off = ms == -INFINITY ? 0.0f : 8.0f - ms;
          float sum = 0.0f;
          uint32_t wh[4], wl[4];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const float u = exp2_approx(fmaf(x[h][2 * r], gk, off)), v = exp2_approx(fmaf(x[h][2 * r + 1], gk, off));
            sum += u + v;
            split2(u, v, 16.0f, wh[h], wl[h]);
          }
          const float k = ms == -INFINITY ? 0.0f : exp2_approx(ms - m[r] - 8.0f);
          l[r] = fmaf(sum, k, l[r]);
          fac[r] = k * sc.y;
          const uint32_t h0 = wh[0] | (wh[1] << 16), h1 = wh[2] | (wh[3] << 16);
          const uint32_t l0 = wl[0] | (wl[1] << 16), l1 = wl[2] | (wl[3] << 16);
          if (R == 8) {
            ph = make_uint4(h0, l0, h1, l1);
          } else if (r == 0) {
            ph.x = h0;
            ph.z = h1;
            pl.x = l0;
            pl.z = l1;
          } else {
            ph.y = h0;
            ph.w = h1;
            pl.y = l0;
            pl.w = l1;
          }
        }
        // ---- o += fac * P V
        const uint32_t v0 = vb + (((2 * wsl) ^ swz) << 4), v1 = vb + (((2 * wsl + 1) ^ swz) << 4);
#pragma unroll
        for (int jj = 0; jj < D / 8; ++jj) {
          const uint32_t b0 = lds32(v0 + jj * 512), b1 = lds32(v1 + jj * 512);
          float y[4] = {};
          if (R != 8) {
            mma_e4m3(y, pl, b0, b1);
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] *= 0.0625f;
          }
          mma_e4m3(y, ph, b0, b1);
          if (R == 8) {
            o[jj][0] = fmaf(fmaf(y[2], 0.0625f, y[0]), fac[0], o[jj][0]);
            o[jj][1] = fmaf(fmaf(y[3], 0.0625f, y[1]), fac[0], o[jj][1]);
          } else {
#pragma unroll
            for (int c = 0; c < 2 * kRows; ++c) o[jj][c] = fmaf(y[c], fac[c >> 1], o[jj][c]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * s);
    }

    // ---- the eight warps' results
    float2* ml = reinterpret_cast<float2*>(smem + S::ml);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (t == 0) ml[warp * R + gq + 8 * r] = make_float2(m[r], l[r]);
    }
    named_bar_sync(1, kWarps * 32);
    float fac[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float mm = -INFINITY;
      for (int i = 0; i < kWarps; ++i) mm = fmaxf(mm, ml[i * R + gq + 8 * r].x);
      fac[r] = m[r] == -INFINITY ? 1.0f : exp2_approx(m[r] - mm);
    }
    // this thread's output: row rr, kCols columns of each round of S::cols
    constexpr int kCols = R * S::cols / (kWarps * 32);
    const int rr = threadIdx.x / (S::cols / kCols), cc = (threadIdx.x % (S::cols / kCols)) * kCols;
    float mm = -INFINITY, ll = 0.0f;
    for (int i = 0; i < kWarps; ++i) mm = fmaxf(mm, ml[i * R + rr].x);
    for (int i = 0; i < kWarps; ++i) {
      const float2 v = ml[i * R + rr];
      ll += v.y * (v.x == -INFINITY ? 1.0f : exp2_approx(v.x - mm));
    }
    const float norm = ll == 0.0f ? 0.0f : 1.0f / ll;
    const int row = r0 + rr;
    const int qi = row / p.group, qh = g.head * p.group + row % p.group;
    const int slot = 2 * blockIdx.x + (g.first ? 0 : 1);
    float* ws = p.ws + (static_cast<size_t>(slot) * R + rr) * D;
    __nv_bfloat16* dst = p.out + g.b * p.o_st[0] + qi * p.o_st[1] + qh * p.o_st[2];
    float* xb = reinterpret_cast<float*>(smem + S::xch);
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += S::cols) {
#pragma unroll
      for (int jj = 0; jj < S::cols / 8; ++jj)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          *reinterpret_cast<float2*>(xb + (warp * R + gq + 8 * r) * S::cols + jj * 8 + 2 * t) =
              make_float2(o[c0 / 8 + jj][2 * r] * fac[r], o[c0 / 8 + jj][2 * r + 1] * fac[r]);
      named_bar_sync(1, kWarps * 32);
      if (rr < rows) {
        float v[kCols] = {};
#pragma unroll
        for (int i = 0; i < kWarps; ++i)
#pragma unroll
          for (int c = 0; c < kCols; ++c) v[c] += xb[(i * R + rr) * S::cols + cc + c];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const int d = c0 + cc + c;
          if (!g.whole) ws[d] = v[c];
          else if (d < p.c.D) dst[d] = __float2bfloat16_rn(v[c] * norm);
        }
      }
      named_bar_sync(1, kWarps * 32);
    }
    if (cc == 0 && rr < rows) {
      if (!g.whole)
        p.ws_ml[slot * R + rr] = make_float2(mm, ll);
      else if (p.lse)
        p.lse[(static_cast<size_t>(g.b) * p.n_q + qi) * p.n_heads + qh] =
            ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
    }
  }
}

// Merges the parts of the items that more than one CTA worked on. CTA (x, y) looks at the cut
// before part y + 1: if it is the first cut inside an item, it merges kMergeWarps / W rows of
// that item, W warps a row (W = 1 for the many rows of few parts, all for few rows of many
// parts): each warp sums every W-th part, a lane D / 32 columns, and the W sums are joined in
// order in shared memory.
constexpr int kMergeWarps = 8;
template <int D, int W>
__global__ void __launch_bounds__(kMergeWarps * 32) kv8_merge_kernel(const Kv8AttendParams p) {
  constexpr int kPl = D / 32 >= 4 ? D / 32 : 4;          // columns a lane, in groups of 4
  constexpr int kLanes = D / kPl;
  constexpr int kG = kPl / 4;
  __shared__ float2 sml[kMergeWarps];
  __shared__ float4 so[W > 1 ? kMergeWarps : 1][kG][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Kv8Line line = kv8_line(p);
  const int cut = blockIdx.y + 1, uc = kv8_begin(line, cut);
  int inside = 0, e = 0, u0 = uc, u1 = uc;
  Kv8Tile row{};
  if (uc < line.total) {
    e = kv8_find(p, line, uc, &inside);
    row = kv8_tile(p, e / p.tiles, e % p.tiles);
    u0 = uc - inside % row.units;
    u1 = u0 + row.units;
  }
  pdl_wait();
  // the first cut inside the item (parts without units have their cuts at the same unit)
  if (uc == u0 || kv8_begin(line, cut - 1) > u0) return;
  const int b = e / p.tiles, tile = e % p.tiles, head = inside / row.units;
  const int rows = min(p.tile_rows, row.cnt * p.group - tile * p.tile_rows);
  const int r = blockIdx.x * (kMergeWarps / W) + warp / W, share = warp % W;
  if (blockIdx.x * (kMergeWarps / W) >= rows) return;
  // parts cut - 1 .. c1 - 1 meet the item; all have units, as the cuts inside an item differ
  int c1 = min(p.grid, cut + (line.per > 0 ? (u1 - uc - 1) / line.per + 1 : u1 - uc));
  while (c1 > cut && kv8_begin(line, c1 - 1) >= u1) --c1;
  float mm = -INFINITY, ll = 0.0f;
  float4 v[kG] = {};
  if (r < rows) {
    for (int c0 = cut - 1 + share; c0 < c1; c0 += 32 * W) {
      // 32 parts' maxima and sums at once, a lane each
      const int c = c0 + lane * W;
      float2 ml = make_float2(-INFINITY, 0.0f);
      int at = 0;
      if (c < c1) {
        // the item in which a CTA's range starts is its first; one that starts later, its second
        at = (2 * c + (kv8_begin(line, c) >= u0 ? 0 : 1)) * p.tile_rows + r;
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
      const int n = min(32, (c1 - c0 + W - 1) / W);
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
  }
  if (W > 1) {
    if (lane == 0) sml[warp] = make_float2(mm, ll);
#pragma unroll
    for (int j = 0; j < kG; ++j) so[W > 1 ? warp : 0][j][lane] = v[j];
    __syncthreads();
    if (share != 0 || r >= rows) return;
    float m0 = mm;
    for (int i = 1; i < W; ++i) m0 = fmaxf(m0, sml[warp + i].x);
    float k = mm == -INFINITY ? 1.0f : exp2_approx(mm - m0);
    ll *= k;
#pragma unroll
    for (int j = 0; j < kG; ++j) v[j] = make_float4(v[j].x * k, v[j].y * k, v[j].z * k, v[j].w * k);
    for (int i = 1; i < W; ++i) {
      const float2 y = sml[warp + i];
      k = y.x == -INFINITY ? 1.0f : exp2_approx(y.x - m0);
      ll = fmaf(y.y, k, ll);
#pragma unroll
      for (int j = 0; j < kG; ++j) {
        const float4 z = so[W > 1 ? warp + i : 0][j][lane];
        v[j] = make_float4(fmaf(z.x, k, v[j].x), fmaf(z.y, k, v[j].y), fmaf(z.z, k, v[j].z), fmaf(z.w, k, v[j].w));
      }
    }
    mm = m0;
  }
  if (r >= rows) return;
  const int q = tile * p.tile_rows + r;
  const int qi = q / p.group, qh = head * p.group + q % p.group;
  const float norm = ll == 0.0f ? 0.0f : 1.0f / ll;
  __nv_bfloat16* dst = p.out + b * p.o_st[0] + qi * p.o_st[1] + qh * p.o_st[2];
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
    p.lse[(static_cast<size_t>(b) * p.n_q + qi) * p.n_heads + qh] =
        ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
}

template <int D, int W>
static cudaError_t launch_merge(const Kv8AttendParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.tile_rows + kMergeWarps / W - 1) / (kMergeWarps / W), p.grid - 1);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_merge_kernel<D, W>, p);
}

cudaError_t launch_kv8_merge(const Kv8AttendParams& p, cudaStream_t s) {
  if (p.grid < 2) return cudaSuccess;
  const bool few = p.tile_rows <= 16;
  if (p.c.Ds == 64) return few ? launch_merge<64, 8>(p, s) : launch_merge<64, 1>(p, s);
  if (p.c.Ds == 128) return few ? launch_merge<128, 8>(p, s) : launch_merge<128, 1>(p, s);
  return few ? launch_merge<256, 8>(p, s) : launch_merge<256, 1>(p, s);
}

template <int D, int R>
static cudaError_t launch_rows(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Kv8AttendParams& p,
                               cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = RowsSmem<D, R>::total + 1024;
  cfg.stream = s;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_attend_rows_kernel<D, R>, tm_k, tm_v, p);
  return e != cudaSuccess ? e : launch_kv8_merge(p, s);
}

cudaError_t launch_kv8_attend_rows(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Kv8AttendParams& p,
                                   cudaStream_t s) {
  const bool r8 = p.tile_rows == 8;
  if (p.c.Ds == 64) return r8 ? launch_rows<64, 8>(tm_k, tm_v, p, s) : launch_rows<64, 16>(tm_k, tm_v, p, s);
  if (p.c.Ds == 128) return r8 ? launch_rows<128, 8>(tm_k, tm_v, p, s) : launch_rows<128, 16>(tm_k, tm_v, p, s);
  return r8 ? launch_rows<256, 8>(tm_k, tm_v, p, s) : launch_rows<256, 16>(tm_k, tm_v, p, s);
}

template <int D, int R>
static cudaError_t configure_rows() {
  static_assert(RowsSmem<D, R>::total + 1024 <= 232448, "shared memory of a CTA");
  return cudaFuncSetAttribute(kv8_attend_rows_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              RowsSmem<D, R>::total + 1024);
}

cudaError_t configure_kv8_kernels() {
  cudaError_t e;
  if ((e = configure_rows<64, 8>()) != cudaSuccess || (e = configure_rows<64, 16>()) != cudaSuccess) return e;
  if ((e = configure_rows<128, 8>()) != cudaSuccess || (e = configure_rows<128, 16>()) != cudaSuccess) return e;
  if ((e = configure_rows<256, 8>()) != cudaSuccess) return e;
  return configure_rows<256, 16>();
}

}  // namespace vla
