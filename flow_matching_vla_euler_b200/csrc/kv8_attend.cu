// kv8_attend.cu -- attention over the 8-bit K/V cache for few query rows.
//
// For each row b, K/V head h and query token i, over the visible keys j:
//   o = sum_j softmax_j(scale * q . k_j) v_j,   k_j = s_K e4m3, v_j = s_V e4m3 (block scales)
// The query rows of one K/V head are its tokens times its group of heads; a tile has 16.
//
// Few rows leave the cache bytes as the bound, so the work is split over the tokens alone:
// the blocks of all (row, head, tile) items in a line are cut into equal parts, one per CTA
// (grid <= SMs), whatever the rows' lengths. One warp feeds a ring of 32 KB stages with TMA;
// eight warps each take 16 tokens of a stage at a time with a softmax of their own (running
// maximum, sum and 16 x D output in registers), and the eight partial results meet in shared
// memory once per item. An item that lies in one CTA is finished there; parts of an item go
// to a workspace that a second kernel merges.
//
// Numbers: E4M3 widens to fp16 exactly. Q (bf16) becomes fp16 after a power of two for each
// row brings its largest magnitude to [128, 256): exact for every value above 2^-24 of that.
// The V scale enters through the exponent: the running maximum is that of s + log2(s_V), so
// the weight fp16(exp2(s + log2 s_V - m)) carries it, and the sum of weights takes it out
// again in fp32. The weight's rounding to fp16 (2^-11) is the only one before the output's.
#include "kernels.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace vla {

namespace {

constexpr int kRows = 16;                    // query rows of a tile
constexpr int kWarps = 8;                    // consumer warps; warp 8 feeds the ring
// Threads of a CTA: three warpgroups, the last one only for the ring's feeder. Registers: 168
// a thread at launch; the feeder's group goes down to 40 and the two others up to 224
// (2 x 128 x 224 + 128 x 40 = 62464 of 384 x 168 = 64512), which holds 16 x 256 outputs.
constexpr int kThreads = 384;
constexpr int kStageK = 16384;               // K bytes of a stage; V follows
constexpr int kStage = 2 * kStageK;
constexpr int kStages = 6;

template <int D>
struct RowsSmem {
  static constexpr int qpitch = D * 2 + 32;                       // bytes: 4 rows x 32 bytes touch all banks
  static constexpr int q = kStages * kStage;
  static constexpr int xch = q + kRows * qpitch;                  // [8 warps][16 rows][32 columns] fp32
  static constexpr int ml = xch + kWarps * kRows * 32 * 4;        // [8 warps][16 rows] (maximum, sum)
  static constexpr int misc = ml + kWarps * kRows * 8;            // row factors, limits, scan
  static constexpr int scale = misc + 1024;                       // [stages][4 blocks] float4
  static constexpr int bar = scale + kStages * 4 * 16;
  static constexpr int total = bar + kStages * 16;
};

// Where a CTA's part of the work begins: the row, the unit inside the row, and the number of
// units left. A row's units are (K/V head, tile, block), block innermost.
struct Part {
  int b;
  long long unit, left, total;
};

// Sum over the CTA's threads, the same value in all of them (red: one slot per warp).
__device__ __forceinline__ long long cta_sum(long long v, long long* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  long long s = 0;
  for (int i = 0; i < static_cast<int>(blockDim.x + 31) / 32; ++i) s += red[i];
  return s;
}

// First unit of CTA c when `total` units are cut into `grid` parts.
__device__ __forceinline__ long long part_begin(long long total, int grid, int c) { return total * c / grid; }

// Units of all rows before row b (b = batch: of all rows).
__device__ __forceinline__ long long units_before(const Kv8AttendParams& p, int b, int per, long long* red) {
  long long n = 0;
  for (int i = threadIdx.x; i < b; i += blockDim.x) n += kv8_row(p, i).nblk;
  return cta_sum(n, red) * per;
}

__device__ __forceinline__ Part find_part(const Kv8AttendParams& p, int per, long long* red) {
  Part r;
  r.total = units_before(p, p.batch, per, red);
  const long long u0 = part_begin(r.total, gridDim.x, blockIdx.x);
  r.left = part_begin(r.total, gridDim.x, blockIdx.x + 1) - u0;
  r.b = 0;
  r.unit = 0;
  if (r.left == 0) return r;
  // chunks of rows until the one that holds u0, then row by row
  long long at = 0;
  int b = 0;
  while (b + 32 < p.batch) {
    long long n = static_cast<long long>(kv8_row(p, b + (threadIdx.x & 31)).nblk) * per;
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (at + n > u0) break;
    at += n;
    b += 32;
  }
  long long mine = b + static_cast<int>(threadIdx.x & 31) < p.batch
                       ? static_cast<long long>(kv8_row(p, b + (threadIdx.x & 31)).nblk) * per : 0;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (static_cast<int>(threadIdx.x & 31) >= o) inc += v;
  }
  const unsigned past = __ballot_sync(0xffffffffu, at + inc > u0);
  const int k = __ffs(past) - 1;
  r.b = b + k;
  r.unit = u0 - (at + __shfl_sync(0xffffffffu, inc - mine, k));
  return r;
}

// The segments of a CTA's part: maximal runs of blocks of one item.
struct Segment {
  Kv8Row row;
  int b, head, tile, blk, n;      // blocks [blk, blk + n) of the slot
  bool whole, first;              // the item's only part; the part that starts the CTA's range
};

struct Walk {
  Part at;
  Kv8Row row;
  bool begun = false;
};

__device__ __forceinline__ bool next_segment(const Kv8AttendParams& p, int per, Walk& w, Segment& g) {
  if (w.at.left == 0) return false;
  if (!w.begun) w.row = kv8_row(p, w.at.b);
  while (w.at.unit >= static_cast<long long>(w.row.nblk) * per) {
    w.at.unit = 0;
    w.row = kv8_row(p, ++w.at.b);
  }
  const int item = static_cast<int>(w.at.unit / w.row.nblk), off = static_cast<int>(w.at.unit % w.row.nblk);
  g.row = w.row;
  g.b = w.at.b;
  g.head = item / p.tiles;
  g.tile = item % p.tiles;
  g.blk = w.row.blk0 + off;
  g.n = static_cast<int>(min(static_cast<long long>(w.row.nblk - off), w.at.left));
  g.whole = off == 0 && g.n == w.row.nblk;
  g.first = !w.begun;
  w.begun = true;
  w.at.unit += g.n;
  w.at.left -= g.n;
  return true;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_attend_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const Kv8AttendParams p) {
  using S = RowsSmem<D>;
  constexpr int kPer = 256 / D;                 // blocks of a stage
  constexpr int kSlices = 4 * kPer;             // 16-token slices of a stage
  constexpr int kArrive = kSlices < kWarps ? kSlices : kWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sm = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* rowf = reinterpret_cast<float*>(smem + S::misc);         // [16] score factors
  long long* red = reinterpret_cast<long long*>(smem + S::misc + 64);
  const uint32_t full0 = sm + S::bar, empty0 = full0 + 8 * kStages;
  const int per = p.c.n_kv * p.tiles;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, kArrive);
    }
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    pdl_trigger();
  }
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.batch; b += blockDim.x)
      if (kv8_row(p, b).slot < 0) report(p.err, kKv8BadRow);
  Walk w;
  w.at = find_part(p, per, red);
  __syncthreads();

  Segment g;
  int it = 0;                                   // stages so far
  bool ok = true;
  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == kWarps && lane == 0) {
      const uint64_t pol = policy_evict_first();
      while (ok && next_segment(p, per, w, g)) {
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
  asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");

  const int gq = lane >> 2, t = lane & 3;       // fragment row (and column of B), and quad lane
  const int swz = (gq >> 1) & 3;                // 64-byte swizzle of the rows this lane reads
  while (next_segment(p, per, w, g)) {
    // ---- Q tile to fp16, each row by its power of two
    const int rows = min(kRows, g.row.cnt * p.group - g.tile * kRows);   // may be <= 0 behind q_count
    named_bar_sync(1, kWarps * 32);             // the last segment's readers of Q are done
    for (int r = warp; r < kRows; r += kWarps) {
      constexpr int kPl = D / 32;               // values a lane
      float x[kPl];
      float am = 0.0f;
      const int row = g.tile * kRows + r;
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
      for (int i = 0; i < kPl; i += 2)
        *reinterpret_cast<uint32_t*>(smem + S::q + r * S::qpitch + (i * 32 + lane * 2) * 2) =
            pack_h2(x[i] * inv, x[i + 1] * inv);
      if (lane == 0) rowf[r] = exp2i(e) * p.scale_log2;
    }
    named_bar_sync(1, kWarps * 32);

    // ---- the visible ranges of this lane's two rows, and of the tile
    const int r0 = g.tile * kRows + gq, last = g.tile * kRows + max(rows, 1) - 1;
    int lo[2], hi[2], lo_first, hi_first, lo_last, hi_last;
    kv8_seen(p, g.row, r0 / p.group, lo[0], hi[0]);
    kv8_seen(p, g.row, (r0 + 8) / p.group, lo[1], hi[1]);
    kv8_seen(p, g.row, g.tile * kRows / p.group, lo_first, hi_first);
    kv8_seen(p, g.row, last / p.group, lo_last, hi_last);
    const float f0 = rowf[gq], f1 = rowf[gq + 8];

    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    for (int j = 0; j < g.n; j += kPer, ++it) {
      const int s = it % kStages;
      const int base = (j / kPer) * kSlices;    // the segment's slices go round the warps
      const int mine = (warp - base % kWarps + kWarps) % kWarps;
      if (mine >= kSlices) continue;
      if (!ok || !mbar_wait(full0 + 8 * s, (it / kStages) & 1, p.err)) {
        ok = false;
        continue;
      }
      for (int sl = mine; sl < kSlices; sl += kWarps) {
        const int bi = sl >> 2, wsl = sl & 3;
        const int tok = (g.blk + j + bi) * kKv8Block + wsl * 16;
        if (j + bi >= g.n || tok >= hi_last || tok + 16 <= lo_first) continue;
        const uint32_t kb = sm + s * kStage + bi * D * 64 + (wsl * 16 + gq) * 64 + 4 * t;
        const uint32_t vb = sm + s * kStage + kStageK + bi * D * 64 + gq * 64 + ((wsl ^ swz) << 4) + 4 * t;
        const float4 sc = *reinterpret_cast<const float4*>(smem + S::scale + s * 64 + bi * 16);
        float x[2][4] = {};
        const uint32_t qa = sm + S::q + gq * S::qpitch + 8 * t;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint2 a = lds64(qa + kk * 32), b = lds64(qa + 8 * S::qpitch + kk * 32);
          const uint32_t ko = (kk >> 2) * 4096 + (((kk & 3) ^ swz) << 4);
          const uint32_t k0 = lds32(kb + ko), k1 = lds32(kb + ko + 512);
          mma_f16(x[0], a.x, b.x, a.y, b.y, e4m3x2_to_h2(static_cast<uint16_t>(k0)),
                  e4m3x2_to_h2(static_cast<uint16_t>(k0 >> 16)));
          mma_f16(x[1], a.x, b.x, a.y, b.y, e4m3x2_to_h2(static_cast<uint16_t>(k1)),
                  e4m3x2_to_h2(static_cast<uint16_t>(k1 >> 16)));
        }
        // scores in the exp2 domain, plus the exponent of the block's V scale
        const int ev = exp_of(sc.y);
        const float fv = static_cast<float>(ev), g0 = f0 * sc.x, g1 = f1 * sc.x;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[h][0] = fmaf(x[h][0], g0, fv);
          x[h][1] = fmaf(x[h][1], g0, fv);
          x[h][2] = fmaf(x[h][2], g1, fv);
          x[h][3] = fmaf(x[h][3], g1, fv);
        }
        if (tok < lo_last || tok + 16 > hi_first) {      // some row does not see all of the slice
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int k = tok + 8 * h + 2 * t + (c & 1), r = c >> 1;
              if (k < lo[r] || k >= hi[r]) x[h][c] = -INFINITY;
            }
        }
        float mx[2] = {fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1])),
                       fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]))};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        }
        // the reference maximum moves only when it is passed by more than 8 (weights <= 2^8)
        const bool move = mx[0] > m[0] + 8.0f || mx[1] > m[1] + 8.0f || (m[0] == -INFINITY && mx[0] > m[0]) ||
                          (m[1] == -INFINITY && mx[1] > m[1]);
        if (__any_sync(0xffffffffu, move)) {
          float fac[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float nm = fmaxf(m[r], mx[r]);
            fac[r] = m[r] == -INFINITY ? 1.0f : exp2_approx(m[r] - nm);   // nothing summed yet: 1
            m[r] = nm;
            l[r] *= fac[r];
          }
#pragma unroll
          for (int jj = 0; jj < D / 8; ++jj) {
            o[jj][0] *= fac[0];
            o[jj][1] *= fac[0];
            o[jj][2] *= fac[1];
            o[jj][3] *= fac[1];
          }
        }
        const float m0 = m[0] == -INFINITY ? 0.0f : m[0], m1 = m[1] == -INFINITY ? 0.0f : m[1];
        float pr[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          pr[h][0] = exp2_approx(x[h][0] - m0);
          pr[h][1] = exp2_approx(x[h][1] - m0);
          pr[h][2] = exp2_approx(x[h][2] - m1);
          pr[h][3] = exp2_approx(x[h][3] - m1);
        }
        const float un = exp2i(-ev);
        l[0] = fmaf(pr[0][0] + pr[0][1] + pr[1][0] + pr[1][1], un, l[0]);
        l[1] = fmaf(pr[0][2] + pr[0][3] + pr[1][2] + pr[1][3], un, l[1]);
        const uint32_t a0 = pack_h2(pr[0][0], pr[0][1]), a1 = pack_h2(pr[0][2], pr[0][3]);
        const uint32_t a2 = pack_h2(pr[1][0], pr[1][1]), a3 = pack_h2(pr[1][2], pr[1][3]);
#pragma unroll
        for (int jj = 0; jj < D / 8; ++jj) {
          const uint32_t v = lds32(vb + jj * 512);
          mma_f16(o[jj], a0, a1, a2, a3, e4m3x2_to_h2(static_cast<uint16_t>(v)),
                  e4m3x2_to_h2(static_cast<uint16_t>(v >> 16)));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * s);
    }

    // ---- the eight warps' results
    float2* ml = reinterpret_cast<float2*>(smem + S::ml);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (t == 0) ml[warp * kRows + gq + 8 * r] = make_float2(m[r], l[r]);
    }
    named_bar_sync(1, kWarps * 32);
    float fac[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mm = -INFINITY;
      for (int i = 0; i < kWarps; ++i) mm = fmaxf(mm, ml[i * kRows + gq + 8 * r].x);
      fac[r] = m[r] == -INFINITY ? 1.0f : exp2_approx(m[r] - mm);
    }
    // this thread's output: row rr, two columns of each 32
    const int rr = threadIdx.x >> 4, cc = (threadIdx.x & 15) * 2;
    float mm = -INFINITY, ll = 0.0f;
    for (int i = 0; i < kWarps; ++i) mm = fmaxf(mm, ml[i * kRows + rr].x);
    for (int i = 0; i < kWarps; ++i) {
      const float2 v = ml[i * kRows + rr];
      ll += v.y * (v.x == -INFINITY ? 1.0f : exp2_approx(v.x - mm));
    }
    const float norm = g.whole ? (ll == 0.0f ? 0.0f : 1.0f / ll) : 1.0f;
    const int row = g.tile * kRows + rr;
    const int qi = row / p.group, qh = g.head * p.group + row % p.group;
    const int slot = 2 * blockIdx.x + (g.first ? 0 : 1);
    float* ws = p.ws + (static_cast<size_t>(slot) * kRows + rr) * D;
    __nv_bfloat16* dst = p.out + g.b * p.o_st[0] + qi * p.o_st[1] + qh * p.o_st[2];
    float* xb = reinterpret_cast<float*>(smem + S::xch);
#pragma unroll
    for (int c0 = 0; c0 < D / 32; ++c0) {
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        float* a = xb + (warp * kRows + gq) * 32 + jj * 8 + 2 * t;
        *reinterpret_cast<float2*>(a) = make_float2(o[c0 * 4 + jj][0] * fac[0], o[c0 * 4 + jj][1] * fac[0]);
        *reinterpret_cast<float2*>(a + 8 * 32) = make_float2(o[c0 * 4 + jj][2] * fac[1], o[c0 * 4 + jj][3] * fac[1]);
      }
      named_bar_sync(1, kWarps * 32);
      if (rr < rows) {
        float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float2 y = *reinterpret_cast<const float2*>(xb + (i * kRows + rr) * 32 + cc);
          v.x += y.x;
          v.y += y.y;
        }
        if (!g.whole) {
          *reinterpret_cast<float2*>(ws + c0 * 32 + cc) = v;
        } else if (c0 * 32 + cc < p.c.D) {
          const __nv_bfloat162 y = __floats2bfloat162_rn(v.x * norm, v.y * norm);
          *reinterpret_cast<__nv_bfloat162*>(dst + c0 * 32 + cc) = y;
        }
      }
      named_bar_sync(1, kWarps * 32);
    }
    if ((threadIdx.x & 15) == 0 && rr < rows) {
      if (!g.whole)
        p.ws_ml[slot * kRows + rr] = make_float2(mm, ll);
      else if (p.lse)
        p.lse[(static_cast<size_t>(g.b) * p.n_q + qi) * p.n_heads + qh] =
            ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
    }
  }
}

// Merges the parts of the items that more than one CTA worked on. One CTA per (tile row, item,
// batch row); Ds threads, a column each.
__global__ void kv8_merge_kernel(const Kv8AttendParams p, int tile_rows, int ds) {
  __shared__ long long red[8];
  const int per = p.c.n_kv * p.tiles;
  const int r = blockIdx.x, item = blockIdx.y, b = blockIdx.z;
  const Kv8Row row = kv8_row(p, b);
  const int head = item / p.tiles, tile = item % p.tiles;
  if (row.cnt * p.group <= tile * tile_rows + r) {
    pdl_wait();
    return;
  }
  const long long before = units_before(p, b, per, red);
  const long long total = units_before(p, p.batch, per, red);
  const long long u0 = before + static_cast<long long>(item) * row.nblk, u1 = u0 + row.nblk;
  // CTAs whose parts meet [u0, u1)
  int c = static_cast<int>(u0 * p.grid / total);
  while (part_begin(total, p.grid, c) > u0) --c;
  while (part_begin(total, p.grid, c + 1) <= u0) ++c;
  pdl_wait();
  if (part_begin(total, p.grid, c + 1) >= u1) return;      // one CTA finished the item
  const int c0 = c;
  float mm = -INFINITY;
  for (; c < p.grid && part_begin(total, p.grid, c) < u1; ++c) {
    const long long s = part_begin(total, p.grid, c);
    if (s == part_begin(total, p.grid, c + 1)) continue;   // an empty part
    mm = fmaxf(mm, p.ws_ml[(2 * c + (s >= u0 ? 0 : 1)) * tile_rows + r].x);
  }
  float ll = 0.0f, v = 0.0f;
  for (int i = c0; i < c; ++i) {
    const long long s = part_begin(total, p.grid, i);
    if (s == part_begin(total, p.grid, i + 1)) continue;
    // the part in which CTA i's range starts is its first; an item that starts later, its second
    const int slot = (2 * i + (s >= u0 ? 0 : 1)) * tile_rows + r;
    const float2 y = p.ws_ml[slot];
    const float f = y.x == -INFINITY ? 1.0f : exp2_approx(y.x - mm);
    ll = fmaf(y.y, f, ll);
    v = fmaf(p.ws[static_cast<size_t>(slot) * ds + threadIdx.x], f, v);
  }
  const int at = tile * tile_rows + r;
  const int qi = at / p.group, qh = head * p.group + at % p.group;
  if (static_cast<int>(threadIdx.x) < p.c.D)
    p.out[b * p.o_st[0] + qi * p.o_st[1] + qh * p.o_st[2] + threadIdx.x] =
        __float2bfloat16_rn(ll == 0.0f ? 0.0f : v / ll);
  if (threadIdx.x == 0 && p.lse)
    p.lse[(static_cast<size_t>(b) * p.n_q + qi) * p.n_heads + qh] =
        ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
}

template <int D>
static cudaError_t launch_rows(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Kv8AttendParams& p,
                               cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = RowsSmem<D>::total + 1024;
  cfg.stream = s;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_attend_rows_kernel<D>, tm_k, tm_v, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(kRows, p.c.n_kv * p.tiles, p.batch);
  cfg.blockDim = dim3(D);
  cfg.dynamicSmemBytes = 0;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_merge_kernel, p, kRows, D);
}

cudaError_t launch_kv8_attend_rows(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Kv8AttendParams& p,
                                   cudaStream_t s) {
  if (p.c.Ds == 64) return launch_rows<64>(tm_k, tm_v, p, s);
  if (p.c.Ds == 128) return launch_rows<128>(tm_k, tm_v, p, s);
  return launch_rows<256>(tm_k, tm_v, p, s);
}

cudaError_t configure_kv8_kernels() {
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(kv8_attend_rows_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                RowsSmem<64>::total + 1024)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(kv8_attend_rows_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                RowsSmem<128>::total + 1024)) != cudaSuccess) return e;
  return cudaFuncSetAttribute(kv8_attend_rows_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              RowsSmem<256>::total + 1024);
}

}  // namespace vla
