// kv8_attend_tc.cu -- attention over the 8-bit K/V cache for many query rows (an action chunk,
// a prompt piece), on the tcgen05 tensor cores.
//
// Same formula and the same equal division of the work as kv8_attend.cu, in tiles of 128
// query rows (head_dim 256) or 256 (smaller head_dim) and units of 64 keys. What bounds it
// is the tensor pipe and, at head_dim 64 and 128, the exponentials (16 a clock and SM).
//
//   S = Q K^T   kind::f8f6f4, K as the cache holds it (its block is already the operand's
//               64-byte swizzled K-major layout), Q as two E4M3 terms accumulated in one
//               sum: a row times the power of two that brings its largest magnitude to
//               [128, 256), hi = e4m3(q), lo = e4m3(q - hi). Exact for bf16 values above
//               2^-9 of the largest, else to 2^-17 of it. Two E4M3 products take as long as
//               one 16-bit product, and K needs no widening.
//   P           bf16, exp2(s + log2 s_V - m): the V scale enters through the exponent and leaves
//               the sum in fp32; off by at most 2^-8 of itself; written over S in tensor memory,
//               from where the second product takes it.
//   O += P V    kind::f16 on bf16. Four warps widen V blocks to bf16 (exact) in the 128-byte
//               swizzled K-major layout; both query tiles use each widened block.
// bf16 has fp32's exponents, so the row's reference m comes from the first block it sees
// and stays unless a block passes it by far (then O in tensor memory is rescaled). At head_dim 64
// and 128 no other maximum is looked for: the weights' sum shows whether they were too large, and
// then the block is done once more. With fp16 weights, whose reference may lag by 2^13 at most,
// one step in five rescaled O on keys of unlike norms.
//
// The tensor pipe and the softmax of a lane depend on each other, so there are two lanes with
// two S buffers of 64 keys each: a buffer's next scores are issued when the output of its last
// weights is done, and a softmax group always has its next scores waiting.
//   head_dim <= 128, more than 128 rows: lane i is query tile i (128 rows), all blocks.
//   head_dim <= 128, up to 128 rows: lane i takes every second block for the same rows, with an
//     output of its own; the two outputs are joined at the end.
//   head_dim 256: lane i takes every second block; one output (256 columns), for which the row's
//     reference maximum goes from block to block between the two groups.
// 2 x 2048 queries of 32 heads (8 K/V heads, head_dim 128) behind 4096 stored tokens: 0.42 ms, 49 %
// of the measured bf16 rate counted on the formula's products. A step of 64 keys for both tiles
// takes 1.1 us (2100 clocks) of an SM at head_dim 128 and 1.05 at 64, so it is not the products that
// bound it: the softmax groups' way through a step does, of which the exponentials fill half (1030
// clocks for two warps a scheduler) and the loads, stores and waits of a warp the rest. Each new tile
// costs 8 us more (Q, start of the lanes, output) and a part of one the merge. (The softmax groups'
// code, at 168 registers, spills 200 to 390 bytes a thread.)
// Warps: 0 and 1 scores, 2 and 3 outputs of lane 0 and 1, 4..7 and 8..11 softmax of lane 0 and 1
// (one thread a row), 12..15 widening of V, 16 loads of K, 17 loads of V.
#include <float.h>

#include "kernels.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace vla {

namespace {

constexpr int kThreads = 640;
// Registers: 96 a thread at launch; the softmax groups go up to 168, the three others down to
// 48 (2 x 128 x 168 + 3 x 128 x 48 = 61440 = 640 x 96).

// A row's reference m is the largest score of a block, to a multiple of 2^-12: taking it off ev - 32
// rounds nothing then, and the largest weight is a power of two to 2^-13 of itself, so that bf16 has
// it (a row of one key is exact). It does not look at V's scales 2^ev, -60 <= ev <= 120: a weight
// 2^(s + ev - 32 - m) (kKv8Lift = 32) is within fp32's and bf16's range for each of them, down to 2^-34 of
// the reference's key at ev = -60 (2^-86 at 2^-8, ordinary values) and, with V's 448 * 2^ev below 2^128, with sums
// over 2^29 keys below 2^127. The reference moves when a block's largest score is above it by more
// than kLag (head_dim 256), or the weights of a block sum to more than 2^kMaxSum without V's scale
// (else); by less where V's scale leaves no room for that (kTop: a block's weights stay below 2^kTop).
constexpr int kLag = 32, kMaxSum = 40 - kKv8Lift, kTop = 95;
// Factor from which on a block's scores can reach 2^23 bits (its sums of products are below 2^25),
// where fp32 has no bits left for the fraction and soon none for ev: these are rounded first, the
// reference is taken off, and then ev is added. (Fused with the subtraction, a product of 2^31 can
// miss its own rounded value by more than the range of the weights.)
constexpr float kFarFactor = 0.25f;
__device__ __forceinline__ float on_grid(float s) {      // (from 2^11 on fp32's own steps are wide enough)
  return fabsf(s) < 2048.0f ? rintf(s * 4096.0f) * (1.0f / 4096.0f) : s;
}

template <int D>
struct Tc {
  static constexpr bool two = D <= 128;                  // two query tiles, or two outputs
  static constexpr int rows = two ? 256 : 128;
  static constexpr int nk = D == 256 ? 4 : 6;            // K blocks
  static constexpr int nv = D == 256 ? 2 : 4;            // V blocks as stored, and widened
  static constexpr int q_half = 128 * D;                 // one term of one tile
  static constexpr int v16 = 0;                          // 128-byte swizzle: 1024-byte aligned
  static constexpr int q = v16 + nv * D * 128;           // [tile][term][D / 64 panels][128 rows][64]
  static constexpr int k = q + (two ? 2 : 1) * 2 * q_half;
  static constexpr int v8 = k + nk * D * 64;
  static constexpr int xch = v8 + nv * D * 64;           // [2][128] reference maxima; (maximum, sum) at the end
  static constexpr int bar = xch + 2048;
  static constexpr int total = bar + 512;
  static constexpr int o_col = 256;                      // tensor memory: S buffers 0, 64, 128, 192; O
};

// Operand descriptors in two words. Low: start address >> 4 and leading offset (unused, 1);
// high: stride between 8-row groups >> 4, version 1, swizzle. K-major rows of 64 bytes (64-byte
// swizzle, groups 512 bytes apart) and of 128 bytes (128-byte swizzle, 1024).
constexpr uint32_t kDescSw64 = (512 >> 4) | (1u << 14) | (4u << 29);
constexpr uint32_t kDescSw128 = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr & 0x3FFFF) >> 4) | (1u << 16); }

// One lane of a converged warp: 1 in it, 0 in the others. The products are issued by the whole
// warp under this predicate, so that their operands stay in uniform registers (issued from a
// branch of one lane, a product took 110 to 190 clocks, here the tensor pipe's own time).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
  return r;
}
// The same value in every lane, as one the compiler knows to be uniform.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
// E4M3 x E4M3 (kind::f8f6f4): format fields 0, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_fmt0(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void umma_f8(uint32_t lead, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                        uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %0, 0;\n\tmov.b64 a, {%2, %6};\n\tmov.b64 b, {%3, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%1], a, b, %4, p;\n\t}\n" ::"r"(lead), "r"(d_tmem), "r"(a_lo),
      "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescSw64)
      : "memory");
}
__device__ __forceinline__ void umma_f16_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                            uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %0, 0;\n\tmov.b64 b, {%3, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], b, %4, p;\n\t}\n" ::"r"(lead), "r"(d_tmem), "r"(a_tmem),
      "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescSw128)
      : "memory");
}
__device__ __forceinline__ void umma_commit_if(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}\n" ::"r"(lead), "r"(bar)
      : "memory");
}
// A bounded wait of a whole converged warp. What depends on it, like every choice of the softmax
// groups that is the same for a warp, goes through a vote, so that the compiler keeps no path for
// lanes that part (406 -> 397 us for 2 x 2048 queries behind 4096 tokens).
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, int* err) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = globaltimer_ns();
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitLimitNs)) {
      report(err, kDevTimeout);
      return false;
    }
  }
}
// Two fp32 lanes in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two E4M3 bytes, each in the upper byte of a half word, to bf16: exponent and mantissa move to
// bf16's places (a value 2^-120 of the right one, E4M3's subnormals among bf16's), times 2^120.
__device__ __forceinline__ uint32_t e4m3_to_bf2(uint32_t v) {
  const uint32_t u = ((v >> 4) & 0x07f007f0u) | (v & 0x80008000u);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x7b807b80u));
  return r;
}
// Exponent that Q's row of largest magnitude `am` is divided by.
__device__ __forceinline__ int q_exp(float am) { return am > 0.0f ? min(max(exp_of(am) - 7, -118), 120) : 0; }
// 32 columns of this warp's 32 lanes; the caller waits (tmem_wait_ld).
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32_async(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_global_32(void* p, const uint32_t* r) {   // one 32-byte sector
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// How the lanes share a segment. Step k of lane i works in S buffer 2 i + (k & 1); scores and
// outputs are issued in the order (lane 0, 0), (lane 1, 0), (lane 0, 1), ... (t = 2 k + lane).
struct Plan {
  bool tiles;            // lane = query tile, every block a step of both; else every second block
  int steps[2];          // of each lane
};
template <int D>
__device__ __forceinline__ Plan make_plan(const Kv8AttendParams& p, const Kv8Segment& g) {
  Plan r;
  r.tiles = Tc<D>::two && g.row.cnt * p.group - g.tile * Tc<D>::rows > 128;
  r.steps[0] = r.tiles ? g.n : (g.n + 1) / 2;
  r.steps[1] = r.tiles ? g.n : g.n / 2;
  return r;
}
// Parities of the buffers' barriers: bit b of `ph` is that of buffer b's first use in a segment.
__device__ __forceinline__ uint32_t buf_parity(uint32_t ph, int lane_of, int k) {
  return ((ph >> (2 * lane_of + (k & 1))) ^ (k >> 1)) & 1;
}
__device__ __forceinline__ uint32_t next_phases(uint32_t ph, const Plan& pl) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    ph ^= (((pl.steps[i] + 1) >> 1) & 1) << (2 * i) | ((pl.steps[i] >> 1) & 1) << (2 * i + 1);
  return ph;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_attend_tc_kernel(const Kv8AttendParams p) {
  using S = Tc<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sm = smem_u32(smem);
  const uint32_t kfull = sm + S::bar, kempty = kfull + 8 * S::nk;
  const uint32_t rfull = kempty + 8 * S::nk, rempty = rfull + 8 * S::nv;      // V as stored
  const uint32_t vfull = rempty + 8 * S::nv, vempty = vfull + 8 * S::nv;      // V widened
  const uint32_t sfull = vempty + 8 * S::nv, pfull = sfull + 32, odone = pfull + 32;   // [buffer]
  const uint32_t qfull = odone + 32;            // [score warp]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::bar + 504);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::nk; ++i) {
      mbar_init(kfull + 8 * i, 1);
      mbar_init(kempty + 8 * i, 2);
    }
    for (int i = 0; i < S::nv; ++i) {
      mbar_init(rfull + 8 * i, 1);
      mbar_init(rempty + 8 * i, 4);
      mbar_init(vfull + 8 * i, 4);
      mbar_init(vempty + 8 * i, S::two ? 2 : 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(sfull + 8 * i, 1);
      mbar_init(pfull + 8 * i, 4);
      mbar_init(odone + 8 * i, 1);
    }
    mbar_init(qfull, 8);
    mbar_init(qfull + 8, 8);
    fence_mbar_init();
    pdl_trigger();
  }
  if (warp == 18) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (blockIdx.x == 0 && warp == 19)
    for (int b = lane; b < p.batch; b += 32)
      if (kv8_tile(p, b, 0).slot < 0) report(p.err, kKv8BadRow);
  Kv8Walk w = kv8_walk(p);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  Kv8Segment g;
  bool ok = true;
  if (warp < 4) {
    // ---- products, each by a converged warp: warps 0 and 1 the scores of lane 0 and 1, warps 2
    // and 3 the outputs (head_dim 256: warp 2 both lanes', in turn, as they share an output)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    const uint32_t lead = elect_one();
    // the warp stays together when a wait gives up
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, parity, p.err)) != 0;
    };
    const uint32_t tm = uniform(tmem);
    uint32_t ph = 0, rph = 0;                             // rph, rs: the ring of K or V
    int rs = 0;
    if (warp < 2) {
      constexpr uint32_t id_s = idesc_fmt0(128, 64);
      constexpr uint32_t kTile = (2 * S::q_half) >> 4;    // from one query tile to the next
      const int i = warp;
      const uint32_t q0 = uniform(desc_lo(sm + S::q)), k0 = uniform(desc_lo(sm + S::k));
      uint32_t qph = 0;
      while (ok && kv8_next(p, w, g)) {
        const Plan pl = make_plan<D>(p, g);
        // Each score warp has a barrier for Q, which goes round only in the segments where the warp
        // has scores to make (lane 1 has none in a segment of one block): the softmax groups cannot
        // complete its next phase before they have had those scores, so no phase is passed unseen.
        if ((i ? pl.steps[1] : pl.steps[0]) > 0) {
          wait_all(qfull + 8 * i, qph);
          qph ^= 1;
        }
        const uint32_t a0 = uniform(q0 + (pl.tiles && i ? kTile : 0));
        // every block in turn, also those of the other lane: a warp that skipped one could take its
        // slot's last phase for the next
        for (int j = 0; j < g.n && ok; ++j) {
          wait_all(kfull + 8 * rs, rph);
          if (pl.tiles || (j & 1) == i) {
            const int k = pl.tiles ? j : j >> 1, buf = 2 * i + (k & 1);
            // the buffer's last weights have been used
            if (k >= 2) wait_all(odone + 8 * buf, buf_parity(ph, i, k - 2));
            tc_fence_after();
            if (!ok) break;
            const uint32_t b0 = k0 + rs * (D * 64 >> 4);
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                umma_f8(lead, tm + buf * 64, a0 + ((term * S::q_half + (kk >> 1) * 8192) >> 4) + 2 * (kk & 1),
                        b0 + (((kk >> 1) * 4096) >> 4) + 2 * (kk & 1), id_s, (term | kk) != 0 ? 1u : 0u);
            umma_commit_if(lead, sfull + 8 * buf);
            umma_commit_if(lead, kempty + 8 * rs);
          } else if (lead) {
            mbar_arrive(kempty + 8 * rs);
          }
          if (++rs == S::nk) {
            rs = 0;
            rph ^= 1;
          }
        }
        ph = next_phases(ph, pl);
      }
    } else if (S::two || warp == 2) {
      constexpr uint32_t id_o = idesc_bf16_f32(128, D);
      const uint32_t v0 = uniform(desc_lo(sm + S::v16));
      while (ok && kv8_next(p, w, g)) {
        const Plan pl = make_plan<D>(p, g);
        for (int j = 0; j < g.n && ok; ++j) {
          wait_all(vfull + 8 * rs, rph);
          const int i = S::two ? warp - 2 : j & 1;
          if (pl.tiles || (j & 1) == i) {
            const int k = pl.tiles ? j : j >> 1, buf = 2 * i + (k & 1);
            wait_all(pfull + 8 * buf, buf_parity(ph, i, k));
            tc_fence_after();
            if (!ok) break;
            const uint32_t acc = (S::two ? k : j) == 0 ? 0u : 1u, b0 = v0 + rs * (D * 128 >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f16_ts(lead, tm + S::o_col + (S::two ? i * D : 0), tm + buf * 64 + kk * 8, b0 + 2 * kk, id_o,
                          kk == 0 ? acc : 1u);
            // (no commit follows the last output's own, for which the CTA waits before it ends)
            umma_commit_if(lead, vempty + 8 * rs);
            umma_commit_if(lead, odone + 8 * buf);
          } else if (lead) {
            mbar_arrive(vempty + 8 * rs);
          }
          if (++rs == S::nv) {
            rs = 0;
            rph ^= 1;
          }
        }
        ph = next_phases(ph, pl);
      }
    }
    __syncwarp();
  } else if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp < 18 && lane == 0) {
      // ---- loads: warp 16 the K blocks, warp 17 the V blocks
      const uint8_t* src = warp == 16 ? p.c.k : p.c.v;
      const uint32_t full = warp == 16 ? kfull : rfull, empty = warp == 16 ? kempty : rempty;
      const uint32_t dst = sm + (warp == 16 ? S::k : S::v8);
      const int ring = warp == 16 ? S::nk : S::nv;
      int n = 0, s = 0;
      uint32_t ph = 1;
      while (ok && kv8_next(p, w, g)) {
        const size_t blk0 =
            ((static_cast<size_t>(p.layer) * p.c.n_slots + g.row.slot) * p.c.n_kv + g.head) * p.c.nblk + g.blk;
        for (int j = 0; j < g.n; ++j, ++n) {
          if (n >= ring && !mbar_wait(empty + 8 * s, ph, p.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(full + 8 * s, D * 64);
          bulk_load_g2s(dst + s * D * 64, src + (blk0 + j) * (D * 64), D * 64, full + 8 * s);
          if (++s == ring) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // no copies left in flight
      for (int i = n > ring ? n - ring : 0; i < n; ++i) mbar_wait(full + 8 * (i % ring), (i / ring) & 1, p.err);
    }
    __syncwarp();
  } else if (warp >= 12) {
    // ---- V blocks to bf16: [D rows][64 positions] bytes, 64-byte swizzle, to 128-byte rows
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    const int tid = threadIdx.x - 384;
    int vt = 0;
    while (kv8_next(p, w, g)) {
      for (int j = 0; j < g.n; ++j, ++vt) {
        const int r = vt % S::nv;
        ok = ok && mbar_wait(rfull + 8 * r, (vt / S::nv) & 1, p.err);
        ok = ok && (vt < S::nv || mbar_wait(vempty + 8 * r, (vt / S::nv - 1) & 1, p.err));
        if (ok) {
          const uint8_t* src = smem + S::v8 + r * D * 64;
          uint8_t* dst = smem + S::v16 + r * D * 128;
#pragma unroll 4
          for (int i = tid; i < D * 4; i += 128) {
            const int d = i >> 2, c = i & 3;
            const uint4 x = *reinterpret_cast<const uint4*>(src + d * 64 + ((c ^ ((d >> 1) & 3)) << 4));
            uint4 y, z;
            y.x = e4m3_to_bf2(__byte_perm(x.x, 0, 0x1404));
            y.y = e4m3_to_bf2(__byte_perm(x.x, 0, 0x3424));
            y.z = e4m3_to_bf2(__byte_perm(x.y, 0, 0x1404));
            y.w = e4m3_to_bf2(__byte_perm(x.y, 0, 0x3424));
            z.x = e4m3_to_bf2(__byte_perm(x.z, 0, 0x1404));
            z.y = e4m3_to_bf2(__byte_perm(x.z, 0, 0x3424));
            z.z = e4m3_to_bf2(__byte_perm(x.w, 0, 0x1404));
            z.w = e4m3_to_bf2(__byte_perm(x.w, 0, 0x3424));
            *reinterpret_cast<uint4*>(dst + d * 128 + (((2 * c) ^ (d & 7)) << 4)) = y;
            *reinterpret_cast<uint4*>(dst + d * 128 + (((2 * c + 1) ^ (d & 7)) << 4)) = z;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(rempty + 8 * r);
          mbar_arrive(vfull + 8 * r);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    const int grp = (warp - 4) >> 2, qd = warp & 3, r = qd * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(qd * 32) << 16);
    float* xch = reinterpret_cast<float*>(smem + S::xch);
    uint32_t ph = 0;
    bool up = true;                      // no wait for scores gave up: the same in a whole warp, unlike ok
    while (kv8_next(p, w, g)) {
      const Plan pl = make_plan<D>(p, g);
      const int left = g.row.cnt * p.group - g.tile * S::rows;      // rows from the tile's first on
      const int r0 = g.tile * S::rows + (pl.tiles ? grp * 128 : 0); // first row of this group's tile
      const int row = r0 + r, rows = min(128, left - (pl.tiles ? grp * 128 : 0));
      const bool row_ok = r < rows;
      // ---- Q to E4M3 pairs: a load brings whole rows (D / 8 lanes each) of the warp's 32
      // (head_dim 256: of its half of them), and every lane keeps its own row's factor
      float rowf = p.scale_log2;
      {
        constexpr int kLanes = D / 8, kAt = 32 / kLanes, kLoads = (S::two ? 32 : 16) / kAt;
        const int half = S::two ? 0 : grp * 16, d = lane % kLanes * 8;
        const long long at = g.b * p.q_st[0] + p.by_group.div(row) * p.q_st[1] +
                             (g.head * p.group + p.by_group.mod(row)) * p.q_st[2];
        uint8_t* dst = smem + S::q + (pl.tiles ? grp * 2 * S::q_half : 0) + (d >> 6) * 8192 + (d & 8);
        float am = 0.0f;
#pragma unroll 1
        for (int i0 = 0; i0 < kLoads; i0 += 8) {
          uint4 x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = half + (i0 + i) * kAt + lane / kLanes;
            const long long from = __shfl_sync(0xffffffffu, at, rr);
            x[i] = make_uint4(0, 0, 0, 0);
            if (qd * 32 + rr < rows && d < p.c.D) x[i] = *reinterpret_cast<const uint4*>(p.q + from + d);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = half + (i0 + i) * kAt + lane / kLanes;
            const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            // the row's largest magnitude (bf16 bits order like their values; not finite: left out)
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t a = v[c] & 0x7fffu, b = (v[c] >> 16) & 0x7fffu;
              top = max(top, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
            }
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float big = __uint_as_float(top << 16);
            const float inv = exp2i(-q_exp(big));
            if (S::two) {
              const float own = __shfl_sync(0xffffffffu, big, lane % kAt * kLanes);
              if (lane / kAt == i0 + i) am = own;
            } else if (lane == 0) {
              xch[qd * 32 + rr] = big;
            }
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float f[4] = {__uint_as_float(v[2 * c] << 16) * inv, __uint_as_float(v[2 * c] & 0xffff0000u) * inv,
                            __uint_as_float(v[2 * c + 1] << 16) * inv, __uint_as_float(v[2 * c + 1] & 0xffff0000u) * inv};
#pragma unroll
              for (int k = 0; k < 4; ++k) f[k] = fmaf(f[k], 0.0f, f[k]);   // an infinity becomes NaN
              const uint16_t h0 = f2_to_e4m3x2(f[0], f[1]), h1 = f2_to_e4m3x2(f[2], f[3]);
              const uint32_t w0 = e4m3x2_to_h2(h0), w1 = e4m3x2_to_h2(h1);
              const float2 g0 = __half22float2(*reinterpret_cast<const __half2*>(&w0));
              const float2 g1 = __half22float2(*reinterpret_cast<const __half2*>(&w1));
              hi[c] = h0 | (static_cast<uint32_t>(h1) << 16);
              lo[c] = f2_to_e4m3x2(f[0] - g0.x, f[1] - g0.y) |
                      (static_cast<uint32_t>(f2_to_e4m3x2(f[2] - g1.x, f[3] - g1.y)) << 16);
            }
            if (!S::two || pl.tiles || grp == 0) {
              const int t = qd * 32 + rr;
              uint8_t* a = dst + t * 64 + ((((d >> 4) & 3) ^ ((t >> 1) & 3)) << 4);
              *reinterpret_cast<uint2*>(a) = make_uint2(hi[0], hi[1]);
              *reinterpret_cast<uint2*>(a + S::q_half) = make_uint2(lo[0], lo[1]);
            }
          }
        }
        if (!S::two) {                                    // each group has read half of the rows
          named_bar_sync(11 + qd, 64);
          am = xch[r];
          named_bar_sync(11 + qd, 64);
        }
        rowf *= exp2i(q_exp(am));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(qfull);
          if (pl.steps[1] > 0) mbar_arrive(qfull + 8);
        }
      }

      int lo, hi, lo_last, hi_first, t0, t1;
      kv8_seen(p, g.row, p.by_group.div(r0 + max(min(r, rows - 1), 0)), lo, hi);
      kv8_seen(p, g.row, p.by_group.div(r0), t0, hi_first);
      kv8_seen(p, g.row, p.by_group.div(r0 + max(rows, 1) - 1), lo_last, t1);
      const float4* scales = p.c.scale +
          ((static_cast<size_t>(p.layer) * p.c.n_slots + g.row.slot) * p.c.n_kv + g.head) * p.c.nblk + g.blk;
      const int steps = grp ? pl.steps[1] : pl.steps[0];   // (no array indexed at run time: local memory)
      const int stride = pl.tiles ? 1 : 2, first = pl.tiles ? 0 : grp;   // block of step k: first + k * stride
      auto scale_of = [&](int k) {
        return __ldg(reinterpret_cast<const float2*>(scales + min(first + k * stride, g.n - 1)));
      };
      float2 sc = scale_of(0);
      float m = -INFINITY, l = 0.0f;
      // moves the row's reference to nm, and with it l and (if it has begun) this warp's rows of O:
      // after the last product on them
      auto move_to = [&](float nm, int k, int j) {
        const float f = nm == m ? 1.0f : exp2_approx(m - nm);
        m = nm;
        l *= f;
        const int before = S::two ? k - 1 : (j - 1) >> 1, of = S::two ? grp : grp ^ 1;
        if ((S::two ? k : j) > 0) {
          ok = ok && up && mbar_wait(odone + 8 * (2 * of + (before & 1)), buf_parity(ph, of, before), p.err);
          tc_fence_after();
          const uint32_t to = tl + S::o_col + (S::two ? grp * D : 0);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float y[32];
            tmem_ld32_async(to + c, y);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] *= f;
            tmem_st32_async(to + c, reinterpret_cast<uint32_t*>(y));
          }
          tmem_wait_st();
        }
      };
      for (int k = 0; k < steps; ++k) {
        const int buf = 2 * grp + (k & 1), j = first + k * stride, key0 = (g.blk + j) * kKv8Block;
        up = up && wait_warp(sfull + 8 * buf, buf_parity(ph, grp, k), p.err);
        tc_fence_after();
        const float gk = fmaxf(rowf * sc.x, FLT_MIN);       // (never 0: a masked score stays -infinity)
        const int ev = exp_of(sc.y);
        const float fv = static_cast<float>(ev - kKv8Lift), un = exp2i(-ev);
        sc = scale_of(k + 1);
        float x[64];
        auto load = [&] {
          tmem_ld32_async(tl + buf * 64, x);
          tmem_ld32_async(tl + buf * 64 + 32, x + 32);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 64; ++c) asm volatile("" : "+f"(x[c]));   // x is not used before the wait
          if (__builtin_expect(__any_sync(0xffffffffu, key0 < lo_last || key0 + 64 > hi_first), 0)) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c < lo - key0 || c >= hi - key0) x[c] = -INFINITY;
          }
        };
        // the reference that the block asks for (-infinity times gk stays -infinity: gk > 0)
        auto largest = [&] {
          float h[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int c = 4; c < 60; c += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = max3(h[i], x[c + i], x[c + 4 + i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = fmaxf(h[i], x[60 + i]);
          return on_grid(max3(h[0], h[1], fmaxf(h[2], h[3])) * gk);
        };
        load();
        if (!S::two) {
          // head_dim 256: the reference of the block before comes from the other group, this
          // block's goes to it
          const float mx = largest();
          if (j > 0) {
            named_bar_sync(1 + (grp ^ 1) * 4 + qd, 64);
            const float old = xch[((j - 1) & 1) * 128 + r];
            if (old != m) l *= exp2_approx(m - old);        // (m = -infinity: l is 0)
            m = old;
          }
          const float lag = static_cast<float>(min(kLag, kTop - 6 + kKv8Lift - ev));
          const bool move = mx > m + lag || (m == -INFINITY && mx > m);
          if (j + 1 < g.n) {
            xch[(j & 1) * 128 + r] = move ? mx : m;
            asm volatile("bar.arrive %0, 64;" ::"r"(1 + grp * 4 + qd) : "memory");
          }
          if (__any_sync(0xffffffffu, move)) move_to(move ? mx : m, k, j);
        }
        uint32_t pk[32];                                    // positions 2 i, 2 i + 1 of the block
        float sum;
        bool move = S::two && m == -INFINITY;
        bool check = S::two;
        // the weights of scores that `score` leaves relative to the reference
        auto weigh = [&](auto score) {
          float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            const float2 e = score(make_float2(x[c], x[c + 1]));
            const float2 w2 = make_float2(exp2_approx(e.x), exp2_approx(e.y));
            s2 = add2(s2, w2);
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(w2.x, w2.y);
            // tokens 16 w + 8 h + 2 t, + 1 stand at positions 16 t + 4 w + 2 h, + 1
            pk[((c >> 1) & 3) * 8 + (c >> 4) * 2 + ((c >> 3) & 1)] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          sum = s2.x + s2.y;
        };
        if (__builtin_expect(__any_sync(0xffffffffu, gk >= kFarFactor), 0)) {
          if (S::two) {
            const float mx = largest();
            if (__any_sync(0xffffffffu, mx > m)) move_to(fmaxf(m, mx), k, j);
          }
          const float ref = m == -INFINITY ? 0.0f : m;
          weigh([&](float2 v) {
            return make_float2((__fmul_rn(v.x, gk) - ref) + fv, (__fmul_rn(v.y, gk) - ref) + fv);
          });
        } else while (true) {
          if (S::two && __any_sync(0xffffffffu, move)) {
            const float mx = largest();
            move_to(move ? fmaxf(m, mx) : m, k, j);
          }
          const float off = fv - (m == -INFINITY ? 0.0f : m);
          weigh([&](float2 v) { return fma2(v, make_float2(gk, gk), make_float2(off, off)); });
          // head_dim <= 128: if the weights are too large for the reference as it stood, once
          // more with the scores read again (a NaN among them comes here too, and stays)
          move = !(sum <= exp2i(min(kTop, kMaxSum + ev)));
          if (__builtin_expect(!check || !__any_sync(0xffffffffu, move), 1)) break;
          check = false;
          load();
        }
        l = fmaf(sum, un, l);
        tmem_st32_async(tl + buf * 64, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull + 8 * buf);
      }

      // ---- the output
      const bool join = S::two && !pl.tiles;              // group 0 joins both lanes' outputs
      const int slot = g.slot, tr = row - g.tile * S::rows;
      float k0 = 1.0f, k1 = 0.0f;
      if (join) {
        float2* x = reinterpret_cast<float2*>(xch);
        if (grp == 1) x[r] = make_float2(m, l);
        named_bar_sync(9, 256);
        if (grp == 0) {
          const float2 y = x[r];
          const float mm = fmaxf(m, y.x);
          k0 = m == -INFINITY ? 1.0f : exp2_approx(m - mm);
          k1 = y.x == -INFINITY ? 1.0f : exp2_approx(y.x - mm);
          l = l * k0 + y.y * k1;
          m = mm;
        }
      } else if (!S::two) {
        named_bar_sync(10, 256);         // no reference in xch is read any more
        float2* x = reinterpret_cast<float2*>(xch);
        x[grp * 128 + r] = make_float2(m, l);
        named_bar_sync(10, 256);
        const float2 y = x[(grp ^ 1) * 128 + r];
        const float mm = fmaxf(m, y.x);  // the last block's, which the output is relative to
        l = l * (m == -INFINITY ? 1.0f : exp2_approx(m - mm)) + y.y * (y.x == -INFINITY ? 1.0f : exp2_approx(y.x - mm));
        m = mm;
      }
      if (!join || grp == 0) {
        // the last products on the outputs read here. A wait may look one phase ahead only, so the
        // groups of head_dim 256 wait for the last two blocks in order.
        if (S::two) {
          ok = ok && up && mbar_wait(odone + 8 * (2 * grp + ((steps - 1) & 1)), buf_parity(ph, grp, steps - 1), p.err);
          if (join && pl.steps[1] > 0) {
            const int e = pl.steps[1] - 1;
            ok = ok && up && mbar_wait(odone + 8 * (2 + (e & 1)), buf_parity(ph, 1, e), p.err);
          }
        } else {
          for (int t = max(0, g.n - 2); t < g.n; ++t)
            ok = ok && up && mbar_wait(odone + 8 * (2 * (t & 1) + ((t >> 1) & 1)), buf_parity(ph, t & 1, t >> 1), p.err);
        }
        tc_fence_after();
        const bool have1 = join && pl.steps[1] > 0;
        const float norm = l == 0.0f ? 0.0f : 1.0f / l;
        const int qi = p.by_group.div(row), qh = g.head * p.group + p.by_group.mod(row);
        __nv_bfloat16* dst = p.out + g.b * p.o_st[0] + qi * p.o_st[1] + qh * p.o_st[2];
        // a part's outputs: [D / 4][rows][4], so that neighbouring rows are neighbours
        float4* ws = reinterpret_cast<float4*>(p.ws + static_cast<size_t>(slot) * S::rows * D) + tr;
        const int c_from = S::two ? 0 : grp * (D / 2), c_to = S::two ? D : c_from + D / 2;
#pragma unroll 1
        for (int c = c_from; c < c_to; c += 32) {
          float y[32];
          tmem_ld32_async(tl + S::o_col + (S::two ? grp * D : 0) + c, y);
          if (have1) {
            float z[32];
            tmem_ld32_async(tl + S::o_col + D + c, z);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = fmaf(z[i], k1, y[i] * k0);
          } else {
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(y[i]));
          }
          if (row_ok && !g.whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              ws[(c + i) / 4 * S::rows] = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
          } else if (row_ok && c < p.c.D) {
            uint32_t o[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i] * norm, y[2 * i + 1] * norm);
              o[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
              st_global_32(dst + c, o);
              st_global_32(dst + c + 16, o + 8);
            } else {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<uint4*>(dst + c + 2 * i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
          }
        }
        if (row_ok && (S::two || grp == 0)) {
          if (!g.whole) p.ws_ml[slot * S::rows + tr] = make_float2(m, l);
          else if (p.lse) p.lse[(static_cast<size_t>(g.b) * p.n_q + qi) * p.n_heads + qh] = kv8_lse(m, l);
        }
        tc_fence_before();
      }
      // group 1 keeps its output and Q until group 0 has read them; at head_dim 256 neither group
      // goes on to a new output, Q or exchange before the other has read
      if (join || !S::two) named_bar_sync(join ? 9 : 10, 256);
      ph = next_phases(ph, pl);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 18) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
static cudaError_t launch_tc(const Kv8AttendParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Tc<D>::total;
  cfg.stream = s;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_attend_tc_kernel<D>, p);
  return e != cudaSuccess ? e : launch_kv8_merge(p, s);
}

cudaError_t launch_kv8_attend_tc(const Kv8AttendParams& p, cudaStream_t s) {
  if (p.c.Ds == 64) return launch_tc<64>(p, s);
  if (p.c.Ds == 128) return launch_tc<128>(p, s);
  return launch_tc<256>(p, s);
}

template <int D>
static cudaError_t configure_tc() {
  static_assert(Tc<D>::total <= 232448, "shared memory of a CTA");
  return cudaFuncSetAttribute(kv8_attend_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D>::total);
}

cudaError_t configure_kv8_tc_kernels() {
  cudaError_t e;
  if ((e = configure_tc<64>()) != cudaSuccess || (e = configure_tc<128>()) != cudaSuccess) return e;
  return configure_tc<256>();
}

}  // namespace vla
