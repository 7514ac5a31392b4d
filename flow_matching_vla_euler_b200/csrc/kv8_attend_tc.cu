// kv8_attend_tc.cu -- attention over the 8-bit K/V cache for many query rows (an action chunk,
// a prompt piece), on the tcgen05 tensor cores.
//
// Same formula and the same equal division of the work as kv8_attend.cu, in tiles of 128
// query rows (head_dim 256) or 256 (smaller head_dim) and units of 128 keys. What bounds it
// is the tensor pipe and, at head_dim 64 and 128, the exponentials (16 a clock and SM).
//
//   S = Q K^T   kind::f8f6f4, K as the cache holds it (its block is already the operand's
//               64-byte swizzled K-major layout), Q as two E4M3 terms accumulated in one
//               sum: a row times the power of two that brings its largest magnitude to
//               [128, 256), hi = e4m3(q), lo = e4m3(q - hi). Exact for bf16 values above
//               2^-10 of the largest, else to 2^-17 of it. Two E4M3 products take as long as
//               one 16-bit product, and K needs no widening.
//   P           fp16, exp2(s + log2 s_V - m + 7): the V scale enters through the exponent and
//               leaves the sum in fp32; written over S in tensor memory, from where the
//               second product takes it. 2^7 lifts the range: weights down to 2^-31 of the
//               largest keep their place.
//   O += P V    kind::f16. Four warps widen V blocks to fp16 (exact) in the 128-byte swizzled
//               K-major layout; both query tiles use each widened block.
// m moves only when a tile's maximum passes it by more than 2^8 (then O in tensor memory is
// rescaled), so P stays below 2^15.
//
// Two lanes of work keep the tensor pipe busy while the softmax of the other lane runs:
//   head_dim <= 128, more than 128 rows: lane i is query tile i (128 rows), all keys.
//   head_dim <= 128, up to 128 rows: lane i takes every second unit of keys for the same rows,
//     with an output of its own; the two outputs are joined at the end.
//   head_dim 256: one tile and one output (256 columns); lane i is one of two S buffers, the
//     two softmax groups each take half of a unit's keys.
// Warps: 0 TMA, 1 MMA, 4..7 and 8..11 softmax (one thread a row), 12..15 widening of V.
#include "kernels.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace vla {

namespace {

constexpr int kKeys = 128;                   // keys of a unit (two blocks)
constexpr int kThreads = 512;
// Registers: 128 a thread at launch; the softmax groups go up to 200, the two others down to
// 56 (2 x 128 x 200 + 2 x 128 x 56 = 65536 = 512 x 128).
constexpr float kLift = 7.0f;

template <int D>
struct Tc {
  static constexpr bool two = D <= 128;                  // two query tiles a CTA
  static constexpr int rows = two ? 256 : 128;
  static constexpr int nk = D == 256 ? 2 : 3;            // K stages of a unit
  static constexpr int nv = D == 256 ? 2 : 4;            // V blocks as stored, and widened
  static constexpr int q_half = 128 * D;                 // one term of one tile
  static constexpr int v16 = 0;                          // 128-byte swizzle: 1024-byte aligned
  static constexpr int q = v16 + nv * D * 128;           // [tile][term][D / 64 panels][128 rows][64]
  static constexpr int k = q + (two ? 2 : 1) * 2 * q_half;
  static constexpr int v8 = k + nk * D * kKeys;
  static constexpr int xch = v8 + nv * D * 64;           // [2][2][128] floats
  static constexpr int bar = xch + 2048;
  static constexpr int total = bar + 512;
  static constexpr int o_col = 256;                      // tensor memory: S 0 and 128, O from 256
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
// E4M3 x E4M3 (kind::f8f6f4) and fp16 x fp16 (kind::f16): format fields 0, fp32 accumulator.
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
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

// A segment's units and how the lanes share them.
struct Plan {
  int units;
  bool tiles;            // lane = query tile (else: lane = every second unit, or S buffer)
};
template <int D>
__device__ __forceinline__ Plan make_plan(const Kv8AttendParams& p, const Kv8Segment& g) {
  Plan r;
  r.units = (g.n + 1) / 2;
  r.tiles = Tc<D>::two && g.row.cnt * p.group - g.tile * Tc<D>::rows > 128;
  return r;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_attend_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const Kv8AttendParams p) {
  using S = Tc<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sm = smem_u32(smem);
  const uint32_t kfull = sm + S::bar, kempty = kfull + 8 * S::nk;
  const uint32_t rfull = kempty + 8 * S::nk, rempty = rfull + 8 * S::nv;      // V as stored
  const uint32_t vfull = rempty + 8 * S::nv, vempty = vfull + 8 * S::nv;      // V widened
  const uint32_t sfull = vempty + 8 * S::nv, pfull = sfull + 16, odone = pfull + 32, qfull = odone + 16;   // pfull: [lane][block]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::bar + 504);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::nk; ++i) {
      mbar_init(kfull + 8 * i, 1);
      mbar_init(kempty + 8 * i, 1);
    }
    for (int i = 0; i < S::nv; ++i) {
      mbar_init(rfull + 8 * i, 1);
      mbar_init(rempty + 8 * i, 4);
      mbar_init(vfull + 8 * i, 4);
      mbar_init(vempty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull + 8 * i, 1);
      mbar_init(pfull + 16 * i, 4);
      mbar_init(pfull + 16 * i + 8, 4);
      mbar_init(odone + 8 * i, 1);
    }
    mbar_init(qfull, 8);
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    pdl_trigger();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (blockIdx.x == 0 && warp == 2)
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
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      // ---- loads: a unit of K, its blocks of V, in the order they are used
      const uint64_t pol = policy_evict_last();
      int kt = 0, vt = 0;
      while (ok && kv8_next(p, w, g)) {
        const size_t blk0 =
            ((static_cast<size_t>(p.layer) * p.c.n_slots + g.row.slot) * p.c.n_kv + g.head) * p.c.nblk + g.blk;
        for (int j = 0; j < g.n && ok; j += 2, ++kt) {
          const int n = min(2, g.n - j), s = kt % S::nk;
          if (kt >= S::nk && !mbar_wait(kempty + 8 * s, (kt / S::nk - 1) & 1, p.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(kfull + 8 * s, n * D * 64);
          for (int i = 0; i < n; ++i)
            // block i of panel c stands behind block 0's: rows of one panel of 128 keys are in line
            for (int c = 0; c < D / 64; ++c)
              tma_load_2d(sm + S::k + s * D * kKeys + (c * 128 + i * 64) * 64, &tm_k, kfull + 8 * s, 0,
                          static_cast<int>((blk0 + j + i) * D + c * 64), pol);
          for (int i = 0; i < n; ++i, ++vt) {
            const int r = vt % S::nv;
            if (vt >= S::nv && !mbar_wait(rempty + 8 * r, (vt / S::nv - 1) & 1, p.err)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(rfull + 8 * r, D * 64);
            tma_load_2d(sm + S::v8 + r * D * 64, &tm_v, rfull + 8 * r, 0, static_cast<int>((blk0 + j + i) * D), pol);
          }
        }
      }
      // no copies left in flight
      for (int i = kt > S::nk ? kt - S::nk : 0; i < kt; ++i) mbar_wait(kfull + 8 * (i % S::nk), (i / S::nk) & 1, p.err);
      for (int i = vt > S::nv ? vt - S::nv : 0; i < vt; ++i) mbar_wait(rfull + 8 * (i % S::nv), (i / S::nv) & 1, p.err);
    } else if (warp == 1) {
      // ---- products, by the converged warp. All that can wait before P arrives is done before:
      // once per unit the V blocks, the next unit's K and the operands' words
      const uint32_t lead = elect_one();
      // the warp stays together when a wait gives up
      auto wait_all = [&](uint32_t bar, uint32_t parity) {
        ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, parity, p.err)) != 0;
      };
      constexpr uint32_t id_s = idesc_fmt0(128, kKeys), id_o = idesc_fmt0(128, D);
      const uint32_t tm = uniform(tmem), q0 = uniform(desc_lo(sm + S::q));
      int ks = 0, vs = 0;                                 // next K stage and V block of the rings
      uint32_t kph = 0, vph = 0, qph = 0, pph = 0;        // phases; pph: bit i of lane i
      // scores of lane i: query tile at a0, K stage at b0
      auto scores = [&](int i, uint32_t a0, uint32_t b0) {
        if (!ok) return;
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            umma_f8(lead, tm + i * 128, a0 + ((term * S::q_half + (kk >> 1) * 8192) >> 4) + 2 * (kk & 1),
                    b0 + (((kk >> 1) * 8192) >> 4) + 2 * (kk & 1), id_s, (term | kk) != 0 ? 1u : 0u);
        umma_commit_if(lead, sfull + 8 * i);
      };
      // output of lane i: += P V over the unit's one or two blocks at b[]
      // (the blocks are free after it when `ve` is given; no commit follows the output's own, for
      // which the CTA waits before it ends)
      auto output = [&](int i, int n, const uint32_t (&b)[2], uint32_t acc, const uint32_t* ve) {
        const uint32_t d0 = tm + S::o_col + (S::two ? i * D : 0), a0 = tm + i * 128;
        wait_all(pfull + 16 * i, (pph >> i) & 1);
        tc_fence_after();
        if (ok)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) umma_f16_ts(lead, d0, a0 + kk * 8, b[0] + 2 * kk, id_o, kk == 0 ? acc : 1u);
        wait_all(pfull + 16 * i + 8, (pph >> i) & 1);
        tc_fence_after();
        if (ok && n == 2)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) umma_f16_ts(lead, d0, a0 + 32 + kk * 8, b[1] + 2 * kk, id_o, 1u);
        if (ok && ve) umma_commit_if(lead, ve[0]);
        if (ok && ve && n == 2) umma_commit_if(lead, ve[1]);
        if (ok) umma_commit_if(lead, odone + 8 * i);
        pph ^= 1u << i;
      };
      auto next_k = [&](uint32_t& b0, uint32_t& empty) {
        wait_all(kfull + 8 * ks, kph);
        b0 = uniform(desc_lo(sm + S::k + ks * D * kKeys));
        empty = kempty + 8 * ks;
        if (++ks == S::nk) {
          ks = 0;
          kph ^= 1;
        }
      };
      while (ok && kv8_next(p, w, g)) {
        const Plan pl = make_plan<D>(p, g);
        constexpr uint32_t kTile = (2 * S::q_half) >> 4;  // from one query tile to the next
        wait_all(qfull, qph);
        qph ^= 1;
        tc_fence_after();
        uint32_t kb = 0, ke = 0;
        next_k(kb, ke);
        scores(0, q0, kb);
        if (pl.tiles) {
          scores(1, q0 + kTile, kb);
        } else if (pl.units > 1) {
          if (ok) umma_commit_if(lead, ke);
          next_k(kb, ke);
          scores(1, q0, kb);
        }
        if (ok) umma_commit_if(lead, ke);
        for (int u = 0; u < pl.units && ok; ++u) {
          const int n = min(2, g.n - 2 * u);
          uint32_t vb[2] = {0, 0}, ve[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (c < n) {
              wait_all(vfull + 8 * vs, vph);
              vb[c] = uniform(desc_lo(sm + S::v16 + vs * D * 128));
              ve[c] = vempty + 8 * vs;
              if (++vs == S::nv) {
                vs = 0;
                vph ^= 1;
              }
            }
          const bool more = u + (pl.tiles ? 1 : 2) < pl.units;
          if (more) next_k(kb, ke);
          if (pl.tiles) {
            const uint32_t acc = u == 0 ? 0u : 1u;
            output(0, n, vb, acc, nullptr);
            if (more) scores(0, q0, kb);
            output(1, n, vb, acc, ve);
            if (more) scores(1, q0 + kTile, kb);
          } else {
            const int i = u & 1;
            const uint32_t acc = u < (S::two ? 2 : 1) ? 0u : 1u;
            output(i, n, vb, acc, ve);
            if (more) scores(i, q0, kb);
          }
          if (ok && more) umma_commit_if(lead, ke);
        }
      }
    }
    __syncwarp();
  } else if (warp >= 12) {
    // ---- V blocks to fp16: [D rows][64 positions] bytes, 64-byte swizzle, to halves, 128-byte
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
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
            y.x = e4m3x2_to_h2(static_cast<uint16_t>(x.x));
            y.y = e4m3x2_to_h2(static_cast<uint16_t>(x.x >> 16));
            y.z = e4m3x2_to_h2(static_cast<uint16_t>(x.y));
            y.w = e4m3x2_to_h2(static_cast<uint16_t>(x.y >> 16));
            z.x = e4m3x2_to_h2(static_cast<uint16_t>(x.z));
            z.y = e4m3x2_to_h2(static_cast<uint16_t>(x.z >> 16));
            z.z = e4m3x2_to_h2(static_cast<uint16_t>(x.w));
            z.w = e4m3x2_to_h2(static_cast<uint16_t>(x.w >> 16));
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    constexpr int kCols = S::two ? kKeys : kKeys / 2;     // keys of a unit a thread takes
    const int grp = (warp - 4) >> 2, qd = warp & 3, r = qd * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(qd * 32) << 16);
    float* xch = reinterpret_cast<float*>(smem + S::xch);
    int step[2] = {0, 0};                                 // S buffers (lanes) consumed so far
    while (kv8_next(p, w, g)) {
      const Plan pl = make_plan<D>(p, g);
      const int left = g.row.cnt * p.group - g.tile * S::rows;      // rows from the tile's first on
      const int r0 = g.tile * S::rows + (pl.tiles ? grp * 128 : 0); // first row of this group's tile
      const int row = r0 + r, rows = min(128, left - (pl.tiles ? grp * 128 : 0));
      const bool row_ok = r < rows;
      // ---- Q to E4M3 pairs: this thread's row (head_dim 256: half of it)
      float rowf = p.scale_log2;
      {
        constexpr int kQ = S::two ? D : D / 2;
        const int d0 = S::two ? 0 : grp * kQ;
        const bool load = S::two ? (pl.tiles || grp == 0) : true;
        const __nv_bfloat16* q = p.q + g.b * p.q_st[0] + (row / p.group) * p.q_st[1] +
                                 (g.head * p.group + row % p.group) * p.q_st[2] + d0;
        uint4 x[kQ / 8];
        float am = 0.0f;
        // the second group of a one-tile segment needs the row's factor only, from the same values
#pragma unroll
        for (int i = 0; i < kQ / 8; ++i) {
          x[i] = make_uint4(0, 0, 0, 0);
          if (row_ok && d0 + i * 8 < p.c.D) x[i] = *reinterpret_cast<const uint4*>(q + i * 8);
          const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float a = fabsf(__uint_as_float(v[c] << 16)), b = fabsf(__uint_as_float(v[c] & 0xffff0000u));
            am = fmaxf(am, fmaxf(a < INFINITY ? a : 0.0f, b < INFINITY ? b : 0.0f));
          }
        }
        if (!S::two) {
          xch[grp * 128 + r] = am;
          named_bar_sync(1 + qd, 64);
          am = fmaxf(am, xch[(grp ^ 1) * 128 + r]);
          named_bar_sync(1 + qd, 64);
        }
        const int e = am > 0.0f ? min(max(exp_of(am) - 7, -118), 120) : 0;
        const float inv = exp2i(-e);
        rowf *= exp2i(e);
        if (load) {
          uint8_t* dst = smem + S::q + (pl.tiles ? grp * 2 * S::q_half : 0) + r * 64;
#pragma unroll
          for (int i = 0; i < kQ / 16; ++i) {             // 16 dims: one 16-byte chunk of each term
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint4 y = x[2 * i + (c >> 1)];
              const uint32_t v0 = (c & 1) ? y.z : y.x, v1 = (c & 1) ? y.w : y.y;
              float f[4] = {__uint_as_float(v0 << 16) * inv, __uint_as_float(v0 & 0xffff0000u) * inv,
                            __uint_as_float(v1 << 16) * inv, __uint_as_float(v1 & 0xffff0000u) * inv};
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
            const int d = d0 + i * 16;
            uint8_t* a = dst + (d >> 6) * 8192 + ((((d >> 4) & 3) ^ ((r >> 1) & 3)) << 4);
            *reinterpret_cast<uint4*>(a) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(a + S::q_half) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(qfull);
      }

      int lo, hi, lo_last, hi_first, t0, t1;
      kv8_seen(p, g.row, row / p.group, lo, hi);
      kv8_seen(p, g.row, r0 / p.group, t0, hi_first);
      kv8_seen(p, g.row, (r0 + max(rows, 1) - 1) / p.group, lo_last, t1);
      const float4* scales = p.c.scale +
          ((static_cast<size_t>(p.layer) * p.c.n_slots + g.row.slot) * p.c.n_kv + g.head) * p.c.nblk;
      const int last_blk = g.blk + g.n - 1;
      const int u_step = S::two && !pl.tiles ? 2 : 1;
      int u = S::two && !pl.tiles ? grp : 0;
      float4 sc[2];                                       // scales of the next unit's blocks
      auto load_scales = [&](int unit) {
        const int b = g.blk + 2 * unit;
        if (S::two) {
          sc[0] = __ldg(scales + min(b, last_blk));
          sc[1] = __ldg(scales + min(b + 1, last_blk));
        } else {
          sc[0] = __ldg(scales + min(b + grp, last_blk));
        }
      };
      load_scales(min(u, pl.units - 1));
      float m = -INFINITY, l = 0.0f;
      bool begun = false;                                 // this output holds something
      int buf = S::two ? grp : 0;
      for (; u < pl.units; u += u_step) {
        if (!S::two) buf = u & 1;
        ok = ok && mbar_wait(sfull + 8 * buf, step[buf] & 1, p.err);
        tc_fence_after();
        float x[kCols];
        const uint32_t ts = tl + buf * 128 + (S::two ? 0 : grp * 64);
#pragma unroll
        for (int c = 0; c < kCols; c += 32) tmem_ld32_async(ts + c, x + c);
        float gk[S::two ? 2 : 1], fv[S::two ? 2 : 1], un[S::two ? 2 : 1];
#pragma unroll
        for (int i = 0; i < (S::two ? 2 : 1); ++i) {
          gk[i] = rowf * sc[i].x;
          const int ev = exp_of(sc[i].y);
          fv[i] = static_cast<float>(ev);
          un[i] = exp2i(-ev);
        }
        load_scales(min(u + u_step, pl.units - 1));
        const int key0 = (g.blk + 2 * u) * kKv8Block + (S::two ? 0 : grp * 64);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kCols; ++c) asm volatile("" : "+f"(x[c]));   // not used before the wait
        if (key0 < lo_last || key0 + kCols > hi_first) {
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (c < lo - key0 || c >= hi - key0) x[c] = -INFINITY;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < kCols / 64; ++i) {
          float h[4] = {x[64 * i], x[64 * i + 1], x[64 * i + 2], x[64 * i + 3]};
#pragma unroll
          for (int c = 4; c < 60; c += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = max3(h[k], x[64 * i + c + k], x[64 * i + c + 4 + k]);
#pragma unroll
          for (int k = 0; k < 4; ++k) h[k] = fmaxf(h[k], x[64 * i + 60 + k]);
          mx = fmaxf(mx, fmaf(fmaxf(fmaxf(h[0], h[1]), fmaxf(h[2], h[3])), gk[i], fv[i]));
        }
        if (!S::two) {                                    // the row's maximum over both halves
          xch[((u & 1) * 2 + grp) * 128 + r] = mx;
          named_bar_sync(1 + qd, 64);
          mx = fmaxf(mx, xch[((u & 1) * 2 + (grp ^ 1)) * 128 + r]);
        }
        const bool move = mx > m + 8.0f || (m == -INFINITY && mx > m);
        if (__any_sync(0xffffffffu, move)) {
          const float nm = move ? mx : m;
          const float k = nm == m ? 1.0f : exp2_approx(m - nm);
          m = nm;
          l *= k;
          if (begun) {                                    // rescale this warp's rows of O
            const int ob = S::two ? buf : (u - 1) & 1;
            ok = ok && mbar_wait(odone + 8 * ob, (step[ob] - 1) & 1, p.err);
            tc_fence_after();
            const uint32_t to = tl + S::o_col + (S::two ? grp * D : grp * (D / 2));
#pragma unroll 1
            for (int c = 0; c < (S::two ? D : D / 2); c += 32) {
              float y[32];
              tmem_ld32_async(to + c, y);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] *= k;
              tmem_st32_async(to + c, reinterpret_cast<uint32_t*>(y));
            }
            tmem_wait_st();
          }
        }
        begun = true;
        const float base = m == -INFINITY ? 0.0f : kLift - m;
#pragma unroll
        for (int i = 0; i < kCols / 64; ++i) {
          const float off = fv[i] + base;
          float s0 = 0.0f, s1 = 0.0f;
          uint32_t pk[32];                                // positions 2 k, 2 k + 1 of the block
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            const float a = exp2_approx(fmaf(x[64 * i + c], gk[i], off));
            const float b = exp2_approx(fmaf(x[64 * i + c + 1], gk[i], off));
            s0 += a;
            s1 += b;
            const __half2 h2 = __floats2half2_rn(a, b);
            // tokens 8 h + 2 t, + 1 of a 16-token group stand at positions 4 t + 2 h, + 1
            const int k = (c >> 4) * 8 + ((c >> 1) & 3) * 2 + ((c >> 3) & 1);
            pk[k] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          l = fmaf(s0 + s1, un[i], l);
          const int blk = S::two ? i : grp;
          tmem_st32_async(tl + buf * 128 + blk * 32, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(pfull + 16 * buf + 8 * blk);
        }
        ++step[buf];
      }

      // ---- the output. One tile on two lanes (head_dim <= 128): group 0 joins both outputs
      const bool join = S::two && !pl.tiles;
      if (!S::two) {                     // in the half of xch that the last unit did not use
        float* x = xch + (pl.units & 1) * 256;
        x[grp * 128 + r] = l;
        named_bar_sync(1 + qd, 64);
        l += x[(grp ^ 1) * 128 + r];
        named_bar_sync(1 + qd, 64);
      }
      float k0 = 1.0f, k1 = 0.0f;
      bool have1 = false;
      if (join) {
        if (grp == 1) {
          xch[r] = m;
          xch[128 + r] = l;
        }
        named_bar_sync(5, 256);
        if (grp == 0) {
          have1 = pl.units > 1;
          const float m1 = xch[r], l1 = xch[128 + r];
          const float mm = fmaxf(m, m1);
          k0 = m == -INFINITY ? 1.0f : exp2_approx(m - mm);
          k1 = m1 == -INFINITY ? 1.0f : exp2_approx(m1 - mm);
          l = l * k0 + l1 * k1;
          m = mm;
          if (have1) ok = ok && mbar_wait(odone + 8, (step[1] + pl.units / 2 - 1) & 1, p.err);
        }
      }
      if (!join || grp == 0) {
        const int ob = S::two ? buf : (pl.units - 1) & 1;
        ok = ok && mbar_wait(odone + 8 * ob, (step[ob] - 1) & 1, p.err);
        tc_fence_after();
        const float norm = g.whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
        const int qi = row / p.group, qh = g.head * p.group + row % p.group;
        const int slot = 2 * blockIdx.x + (g.first ? 0 : 1), tr = row - g.tile * S::rows;
        __nv_bfloat16* dst = p.out + g.b * p.o_st[0] + qi * p.o_st[1] + qh * p.o_st[2];
        float* ws = p.ws + (static_cast<size_t>(slot) * S::rows + tr) * D;
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
          }
          if (row_ok && !g.whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(ws + c + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
          } else if (row_ok && c < p.c.D) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t o[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(y[i + 2 * k] * norm, y[i + 2 * k + 1] * norm);
                o[k] = *reinterpret_cast<const uint32_t*>(&h);
              }
              *reinterpret_cast<uint4*>(dst + c + i) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
        if (row_ok && (S::two || grp == 0)) {
          if (!g.whole) p.ws_ml[slot * S::rows + tr] = make_float2(m - kLift, l);
          else if (p.lse)
            p.lse[(static_cast<size_t>(g.b) * p.n_q + qi) * p.n_heads + qh] =
                l == 0.0f ? -INFINITY : (m - kLift + log2f(l)) * 0.6931471805599453f;
        }
        tc_fence_before();
      }
      if (join) {
        named_bar_sync(5, 256);          // group 1 keeps its output and Q until group 0 has read them
      }
      if (S::two && !pl.tiles && grp == 0) step[1] += pl.units / 2;
      if (S::two && !pl.tiles && grp == 1) step[0] += (pl.units + 1) / 2;
      if (S::two && pl.tiles) step[grp ^ 1] += pl.units;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
static cudaError_t launch_tc(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Kv8AttendParams& p,
                             cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Tc<D>::total;
  cfg.stream = s;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_attend_tc_kernel<D>, tm_k, tm_v, p);
  return e != cudaSuccess ? e : launch_kv8_merge(p, s);
}

cudaError_t launch_kv8_attend_tc(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Kv8AttendParams& p,
                                 cudaStream_t s) {
  if (p.c.Ds == 64) return launch_tc<64>(tm_k, tm_v, p, s);
  if (p.c.Ds == 128) return launch_tc<128>(tm_k, tm_v, p, s);
  return launch_tc<256>(tm_k, tm_v, p, s);
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
