// kv8.cuh -- the 8-bit K/V cache: layout, device helpers and kernel launchers (internal).
//
// Layout. For each (layer, slot, K/V head) the tokens are kept in blocks of 64. A block of K
// and a block of V are Ds rows of 64 bytes each (Ds = head_dim, at least 64), E4M3:
//   K  row p * 64 + i, byte c    = token i, dim 64 p + c          (panels of 64 dims)
//   V  row d, byte pos           = dim d, token tok(pos)          (transposed)
// with tok(16t + 4w + 2h + e) = 16w + 8h + 2t + e (t, w < 4; h, e < 2): the sixteen tokens that
// one lane of a matrix instruction needs of a row are one 16-byte chunk. Chunk c of row r stands
// at chunk c ^ ((r >> 1) & 3) of its row: the 64-byte swizzle of tcgen05.mma's K-major operands.
// So a block, or several in a row, comes to shared memory ready for use by one plain bulk copy.
// Scales: float4 (K scale, V scale, 0, 0) per block, powers of two, value = scale * e4m3.
// V never holds the E4M3 NaN: a token whose K or V row is not finite has a K row of NaN and
// a V row of zeros, so that a weight of zero makes a stored token count for nothing.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace vla {

// Byte of chunk c (16 bytes) of row r of a block.
__host__ __device__ constexpr int kv8_chunk(int r, int c) { return r * 64 + ((c ^ ((r >> 1) & 3)) << 4); }

constexpr int kKv8Block = 64;        // tokens per block
constexpr int kKv8MinExp = -60;      // smallest scale 2^-60
constexpr int kKv8BadRow = 2;        // device status: a row's slot, position or length is out of range

struct Kv8Cache {
  uint8_t* k;          // [L][slots][n_kv][nblk] blocks of Ds * 64 bytes
  uint8_t* v;
  float4* scale;       // [L][slots][n_kv][nblk]
  int n_layers, n_slots, n_kv, nblk, capacity, D, Ds;
};

// n / d for 0 <= n < 2^31 and a divisor d >= 1 fixed on the host: with 2^s >= d and
// m = ceil(2^(32 + s) / d) - 2^32, the quotient is (mulhi(n, m) + n) >> s.
struct FastDiv {
  uint32_t mul, shift;
  int d;
  FastDiv() = default;
  explicit FastDiv(int div) : d(div) {
    shift = 0;
    while ((1ull << shift) < static_cast<unsigned long long>(div)) ++shift;
    const unsigned long long m = ((1ull << shift) - static_cast<unsigned>(div)) << 32;
    mul = static_cast<uint32_t>((m + static_cast<unsigned>(div) - 1) / static_cast<unsigned>(div));
  }
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >> shift);
  }
  __device__ __forceinline__ int mod(int n) const { return n - div(n) * d; }
};

// Rows of a write or a read: row b holds tokens pos[b] .. pos[b] + count[b] - 1 of slots[b]
// (null: slot b, position 0, n_tokens tokens).
struct Kv8RowsParams {
  Kv8Cache c;
  const __nv_bfloat16 *k_in, *v_in;    // write
  __nv_bfloat16 *k_out, *v_out;        // read
  long long st_layer, st_row, st_tok;  // element strides of the bf16 side
  const int *slots, *pos, *count;
  int layer0, n_layers, batch, n_tokens, nblk_row;   // nblk_row: blocks a row can touch
  int sm_count;
  int* err;
};
cudaError_t launch_kv8_write(const Kv8RowsParams& p, cudaStream_t s);
cudaError_t launch_kv8_read(const Kv8RowsParams& p, cudaStream_t s);
cudaError_t configure_kv8_store_kernels();
cudaError_t launch_kv8_init(const Kv8Cache& c, cudaStream_t s);   // every scale to 2^-60

struct Kv8AttendParams {
  Kv8Cache c;
  const __nv_bfloat16* q;              // [batch][n_q][n_heads][D]
  __nv_bfloat16* out;
  float* lse;                          // [batch][n_q][n_heads] or null
  long long q_st[3], o_st[3];          // element strides: batch, token, head
  const int *slots, *kv_len, *q_pos, *q_count;   // slots, q_pos, q_count may be null
  int layer, batch, n_q, n_heads, group;         // group = n_heads / n_kv
  FastDiv by_group, by_tiles;
  int causal, window;
  float scale_log2;                    // softmax scale * log2(e)
  int tile_rows, tiles;                // query rows of a tile, tiles of a (row, K/V head)
  float* ws;                           // partial outputs [2 * CTAs][tile_rows][Ds]
  float2* ws_ml;                       // [2 * CTAs][tile_rows] (reference maximum, sum)
  int grid;                            // CTAs of the attention kernel
  int* err;
};

// ---- the division of the work
// An item is a tile of query rows of one (batch row, K/V head), its units the blocks of 64
// tokens that any of its queries can see. All units stand in a line (batch row, tile, K/V head, block),
// which `grid` - 1 cuts part into equal shares, one a CTA. So the CTAs have equal work for any
// lengths, and at most two of a CTA's items are shared with others. With many rows a cut costs as
// much as some units do (an output in 32 bits to write and to merge, one more tile of Q to bring
// in): there a cut that lies within `snap` units of an item's end moves to it. 400 rows in tiles of
// 128 against 64 slots of 788 keys (256 items of up to 13 units, 22 a CTA): 90.1 us with no cut
// moved, 88.1 with 4 units, 77.8 with 6 and with 12. Items of 64 to 96 units are the same either way;
// sizes between were not measured.

constexpr int kKv8Snap = 6;        // and no more than a third of a CTA's share

struct Kv8Tile {
  int slot, len, pos, cnt;             // slot < 0: refused, nothing of the row is written
  int blk0, units;                     // blocks any of its queries can see; units 0: no queries
};

__device__ __forceinline__ Kv8Tile kv8_tile(const Kv8AttendParams& p, int b, int tile) {
  Kv8Tile r;
  r.slot = p.slots ? p.slots[b] : b;
  r.len = p.kv_len[b];
  r.cnt = p.q_count ? p.q_count[b] : p.n_q;
  r.pos = p.q_pos ? p.q_pos[b] : r.len - r.cnt;
  r.blk0 = r.units = 0;
  if (r.cnt == 0) {                    // padding: names no slot, length or position
    r.slot = 0;
    return r;
  }
  if (r.slot < 0 || r.slot >= p.c.n_slots || r.len < 0 || r.len > p.c.capacity || r.cnt < 0 || r.cnt > p.n_q ||
      r.pos < -p.n_q || r.pos > p.c.capacity) {
    r.slot = -1;
    r.cnt = 0;
    return r;
  }
  const int i0 = p.by_group.div(tile * p.tile_rows);
  if (i0 >= r.cnt) return r;
  const int i1 = min(r.cnt - 1, p.by_group.div((tile + 1) * p.tile_rows - 1));
  const int hi = p.causal ? min(r.len, r.pos + i1 + 1) : r.len;
  const int lo = p.window ? max(0, r.pos + i0 - p.window + 1) : 0;
  r.blk0 = min(lo / kKv8Block, p.c.nblk - 1);
  r.units = max(1, (hi + kKv8Block - 1) / kKv8Block - r.blk0);   // one block even if no key is seen
  return r;
}

// Visible keys [lo, hi) of query token i of a row.
__device__ __forceinline__ void kv8_seen(const Kv8AttendParams& p, const Kv8Tile& r, int i, int& lo, int& hi) {
  hi = p.causal ? min(r.len, r.pos + i + 1) : r.len;
  lo = p.window ? max(0, r.pos + i - p.window + 1) : 0;
}

// Units of entry e = (batch row, tile), all K/V heads; 0 behind the last entry.
__device__ __forceinline__ int kv8_weight(const Kv8AttendParams& p, int e) {
  if (e >= p.batch * p.tiles) return 0;
  return kv8_tile(p, p.by_tiles.div(e), p.by_tiles.mod(e)).units * p.c.n_kv;
}

// The line of units of a call (fewer than 2^31: the host sees to it), as a warp sees it: every
// warp works it out for itself, up to 128 entries from one round of loads.
struct Kv8Line {
  int total, per, rem, snap;
  int w[4];                       // this lane's entries lane, lane + 32, ... (of the first 128)
};

__device__ __forceinline__ Kv8Line kv8_line(const Kv8AttendParams& p) {
  Kv8Line n;
  const int lane = threadIdx.x & 31;
  int sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    n.w[i] = kv8_weight(p, 32 * i + lane);
    sum += n.w[i];
  }
#pragma unroll 1
  for (int e = 128 + lane; e < p.batch * p.tiles; e += 32) sum += kv8_weight(p, e);
  n.total = __reduce_add_sync(0xffffffffu, sum);
  n.per = n.total / p.grid;
  n.rem = n.total % p.grid;
  n.snap = p.tile_rows > 16 ? min(kKv8Snap, n.per / 3) : 0;
  return n;
}

// Cut c, the first unit of part c, before it is moved: the parts differ by at most one unit.
__device__ __forceinline__ int kv8_begin(const Kv8Line& n, int c) { return c * n.per + min(c, n.rem); }

// The entry that holds unit u < total, and the unit's number inside it.
__device__ __forceinline__ int kv8_find(const Kv8AttendParams& p, const Kv8Line& n, int u, int* inside) {
  const int lane = threadIdx.x & 31;
  int at = 0;
#pragma unroll 1
  for (int i = 0;; ++i) {
    const int mine = i == 0 ? n.w[0] : i == 1 ? n.w[1] : i == 2 ? n.w[2] : i == 3 ? n.w[3] : kv8_weight(p, 32 * i + lane);
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, at + inc > u);
    if (past) {
      const int k = __ffs(past) - 1;
      *inside = u - at - __shfl_sync(0xffffffffu, inc - mine, k);
      return 32 * i + k;
    }
    at += __shfl_sync(0xffffffffu, inc, 31);
    if (32 * i + 32 >= p.batch * p.tiles) {   // u >= total: not reached
      *inside = 0;
      return 0;
    }
  }
}

// The segments of a CTA's part: its share of one item after the other.
struct Kv8Segment {
  Kv8Tile row;
  int b, head, tile;
  int blk, n;                     // blocks [blk, blk + n) of the slot
  bool whole;                     // the item's only part
  int slot;                       // its place in the workspace if it is not
};
// A CTA has at most one part that begins inside an item and one that begins with it and ends inside.
__device__ __forceinline__ int kv8_slot(int cta, bool begins) { return 2 * cta + (begins ? 1 : 0); }

// Where cut u lies, moved to an end of its item that is near.
__device__ __forceinline__ int kv8_place(const Kv8AttendParams& p, const Kv8Line& n, int u, Kv8Tile& row, int& e,
                                         int& inside) {
  e = kv8_find(p, n, u, &inside);
  row = kv8_tile(p, p.by_tiles.div(e), p.by_tiles.mod(e));
  if (n.snap) {
    const int off = inside % row.units, up = row.units - off;
    const int by = off <= min(n.snap, up) ? -off : up <= n.snap ? up : 0;
    inside += by;
    u += by;
  }
  return u;
}

struct Kv8Walk {
  int e, unit, left;
  Kv8Tile row;
};

__device__ __forceinline__ Kv8Walk kv8_walk(const Kv8AttendParams& p) {
  Kv8Walk w;
  const Kv8Line n = kv8_line(p);
  const int u0 = kv8_begin(n, blockIdx.x), u1 = kv8_begin(n, blockIdx.x + 1);
  w.left = u1 - u0;
  w.e = 0;
  w.unit = 0;
  if (w.left) {
    if (n.snap && u1 < n.total) w.left = kv8_place(p, n, u1, w.row, w.e, w.unit) - u0;
    w.left += u0 - kv8_place(p, n, u0, w.row, w.e, w.unit);
  }
  return w;
}

__device__ __forceinline__ bool kv8_next(const Kv8AttendParams& p, Kv8Walk& w, Kv8Segment& g) {
  if (w.left == 0) return false;
#pragma unroll 1
  while (w.unit >= w.row.units * p.c.n_kv) {
    ++w.e;
    w.unit = 0;
    w.row = kv8_tile(p, p.by_tiles.div(w.e), p.by_tiles.mod(w.e));
  }
  g.head = 0;                     // (a few K/V heads: subtraction is shorter than division)
  int off = w.unit;
#pragma unroll 1
  while (off >= w.row.units) {
    off -= w.row.units;
    ++g.head;
  }
  const int n = min(w.row.units - off, w.left);
  g.row = w.row;
  g.b = p.by_tiles.div(w.e);
  g.tile = w.e - g.b * p.tiles;
  g.blk = w.row.blk0 + off;
  g.n = n;
  g.whole = n == w.row.units;
  g.slot = kv8_slot(blockIdx.x, off == 0);
  w.unit += n;
  w.left -= n;
  return true;
}

// The merges look for the cuts of each item, if there are fewer items than cuts and a warp holds
// all entries; else for the item of each cut.
__host__ __device__ __forceinline__ bool kv8_merge_by_items(const Kv8AttendParams& p) {
  return p.batch * p.tiles <= 128 && p.batch * p.tiles * p.c.n_kv < p.grid - 1;
}

// A row's partial result is (m, l, o): m its reference, a score in bits (base 2); l the sum of
// 2^(s - m - kKv8Lift), o that of 2^(s - m - kKv8Lift) v. The lift keeps sums of V's largest values
// within fp32.
constexpr int kKv8Lift = 32;
// Natural logarithm of the sum of exp(score).
__device__ __forceinline__ float kv8_lse(float m, float l) {
  constexpr float up = 4294967296.0f;
  static_assert(up == static_cast<float>(1ull << kKv8Lift), "2^kKv8Lift");
  return l == 0.0f ? -INFINITY : (m + log2f(l * up)) * 0.6931471805599453f;
}

// Few rows (tile_rows 8 or 16) and many (128 or 256).
cudaError_t launch_kv8_attend_rows(const Kv8AttendParams& p, cudaStream_t s);
cudaError_t launch_kv8_attend_tc(const Kv8AttendParams& p, cudaStream_t s);
cudaError_t configure_kv8_tc_kernels();
cudaError_t launch_kv8_merge(const Kv8AttendParams& p, cudaStream_t s);
cudaError_t configure_kv8_kernels();

// E4M3 pairs (two bytes, low byte first) to and from half and float pairs.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ uint16_t f2_to_e4m3x2(float lo, float hi) {   // to nearest even, saturating; NaN stays NaN
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Exponent of the smallest power of two s >= 2^-60 with amax / s <= 448 = 1.75 * 2^8.
__device__ __forceinline__ int kv8_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffff) > 0x600000 ? 1 : 0);
  return max(e, kKv8MinExp);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ int exp_of(float s) { return static_cast<int>((__float_as_uint(s) >> 23) & 255) - 127; }

}  // namespace vla
