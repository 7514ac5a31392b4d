// kv8.cuh -- the 8-bit K/V cache: layout, device helpers and kernel launchers (internal).
//
// Layout. For each (layer, slot, K/V head) the tokens are kept in blocks of 64. A block of K
// and a block of V are Ds rows of 64 bytes each (Ds = head_dim, at least 64), E4M3:
//   K  row p * 64 + i, byte c    = token i, dim 64 p + c          (panels of 64 dims)
//   V  row d, byte 16 w + pos    = dim d, token 16 w + tok(pos)   (transposed)
// with tok(4t + 2h + e) = 8h + 2t + e (t < 4, h, e < 2): the four tokens that one lane of a
// 16 x 8 x 16 matrix instruction needs of a 16-token group are one 32-bit word. Both block
// kinds are one TMA box of Ds rows x 64 bytes under the 64-byte swizzle, which is also the
// K-major operand layout of tcgen05.mma, and a 32-bit read of 8 rows x 4 words of one chunk
// touches all 32 banks.
// Scales: float4 (K scale, V scale, 0, 0) per block, powers of two, value = scale * e4m3.
// V never holds the E4M3 NaN: a token whose K or V row is not finite has a K row of NaN and
// a V row of zeros, so that a weight of zero makes a stored token count for nothing.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace vla {

constexpr int kKv8Block = 64;        // tokens per block
constexpr int kKv8MinExp = -60;      // smallest scale 2^-60
constexpr int kKv8BadRow = 2;        // device status: a row's slot, position or length is out of range

struct Kv8Cache {
  uint8_t* k;          // [L][slots][n_kv][nblk] blocks of Ds * 64 bytes
  uint8_t* v;
  float4* scale;       // [L][slots][n_kv][nblk]
  int n_layers, n_slots, n_kv, nblk, capacity, D, Ds;
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
  int* err;
};
cudaError_t launch_kv8_write(const Kv8RowsParams& p, cudaStream_t s);
cudaError_t launch_kv8_read(const Kv8RowsParams& p, cudaStream_t s);
cudaError_t launch_kv8_init(const Kv8Cache& c, cudaStream_t s);   // every scale to 2^-60

struct Kv8AttendParams {
  Kv8Cache c;
  const __nv_bfloat16* q;              // [batch][n_q][n_heads][D]
  __nv_bfloat16* out;
  float* lse;                          // [batch][n_q][n_heads] or null
  long long q_st[3], o_st[3];          // element strides: batch, token, head
  const int *slots, *kv_len, *q_pos, *q_count;   // slots, q_pos, q_count may be null
  int layer, batch, n_q, n_heads, group;         // group = n_heads / n_kv
  int causal, window;
  float scale_log2;                    // softmax scale * log2(e)
  int tiles;                           // row tiles per (row, K/V head)
  float* ws;                           // partial outputs [2 * CTAs][tile rows][Ds]
  float2* ws_ml;                       // [2 * CTAs][tile rows] (running maximum, sum)
  int grid;                            // CTAs of the attention kernel
  int* err;
};

// One batch row as the attention kernels see it.
struct Kv8Row {
  int slot, len, pos, cnt;             // slot < 0: refused or empty, nothing is written
  int blk0, nblk;                      // blocks any of its queries can see (at least 1 if cnt > 0)
};

__device__ __forceinline__ Kv8Row kv8_row(const Kv8AttendParams& p, int b) {
  Kv8Row r;
  r.slot = p.slots ? p.slots[b] : b;
  r.len = p.kv_len[b];
  r.cnt = p.q_count ? p.q_count[b] : p.n_q;
  r.pos = p.q_pos ? p.q_pos[b] : r.len - r.cnt;
  r.blk0 = 0;
  r.nblk = 0;
  if (r.slot < 0 || r.slot >= p.c.n_slots || r.len < 0 || r.len > p.c.capacity || r.cnt < 0 || r.cnt > p.n_q ||
      r.pos < -p.n_q || r.pos > p.c.capacity) {
    r.slot = -1;
    r.cnt = 0;
    return r;
  }
  if (r.cnt == 0) return r;
  int hi = r.len, lo = 0;
  if (p.causal) hi = min(hi, r.pos + r.cnt);
  if (p.window) lo = max(0, r.pos - p.window + 1);
  r.blk0 = min(lo / kKv8Block, p.c.nblk - 1);
  r.nblk = max(1, (hi + kKv8Block - 1) / kKv8Block - r.blk0);
  return r;
}

// Visible keys [lo, hi) of query token i of a row.
__device__ __forceinline__ void kv8_seen(const Kv8AttendParams& p, const Kv8Row& r, int i, int& lo, int& hi) {
  hi = p.causal ? min(r.len, r.pos + i + 1) : r.len;
  lo = p.window ? max(0, r.pos + i - p.window + 1) : 0;
}

// The few-rows kernel: 16 query rows a tile. tm_k, tm_v: the whole cache as rows of 64 bytes.
cudaError_t launch_kv8_attend_rows(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Kv8AttendParams& p,
                                   cudaStream_t s);
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
