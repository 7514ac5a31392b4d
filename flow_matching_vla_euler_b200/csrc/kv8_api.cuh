// kv8_api.cuh -- host runtime of the 8-bit K/V cache (vla_kv8_* in include/vla.h).
//
// Part of the api.cu translation unit (included at its end): it reuses that file's
// allocation and error helpers. The handle owns the blocks, their scales, the attention
// workspace and a status word; every call after create only launches kernels, so all of
// them can be captured into a graph.

struct vla_kv8 {
  vla_kv8_config cfg;
  int dev = 0, sm_count = 148;
  std::vector<void*> allocs;
  Kv8Cache c{};
  float* ws = nullptr;
  float2* ws_ml = nullptr;
  int* err = nullptr;
};

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Query rows of a tile of the many-rows kernel.
int kv8_tc_rows(const Kv8Cache& c) { return c.Ds == 256 ? 128 : 256; }

int kv8_validate(const vla_kv8_config* c) {
  if (!c) return fail(VLA_ERR_ARG, "null config");
  if (c->flags) return fail(VLA_ERR_ARG, "unknown flag bits 0x%x", c->flags);
  if (c->n_layers < 1 || c->n_kv_heads < 1 || c->n_slots < 1 || c->capacity < 1)
    return fail(VLA_ERR_SHAPE, "n_layers, n_kv_heads, n_slots and capacity must be >= 1");
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(VLA_ERR_SHAPE, "head_dim %d: 32, 64, 128 or 256", c->head_dim);
  if (c->capacity > (1 << 30)) return fail(VLA_ERR_SHAPE, "capacity %d: at most 2^30 tokens", c->capacity);
  const double blocks = static_cast<double>(c->n_layers) * c->n_slots * c->n_kv_heads *
                        ((c->capacity + kKv8Block - 1) / kKv8Block);
  if (blocks > 2147483647.0) return fail(VLA_ERR_SHAPE, "%.0f blocks of 64 tokens, at most 2^31 - 1", blocks);
  return VLA_OK;
}

// The checks that write and read share. A row touches at most *nblk_row blocks.
int kv8_rows(vla_kv8* h, const vla_kv8_rows* r, const void* K, const void* V, bool out, Kv8RowsParams* p) {
  if (!h || !r || !K || !V) return fail(VLA_ERR_ARG, "null argument");
  if ((reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(V)) & 15)
    return fail(VLA_ERR_ARG, "K and V must be 16-byte aligned");
  int dev = 0;
  CU(cudaGetDevice(&dev));
  if (dev != h->dev) return fail(VLA_ERR_STATE, "the cache is on device %d, the current device is %d", h->dev, dev);
  if (r->layer < 0 || r->n_layers < 1 || r->n_layers > h->cfg.n_layers - r->layer)
    return fail(VLA_ERR_SHAPE, "layers %d to %d of %d", r->layer, r->layer + r->n_layers - 1, h->cfg.n_layers);
  if (r->batch < 1 || (!r->slots && r->batch > h->cfg.n_slots))
    return fail(VLA_ERR_SHAPE, "batch %d: at least 1, at most %d slots", r->batch, h->cfg.n_slots);
  if (r->n_tokens < 1 || r->n_tokens > h->cfg.capacity)
    return fail(VLA_ERR_SHAPE, "n_tokens %d outside [1, %d]", r->n_tokens, h->cfg.capacity);
  const long long w = static_cast<long long>(h->c.n_kv) * h->c.D;
  const bool packed = !r->stride[0] && !r->stride[1] && !r->stride[2];
  p->st_tok = packed ? w : r->stride[2];
  p->st_row = packed ? w * r->n_tokens : r->stride[1];
  p->st_layer = packed ? w * r->n_tokens * r->batch : r->stride[0];
  if (p->st_tok < 0 || p->st_row < 0 || p->st_layer < 0 || (p->st_tok | p->st_row | p->st_layer) % 8)
    return fail(VLA_ERR_ARG, "strides must be multiples of 8 elements, none negative");
  if (out && ((!p->st_tok && r->n_tokens > 1) || (!p->st_row && r->batch > 1) || (!p->st_layer && r->n_layers > 1)))
    return fail(VLA_ERR_ARG, "an output stride of 0");
  const int nb = (r->n_tokens + kKv8Block - 1) / kKv8Block;
  p->sm_count = h->sm_count;
  p->nblk_row = std::min(h->c.nblk, r->pos ? (r->n_tokens + 2 * kKv8Block - 2) / kKv8Block : nb);
  const double units = static_cast<double>(r->n_layers) * r->batch * h->c.n_kv * p->nblk_row;
  if (units > 2147483647.0) return fail(VLA_ERR_SHAPE, "%.0f blocks in one call, at most 2^31 - 1", units);
  p->c = h->c;
  p->slots = r->slots;
  p->pos = r->pos;
  p->count = r->count;
  p->layer0 = r->layer;
  p->n_layers = r->n_layers;
  p->batch = r->batch;
  p->n_tokens = r->n_tokens;
  p->err = h->err;
  return VLA_OK;
}

}  // namespace

extern "C" {

int vla_kv8_create(const vla_kv8_config* cfg, vla_kv8** out) {
  g_err.clear();
  if (!out) return fail(VLA_ERR_ARG, "null out");
  *out = nullptr;
  int rc = kv8_validate(cfg);
  if (rc) return rc;
  int dev = 0, major = 0, sm_count = 0;
  CU(cudaGetDevice(&dev));
  CU(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
  if (major != 10) return fail(VLA_ERR_UNSUPPORTED, "device is sm_%d0; this library is built for sm_100a", major);
  CU(cudaDeviceGetAttribute(&sm_count, cudaDevAttrMultiProcessorCount, dev));
  vla_kv8* h = new (std::nothrow) vla_kv8();
  if (!h) return fail(VLA_ERR_OOM, "host allocation failed");
  h->cfg = *cfg;
  h->dev = dev;
  h->sm_count = sm_count;
  auto cleanup = [&](int code) {
    vla_kv8_destroy(h);
    cudaGetLastError();   // a failed allocation is reported here, not by the next launch
    return code;
  };
  try {
    h->allocs.reserve(8);
  } catch (const std::bad_alloc&) {
    return cleanup(fail(VLA_ERR_OOM, "host allocation failed"));
  }
  Kv8Cache& c = h->c;
  c.n_layers = cfg->n_layers;
  c.n_slots = cfg->n_slots;
  c.n_kv = cfg->n_kv_heads;
  c.capacity = cfg->capacity;
  c.nblk = cdiv(cfg->capacity, kKv8Block);
  c.D = cfg->head_dim;
  c.Ds = std::max(64, cfg->head_dim);
  const size_t blocks = static_cast<size_t>(c.n_layers) * c.n_slots * c.n_kv * c.nblk;
  if ((rc = dalloc(h, &c.k, blocks * c.Ds * 64))) return cleanup(rc);
  if ((rc = dalloc(h, &c.v, blocks * c.Ds * 64))) return cleanup(rc);
  if ((rc = dalloc(h, &c.scale, blocks))) return cleanup(rc);
  if ((rc = dalloc(h, &h->ws, static_cast<size_t>(2) * sm_count * kv8_tc_rows(c) * c.Ds))) return cleanup(rc);
  if ((rc = dalloc(h, &h->ws_ml, static_cast<size_t>(2) * sm_count * kv8_tc_rows(c)))) return cleanup(rc);
  if ((rc = dalloc(h, &h->err, 1))) return cleanup(rc);
  CU_CLEANUP(configure_kv8_store_kernels());
  CU_CLEANUP(configure_kv8_kernels());
  CU_CLEANUP(configure_kv8_tc_kernels());
  CU_CLEANUP(launch_kv8_init(c, 0));
  CU_CLEANUP(cudaDeviceSynchronize());
  *out = h;
  return VLA_OK;
}

void vla_kv8_destroy(vla_kv8* h) {
  if (!h) return;
  cudaDeviceSynchronize();
  for (void* p : h->allocs) cudaFree(p);
  delete h;
}

int vla_kv8_write(vla_kv8* h, const uint16_t* K, const uint16_t* V, const vla_kv8_rows* rows, void* cuda_stream) {
  g_err.clear();
  Kv8RowsParams p{};
  int rc = kv8_rows(h, rows, K, V, false, &p);
  if (rc) return rc;
  p.k_in = reinterpret_cast<const bf16*>(K);
  p.v_in = reinterpret_cast<const bf16*>(V);
  CU(launch_kv8_write(p, static_cast<cudaStream_t>(cuda_stream)));
  return VLA_OK;
}

int vla_kv8_read(vla_kv8* h, uint16_t* K_out, uint16_t* V_out, const vla_kv8_rows* rows, void* cuda_stream) {
  g_err.clear();
  Kv8RowsParams p{};
  int rc = kv8_rows(h, rows, K_out, V_out, true, &p);
  if (rc) return rc;
  p.k_out = reinterpret_cast<bf16*>(K_out);
  p.v_out = reinterpret_cast<bf16*>(V_out);
  CU(launch_kv8_read(p, static_cast<cudaStream_t>(cuda_stream)));
  return VLA_OK;
}

int vla_kv8_attend(vla_kv8* h, const uint16_t* q, uint16_t* out, float* lse, const vla_kv8_query* a,
                   void* cuda_stream) {
  g_err.clear();
  if (!h || !q || !out || !a || !a->kv_len) return fail(VLA_ERR_ARG, "null argument");
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15)
    return fail(VLA_ERR_ARG, "q and out must be 16-byte aligned");
  int dev = 0;
  CU(cudaGetDevice(&dev));
  if (dev != h->dev) return fail(VLA_ERR_STATE, "the cache is on device %d, the current device is %d", h->dev, dev);
  if (a->layer < 0 || a->layer >= h->cfg.n_layers)
    return fail(VLA_ERR_SHAPE, "layer %d of %d", a->layer, h->cfg.n_layers);
  if (a->batch < 1 || (!a->slots && a->batch > h->cfg.n_slots))
    return fail(VLA_ERR_SHAPE, "batch %d: at least 1, at most %d slots", a->batch, h->cfg.n_slots);
  if (a->n_heads < 1 || a->n_heads % h->c.n_kv)
    return fail(VLA_ERR_SHAPE, "n_heads %d: a positive multiple of %d K/V heads", a->n_heads, h->c.n_kv);
  if (a->n_q < 1 || a->n_q > (1 << 20)) return fail(VLA_ERR_SHAPE, "n_q %d outside [1, 2^20]", a->n_q);
  if (a->causal != 0 && a->causal != 1) return fail(VLA_ERR_ARG, "causal %d: 0 or 1", a->causal);
  if (a->window < 0 || a->window > (1 << 30)) return fail(VLA_ERR_ARG, "window %d outside [0, 2^30]", a->window);
  if (!(a->scale >= 0.0f) || std::isinf(a->scale * kLog2e))
    return fail(VLA_ERR_ARG, "scale must be >= 0, and finite times log2(e)");
  Kv8AttendParams p{};
  const long long w = static_cast<long long>(a->n_heads) * h->c.D;
  for (int i = 0; i < 2; ++i) {
    const long long* st = i ? a->out_stride : a->q_stride;
    long long* d = i ? p.o_st : p.q_st;
    const bool packed = !st[0] && !st[1] && !st[2];
    d[0] = packed ? w * a->n_q : st[0];
    d[1] = packed ? w : st[1];
    d[2] = packed ? h->c.D : st[2];
    if (d[0] < 0 || d[1] < 0 || d[2] < 0 || (d[0] | d[1] | d[2]) % 8)
      return fail(VLA_ERR_ARG, "strides must be multiples of 8 elements, none negative");
    if (i && ((!d[0] && a->batch > 1) || (!d[1] && a->n_q > 1) || (!d[2] && a->n_heads > 1)))
      return fail(VLA_ERR_ARG, "an output stride of 0");
  }
  p.c = h->c;
  p.q = reinterpret_cast<const bf16*>(q);
  p.out = reinterpret_cast<bf16*>(out);
  p.lse = lse;
  p.slots = a->slots;
  p.kv_len = a->kv_len;
  p.q_pos = a->q_pos;
  p.q_count = a->q_count;
  p.layer = a->layer;
  p.batch = a->batch;
  p.n_q = a->n_q;
  p.n_heads = a->n_heads;
  p.group = a->n_heads / h->c.n_kv;
  p.causal = a->causal;
  p.window = a->window;
  p.scale_log2 = (a->scale > 0.0f ? a->scale : 1.0f / sqrtf(static_cast<float>(h->c.D))) * kLog2e;
  p.err = h->err;
  p.ws = h->ws;
  p.ws_ml = h->ws_ml;
  const double rows = static_cast<double>(a->n_q) * p.group;
  // One tile of 16 rows: the kernel for few rows. Two: also, if there are so few of them that its
  // shorter start counts for more than reading the keys twice (20 rows of head_dim 128, 8 K/V heads,
  // few and many: 4 x 512 keys 24.5 and 30.2 us, 4 x 4096 36.9 and 47.1, 16 x 4096 86.0 and 77.8; 32
  // rows of head_dim 256, 32 x 788 41.0 and 45.1, 64 x 788 57.3 and 43.0).
  const bool few = rows <= 16 || (rows <= 32 && static_cast<double>(a->batch) * h->c.n_kv <= 32);
  p.tile_rows = rows <= 8 ? 8 : few ? 16 : kv8_tc_rows(h->c);
  const double tiles = std::ceil(rows / p.tile_rows);
  const double units = tiles * h->c.n_kv * a->batch * h->c.nblk;
  if (units > 2147483647.0)
    return fail(VLA_ERR_SHAPE, "%.0f units of work (tiles of %d query rows times blocks), at most 2^31 - 1 a call", units,
                p.tile_rows);
  // (the kernels number the query rows of a K/V head by an int, to the end of the last tile)
  if (tiles * p.tile_rows > 2147483647.0)
    return fail(VLA_ERR_SHAPE, "%.0f query rows a K/V head (n_q * n_heads / n_kv_heads), fewer than 2^31 a call", rows);
  p.tiles = static_cast<int>(tiles);
  p.by_group = FastDiv(p.group);
  p.by_tiles = FastDiv(p.tiles);
  p.grid = static_cast<int>(std::min(units, static_cast<double>(h->sm_count)));
  if (few) CU(launch_kv8_attend_rows(p, static_cast<cudaStream_t>(cuda_stream)));
  else CU(launch_kv8_attend_tc(p, static_cast<cudaStream_t>(cuda_stream)));
  return VLA_OK;
}

int vla_kv8_status(vla_kv8* h, void* cuda_stream) {
  g_err.clear();
  if (!h) return fail(VLA_ERR_ARG, "null handle");
  CU(cudaStreamSynchronize(static_cast<cudaStream_t>(cuda_stream)));
  int v = 0;
  CU(cudaMemcpy(&v, h->err, sizeof(int), cudaMemcpyDeviceToHost));
  if (v == 0) return VLA_OK;
  CU(cudaMemset(h->err, 0, sizeof(int)));
  CU(cudaDeviceSynchronize());
  if (v == kKv8BadRow)
    return fail(VLA_ERR_SHAPE, "a row's slot, position, length or count was out of range, or two rows of a write "
                               "named one slot; such rows were left out; the status word was cleared");
  return fail(VLA_ERR_TIMEOUT, "a bounded wait gave up inside a cache kernel (device status %d); the word was cleared", v);
}

}  // extern "C"
