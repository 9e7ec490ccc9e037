// kv4_attention.cu -- dspark_kv4_attention (include/dspark_kv4.h): argument
// checks, the workspace, the choice of kernel.
#include <math.h>

#include "kv4_attn.cuh"

namespace dspark {
namespace kv4 {
namespace {

// Rows of a request's tile grid up to which the small kernel serves a call:
// its tiles have up to 16 rows.
constexpr int64_t kSmallRows = 16;

// Partial sums of one call: tiles of up to 16 or 256 rows.
int64_t slots_bytes(int64_t rows, int dim) {
  return 2 * kMaxGrid * (rows <= kSmallRows ? 16 : rows <= 128 ? 128 : 256) * static_cast<int64_t>(dim + 2) * 4;
}

}  // namespace
}  // namespace kv4
}  // namespace dspark

extern "C" {

size_t dspark_kv4_attention_workspace_bytes(const dspark_kv4_cache* cache, const dspark_kv4_batch* batch,
                                            int32_t q_heads) {
  using namespace dspark::kv4;
  Cache c;
  Batch s;
  if (make_cache(cache, &c) != DSPARK_OK || make_batch(batch, c, &s) != DSPARK_OK || q_heads < 1 ||
      q_heads % c.kv_heads != 0)
    return 0;
  return static_cast<size_t>(kCutBytes + slots_bytes(static_cast<int64_t>(batch->max_rows) * (q_heads / c.kv_heads), cache->head_dim));
}

int dspark_kv4_attention(const dspark_kv4_cache* cache, const dspark_kv4_batch* batch,
                         const dspark_kv4_attention_args* args, cudaStream_t stream) {
  using namespace dspark::kv4;
  Attn a{};
  int rc = make_cache(cache, &a.c);
  if (rc != DSPARK_OK) return rc;
  rc = make_batch(batch, a.c, &a.s);
  if (rc != DSPARK_OK) return rc;
  if (!args) return DSPARK_ERR_INVALID_ARG;
  if (args->dtype != DSPARK_DTYPE_BF16 && args->dtype != DSPARK_DTYPE_F16) return DSPARK_ERR_INVALID_ARG;
  if (args->q_heads < 1 || args->q_heads % a.c.kv_heads != 0 || args->window < 0 || !isfinite(args->scale))
    return DSPARK_ERR_INVALID_ARG;
  if (args->q_row < 0 || args->q_head < 0 || args->out_row < 0 || args->out_head < 0) return DSPARK_ERR_INVALID_ARG;
  if (static_cast<int64_t>(a.s.total_rows) * args->q_heads > 0x7FFFFFFF) return DSPARK_ERR_INVALID_ARG;
  if (a.s.batch == 0 || a.s.total_rows == 0) return DSPARK_OK;
  if (!args->q || !args->out || !args->workspace) return DSPARK_ERR_INVALID_ARG;
  if (args->workspace_bytes < dspark_kv4_attention_workspace_bytes(cache, batch, args->q_heads))
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned(args->q, 2) || !aligned(args->out, 2) || !aligned(args->lse, 4) || !aligned(args->workspace, 256))
    return DSPARK_ERR_MISALIGNED;
  a.q = static_cast<const uint16_t*>(args->q);
  a.q_row = args->q_row;
  a.q_head = args->q_head;
  a.out = static_cast<uint16_t*>(args->out);
  a.out_row = args->out_row;
  a.out_head = args->out_head;
  a.lse = args->lse;
  a.heads = a.c.kv_heads;
  a.group = args->q_heads / a.c.kv_heads;
  a.window = args->window;
  a.bf16 = args->dtype == DSPARK_DTYPE_BF16;
  a.q_vec = aligned(args->q, 16) && args->q_row % 8 == 0 && args->q_head % 8 == 0;
  a.out_vec = aligned(args->out, 16) && args->out_row % 8 == 0 && args->out_head % 8 == 0;
  a.scale_log2 = args->scale * kLog2E;
  a.cuts = static_cast<Cut*>(args->workspace);
  a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(args->workspace) + kCutBytes);
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  const int grid = sms < kMaxGrid ? sms : kMaxGrid;
  const auto launch = static_cast<int64_t>(batch->max_rows) * a.group <= kSmallRows ? launch_rows : launch_tiles;
  return launch(a, cache->head_dim, batch->max_rows, grid, stream) == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // extern "C"
