// kv4_attention.cu -- dspark_kv4_attention (include/dspark_kv4.h): argument
// checks, the workspace, the choice of kernel.
#include <math.h>

#include "kv4_attn.cuh"

namespace dspark {
namespace kv4 {
namespace {

// Rows of a tile for a call: 8 or 16 (kv4_rows.cu), 128 or 256 (kv4_tiles.cu),
// whichever should take least.  A call takes about
//   fixed + tiles of a request * cost * blocks of all requests and heads / CTAs,
// the costs as measured for 32 requests of 8 heads and 4 to 8 k tokens, 128 and 64
// dimensions (us a block and CTA), the fixed part for 2 requests of 2 to 4 k
// (us).  Measured / 8, 16, 128, 256 rows a tile, 128 dimensions:
//   32 requests:  8 rows  52 /  70 / 103 / 160 us,  16 rows  92 /  73 / 105 / 163,
//                24 rows 131 / 127 / 106 / 163,    192 rows 1034 / 746 / 221 / 197;
//    2 requests: 16 rows  14 /  14 /  17 /  19 us,  48 rows  17 /  19 /  20 /  23.
// Lengths are on the device: what the page tables can hold stands for them.
// Tiles so small that there could be more positions (kv4_attn.cuh) than 31 bits
// hold are not taken, if there are larger ones: a call that promises fewer rows
// than it has could get them.
struct Choice {
  int32_t rows;
  double fixed, cost;
};
constexpr Choice kChoices[] = {{8, 9.0, 0.26}, {16, 11.0, 0.38}, {128, 18.0, 0.56}, {256, 18.0, 0.90}};
constexpr double kCtas = 152.0;

int32_t tile_rows(const Batch& s, int32_t heads, int32_t group, int64_t rows) {
  const double longest = static_cast<double>((s.max_tokens + kBlock - 1) / kBlock);
  const double blocks = static_cast<double>(s.batch) * heads * longest;
  int32_t best = 0;
  double least = 0.0;
  bool counted = false;
  for (const Choice& c : kChoices) {
    const double units = (static_cast<double>(s.total_rows) * group / c.rows + s.batch) * heads;
    const bool fits = units * (longest + 8.0) < kTooMany;
    const double time = c.fixed + static_cast<double>((rows + c.rows - 1) / c.rows) * c.cost * blocks / kCtas;
    if (best == 0 || (fits && !counted) || (fits == counted && time < least)) best = c.rows, least = time, counted = fits;
  }
  return best;
}

// Partial sums of one call.
int64_t slots_bytes(int32_t rows, int dim) { return 2 * kMaxGrid * static_cast<int64_t>(rows) * (dim + 2) * 4; }

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
  const int32_t group = q_heads / c.kv_heads;
  const int32_t tile = tile_rows(s, c.kv_heads, group, static_cast<int64_t>(batch->max_rows) * group);
  return static_cast<size_t>(kCutBytes + slots_bytes(tile, cache->head_dim));
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
  a.window = args->window < a.s.max_tokens ? args->window : 0;
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
  const int64_t rows = static_cast<int64_t>(batch->max_rows) * a.group;
  const int32_t tile = tile_rows(a.s, a.heads, a.group, rows);
  a.many_tiles = rows > tile;
  const auto launch = tile <= 16 ? launch_rows : launch_tiles;
  return launch(a, cache->head_dim, tile, grid, stream) == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // extern "C"
