// tree_attn.cu - gdn_tree_attention's launch: row tiles, tensor maps and workspace
// (the kernel is in tree_attn.cuh).
#include "tree_attn.cuh"

namespace gdn {

namespace {

constexpr int kMaxRows = 64;

// P x G query rows per (request, kv head) in row tiles of equal size.
void row_tiles(int P, int G, int* rows, int* tiles) {
  const int all = P * G;
  *tiles = (all + kMaxRows - 1) / kMaxRows;
  *rows = (all + *tiles - 1) / *tiles;
  *tiles = (all + *rows - 1) / *rows;
}

// An output group's partial: its rows' maxima and sums, a flag, and rows x 128 values, or rows x 256 where
// one group has both halves of D = 256 (up to 16 rows).
int slot_floats(int rows) { return ((2 * rows + 4) / 4 * 4 + rows * (rows <= 16 ? 256 : 128) + 63) / 64 * 64; }

// Rows of one token and kv head; a box is 128 bytes of `box` tokens, swizzled as the MMAs read it.
bool encode(CUtensorMap* m, void* base, const KvArgs& c, int D, int box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const int es = c.e4m3 ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)c.slots * c.Hkv};
  const cuuint64_t strides[1] = {(cuuint64_t)D * es};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows};
  const cuuint32_t elem[2] = {1, 1};
  return enc(m, c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box,
             elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t tree_attn_workspace_bytes(int P, int G) {
  int rows, tiles;
  row_tiles(P, G, &rows, &tiles);
  return tree_attn::kTicketBytes + (size_t)4 * tree_attn::kMaxCtas * slot_floats(rows) * sizeof(float);
}

cudaError_t launch_tree_attn(const TreeAttnArgs& p, const KvArgs& c, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err != cudaSuccess) return err;
  tree_attn::Args a{};
  a.p = p;
  a.c = c;
  row_tiles(p.P, p.G, &a.rows, &a.row_tiles);
  a.slot_floats = slot_floats(a.rows);
  a.box = 16;
  while (a.box < tree_attn::kTile && c.page % (2 * a.box) == 0) a.box *= 2;
  CUtensorMap tmk{}, tmv{};
  if (!encode(&tmk, c.k, c, p.D, a.box) || !encode(&tmv, c.v, c, p.D, a.box)) return cudaErrorInvalidValue;
  const int grid = sms < tree_attn::kMaxCtas ? sms : tree_attn::kMaxCtas;
  return c.e4m3 ? tree_attn::launch_e4m3(a, tmk, tmv, grid, stream) : tree_attn::launch_bf16(a, tmk, tmv, grid, stream);
}

}  // namespace gdn
