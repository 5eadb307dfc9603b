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

int slot_floats(int rows, int D) { return (tree_attn::head_floats(rows) + rows * D + 63) / 64 * 64; }

// The partial results of the units that several CTAs share, one after the other in the order of their tiles:
// blockIdx.x is the CTA with a unit's first tile, blockIdx.y 1024 / D of its rows, a thread has four values.
// Bound by its chain of trips to L2, the descriptor, the maxima and the rows: 9.5 us cold for the 11 MB of 64 nodes on
// 131,071 tokens (2432 blocks), set up while the tiles' kernel runs.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const tree_attn::Args a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const TreeAttnArgs& p = a.p;
  const tree_attn::Desc d = static_cast<const tree_attn::Desc*>(p.workspace)[blockIdx.x];
  if (!d.valid) return;
  constexpr int kPer = D / 4;
  const int row = blockIdx.y * (256 / kPer) + threadIdx.x / kPer, col = threadIdx.x % kPer * 4;
  const int r = d.u % a.row_tiles * a.rows + row, j = r / p.G;
  if (row >= a.rows || j >= p.P) return;
  const int head = tree_attn::head_floats(a.rows);
  const size_t at = (((size_t)d.n * p.P + j) * p.Hq + d.u / a.row_tiles * p.G + r % p.G) * D + col;
  uint2 gate = make_uint2(0u, 0u);
  if (p.gate) gate = *reinterpret_cast<const uint2*>(p.gate + at);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  bool bad = false;
  // E4M3: the maxima are those of the weights with the value scales, the sums are not. A sum may hold against a factor
  // that is too small for a number: there a factor is the square of its root, which is 1 for bf16.
  const float part = a.c.e4m3 ? 0.5f : 1.f;
  constexpr int kAtOnce = 4;
  for (int k0 = blockIdx.x; k0 <= d.last; k0 += kAtOnce) {
    float mk[kAtOnce], lk[kAtOnce];
    float4 v[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int k = min(k0 + i, d.last);
      const float* q = tree_attn::partial(a, k, k == blockIdx.x);
      mk[i] = q[row];
      lk[i] = q[a.rows + row];
      bad |= reinterpret_cast<const int*>(q)[2 * a.rows] != 0 || reinterpret_cast<const int*>(q)[2 * a.rows + 1] != 0;
      v[i] = *reinterpret_cast<const float4*>(q + head + (size_t)row * D + col);
      if (k0 + i > d.last) mk[i] = -INFINITY, lk[i] = 0.f, v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mn = m;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) mn = fmaxf(mn, mk[i]);
    const float root = m == -INFINITY ? 0.f : tree_attn::ex2((m - mn) * part), again = a.c.e4m3 ? root : 1.f;
    const float keep = root * again;
    l = l * root * again;
    o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float wr = mk[i] == -INFINITY ? 0.f : tree_attn::ex2((mk[i] - mn) * part), wa = a.c.e4m3 ? wr : 1.f, w = wr * wa;
      l += mk[i] == -INFINITY ? lk[i] : lk[i] * wr * wa;  // a NaN of a row without a maximum stays one
      o = make_float4(fmaf(v[i].x, w, o.x), fmaf(v[i].y, w, o.y), fmaf(v[i].z, w, o.z), fmaf(v[i].w, w, o.w));
    }
    m = mn;
  }
  if (p.lse && col == 0)
    p.lse[((size_t)d.n * p.P + j) * p.Hq + d.u / a.row_tiles * p.G + r % p.G] = bad ? NAN : tree_attn::lse_of(m, l);
  if (bad) return;
  const float f = l == 0.f ? 0.f : __fdividef(1.f, l);
  *reinterpret_cast<uint2*>(p.out + at) = tree_attn::to_out(make_float4(o.x * f, o.y * f, o.z * f, o.w * f), p.gate, gate);
}

}  // namespace

namespace tree_attn {

bool encode_rows(CUtensorMap* m, void* base, const KvArgs& c, int D, int box_rows) {
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

int box_tokens(int page) {
  int box = 16;
  while (box < kTile && page % (2 * box) == 0) box *= 2;
  return box;
}

}  // namespace tree_attn

size_t tree_attn_workspace_bytes(int P, int G, int D) {
  int rows, tiles;
  row_tiles(P, G, &rows, &tiles);
  return tree_attn::kDescBytes + (size_t)2 * tree_attn::kMaxCtas * slot_floats(rows, D) * sizeof(float);
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
  a.slot_floats = slot_floats(a.rows, p.D);
  a.box = tree_attn::box_tokens(c.page);
  CUtensorMap tmk{}, tmv{};
  if (!tree_attn::encode_rows(&tmk, c.k, c, p.D, a.box) || !tree_attn::encode_rows(&tmv, c.v, c, p.D, a.box)) return cudaErrorInvalidValue;
  const int grid = sms < tree_attn::kMaxCtas ? sms : tree_attn::kMaxCtas;
  err = c.e4m3 ? tree_attn::launch_e4m3(a, tmk, tmv, grid, stream) : tree_attn::launch_bf16(a, tmk, tmv, grid, stream);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, (unsigned)((a.rows * p.D + 1023) / 1024), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return p.D == 256 ? cudaLaunchKernelEx(&cfg, join_kernel<256>, a) : cudaLaunchKernelEx(&cfg, join_kernel<128>, a);
}

}  // namespace gdn
