// fp8_matmul.cu — fp8_matmul and fp8_gated_matmul: checks of the arguments,
// tensor maps, the choice of the kernel.
#include <cstdint>

#include "fp8_matmul.cuh"
#include "kvq_experts.h"
#include "kvq_host.h"

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime (no link to the driver library).
EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// Rows of E4M3 codes: boxes of 128 codes x `box_rows` rows (x one expert),
// 128-byte swizzle, zeros outside.
bool encode(CUtensorMap* map, const uint8_t* base, int dims, int64_t k, int64_t rows,
            int64_t experts, int64_t stride, int64_t expert_stride, int box_rows) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t size[3] = {(cuuint64_t)k, (cuuint64_t)rows, (cuuint64_t)experts};
  const cuuint64_t pitch[2] = {(cuuint64_t)stride, (cuuint64_t)expert_stride};
  const cuuint32_t box[3] = {(cuuint32_t)kvq::kGroupK, (cuuint32_t)box_rows, 1};
  const cuuint32_t unit[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, const_cast<uint8_t*>(base), size, pitch, box,
            unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The result's rows for stores of 32 rows x 64 columns: values with a 128-byte swizzle, or
// codes with one of 64 bytes.
bool encode_out(CUtensorMap* map, uint8_t* base, int64_t n, int64_t rows, int64_t pitch, bool codes) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t size[2] = {(cuuint64_t)n, (cuuint64_t)rows};
  const cuuint64_t stride[1] = {(cuuint64_t)pitch};
  const cuuint32_t box[2] = {64, 32}, unit[2] = {1, 1};
  return fn(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, size,
            stride, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
            codes ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Args {
  const uint8_t* a;
  int64_t a_stride;
  const float* a_scales;
  int64_t a_scale_stride, a_groups, a_rows;
  const uint8_t* b;
  int64_t b_stride, b_expert_stride;
  const float* b_scales;
  int64_t b_scale_stride, b_scale_expert_stride, n, k, num_experts;
  const int64_t* offsets;
  const int64_t* rows;
  int64_t num_rows;
  uint8_t* out;
  int64_t out_stride;
  float* out_scales;
  int64_t out_scale_stride;
  int32_t dtype;
  int32_t* status;
};

int run(const Args& a, bool gated, cudaStream_t stream) {
  using namespace kvq;
  constexpr int64_t kMostRows = (1ll << 31) - 1024, kMostWidth = 1 << 24;
  if (a.a_rows < 0 || a.a_rows >= kMostRows || a.num_rows < 0 || a.num_rows >= kMostRows)
    return KVQ_EINVAL;
  if (a.n < 1 || a.n > kMostWidth || a.k < 1 || a.k > kMostWidth || a.k % 16) return KVQ_EINVAL;
  if (gated && a.n % 128) return KVQ_EINVAL;
  if (a.num_experts < 0 || a.num_experts > kMaxExperts) return KVQ_EINVAL;
  if (a.num_experts == 0 && (a.offsets || a.rows || a.num_rows != a.a_rows)) return KVQ_EINVAL;
  if (!gated && a.dtype != KVQ_BF16 && a.dtype != KVQ_FP16) return KVQ_EINVAL;
  const int64_t groups = (a.k + kGroupK - 1) / kGroupK;
  const int64_t columns = gated ? 2 * a.n : a.n;
  const int64_t experts = a.num_experts ? a.num_experts : 1;
  if (a.a_groups != 1 && a.a_groups != groups) return KVQ_EINVAL;
  // (at most 2^31 rows, so no place passes 2^62; tensor maps take strides below 2^40)
  const auto bad = [](int64_t s, int64_t least, int64_t unit) {
    return s < least || s % unit || s > (1ll << 30);
  };
  if (bad(a.a_stride, a.k, 16) || bad(a.a_scale_stride, 0, 1) || bad(a.b_stride, a.k, 16) ||
      bad(a.b_scale_stride, 0, 1) || bad(a.out_stride, a.n, gated ? 16 : 1) ||
      (gated && bad(a.out_scale_stride, a.n / 128, 1)))
    return KVQ_EINVAL;
  const auto bad_expert = [](int64_t s, int64_t least, int64_t unit) {
    return s < least || s % unit || s > (1ll << 39);
  };
  if (experts > 1 &&
      (bad_expert(a.b_expert_stride, 16, 16) || bad_expert(a.b_scale_expert_stride, 0, 1)))
    return KVQ_EINVAL;
  if (a.num_rows == 0) return KVQ_OK;
  if (a.a_rows == 0 || !a.a || !a.a_scales || !a.b || !a.b_scales || !a.out) return KVQ_EINVAL;
  if ((gated && !a.out_scales) || (a.num_experts && !a.offsets)) return KVQ_EINVAL;
  if (!aligned(a.a, 16) || !aligned(a.b, 16) || !aligned(a.out, gated ? 16 : 2) ||
      !aligned(a.a_scales, 4) || !aligned(a.b_scales, 4) || !aligned(a.out_scales, 4) ||
      !aligned(a.offsets, 8) || !aligned(a.rows, 8) || !aligned(a.status, 4))
    return KVQ_EINVAL;
  MatmulParams p;
  p.a = a.a;
  p.a_stride = a.a_stride;
  p.k = a.k;
  p.a_scales = a.a_scales;
  p.b_scales = a.b_scales;
  p.offsets = a.num_experts ? a.offsets : nullptr;
  p.rows = a.rows;
  p.out = a.out;
  p.out_scales = a.out_scales;
  p.status = a.status;
  p.a_scale_stride = a.a_scale_stride;
  p.b_scale_stride = a.b_scale_stride;
  p.b_scale_expert_stride = a.b_scale_expert_stride;
  p.out_pitch = a.out_stride * (gated ? 1 : 2);
  p.out_scale_stride = a.out_scale_stride;
  p.a_rows = (int)a.a_rows;
  p.num_rows = (int)a.num_rows;
  p.experts = (int)experts;
  p.n = (int)a.n;
  p.steps = (int)groups;
  p.a_group_step = a.a_groups == 1 ? 0 : 1;
  p.half = a.dtype == KVQ_FP16;
  p.up_blocks = gated ? (int)(a.n / 128) : 0;
  p.blocks = (int)((columns + 127) / 128);
  p.wide = aligned(a.out, 32) && p.out_pitch % 32 == 0   ? 2
           : aligned(a.out, 16) && p.out_pitch % 16 == 0 ? 1
                                                         : 0;

  // Which kernel, and how many rows a tile of the one for few rows has. One matrix: tiles
  // of the other kernel are 256 x 256, too few where 64 rows by a block of columns are no
  // more than half of the SMs: 128 x 4096 x 4096 takes 13.0 us by the kernel for few rows and
  // 17.1 by the other, 160 x 4096 x 4096 17.1 by both, 128 x 4096 x 16384 30.1 and 21.5.
  // Experts: their rows scatter about the mean. 64 experts, 4096 -> 1024 gated, through an
  // index: a mean of 32 rows 112 and 131 us, 40 rows 134 and 129, 48 rows 150 and 130; 1024 ->
  // 4096 in place: 59 and 69, 68 and 70, 76 and 70. Their row tiles: a mean of 16 rows by
  // tiles of 16, 32 and 64 rows 59, 48 and 50 us, of 24 rows 72, 55 and 54. (The host knows no
  // more than the mean: most rows on one expert of many stay with the kernel for few rows.)
  const int64_t rows_each = (a.num_rows + experts - 1) / experts;
  const bool many = a.num_experts ? rows_each > 40
                                  : rows_each > 64 && (rows_each + 63) / 64 * p.blocks > sm_count() / 2;
  const int64_t likely = a.num_experts ? 2 * rows_each : rows_each;
  const int row_tile = likely <= 16 ? 16 : likely <= 32 ? 32 : 64;
  const int row_box = many ? 128 : row_tile;
  p.row_tiles_dense = (int)((a.num_rows + (many ? 255 : row_tile - 1)) / (many ? 256 : row_tile));
  const int width = many && !gated ? 256 : 128;
  p.column_tiles = (int)((a.n + width - 1) / width);
  const int64_t b_expert = experts > 1 ? a.b_expert_stride : a.b_stride;
  if (!encode(&p.a_map, a.a, 2, a.k, a.a_rows, 1, a.a_stride, 0, p.rows && !many ? 1 : row_box) ||
      !encode(&p.b_map, a.b, 3, a.k, columns, experts, a.b_stride, b_expert, many && gated ? 64 : 128))
    return KVQ_ECUDA;
  if (many && (gated || (p.wide && a.n % 128 == 0)) &&
      !encode_out(&p.out_map, a.out, a.n, a.num_rows, p.out_pitch, gated))
    return KVQ_ECUDA;
  return many ? launch_matmul_tiles(p, gated, stream) : launch_matmul_few(p, gated, row_tile, stream);
}

}  // namespace

extern "C" int fp8_matmul(const uint8_t* a, int64_t a_stride, const float* a_scales,
                          int64_t a_scale_stride, int64_t a_groups, int64_t a_rows,
                          const uint8_t* b, int64_t b_stride, int64_t b_expert_stride,
                          const float* b_scales, int64_t b_scale_stride,
                          int64_t b_scale_expert_stride, int64_t n, int64_t k, int64_t num_experts,
                          const int64_t* offsets, const int64_t* rows, int64_t num_rows, void* out,
                          int64_t out_stride, int32_t dtype, int32_t* status, cudaStream_t stream) {
  return run({a, a_stride, a_scales, a_scale_stride, a_groups, a_rows, b, b_stride, b_expert_stride,
              b_scales, b_scale_stride, b_scale_expert_stride, n, k, num_experts, offsets, rows,
              num_rows, static_cast<uint8_t*>(out), out_stride, nullptr, 0, dtype, status},
             false, stream);
}

extern "C" int fp8_gated_matmul(const uint8_t* a, int64_t a_stride, const float* a_scales,
                                int64_t a_scale_stride, int64_t a_groups, int64_t a_rows,
                                const uint8_t* b, int64_t b_stride, int64_t b_expert_stride,
                                const float* b_scales, int64_t b_scale_stride,
                                int64_t b_scale_expert_stride, int64_t n, int64_t k,
                                int64_t num_experts, const int64_t* offsets, const int64_t* rows,
                                int64_t num_rows, uint8_t* out, int64_t out_stride,
                                float* out_scales, int64_t out_scale_stride, int32_t* status,
                                cudaStream_t stream) {
  return run({a, a_stride, a_scales, a_scale_stride, a_groups, a_rows, b, b_stride, b_expert_stride,
              b_scales, b_scale_stride, b_scale_expert_stride, n, k, num_experts, offsets, rows,
              num_rows, out, out_stride, out_scales, out_scale_stride, KVQ_BF16, status},
             true, stream);
}
