// FP8 linear for bfloat16 outputs with many tiles (fp8_wide.h).
#include "fp8_wide.h"

namespace convrot {
namespace {

template <bool GELU, bool F32>
__global__ __launch_bounds__(256, 1) void fp8_gemm_wide_kernel(const Fp8Params p, int total) {
  fp8_wide<GELU, F32, kPlain>(p, total);
}

}  // namespace

// Whether these tiles take less time than those of 128 x 128 (fp8_gemm.hip),
// which the CUs hold two each.
//
// Power-of-two scales: a round of all CUs takes 1.4 times as long here.
// Measured, here and there (us; 4096 -> 4096 unless stated, rounds in
// brackets): 2048 rows 44.7 (1), 40.5 (1); 2304 44.7 (1), 65.8 (2); 4096 53.9
// (1), 78.8 (2); 4608 89.9 (2), 103.8 (3); 8192 104.9 (2), 151.6 (4); 32768 x
// 5120 -> 128 58.1 (1), 33.8 (1); 65536 x 4096 -> 200 80.5 (1), 97.2 (2); 300 x
// 5120 -> 40000 108.9 (2), 88.3 (2); 129 x 4096 -> 100000 122.3 (2), 171.6 (4).
//
// float32 weight scales: the tiles here are half as large, and a last round
// there that gives each CU one workgroup takes half of a round that gives each
// two, so those count as halves: a round here takes 7/4 of a half there.  2048
// rows 43.2 (1), 47.5 (2); 2304 74.7 (2), 68.9 (3); 2816 76.2 (2), 71.3 (3);
// 3328 77.2 (2), 81.3 (4); 4096 81.9 (2), 87.3 (4); 4608 110.6 (3), 107.6 (5);
// 6144 120.8 (3), 128.4 (6); 1024 42.1 (1), 28.8 (1); 1280 41.4 (1), 42.4 (2);
// 32768 x 5120 -> 128 46.7 (1), 34.6 (1); 300 x 5120 -> 40000 131.8 (3), 98.4
// (4); 129 x 4096 -> 100000 156.0 (4), 174.0 (7).
bool fp8_wide_wanted(const Fp8GemmArgs& a) {
  if (!a.y_bf16 || (a.k + kFp8Block - 1) / kFp8Block < kMinBlocks) return false;
  const int64_t cus = device_cu_count();
  const int bn = a.f32_scale ? WideCfg<true>::BN : WideCfg<false>::BN;
  int64_t tiles = 0, small = 0;
  if (a.gated) {  // (as many rows of W to a tile, half as many columns of Y)
    if (a.w[0].ldy >= kMaxLdy || (a.kept[0] && a.ldk >= kMaxLdy)) return false;
    tiles = ((a.m + kBM - 1) / kBM) * ((a.w[0].n + bn / 2 - 1) / (bn / 2));
    small = ((a.m + 127) / 128) * ((a.w[0].n + 63) / 64);
  }
  for (int i = 0; !a.gated && i < a.count; ++i) {
    if (a.w[i].ldy >= kMaxLdy) return false;
    tiles += ((a.m + kBM - 1) / kBM) * ((a.w[i].n + bn - 1) / bn);
    small += ((a.m + 127) / 128) * ((a.w[i].n + 127) / 128);
  }
  const int64_t here = (tiles + cus - 1) / cus, there = (small + 2 * cus - 1) / (2 * cus);
  if (!a.f32_scale) return 7 * here < 5 * there;
  const int64_t last = small % (2 * cus);
  const int64_t halves = 2 * there - (last > 0 && last <= cus ? 1 : 0);
  return 7 * here <= 4 * halves;
}

namespace {

template <bool GELU, bool F32>
void launch_t(const Fp8GemmArgs& a, hipStream_t stream) {
  const Fp8Params p = fp8_params<kBM, WideCfg<F32>::BN>(a);
  const int total = p.tiles_m * p.tiles_n;
  const int cus = device_cu_count();
  hipLaunchKernelGGL((fp8_gemm_wide_kernel<GELU, F32>), dim3(total < cus ? total : cus), dim3(256), 0, stream, p,
                     total);
}

}  // namespace

hipError_t launch_fp8_gemm_wide(const Fp8GemmArgs& a, hipStream_t stream) {
  if (a.f32_scale)
    a.gelu ? launch_t<true, true>(a, stream) : launch_t<false, true>(a, stream);
  else
    a.gelu ? launch_t<true, false>(a, stream) : launch_t<false, false>(a, stream);
  return hipGetLastError();
}

}  // namespace convrot
