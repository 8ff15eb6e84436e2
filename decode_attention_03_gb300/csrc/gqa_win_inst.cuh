// The launches of gqa_win.cuh for one cache and d_head; a translation unit for each instantiates them.
#pragma once
#include "gqa_host.cuh"
#include "gqa_win.cuh"

namespace gqa {

template <int D, int NT, int RG, bool KV4, bool BF16>
cudaError_t win_prepare_one() {
  constexpr int bytes = WinCfg<D, NT, RG, KV4>::SMEM;
  const cudaError_t e = cudaFuncSetAttribute(gqa_win_kernel<D, NT, RG, KV4, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             bytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(gqa_win_short_kernel<D, NT, RG, KV4, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int D, int NT, int RG, bool KV4, bool BF16>
cudaError_t win_launch_one(const WinParams& p, unsigned grid, cudaStream_t st) {
  using C = WinCfg<D, NT, RG, KV4>;
  if (p.ctas > 0) return launch_pdl_smem(gqa_win_short_kernel<D, NT, RG, KV4, BF16>, grid, C::THREADS, C::SMEM, st, p.ctas, p);
  return launch_pdl_smem(gqa_win_kernel<D, NT, RG, KV4, BF16>, grid, C::THREADS, C::SMEM, st, 1, p);
}

template <int D, bool KV4, bool BF16>
cudaError_t win_prepare_class(int cls) {
  switch (cls) {
    case 0: return win_prepare_one<D, win_rows_nt<KV4>(0), win_rows_rg<KV4>(0), KV4, BF16>();
    case 1: return win_prepare_one<D, win_rows_nt<KV4>(1), win_rows_rg<KV4>(1), KV4, BF16>();
    case 2: return win_prepare_one<D, win_rows_nt<KV4>(2), win_rows_rg<KV4>(2), KV4, BF16>();
    case 3: return win_prepare_one<D, win_rows_nt<KV4>(3), win_rows_rg<KV4>(3), KV4, BF16>();
    case 4: return win_prepare_one<D, win_rows_nt<KV4>(4), win_rows_rg<KV4>(4), KV4, BF16>();
    default: return win_prepare_one<D, win_rows_nt<KV4>(5), win_rows_rg<KV4>(5), KV4, BF16>();
  }
}

template <int D, bool KV4, bool BF16>
cudaError_t win_launch_class(const WinParams& p, int cls, unsigned grid, cudaStream_t st) {
  switch (cls) {
    case 0: return win_launch_one<D, win_rows_nt<KV4>(0), win_rows_rg<KV4>(0), KV4, BF16>(p, grid, st);
    case 1: return win_launch_one<D, win_rows_nt<KV4>(1), win_rows_rg<KV4>(1), KV4, BF16>(p, grid, st);
    case 2: return win_launch_one<D, win_rows_nt<KV4>(2), win_rows_rg<KV4>(2), KV4, BF16>(p, grid, st);
    case 3: return win_launch_one<D, win_rows_nt<KV4>(3), win_rows_rg<KV4>(3), KV4, BF16>(p, grid, st);
    case 4: return win_launch_one<D, win_rows_nt<KV4>(4), win_rows_rg<KV4>(4), KV4, BF16>(p, grid, st);
    default: return win_launch_one<D, win_rows_nt<KV4>(5), win_rows_rg<KV4>(5), KV4, BF16>(p, grid, st);
  }
}

}  // namespace gqa

#define GQA_WIN_INSTANCE(D, KV4, BF16)                                                                              \
  namespace gqa {                                                                                                   \
  template <>                                                                                                       \
  cudaError_t win_prepare<D, KV4, BF16>(int cls) {                                                                  \
    return win_prepare_class<D, KV4, BF16>(cls);                                                                    \
  }                                                                                                                 \
  template <>                                                                                                       \
  cudaError_t win_launch<D, KV4, BF16>(const WinParams& p, int cls, unsigned grid, cudaStream_t st) {               \
    return win_launch_class<D, KV4, BF16>(p, cls, grid, st);                                                        \
  }                                                                                                                 \
  }
