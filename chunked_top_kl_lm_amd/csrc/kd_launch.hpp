// kd_launch.hpp -- host-side launch helpers shared by the library's sources:
// the GEMM's shape and grid, and the error check after a launch.
#pragma once

#include "kd_gemm.hpp"
#include "kd_plan.hpp"

namespace kd {
namespace {

// One block per tile (a multiple of 8 blocks).
template <class TC, class E, class Epi>
hipError_t launch_gemm(const GemmShape& g, const Epi& epi, hipStream_t st) {
  const int nb = g.tiles_m * g.tiles_n * g.splits;
  const int grid = (nb + 7) & ~7;
  hipLaunchKernelGGL((gemm_nt_kernel<E, TC::BM, TC::BN, TC::WM, TC::WN, TC::STAGES, Epi, TC::RB>), dim3(grid),
                     dim3(TC::kThreads), 0, st, g, epi);
  return hipGetLastError();
}

// group_m: row tiles per group of the tile order (see tile_position).  The
// head-gradient GEMM uses 4 (it re-streams its 11.8 MB H_c^T operand once
// per row band otherwise); the others measured best with 1.
template <class TC>
GemmShape make_shape(const void* A, int64_t lda, int M, const void* B, int64_t ldb, int N, int64_t k_bytes,
                     int splits, int group_m) {
  GemmShape g;
  g.group_m = group_m;
  g.A = A; g.B = B; g.lda = lda; g.ldb = ldb; g.M = M; g.N = N;
  g.k_tiles = (int)(k_bytes / TC::RB);
  g.k_tiles_per_split = (int)cdiv(g.k_tiles, splits);
  g.splits = (int)cdiv(g.k_tiles, g.k_tiles_per_split);   // <= splits; no split is empty
  g.tiles_m = (int)cdiv(M, TC::BM);
  g.tiles_n = (int)cdiv(N, TC::BN);
  return g;
}

}  // namespace
}  // namespace kd

#define KD_LAUNCH_CHECK()                         \
  do {                                            \
    if (hipGetLastError() != hipSuccess) return KD_ERR_HIP; \
  } while (0)
