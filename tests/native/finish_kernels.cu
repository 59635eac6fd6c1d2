// The kernels that add the parts of a product, alone, on parts given by a test. Built by the test.
#include "hqq_dense.cu"
#include "hqq_mid_impl.cuh"

#define TEST_EXPORT extern "C" __attribute__((visibility("default")))

TEST_EXPORT unsigned int no_part() { return hqqk::kNoPart; }

// partial [ctas][2][mats][tok][128]; Y, G, U [M][out], bf16
TEST_EXPORT int mid_finish(float* partial, void* Y, void* G, void* U, int M, int out, int tok, int tok_tiles,
                           int row_tiles, int kb, int ctas, int mats) {
  hqqk::MidArgs a = {};
  a.partial = partial;
  a.Y = static_cast<unsigned short*>(Y);
  a.G = static_cast<unsigned short*>(G);
  a.U = static_cast<unsigned short*>(U);
  a.M = M;
  a.out = a.rows = out;
  a.p.tok = tok;
  a.p.tok_tiles = tok_tiles;
  a.p.row_tiles = row_tiles;
  a.p.kb = kb;
  a.p.ctas = ctas;
  const dim3 grid(row_tiles * tok_tiles, (tok + 7) / 8);
  if (mats == 2)
    hqqk::mid_finish_kernel<false, 2><<<grid, 256>>>(a);
  else
    hqqk::mid_finish_kernel<false, 1><<<grid, 256>>>(a);
  return static_cast<int>(cudaDeviceSynchronize());
}

// partial [splits][products][M][N]; D, G, U [M][N], bf16
TEST_EXPORT int dense_finish(float* partial, void* D, void* G, void* U, int M, int N, int splits, int kind) {
  hqqk::DenseArgs a = {};
  a.partial = partial;
  a.D = static_cast<unsigned short*>(D);
  a.G = static_cast<unsigned short*>(G);
  a.U = static_cast<unsigned short*>(U);
  a.M = M;
  a.N = N;
  a.splits = splits;
  const int grid = static_cast<int>((static_cast<int64_t>(M) * N / 4 + 255) / 256);
  if (kind == hqqk::kDenseGated)
    hqqk::dense_finish_kernel<false, hqqk::kDenseGated><<<grid, 256>>>(a);
  else if (kind == hqqk::kDenseForward)
    hqqk::dense_finish_kernel<false, hqqk::kDenseForward><<<grid, 256>>>(a);
  else
    hqqk::dense_finish_kernel<false, hqqk::kDenseBackward><<<grid, 256>>>(a);
  return static_cast<int>(cudaDeviceSynchronize());
}
