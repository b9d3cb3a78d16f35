// cross.h -- host-side declarations of the cross attention kernels.  Not part of
// the ABI.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include "rope.h"

namespace fa4 {

struct CrossParams {
  Strided q, k, v, o, dout, dq, dk, dv;   // the last four: backward only
  float* lse;                             // [B][Hq][Nq]; nullable forward
  const int* lens;                        // [B] or nullptr (Nk)
  unsigned* err;
  int B, Hq, Hkv, Nq, Nk, d;
  float scale, c;                         // softmax scale, fl32(scale * log2 e)
  int keys_log2;                          // forward: Nk <= 2^it
  uint8_t* work;                          // backward workspace
};

// A tiled map of one of the tensors, and whether its heads and sequences have
// places of their own (0: broadcast, all at coordinate 0).
struct HeadsMap {
  CUtensorMap map;
  int own_h, own_b;
};
bool heads_map(HeadsMap* m, const Strided& t, int B, int H, int N, int d, int rows, int heads);
// ... whose boxes end with their kv head's G heads: zeros behind them (tma_group).
bool group_map(HeadsMap* m, const Strided& t, int B, int Hkv, int G, int N, int d, int rows, int heads);

// Few query rows: keys shared among clusters, products of 16 rows.
bool cross_few_rows(const CrossParams& p);
cudaError_t launch_cross_token(const CrossParams& p, cudaStream_t st);
cudaError_t launch_cross_fwd(const CrossParams& p, cudaStream_t st);
size_t cross_bwd_workspace(int B, int Hq, int Hkv, int Nq, int Nk, int d);
cudaError_t launch_cross_bwd(const CrossParams& p, cudaStream_t st);

}  // namespace fa4
