// rope.h -- host-side declarations of the norm and rotation kernels.  Not part
// of the ABI.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#ifdef __CUDACC__
#define FA4_BOTH __host__ __device__ __forceinline__
#else
#define FA4_BOTH inline
#endif

namespace fa4 {

// A strided [B][H][N][d] tensor: element strides, the last dimension dense.
struct Strided {
  void* p;
  long long b, h, n;
};

// Multiprocessors of the current device (1 where there is none).
int sm_count();

// cudaFuncAttributeMaxDynamicSharedMemorySize of a kernel, set once per device (and
// the leave for clusters of 16).
cudaError_t allow_smem(const void* kernel, int bytes, bool clusters = false);

// Launches a kernel; `early`: it may start while its predecessor runs, and waits for it
// itself (griddepcontrol.wait) before it reads what that writes.
template <class... P>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, int smem, bool early, cudaStream_t st, const P&... p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p...);
}

// Division of 0 <= n < 2^31 by a fixed d >= 1: (umulhi(n, m) + n) >> s.
struct Divisor {
  uint32_t m = 0;
  int s = 0, d = 1;
  Divisor() = default;
  explicit Divisor(int d_) : d(d_) {
    while ((1ll << s) < d) ++s;
    m = (uint32_t)((((1ull << s) - (uint64_t)d) << 32) / (uint64_t)d + 1);
  }
};

// A warp's tasks: every `step`th of `all` from `now` on.  Counted without a sign: 2^30 tokens with heads of q
// and of k are 2^31 tasks, and a warp's last step goes behind them.
struct Tasks {
  uint32_t now, step, all;
  FA4_BOTH bool more() const { return now < all; }
  FA4_BOTH void next() { now += step; }
};

struct RopeTensor {            // q or k
  Strided x, dy, out;          // dy: backward only
  const void* w;               // norm weight [d] or nullptr
  float* part;                 // backward: weight gradient partials [CTAs of the tensor][d]
  float* dw;                   // backward: weight gradient [d] or nullptr
  int H;
};
struct RopeParams {
  RopeTensor t[2];
  const int* pos;              // [B or 1][axes][N], or nullptr: no rotation
  long long pos_b;             // its stride between sequences
  uint64_t turn[64];           // turns a position of each channel pair, 0.64 fixed point
  uint8_t axis[64];            // axis of each channel pair
  int B, N, d, norm, w_bf16, pairs, dy_f32;
  int ctas[2];                 // backward: CTAs of each tensor
  float eps;
};
cudaError_t launch_norm_rope(const RopeParams& p, cudaStream_t st);

// CTAs that the backward gives q and k (a rule of shapes and SMs).
void rope_bwd_ctas(int B, int Hq, int Hkv, int N, int d, int* ctas);
cudaError_t launch_norm_rope_bwd(const RopeParams& p, cudaStream_t st);

}  // namespace fa4
