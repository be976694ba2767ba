// join.hip -- sums over rows or batches (dweight and dbias of a norm; ddecay and the biases' gradients of a recurrence) from
// the partial sums that the workgroups of their backward passes leave.
//
// COLS columns per workgroup, the partial sums split over NT / COLS groups of lanes, each in order, then the groups' sums
// in order (1366 sums of 768 columns, 16 at a time: 6 us).  Up to 4096 of them in one go: 64 a lane; more in levels of 512:
// every `step`th of them, `many` to a workgroup, which leaves their sum in the place of the first.  So a lane's chain
// stays short however many there are, and the last call's single sum goes to the output.
#include "block_device.h"

namespace ssm {

// The n sums that are left lie `step` apart.  (Divisions in 32 bits: in 64 they took longer than the
// loads of a short join.)
template <int COLS, int NT>
__global__ __launch_bounds__(NT) void join_kernel(JoinParams p, int64_t step, int64_t n, int many, uint32_t cols,
                                                  uint32_t blocks) {
  constexpr int GROUPS = NT / COLS;
  __shared__ float sm[NT], sn[NT / 4];
  if (block_id() >= blocks) return;
  const uint32_t blk = (uint32_t)xcd_remap((int)block_id(), (int)blocks);  // (neighbours read the same lines)
  const uint32_t col = blk % cols, rest = blk / cols, which = rest % p.kinds;
  const int64_t first = (int64_t)(rest / p.kinds) * many;
  const int here = n - first < many ? (int)(n - first) : many;
  const int64_t c = (int64_t)col * COLS + threadIdx.x % COLS, row = step * p.kinds * p.E;
  const int per = (here + GROUPS - 1) / GROUPS, k0 = threadIdx.x / COLS * per, k1 = k0 + per < here ? k0 + per : here;
  float* q = p.part + first * row + which * p.E + c;
  float s = 0.0f;
  if (c < p.E) {
    for (int k = k0; k < k1; k += 8) {  // (the last few at once, too: one by one they were half of the time)
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = k + e < k1 ? q[(k + e) * row] : 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[e];
    }
  }
  sm[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x < NT / 4) {
    const int at = threadIdx.x / COLS * 4 * COLS + threadIdx.x % COLS;
    sn[threadIdx.x] = (sm[at] + sm[at + COLS]) + (sm[at + 2 * COLS] + sm[at + 3 * COLS]);
  }
  __syncthreads();
  float* out = many < n ? q : which == 0 ? p.out[0] : which == 1 ? p.out[1] : p.out[2];
  if (threadIdx.x < COLS && c < p.E && out) {
    s = 0.0f;
#pragma unroll
    for (int t = 0; t < GROUPS / 4; ++t) s += sn[t * COLS + threadIdx.x];
    out[many < n ? 0 : c] = s;
  }
}

hipError_t launch_join(const JoinParams& p, hipStream_t s) {
  for (int64_t n = p.count, step = 1, many; n; step *= many) {
    many = n <= 4096 ? n : 512;
    const int64_t groups = (n + many - 1) / many;
    auto go = [&](auto kernel, int threads, int64_t width) {
      const int64_t cols = (p.E + width - 1) / width, blocks = cols * p.kinds * groups;
      hipLaunchKernelGGL(kernel, grid_of(blocks), dim3(threads), 0, s, p, step, n, (int)many, (uint32_t)cols,
                         (uint32_t)blocks);
    };
    // (of few sums, four groups of lanes leave fewer of them without one: 64 x 100000, gradients: 83 us, 153 with 64 groups)
    many <= 64 ? go(join_kernel<64, 256>, 256, 64) : go(join_kernel<16, 1024>, 1024, 16);
    n = groups > 1 ? groups : 0;
  }
  return hipGetLastError();
}

}  // namespace ssm
