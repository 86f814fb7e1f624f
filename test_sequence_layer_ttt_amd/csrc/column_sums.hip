// Sums over the rows of a matrix of partial results, in a fixed order (the
// same bits on every run). A workgroup takes 64 columns of one range and
// splits the rows over 16 lanes' worth of threads that meet in LDS. The callers
// keep the partials to a few percent of their own bytes, so a call is bound by
// its launch: 4.1 us for 64 rows of 4480, 4.7 us for 512 rows of 2304.
#include "block.hpp"

namespace ttt {
namespace {

constexpr int CW = 64, RW = 16;  // columns and row subsets of a workgroup

__global__ __launch_bounds__(CW *RW) void column_sums(ColumnSums a) {
    __shared__ float red[RW][CW];
    const ColumnSums::Range q = a.q[blockIdx.y];
    if (static_cast<int>(blockIdx.z) >= q.outer) return;
    const int lane = threadIdx.x % CW, w = threadIdx.x / CW;
    const int rows = a.rows / q.outer;
    const float *p = a.part + static_cast<int64_t>(blockIdx.z) * rows * a.stride + q.off;
    for (int c0 = blockIdx.x * CW; c0 < q.cols; c0 += gridDim.x * CW) {
        const int c = c0 + lane;
        float s[4] = {};
        if (c < q.cols) {
            int r = w;
            for (; r + 3 * RW < rows; r += 4 * RW) {
#pragma unroll
                for (int u = 0; u < 4; ++u) s[u] += p[static_cast<int64_t>(r + u * RW) * a.stride + c];
            }
            for (; r < rows; r += RW) s[0] += p[static_cast<int64_t>(r) * a.stride + c];
        }
        red[w][lane] = (s[0] + s[1]) + (s[2] + s[3]);
        __syncthreads();
        if (w == 0 && c < q.cols) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < RW; ++i) v += red[i][lane];
            q.out[static_cast<int64_t>(blockIdx.z) * q.cols + c] = v;
        }
        __syncthreads();
    }
}

}  // namespace

hipError_t launch_column_sums(const ColumnSums &c, hipStream_t stream) {
    if (c.n == 0) return hipSuccess;
    int cols = 0, outer = 0;
    for (int i = 0; i < c.n; ++i) {
        cols = c.q[i].cols > cols ? c.q[i].cols : cols;
        outer = c.q[i].outer > outer ? c.q[i].outer : outer;
    }
    const int gx = (cols + CW - 1) / CW;
    hipLaunchKernelGGL(column_sums, dim3(gx < 4096 ? gx : 4096, c.n, outer), dim3(CW * RW), 0, stream, c);
    return hipGetLastError();
}

}  // namespace ttt
