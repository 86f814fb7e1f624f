// The state space scan's backward, last part. The gradient of the log-decay
// D_t A of a token is q_t = <g_t, a_t h_{t-1}>: of everything that passes from
// the tokens before t to those from t on. With dy . (strict read of h) = row
// and u . (strict read of g) = col, both without the token's own term,
//     q_t = q_{t+1} + row_t - col_t,
// a running sum from the segment's end, where q is the product of the state
// and its gradient. Rounding errors in such a sum never leave it again, while
// what q_t measures decays; so it starts anew as often as can be.
//  * Walks: a segment has 64 tokens.
//  * Sweeps, in 64-token chunks: with re and co the parts that pass through the
//    state before and behind the chunk, and W (row_i = sum_j W_ij, col_j =
//    sum_i W_ij) what passes within it,
//        q_t = base + sum_{j < t} co_j + sum_{i >= t} re_i + sum_{i >= t > j} W_ij,
//    where base passes the whole chunk: q at its end less all of co, or in
//    the segment's first half q at its start less all of re, and
//    taken as 0 where the chunk's decay is below 2^-24 and that difference is
//    nothing but rounding. The last sum is known at the borders of the
//    16-token tiles from the tiles' sums and runs within a tile.
// All in 64 bits. Then
//     ddt_t = (A q_t + x_t . du_t) sigma(dt_t + dt_bias),
//     dA = sum D_t q_t,  dD = sum dy_t . x_t,  ddt_bias = sum ddt_t,
// and dB, dC are summed over the heads of a group. Bound by the heads' parts,
// which the sweeps have written: 75 MB in 15 us (B=4 L=2048 H=12 N=64).
#include <cmath>

#include "block.hpp"
#include "ssm.hpp"
#include "vec.hpp"

namespace ttt {
namespace {

constexpr int NT = 256;

struct FinishArgs {
    SsmBwdArgs g;
    SsmBwdWs w;
    int rows;  // tokens of a workgroup of head_sums
};

__device__ __forceinline__ double block_sum(double v, double (&red)[NT / 64]) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    __syncthreads();
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// sums over the lanes below (above) this one and it, in groups of W lanes
template <int W> __device__ __forceinline__ double sum_before(double v) {
    const int lane = threadIdx.x % W;
#pragma unroll
    for (int m = 1; m < W; m *= 2) {
        const double o = __shfl_up(v, m, W);
        if (lane >= m) v += o;
    }
    return v;
}
template <int W> __device__ __forceinline__ double sum_behind(double v) {
    const int lane = threadIdx.x % W;
#pragma unroll
    for (int m = 1; m < W; m *= 2) {
        const double o = __shfl_down(v, m, W);
        if (lane + m < W) v += o;
    }
    return v;
}

// a thread's part of the product of two arrays of n
__device__ __forceinline__ double dot(const float *s, const float *g, int64_t n) {
    double e = 0.0;
    if (n % 4 == 0 && ((reinterpret_cast<uintptr_t>(s) | reinterpret_cast<uintptr_t>(g)) & 15) == 0) {
        const float4 *s4 = reinterpret_cast<const float4 *>(s), *g4 = reinterpret_cast<const float4 *>(g);
#pragma unroll 4
        for (int i = threadIdx.x; i < static_cast<int>(n / 4); i += NT) {
            const float4 u = s4[i], v = g4[i];
            e += (static_cast<double>(u.x) * v.x + static_cast<double>(u.y) * v.y) +
                 (static_cast<double>(u.z) * v.z + static_cast<double>(u.w) * v.w);
        }
    } else {
        for (int i = threadIdx.x; i < static_cast<int>(n); i += NT) e += static_cast<double>(s[i]) * g[i];
    }
    return e;
}

// A workgroup takes a segment, a thread a token, a wave a 64-token chunk.
template <typename TIO, bool SWEEPS>
__device__ __forceinline__ void decay_gradient(const FinishArgs &f, int block) {
    const SsmArgs &a = f.g.f;
    __shared__ double red[NT / 64], all_re[NT / 64], all_co[NT / 64], all_l[NT / 64];
    const int seg = block % a.nseg, bh = block / a.nseg, b = bh / a.H, h = bh % a.H;
    const int64_t NP = static_cast<int64_t>(a.N) * a.P;
    const int n = a.lens ? max(0, min(a.lens[b], a.L)) : a.L;
    const int64_t t = static_cast<int64_t>(seg) * a.seglen + threadIdx.x;
    const bool mine = static_cast<int>(threadIdx.x) < a.seglen && t < a.L, live = mine && t < n;
    // <state, its gradient> at the segment's end, and at its start where that is known
    const float *se = seg + 1 < a.nseg ? f.w.sf + (static_cast<int64_t>(bh) * a.nseg + seg + 1) * NP : f.w.last + bh * NP;
    const float *ge = f.w.sr + (static_cast<int64_t>(bh) * a.nseg + seg) * NP;
    const bool both = SWEEPS && seg > 0;
    double e = dot(se, ge, NP), e0 = 0.0;
    if (both) e0 = block_sum(dot(f.w.sf + (static_cast<int64_t>(bh) * a.nseg + seg) * NP, ge - NP, NP), red);
    e = block_sum(e, red);
    const int64_t tok = static_cast<int64_t>(bh) * a.L + t, blk = static_cast<int64_t>(a.B) * a.H * a.L;
    double xdu = 0.0, dyx = 0.0, z = 0.0, step = 0.0, q;
    if (live) {
        z = static_cast<double>(io_traits<TIO>::load(static_cast<const TIO *>(a.dt.p), b * a.dt.sb + t * a.dt.st + h * a.dt.sh)) +
            (a.dt_bias ? a.dt_bias[h] : 0.f);
        step = softplus_f(static_cast<float>(z));
    }
    if constexpr (SWEEPS) {
        double w = 0.0, re = 0.0, co = 0.0;
        if (live) {
            w = static_cast<double>(f.w.row[tok]) - f.w.col[tok];
            re = f.w.row[blk + tok];
            co = f.w.col[blk + tok];
            xdu = f.w.xdu[tok];
            dyx = f.w.dyx[tok];
        }
        const int wv = threadIdx.x / 64, lane = threadIdx.x % 64;
        const double re_behind = sum_behind<64>(re), co_here = sum_before<64>(co), co_before = co_here - co;
        const double l = sum_before<64>(step * a.A[h]);
        double within = sum_behind<16>(w);
        if (mine && lane < 48) {  // what passes the end of this token's tile
            const float *p = f.w.tiles + (static_cast<int64_t>(bh) * ((a.L + 63) / 64) + t / 64) * 8;
            const int tile = lane / 16;
            // the pairs (i, j) with j <= tile < i; those of a tile that has no tokens were never
            // made, so only what the sequence holds is read
            const int held = static_cast<int>((n - (t - lane) + 15) / 16);  // tiles with tokens
            const int place[3][3] = {{0, 1, 2}, {-1, 3, 4}, {-1, -1, 5}};   // [j][i - 1]
#pragma unroll
            for (int j = 0; j < 3; ++j)
#pragma unroll
                for (int i = 1; i < 4; ++i)
                    if (j <= tile && i > tile && i > j && i < held) within += p[place[j][i - 1]];
        }
        if (lane == 0) all_re[wv] = re_behind;
        if (lane == 63) {
            all_co[wv] = co_here;
            all_l[wv] = l;
        }
        __syncthreads();
        double base = 0.0;
        const int held = static_cast<int>((max(0, min(a.seglen, n - seg * a.seglen)) + 63) / 64);  // chunks with tokens
        auto passes = [&](int k, double q_border, double own) {
            return all_l[k] < -24.0 * 0.6931471805599453 ? 0.0 : q_border - own;
        };
        if (both && wv < held / 2) {
            for (int k = 0; k <= wv; ++k) {  // e0: q before chunk k
                base = passes(k, e0, all_re[k]);
                e0 = base + all_co[k];
            }
        } else {
            for (int k = held - 1; k >= wv; --k) {  // e: q behind chunk k
                base = passes(k, e, all_co[k]);
                e = base + all_re[k];
            }
        }
        q = base + co_before + re_behind + within;
    } else {
        double w = 0.0;
        if (live) {
            for (int i = 0; i < f.w.rows; ++i) w += f.w.row[i * blk + tok];
            for (int i = 0; i < f.w.cols; ++i) {
                w -= f.w.col[i * blk + tok];
                xdu += f.w.xdu[i * blk + tok];
                dyx += f.w.dyx[i * blk + tok];
            }
        }
        q = sum_behind<64>(w) + e;  // a segment of 64 tokens: the first wave's
    }
    double dz = 0.0, dA = 0.0;
    if (live) {
        dA = q * step;
        dz = (a.A[h] * q + xdu) / (1.0 + exp(-z));
    }
    if (mine)
        io_traits<TIO>::store(static_cast<TIO *>(const_cast<void *>(f.g.ddt.p)),
                              b * f.g.ddt.sb + t * f.g.ddt.st + h * f.g.ddt.sh, static_cast<float>(dz));
    dA = block_sum(dA, red);
    const double dD = block_sum(dyx, red), db = block_sum(dz, red);
    if (threadIdx.x == 0) {
        float *p = f.w.part + (static_cast<int64_t>(b) * a.nseg + seg) * 3 * a.H + h;
        p[0] = static_cast<float>(dA);
        p[a.H] = static_cast<float>(dD);
        p[2 * a.H] = static_cast<float>(db);
    }
}

// dB (second: dC) from the heads' parts, a group's heads in order: V adjacent
// values of a thread, f.rows tokens of one sequence and group to a workgroup.
template <typename TIO, int V>
__device__ __forceinline__ void head_sums(const FinishArgs &f, int64_t block, bool second) {
    const SsmArgs &a = f.g.f;
    const int runs = (a.L + f.rows - 1) / f.rows, R = a.H / a.G;
    const int run = static_cast<int>(block % runs), bg = static_cast<int>(block / runs), b = bg / a.G, g = bg % a.G;
    const int64_t LN = static_cast<int64_t>(a.L) * a.N;
    const int t0 = run * f.rows, nv = a.N / V, count = min(f.rows, a.L - t0) * nv;
    const float *part = (second ? f.w.dCh : f.w.dBh) + (static_cast<int64_t>(b) * a.H + static_cast<int64_t>(g) * R) * LN +
                        static_cast<int64_t>(t0) * a.N;
    const SsmOperand &o = second ? f.g.dC : f.g.dB;
    TIO *out = static_cast<TIO *>(const_cast<void *>(o.p)) + b * o.sb + g * o.sh;
    for (int i = threadIdx.x; i < count; i += NT) {
        float s[V] = {};
#pragma unroll 4
        for (int r = 0; r < R; ++r) {
            float v[V];
            vec_load<float, V>(part + r * LN + static_cast<int64_t>(i) * V, v);
#pragma unroll
            for (int k = 0; k < V; ++k) s[k] += v[k];
        }
        const int t = i / nv;
        VecIO<TIO, V>::store(out + (t0 + t) * o.st + (i - t * nv) * V, s);
    }
}

// One launch: workgroups of the decay's gradient, then those of dB, of dC.
template <typename TIO, bool SWEEPS, int V>
__global__ __launch_bounds__(NT) void last(FinishArgs f, int decays, int sums) {
    const int64_t i = blockIdx.x;
    if (i < decays)
        decay_gradient<TIO, SWEEPS>(f, static_cast<int>(i));
    else
        head_sums<TIO, V>(f, (i - decays) % sums, i - decays >= sums);
}

template <typename TIO, bool SWEEPS> hipError_t finish(FinishArgs f, hipStream_t s) {
    const SsmArgs &a = f.g.f;
    // a grid's threads are counted in 32 bits: at most 12 million workgroups here
    f.rows = static_cast<int64_t>(a.B) * a.G * a.L < (1 << 24) ? 32 : 256;
    const int decays = a.B * a.H * a.nseg, sums = a.B * a.G * ((a.L + f.rows - 1) / f.rows);
    hipError_t e = hipSuccess;
    if (decays + sums > 0) {
        auto wide = [&](const SsmOperand &o) {
            return (reinterpret_cast<uintptr_t>(o.p) & (4 * sizeof(TIO) - 1)) == 0 && o.sb % 4 == 0 && o.st % 4 == 0 && o.sh % 4 == 0;
        };
        const dim3 grid(static_cast<unsigned>(decays) + 2u * sums);
        if (a.N % 4 == 0 && wide(f.g.dB) && wide(f.g.dC) && (reinterpret_cast<uintptr_t>(a.ws) & 15) == 0)
            hipLaunchKernelGGL((last<TIO, SWEEPS, 4>), grid, dim3(NT), 0, s, f, decays, sums);
        else
            hipLaunchKernelGGL((last<TIO, SWEEPS, 1>), grid, dim3(NT), 0, s, f, decays, sums);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    ColumnSums c{f.w.part, 3 * static_cast<int64_t>(a.H), a.B * a.nseg};
    c.add(0, a.H, 1, f.g.dA);
    c.add(a.H, a.H, 1, f.g.dD);
    c.add(2 * static_cast<int64_t>(a.H), a.H, 1, f.g.ddt_bias);
    return launch_column_sums(c, s);
}

}  // namespace

SsmBwdWs ssm_backward_ws(const SsmArgs &a) {
    const int64_t BH = static_cast<int64_t>(a.B) * a.H, NP = static_cast<int64_t>(a.N) * a.P;
    SsmBwdWs w;
    w.floats = 0;
    auto take = [&](int64_t n) {
        float *q = a.ws ? a.ws + w.floats : nullptr;
        w.floats += static_cast<size_t>((n + 3) / 4 * 4);
        return q;
    };
    w.sf = take(BH * a.nseg * NP);
    w.sr = take(BH * a.nseg * NP);
    w.last = take(BH * NP);
    w.decay = take(BH * a.nseg);
    w.dBh = take(BH * a.L * a.N);
    w.dCh = take(BH * a.L * a.N);
    const int rb = 16 * ssm_lane_values(a.B, a.L, a.H, a.N), cb = 16 * ssm_lane_values(a.B, a.L, a.H, a.P);
    w.rows = (a.N + rb - 1) / rb;
    w.cols = (a.P + cb - 1) / cb;
    w.row = take((w.rows > 2 ? w.rows : 2) * BH * a.L);
    w.col = take((w.cols > 2 ? w.cols : 2) * BH * a.L);
    w.xdu = take(w.cols * BH * a.L);
    w.dyx = take(w.cols * BH * a.L);
    w.tiles = take(BH * ((static_cast<int64_t>(a.L) + 63) / 64) * 8);
    w.part = take(static_cast<int64_t>(a.B) * a.nseg * 3 * a.H);
    w.prep = take(static_cast<int64_t>(ssm_prep_floats(a.B, a.L, a.H)));
    return w;
}

size_t ssm_backward_floats(int B, int L, int H, int P, int N, int nseg) {
    SsmArgs a{};
    a.B = B; a.L = L; a.H = H; a.P = P; a.N = N; a.nseg = nseg;
    return ssm_backward_ws(a).floats;
}

size_t ssm_forward_floats(int B, int L, int H, int P, int N, int nseg) {
    return ssm_prep_floats(B, L, H) +
           (nseg > 1 ? static_cast<size_t>(B) * H * nseg * (static_cast<size_t>(N) * P + 1) : 0);
}

void ssm_segments(int B, int L, int H, int N, bool mfma, bool backward, int *nseg, int *seglen) {
    const int64_t heads = static_cast<int64_t>(B) * H;
    int64_t unit, want, most;  // tokens a segment is a multiple of, segments of a head, units of a segment
    double least;              // where the walk of a segment and the carry over the segments cost the same
    if (mfma) {
        // as many workgroups as run at once (three a compute unit, two where N
        // takes more of its LDS and registers), in whole 64-token chunks; the
        // backward's sums over a segment hold 256 tokens
        unit = 64;
        want = (N > 64 ? 512 : 768) / (heads > 0 ? heads : 1);
        most = INT64_MAX;
        least = std::sqrt(L / 64.0 / 32.0);  // 2 us a chunk, 1 us for 16 segments
        if (backward) {
            // the longest segments, of four chunks at most, that leave the
            // two sweeps 384 workgroups, 1.5 a compute unit: a border costs a
            // share, a carry and its states' product. Whole backward, segments
            // of 1 / 2 / 4 chunks, N = 64: 768 workgroups of four (B=4 L=2048
            // H=12) 109 / 87 / 82 us, 384 (B=2) 70 / 59 / 57, 192 (B=1) 49 /
            // 47 / 49; N = 128, B=4: 214 / 163 / 142
            const int64_t chunks = (static_cast<int64_t>(L) + 63) / 64;
            most = 4;
            while (most > 1 && 2 * heads * ((chunks + most - 1) / most) < 384) --most;
            want = 1;
            least = 1;
        }
    } else {
        // three waves for each SIMD; the backward's sums hold 64 tokens
        unit = 16;
        want = 3 * 1024 / (heads > 0 ? heads : 1);
        most = backward ? 4 : INT64_MAX;
        least = std::fmax(2.0, std::sqrt(L / 6.0) / 16.0);  // 6 us for 16 tokens
    }
    const int64_t units = (static_cast<int64_t>(L) + unit - 1) / unit;
    if (want > units) want = units;
    if (want < 1) want = 1;
    int64_t per = (units + want - 1) / want;
    if (per < static_cast<int64_t>(std::ceil(least)) && units > 1) per = static_cast<int64_t>(std::ceil(least));
    if (per > most) per = most;
    if (per < 1) per = 1;
    *seglen = static_cast<int>(per * unit);
    *nseg = static_cast<int>(units > 0 ? (units + per - 1) / per : 1);
}

hipError_t launch_ssm_bwd_finish(const SsmBwdArgs &g, bool sweeps, hipStream_t stream) {
    const FinishArgs f{g, ssm_backward_ws(g.f), 0};
    if (sweeps) return finish<bf16_t, true>(f, stream);  // bf16 alone
    return g.f.io == 1 ? finish<bf16_t, false>(f, stream) : finish<float, false>(f, stream);
}

}  // namespace ttt
