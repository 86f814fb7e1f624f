// Pieces of the state space scan's MFMA kernels (gfx950): 64-token chunks of
// bf16 operands in LDS, transposed fragment reads, and the chunk's decays.
//
// 16x16x32 products: lane (g = lane / 16, c = lane % 16) gives row or column c
// and, of the contraction, either 32 kb + 8 g .. + 7 (features: 16 bytes of a
// row) or tokens 32 kb + 4 g .. + 3 and 32 kb + 16 + 4 g .. + 3 (the order in
// which two products' outputs lie in a lane, so an output tile is the next
// product's operand as it stands). It receives rows 4 g .. 4 g + 3 of column c.
#pragma once

#include "ssm.hpp"
#include "vec.hpp"

namespace ttt {
namespace ssm {

using namespace tile;

constexpr int Q = 64;       // tokens of a chunk
constexpr int XS = 64 + 8;  // row stride (elements) of 64 features: rows 4 banks apart
constexpr float LOG2E = 1.4426950408889634f;

typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Four tokens' values of one feature for each lane: in a group of 16 lanes,
// lane 4 r + q points at four features of row r; lane 4 q + s receives feature
// s of those that q points at, of rows 0 .. 3.
__device__ __forceinline__ s16x4 read_tr(const uint16_t *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
}
__device__ __forceinline__ bf16x8 join(s16x4 a, s16x4 b) {
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ __forceinline__ bf16x8 read16(const uint16_t *p) {
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4 *>(p));
}

// Transposed fragment (contraction over tokens 32 kb .. + 31) of the 16
// features f0 .. f0 + 15 of a [64 tokens][stride] tile.
__device__ __forceinline__ bf16x8 tokens_frag(const uint16_t *tile, int stride, int kb, int f0, int g, int c) {
    const uint16_t *p = tile + (32 * kb + 4 * g + c / 4) * stride + f0 + 4 * (c % 4);
    return join(read_tr(p), read_tr(p + 16 * stride));
}

// Per token of a chunk: log2 of the decay since the chunk's start, split into
// two floats (their differences are decays between two tokens: one float would
// lose up to |sum| 2^-24 of them), D_t, and the decay to the chunk's end.
struct ChunkDecay {
    alignas(16) float hi[Q], lo[Q], step[Q], tail[Q];
    __device__ __forceinline__ float total() const { return hi[Q - 1]; }  // log2 of the whole chunk's
};
static_assert(sizeof(ChunkDecay) == 4 * Q * sizeof(float), "as ssm_prep writes it");

// x = a + b + c to about 24 bits, each a bf16 (two floats at a time)
__device__ __forceinline__ void split3(float x0, float x1, uint32_t &a, uint32_t &b, uint32_t &c) {
    a = pack2(x0, x1);
    x0 -= lo_bf(a);
    x1 -= hi_bf(a);
    b = pack2(x0, x1);
    c = pack2(x0 - lo_bf(b), x1 - hi_bf(b));
}

// A fragment of a transposed read times one weight for each of its tokens
// (w0: the first four, w1: the others), in one or three bf16 parts.
template <int PARTS>
__device__ __forceinline__ void weigh(bf16x8 f, f32x4 w0, f32x4 w1, bf16x8 (&out)[PARTS]) {
    static_assert(PARTS == 1 || PARTS == 3, "rounded, or to about 24 bits");
    const uint4 r = __builtin_bit_cast(uint4, f);
    const uint32_t in[4] = {r.x, r.y, r.z, r.w};
    uint32_t p[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = lo_bf(in[i]) * (i < 2 ? w0[2 * i] : w1[2 * i - 4]);
        const float b = hi_bf(in[i]) * (i < 2 ? w0[2 * i + 1] : w1[2 * i - 3]);
        if constexpr (PARTS == 1)
            p[0][i] = pack2(a, b);
        else
            split3(a, b, p[0][i], p[1][i], p[2][i]);
    }
#pragma unroll
    for (int k = 0; k < PARTS; ++k)
        out[k] = __builtin_bit_cast(bf16x8, make_uint4(p[k][0], p[k][1], p[k][2], p[k][3]));
}

typedef __attribute__((ext_vector_type(2))) short s16x2;
__device__ __forceinline__ s16x2 as_bf16x2(uint32_t v) { return __builtin_bit_cast(s16x2, v); }

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Feature f of a row of `cols`, 0 behind them (which are not read).
__device__ __forceinline__ uint32_t feature_or_zero(const bf16_t *row, int f, int cols) {
    const uint32_t v = row[min(f, cols - 1)];
    return f < cols ? v : 0u;
}
__device__ __forceinline__ uint2 four(const bf16_t *row, int f, int cols) {
    return make_uint2(feature_or_zero(row, f, cols) | feature_or_zero(row, f + 1, cols) << 16,
                      feature_or_zero(row, f + 2, cols) | feature_or_zero(row, f + 3, cols) << 16);
}
// How a kernel's operands lie in its tiles of 64 x 32, 64 or 128 features.
// FULL: they fill them, in 16-byte accesses. WIDE: multiples of eight features
// in such accesses, the rest of a tile is zeros. SINGLE: any number in any
// place, read one by one.
enum Fit { SINGLE, WIDE, FULL };

// Eight adjacent features of a row.
template <Fit FIT> __device__ __forceinline__ uint4 eight(const bf16_t *row, int f, int cols) {
    if constexpr (FIT == FULL) return *reinterpret_cast<const uint4 *>(row + f);
    if constexpr (FIT == WIDE) {
        const uint4 v = *reinterpret_cast<const uint4 *>(row + min(f, cols - 8));
        return f < cols ? v : make_uint4(0, 0, 0, 0);
    }
    const uint2 a = four(row, f, cols), b = four(row, f + 4, cols);
    return make_uint4(a.x, a.y, b.x, b.y);
}

// Four adjacent features f .. f + 3 to a row of `cols`.
template <Fit FIT> __device__ __forceinline__ void store4(bf16_t *row, int f, int cols, const float (&v)[4]) {
    if constexpr (FIT != SINGLE) {
        if (FIT == FULL || f < cols) VecIO<bf16_t, 4>::store(row + f, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (f + i < cols) row[f + i] = f32_to_bf16(v[i]);
    }
}

// A token's 64 output values, of which a lane holds features 16 u + 4 g .. + 3
// as v[u], to its row of `cols`. Lane rows g and g ^ 1 exchange a quad of two
// tiles, so that each stores eight adjacent features at a time, 64 bytes of the
// row to an instruction (scan outputs, 2 x 8192 tokens, 32 heads: 41 us, 43.5 us with
// quads of 8 bytes as they lie). All lanes of the wave call it.
template <Fit FIT>
__device__ __forceinline__ void store_row(bf16_t *row, bool live, const float (&v)[4][4], int g, int cols) {
    if constexpr (FIT == SINGLE) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (live) store4<SINGLE>(row, 16 * u + 4 * g, cols, v[u]);
    } else {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const float *p = v[2 * a], *q = v[2 * a + 1];
            // odd rows of the first with even rows of the second
            const auto lo = __builtin_amdgcn_permlane16_swap(pack2(p[0], p[1]), pack2(q[0], q[1]), false, false);
            const auto hi = __builtin_amdgcn_permlane16_swap(pack2(p[2], p[3]), pack2(q[2], q[3]), false, false);
            const int f = 32 * a + 16 * (g % 2) + 8 * (g / 2);
            if (live && (FIT == FULL || f < cols))
                *reinterpret_cast<uint4 *>(row + f) = make_uint4(lo[0], hi[0], lo[1], hi[1]);
        }
    }
}

// 64 rows of F features (F = 32, 64, 128) from global memory to LDS by 256
// threads: 16 bytes each, through registers, fetched while the chunk before is
// worked on; single elements are read when they are put (they would take four
// times the registers). Rows at and past `count` are zeros and are
// not read.
template <int F, Fit FIT> struct Stage {
    static constexpr int PER = F / 8;         // accesses of a row
    static constexpr int ROWS = 256 / PER;    // rows of a pass
    static constexpr int NP = Q / ROWS;       // passes
    uint4 r[FIT == SINGLE ? 1 : NP];
    const bf16_t *base;
    int64_t stride;
    int count;
    __device__ __forceinline__ void fetch(const bf16_t *from, int64_t row_stride, int rows, int cols) {
        if constexpr (FIT != SINGLE) {
            const int row = threadIdx.x / PER, f = threadIdx.x % PER * 8;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int t = row + i * ROWS;
                r[i] = make_uint4(0, 0, 0, 0);
                if (t < rows && (FIT == FULL || f < cols)) r[i] = *reinterpret_cast<const uint4 *>(from + t * row_stride + f);
            }
        } else {
            base = from;
            stride = row_stride;
            count = rows;
        }
    }
    __device__ __forceinline__ uint4 values(int i, int cols) const {
        if constexpr (FIT != SINGLE) return r[i];
        const int t = threadIdx.x / PER + i * ROWS, f = threadIdx.x % PER * 8;
        return t < count ? eight<SINGLE>(base + t * stride, f, cols) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void put(uint16_t *tile, int lds_stride, int cols) const {
        const int row = threadIdx.x / PER, f = threadIdx.x % PER * 8;
#pragma unroll
        for (int i = 0; i < NP; ++i) *reinterpret_cast<uint4 *>(tile + (row + i * ROWS) * lds_stride + f) = values(i, cols);
    }
    // The same, with zeros in the place of infinities and NaN. Returns whether
    // the wave has any: then first[feature] is the first row where it found
    // one, Q where it found none.
    __device__ __forceinline__ bool put_finite(uint16_t *tile, int lds_stride, int cols, int *first) const {
        static_assert(F == 64, "a lane for each feature");
        const int row = threadIdx.x / PER, f = threadIdx.x % PER * 8;
        uint4 v[NP];
        float zero = 0.f;  // the sum of all values times 0
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            v[i] = values(i, cols);
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) zero = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(w[k]), as_bf16x2(0), zero, false);
        }
        const bool found = __any(zero != 0.f);
        if (__builtin_expect(found, 0)) {
            first[threadIdx.x % 64] = Q;
            for (int i = 0; i < NP; ++i) {
                uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                for (int k = 0; k < 8; ++k) {
                    const uint32_t mask = 0x7f80u << 16 * (k % 2);
                    if ((w[k / 2] & mask) == mask) {
                        atomicMin(&first[f + k], row + i * ROWS);
                        w[k / 2] &= k % 2 ? 0x0000ffffu : 0xffff0000u;
                    }
                }
                v[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) *reinterpret_cast<uint4 *>(tile + (row + i * ROWS) * lds_stride + f) = v[i];
        return found;
    }
};

// A chunk's decays, which ssm_prep has laid out, to LDS by the first 64 threads.
struct StageDecay {
    uint4 r;
    __device__ __forceinline__ void fetch(const float *base) {
        if (threadIdx.x < Q) r = *reinterpret_cast<const uint4 *>(base + 4 * threadIdx.x);
    }
    __device__ __forceinline__ void put(ChunkDecay &d) const {
        if (threadIdx.x < Q) *reinterpret_cast<uint4 *>(&d.hi[0] + 4 * threadIdx.x) = r;
    }
};

// Workgroup -> (sequence and segment, head) such that the heads of one segment,
// which read the same B and C, run on one XCD (workgroups go to the eight XCDs
// in turn). The last few segments that do not fill a round of eight are spread.
__device__ __forceinline__ void place(int blk, int segs, int heads, int &bs, int &h) {
    const int full = segs / 8 * 8;
    if (blk < full * heads) {
        const int i = blk / 8;
        bs = i / heads * 8 + blk % 8;
        h = i % heads;
    } else {
        bs = blk / heads;
        h = blk % heads;
    }
}

}  // namespace ssm
}  // namespace ttt
