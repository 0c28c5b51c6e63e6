// Max-norm quantization to 8 bits: levels and scale of each row, or of each
// column with the levels transposed. Formulas in include/qsgd_ops.h.
//
// Bound by memory: an element is read once (2 or 4 bytes) and its level written
// (1 byte). Rows of up to 16384 values stay in registers between the maximum and
// the rounding; the column form reads x twice, the second time out of the
// 256 MB last-level cache for the sizes that fit it.
#pragma once

#include "ops_common.h"

namespace qsgd {
namespace ops {

// The maximum of |y| is taken over the magnitudes' bit patterns: they are ordered
// as the magnitudes are, with infinity above every number and NaN above infinity,
// so neither is lost.
__device__ __forceinline__ uint32_t magnitude(float y) { return __float_as_uint(y) & 0x7fffffffu; }

struct RowScale {
    float scale, inv;
    bool ok;    // finite and not 0
    bool safe;  // y * inv is near y / scale
};

__device__ __forceinline__ RowScale row_scale(uint32_t amax) {
    RowScale r;
    r.scale = __uint_as_float(amax) / 127.0f;
    r.ok = r.scale > 0.0f && r.scale < INFINITY;
    r.safe = r.scale > 0x1p-100f && r.scale < 0x1p100f;
    r.inv = 1.0f / r.scale;
    return r;
}

// RNE(RN32(y / scale)) without a division where it cannot matter. y * inv lies
// within 127 * 2^-23 < 2e-5 of the real quotient (two roundings), RN32(y / scale)
// within half of that, so they round to the same integer unless y * inv is within
// 1e-4 of a half; then the quotient itself is taken. About one value in 5000
// takes it with fp32 inputs.
__device__ __forceinline__ int level_of(float y, const RowScale &s) {
    float r = y * s.inv, k = rintf(r);
    if (!s.safe || fabsf(fabsf(r - k) - 0.5f) < 1e-4f) k = rintf(y / s.scale);
    k = fminf(fmaxf(k, -127.0f), 127.0f);  // a subnormal scale may be far below max |y| / 127
    return s.ok ? (int)k : 0;
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)d << 24;
}

struct QuantizeParams {
    const void *x;
    const float *fold;
    int8_t *levels;
    float *scale;
    uint64_t ldx, ldl;
    uint32_t rows, cols;
    uint32_t wide;  // columns written: cols, or up to a multiple of 16 (zeros past cols)
};

// Eight levels to columns [c, c + 8) of a row, those below `wide`.
__device__ __forceinline__ void put_levels(int8_t *row, uint32_t c, uint32_t wide, const float (&y)[8],
                                           const RowScale &s) {
    int k[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = level_of(y[i], s);
    if (c + 8 <= wide) {
        const uint32_t w[2] = {pack4(k[0], k[1], k[2], k[3]), pack4(k[4], k[5], k[6], k[7])};
        __builtin_memcpy(row + c, w, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < wide) row[c + i] = (int8_t)k[i];
    }
}

// TPR threads take a row (a wave or the workgroup), each NV chunks of 8 values
// that stay in registers; NV = 0 takes rows of any length, reading them twice.
template <class T, int TPR, int NV>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantizeParams p) {
    __shared__ uint32_t part[4];
    const uint32_t row = (uint32_t)block_index() * (256 / TPR) + threadIdx.x / TPR;
    const uint32_t t = threadIdx.x % TPR;
    if (row >= p.rows) return;  // a whole wave, or the workgroup
    const T *x = (const T *)p.x + (uint64_t)row * p.ldx;
    const auto get = [&](uint32_t c, float (&y)[8]) {
        load_upto8(x + c, (int64_t)p.cols - c, 0.0f, y);
        if (p.fold) {
            float f[8];
            load_upto8(p.fold + c, (int64_t)p.cols - c, 0.0f, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= f[i];
        }
    };
    uint32_t amax = 0;
    float y[NV > 0 ? NV : 1][8];
    if (NV > 0) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const uint32_t c = (v * TPR + t) * 8;
            if (c < p.cols) get(c, y[v]);
            else for (int i = 0; i < 8; ++i) y[v][i] = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = max(amax, magnitude(y[v][i]));
        }
    } else {
        for (uint64_t c = t * 8; c < p.cols; c += TPR * 8) {
            get((uint32_t)c, y[0]);
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = max(amax, magnitude(y[0][i]));
        }
    }
    amax = wave_max(amax);
    if (TPR == 256) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = amax;
        __syncthreads();
        amax = max(max(part[0], part[1]), max(part[2], part[3]));
    }
    const RowScale s = row_scale(amax);
    if (t == 0) p.scale[row] = s.scale;
    int8_t *out = p.levels + (uint64_t)row * p.ldl;
    if (NV > 0) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const uint32_t c = (v * TPR + t) * 8;
            if (c < p.wide) put_levels(out, c, p.wide, y[v], s);
        }
    } else {
        for (uint64_t c = t * 8; c < p.wide; c += TPR * 8) {
            if (c < p.cols) get((uint32_t)c, y[0]);
            else for (int i = 0; i < 8; ++i) y[0][i] = 0.0f;
            put_levels(out, (uint32_t)c, p.wide, y[0], s);
        }
    }
}

struct TransposeParams {
    const void *x;
    const float *fold;
    int8_t *levels;
    float *scale;
    uint32_t *part;  // [splits, cols]: the column maxima of each run of rows
    uint64_t ldx, ldl;
    uint32_t rows, cols;
    uint32_t wide;  // rows written: rows, or up to a multiple of 16 (zeros past rows)
    uint32_t splits, rows_per_split;
    uint32_t row_tiles, col_tiles;
};

constexpr uint32_t kMaxSplits = 32;

// Column maxima of a run of rows: a wave takes every fourth row, a lane 8 columns.
template <class T>
__global__ __launch_bounds__(256) void column_max_kernel(TransposeParams p) {
    __shared__ uint32_t part[3][512];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t c = blockIdx.x * 512 + lane * 8;
    const uint32_t lo = blockIdx.y * p.rows_per_split, hi = min(p.rows, lo + p.rows_per_split);
    uint32_t amax[8] = {};
    if (c < p.cols) {
        const T *x = (const T *)p.x + c;
#pragma unroll 4
        for (uint32_t r = lo + wave; r < hi; r += 4) {
            float y[8];
            load_upto8(x + (uint64_t)r * p.ldx, (int64_t)p.cols - c, 0.0f, y);
            const float f = p.fold ? p.fold[r] : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax[i] = max(amax[i], magnitude(y[i] * f));
        }
    }
    if (wave) {
#pragma unroll
        for (int i = 0; i < 8; ++i) part[wave - 1][i * 64 + lane] = amax[i];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t m = max(max(amax[i], part[0][i * 64 + lane]), max(part[1][i * 64 + lane], part[2][i * 64 + lane]));
            if (c + i < p.cols) p.part[(uint64_t)blockIdx.y * p.cols + c + i] = m;
        }
    }
}

// A tile of 128 rows and 64 columns, transposed through LDS. A thread takes four
// rows of eight columns, so a column's four levels make one LDS word: the tile's
// columns have 33 words, which spreads a wave's writes over all banks. T = int8_t
// moves bytes as they are.
template <class T>
__global__ __launch_bounds__(256) void transpose_kernel(TransposeParams p) {
    constexpr bool kBytes = sizeof(T) == 1;
    __shared__ uint32_t tile[64 * 33];
    __shared__ uint32_t cmax[4][64];
    const uint32_t t = threadIdx.x;
    const uint64_t block = block_index();
    if (block >= (uint64_t)p.row_tiles * p.col_tiles) return;
    const uint32_t r0 = (uint32_t)(block % p.row_tiles) * 128, c0 = (uint32_t)(block / p.row_tiles) * 64;
    const uint32_t c = c0 + (t & 7) * 8, r = r0 + (t >> 3) * 4;
    if (!kBytes) {
        const uint32_t cc = c0 + (t & 63);
        uint32_t m = 0;
        if (cc < p.cols)
            for (uint32_t s = t >> 6; s < p.splits; s += 4) m = max(m, p.part[(uint64_t)s * p.cols + cc]);
        cmax[t >> 6][t & 63] = m;
    }
    float y[4][8];
    uint8_t b[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool there = r + j < p.rows && c < p.cols;
        const T *x = (const T *)p.x + (uint64_t)(r + j) * p.ldx + c;
        if (kBytes) {
            if (there && c + 8 <= p.cols) __builtin_memcpy(b[j], x, 8);
            else
                for (int i = 0; i < 8; ++i) b[j][i] = there && c + i < p.cols ? (uint8_t)x[i] : 0;
        } else {
            if (there) load_upto8(x, (int64_t)p.cols - c, 0.0f, y[j]);
            else for (int i = 0; i < 8; ++i) y[j][i] = 0.0f;
            const float f = p.fold && there ? p.fold[r + j] : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[j][i] *= f;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t k = (t & 7) * 8 + i;
        uint32_t w;
        if (kBytes) {
            w = pack4(b[0][i], b[1][i], b[2][i], b[3][i]);
        } else {
            const RowScale s = row_scale(max(max(cmax[0][k], cmax[1][k]), max(cmax[2][k], cmax[3][k])));
            if (r0 == 0 && t < 8 && c + i < p.cols) p.scale[c + i] = s.scale;
            w = pack4(level_of(y[0][i], s), level_of(y[1][i], s), level_of(y[2][i], s), level_of(y[3][i], s));
        }
        tile[k * 33 + (t >> 3)] = w;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t k = h * 32 + (t >> 3), q = (t & 7) * 4;
        const uint32_t rr = r0 + q * 4;
        if (c0 + k >= p.cols || rr >= p.wide) continue;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = tile[k * 33 + q + i];
        int8_t *out = p.levels + (uint64_t)(c0 + k) * p.ldl + rr;
        if (rr + 16 <= p.wide) {
            __builtin_memcpy(out, w, 16);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (rr + i < p.wide) out[i] = (int8_t)(w[i / 4] >> (8 * (i % 4)));
        }
    }
}

// Bytes of a row of levels in LDS: whole 64-byte steps, and 16 more so that rows
// begin in different banks.
__host__ __device__ __forceinline__ uint32_t fused_pitch(uint32_t k) { return (k + 63) / 64 * 64 + 16; }

// The levels of m rows of x into LDS and their scales into sx, by a workgroup of
// eight waves; ends with a barrier. A row is taken by eight waves, or by fewer
// where there are more rows. `part` holds 16 words.
template <class X>
__device__ __forceinline__ void quantize_to_lds(const X *x, uint64_t ldx, uint32_t m, uint32_t k, uint32_t pitch,
                                                int8_t *levels, float *sx, uint32_t *part) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t share = m == 1 ? 8 : m == 2 ? 4 : m <= 4 ? 2 : 1;  // waves of a row
    const uint32_t at = wave % share * 512 + lane * 8, step = share * 512;
    for (uint32_t r0 = 0; r0 < m; r0 += 8 / share) {
        const uint32_t row = r0 + wave / share;
        const X *from = x + (uint64_t)row * ldx;
        uint32_t amax = 0;
        if (row < m)
            for (uint32_t c = at; c < k; c += step) {
                float y[8];
                load_upto8(from + c, (int64_t)k - c, 0.0f, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = max(amax, magnitude(y[i]));
            }
        amax = wave_max(amax);
        if (lane == 0) part[wave] = amax;
        __syncthreads();
        for (uint32_t i = 0; i < share; ++i) amax = max(amax, part[wave / share * share + i]);
        const RowScale s = row_scale(amax);
        if (row < m) {
            if (at == 0) sx[row] = s.scale;
            for (uint32_t c = at; c < pitch; c += step) {
                float y[8] = {};
                if (c < k) load_upto8(from + c, (int64_t)k - c, 0.0f, y);
                put_levels(levels + (uint64_t)row * pitch, c, pitch, y, s);
            }
        }
        __syncthreads();
    }
}

// Copies rows of bytes to a row stride that is a multiple of 16, zeros past the
// row's end, so that the product's tiles can be loaded 16 bytes at a time.
struct RepackParams {
    const int8_t *src;
    int8_t *dst;
    uint64_t lds, ldd;
    uint32_t rows, cols;
};

static __global__ __launch_bounds__(256) void repack_kernel(RepackParams p) {
    const uint64_t per_row = p.ldd / 16;
    const uint64_t at = block_index() * 256 + threadIdx.x;
    if (at >= per_row * p.rows) return;
    const uint64_t row = at / per_row, c = at % per_row * 16;
    const int8_t *s = p.src + row * p.lds + c;
    uint32_t w[4] = {0, 0, 0, 0};
    if (c + 16 <= p.cols) {
        __builtin_memcpy(w, s, 16);
    } else {
        for (int i = 0; i < 16; ++i)
            if (c + i < p.cols) w[i / 4] |= (uint32_t)(uint8_t)s[i] << (8 * (i % 4));
    }
    *(uint4 *)(p.dst + row * p.ldd + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace ops
}  // namespace qsgd
