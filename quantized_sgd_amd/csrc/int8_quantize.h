// Max-norm quantization to 8 bits: levels and scale of each row, or of each
// column with the levels transposed. Formulas in include/qsgd_ops.h.
//
// Bound by memory: an element is read once (2 or 4 bytes) and its level written
// (1 byte). Rows of up to 16384 values stay in registers between the maximum and
// the rounding (4096 x 4096 in bfloat16: 11.2 us, 4.5 TB/s; 8192 x 4096: 23.1 us, 4.4
// TB/s); the column form reads x twice, the second time out of the 256 MB last-level
// cache for the sizes that fit it. Rows and columns in one kernel (tiles of whole
// columns held in LDS) took 47 us at 8192 x 4096, 24 and 22 apart.
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

__device__ __forceinline__ RowScale with_inverse(float2 v) {
    return {v.x, v.y, v.x > 0.0f && v.x < INFINITY, v.x > 0x1p-100f && v.x < 0x1p100f};
}
__device__ __forceinline__ RowScale row_scale(uint32_t amax) {
    const float scale = __uint_as_float(amax) / 127.0f;
    return with_inverse(make_float2(scale, 1.0f / scale));
}

// Eight levels RNE(RN32(y / scale)), packed, without a division where it cannot
// matter. y * inv lies within 127 * 2^-23 < 2e-5 of the real quotient (two
// roundings), RN32(y / scale) within half of that, so they round to the same integer
// unless y * inv is within 1e-4 of a half; then the quotient itself is taken.
// Adding 1.5 * 2^23 rounds to the nearest integer (ties to even) and leaves its two's
// complement in the sum's low bits, so a level costs five operations and three
// byte permutes for four of them pack it. A safe scale is max |y| / 127 to 2^-24, so no
// level passes 127; an unsafe one (subnormal) may be far from it.
// The first four have scale s[0], the others s[1].
__device__ __forceinline__ void levels8(const float (&y)[8], const RowScale (&s)[2], uint32_t (&w)[2]) {
    constexpr float kMagic = 12582912.0f;
    float b[8], d[8], far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float r = y[i] * s[i / 4].inv;
        b[i] = r + kMagic;
        d[i] = r - (b[i] - kMagic);
        far = fmaxf(far, fabsf(d[i]));
    }
    if (far > 0.4999f || !s[0].safe || !s[1].safe) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(d[i]) > 0.4999f || !s[i / 4].safe)
                b[i] = fminf(fmaxf(rintf(y[i] / s[i / 4].scale), -127.0f), 127.0f) + kMagic;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(b[4 * h + 1]), __float_as_uint(b[4 * h]), 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(b[4 * h + 3]), __float_as_uint(b[4 * h + 2]), 0x0c0c0400u);
        w[h] = s[h].ok ? lo | hi << 16 : 0u;
    }
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
    uint32_t w[2];
    levels8(y, {s, s}, w);
    if (c + 8 <= wide) {
        __builtin_memcpy(row + c, w, 8);
    } else {
        for (uint32_t i = 0; c + i < wide; ++i) row[c + i] = (int8_t)((i < 4 ? w[0] : w[1]) >> (8 * (i & 3)));
    }
}

__device__ __forceinline__ uint32_t largest(uint32_t amax, const float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) amax = max(max(amax, magnitude(y[i])), magnitude(y[i + 1]));
    return amax;
}

// TPR threads take a row (a wave or the workgroup), each NV chunks of 8 values
// that stay in registers; NV = 0 takes rows of any length, reading them twice.
template <class T, int TPR, int NV>
__device__ __forceinline__ void quantize_rows_block(const QuantizeParams &p, uint64_t block, uint32_t *part) {
    const uint32_t row = (uint32_t)block * (256 / TPR) + threadIdx.x / TPR;
    const uint32_t t = threadIdx.x % TPR;
    if (row >= p.rows) return;  // a whole wave, or the workgroup
    const T *x = (const T *)p.x + (uint64_t)row * p.ldx;
    const auto values = [&](uint32_t c, Eight<T> &raw, Eight<float> &raw_fold, float (&y)[8]) {
        settle(c, p.cols, raw, y);
        if (p.fold) {
            float f[8];
            settle(c, p.cols, raw_fold, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= f[i];
        }
    };
    uint32_t amax = 0;
    float y[NV > 0 ? NV : 1][8];
    if (NV > 0) {
        Eight<T> raw[NV > 0 ? NV : 1];
        Eight<float> raw_fold[NV > 0 ? NV : 1];
#pragma unroll
        for (int v = 0; v < NV; ++v) fetch(x, (v * TPR + t) * 8, p.cols, raw[v]);
        if (p.fold) {
#pragma unroll
            for (int v = 0; v < NV; ++v) fetch(p.fold, (v * TPR + t) * 8, p.cols, raw_fold[v]);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            values((v * TPR + t) * 8, raw[v], raw_fold[v], y[v]);
            amax = largest(amax, y[v]);
        }
    } else {
#pragma unroll 4
        for (uint32_t c = t * 8; c < p.cols; c += TPR * 8) {
            Eight<T> raw;
            Eight<float> raw_fold;
            fetch(x, c, p.cols, raw);
            if (p.fold) fetch(p.fold, c, p.cols, raw_fold);
            values(c, raw, raw_fold, y[0]);
            amax = largest(amax, y[0]);
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
        for (uint32_t c = t * 8; c < p.wide; c += TPR * 8) {
            Eight<T> raw;
            Eight<float> raw_fold;
            fetch(x, c, p.cols, raw);
            if (p.fold) fetch(p.fold, c, p.cols, raw_fold);
            values(c, raw, raw_fold, y[0]);
            put_levels(out, c, p.wide, y[0], s);
        }
    }
}

template <class T, int TPR, int NV>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantizeParams p) {
    __shared__ uint32_t part[4];
    quantize_rows_block<T, TPR, NV>(p, block_index(), part);
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

constexpr uint32_t kMaxSplits = 256;
constexpr uint32_t kFewSplits = 32;  // joined by the kernel that uses them

// Column maxima of a run of rows: a wave takes every fourth row, a lane 8 columns.
template <class T>
__device__ __forceinline__ void column_max_block(const TransposeParams &p, uint32_t block, uint32_t (*part)[512]) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t wide = (p.cols + 511) / 512, split = block / wide;
    const uint32_t c = block % wide * 512 + lane * 8;
    const uint32_t lo = split * p.rows_per_split, hi = min(p.rows, lo + p.rows_per_split);
    uint32_t amax[8] = {};
    if (c < p.cols) {
        const T *x = (const T *)p.x;
        constexpr int kRows = 4;  // loads in flight
        for (uint32_t r = lo + wave; r < hi; r += 4 * kRows) {
            Eight<T> raw[kRows];
            float f[kRows];
#pragma unroll
            for (int g = 0; g < kRows; ++g) {
                const uint32_t at = min(r + 4 * g, hi - 1);  // past the run: its last row again
                fetch(x + (uint64_t)at * p.ldx, c, p.cols, raw[g]);
                f[g] = p.fold ? p.fold[at] : 1.0f;
            }
#pragma unroll
            for (int g = 0; g < kRows; ++g) {
                float y[8];
                settle(c, p.cols, raw[g], y);
#pragma unroll
                for (int i = 0; i < 8; ++i) amax[i] = max(amax[i], magnitude(y[i] * f[g]));
            }
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
            if (c + i < p.cols) p.part[(uint64_t)split * p.cols + c + i] = m;
        }
    }
}
// 1021 x 5003 in fp32: 7.0 us, bound by the latency of a run's loads.
template <class T>
__global__ __launch_bounds__(256) void column_max_kernel(TransposeParams p) {
    __shared__ uint32_t part[3][512];
    column_max_block<T>(p, blockIdx.x, part);
}

// Joins the runs' column maxima where there are more than kFewSplits: a column's
// scale. 64 columns a workgroup, sixteen threads a column (4096 columns of 128 runs:
// 4.7 us, a launch and two loads' latency).
static __global__ __launch_bounds__(1024) void column_scale_kernel(TransposeParams p) {
    __shared__ uint32_t part[16][64];
    const uint64_t block = block_index();
    if (block * 64 >= p.cols) return;
    const uint32_t c = (uint32_t)block * 64 + (threadIdx.x & 63), g = threadIdx.x >> 6;
    uint32_t m = 0;
    if (c < p.cols) {
#pragma unroll 8
        for (uint32_t s = g; s < p.splits; s += 16) m = max(m, p.part[(uint64_t)s * p.cols + c]);
    }
    part[g][threadIdx.x & 63] = m;
    __syncthreads();
    if (g == 0 && c < p.cols) {
#pragma unroll
        for (int i = 1; i < 16; ++i) m = max(m, part[i][threadIdx.x]);
        p.scale[c] = row_scale(m).scale;
    }
}

// A tile of 128 rows and 64 columns, transposed through LDS. A thread takes four
// rows of eight columns, so a column's four levels make one LDS word: the tile's
// columns have 33 words, which spreads a wave's writes over all banks. T = int8_t
// moves bytes as they are.
template <class T>
__device__ __forceinline__ void transpose_block(const TransposeParams &p, uint64_t block, uint32_t *tile, float2 *scales) {
    constexpr bool kBytes = sizeof(T) == 1;
    const uint32_t t = threadIdx.x;
    if (block >= (uint64_t)p.row_tiles * p.col_tiles) return;
    const uint32_t r0 = (uint32_t)(block % p.row_tiles) * 128, c0 = (uint32_t)(block / p.row_tiles) * 64;
    const uint32_t c = c0 + (t & 7) * 8, r = r0 + (t >> 3) * 4;
    float y[4][8];
    uint8_t b[4][8];
    if constexpr (kBytes) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool there = r + j < p.rows && c < p.cols;
            const T *x = (const T *)p.x + (uint64_t)(r + j) * p.ldx + c;
            if (there && c + 8 <= p.cols) __builtin_memcpy(b[j], x, 8);
            else
                for (int i = 0; i < 8; ++i) b[j][i] = there && c + i < p.cols ? (uint8_t)x[i] : 0;
        }
    } else {
        Eight<T> raw[4];
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t at = min(r + j, p.rows - 1);
            fetch((const T *)p.x + (uint64_t)at * p.ldx, c, p.cols, raw[j]);
            f[j] = p.fold ? p.fold[at] : 1.0f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            settle(c, p.cols, raw[j], y[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[j][i] = r + j < p.rows ? y[j][i] * f[j] : 0.0f;
        }
    }
    if (kBytes) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            tile[((t & 7) * 8 + i) * 33 + (t >> 3)] =
                (uint32_t)b[0][i] | (uint32_t)b[1][i] << 8 | (uint32_t)b[2][i] << 16 | (uint32_t)b[3][i] << 24;
    } else {
        if (p.splits <= kFewSplits) {  // this tile's columns' scales, joined here
            const uint32_t col = c0 + (t & 63);
            uint32_t m = 0;
            if (col < p.cols) {
#pragma unroll
                for (uint32_t s = 0; s < kFewSplits; s += 4)
                    if (s + (t >> 6) < p.splits) m = max(m, p.part[(uint64_t)(s + (t >> 6)) * p.cols + col]);
            }
            tile[t] = m;
            __syncthreads();
            if (t < 64) {
                const RowScale s = row_scale(max(max(tile[t], tile[64 + t]), max(tile[128 + t], tile[192 + t])));
                scales[t] = make_float2(s.scale, s.inv);
                if (r0 == 0 && col < p.cols) p.scale[col] = s.scale;
            }
        } else if (t < 64) {
            const float s = c0 + t < p.cols ? p.scale[c0 + t] : 0.0f;
            scales[t] = make_float2(s, 1.0f / s);
        }
        __syncthreads();
        // two columns at a time: four levels of each
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint32_t k = (t & 7) * 8 + i;
            uint32_t w[2];
            levels8({y[0][i], y[1][i], y[2][i], y[3][i], y[0][i + 1], y[1][i + 1], y[2][i + 1], y[3][i + 1]},
                    {with_inverse(scales[k]), with_inverse(scales[k + 1])}, w);
            tile[k * 33 + (t >> 3)] = w[0];
            tile[(k + 1) * 33 + (t >> 3)] = w[1];
        }
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

// 8192 x 4096 in bfloat16: 23.4 us, 4.3 TB/s of values read and levels written; tiles of
// 128 x 64 pass through LDS, so that both sides go by whole cache lines. 1021 x 5003 in
// fp32: 11.6 us (strided, odd rows: 4-byte loads).
template <class T>
__global__ __launch_bounds__(256) void transpose_kernel(TransposeParams p) {
    __shared__ uint32_t tile[64 * 33];
    __shared__ float2 scales[64];  // with its inverse
    transpose_block<T>(p, block_index(), tile, scales);
}

// What the gradient's products need, in one launch of workgroups of four kinds: the
// column maxima of gy, its rows' levels, w and xq transposed (8192 x 4096 x 4096 in
// bfloat16: 49 us for 236 MB, 4.8 TB/s; the gradient of 1000 x 777 x 1537 takes 12 us
// less than with a launch each).
struct GradientParams {
    QuantizeParams rows;
    TransposeParams columns, w, x;
    uint64_t n_max, n_rows, n_w, n_x;  // workgroups of each
};
template <class T, int TPR, int NV>
__global__ __launch_bounds__(256) void gradient_inputs_kernel(GradientParams p) {
    __shared__ uint32_t lds[64 * 33];
    uint64_t block = block_index();
    if (block < p.n_max) return column_max_block<T>(p.columns, (uint32_t)block, (uint32_t(*)[512])lds);
    block -= p.n_max;
    if (block < p.n_rows) return quantize_rows_block<T, TPR, NV>(p.rows, block, lds);
    block -= p.n_rows;
    if (block < p.n_w) return transpose_block<int8_t>(p.w, block, lds, nullptr);
    block -= p.n_w;
    if (block < p.n_x) transpose_block<int8_t>(p.x, block, lds, nullptr);
}

// Bytes of a row of levels in LDS: whole 64-byte steps, and 16 more so that rows
// begin in different banks (never read).
__host__ __device__ __forceinline__ uint32_t fused_pitch(uint32_t k) { return (k + 63) / 64 * 64 + 16; }

// Few rows of x quantized into LDS by a workgroup of eight waves: a row is taken by
// eight waves, or by fewer where there are more rows, and is held in registers
// between the maximum and the levels (kHeld chunks a thread).
constexpr int kHeld = 4;
__host__ __device__ __forceinline__ uint32_t waves_of_row(uint32_t m) { return m == 1 ? 8 : m == 2 ? 4 : m <= 4 ? 2 : 1; }
// Whether that takes m rows of k.
inline bool holds_rows(uint64_t m, uint64_t k) { return m <= 8 && k <= waves_of_row((uint32_t)m) * 512 * kHeld; }

template <class X>
struct HeldRow {
    Eight<X> v[kHeld];
    uint32_t row, at, step;  // the wave's row; the lane's first column and the next one's distance
};
template <class X>
__device__ __forceinline__ void load_row(const X *x, uint64_t ldx, uint32_t m, uint32_t k, HeldRow<X> &h) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, share = waves_of_row(m);
    h.row = wave / share;
    h.at = wave % share * 512 + lane * 8;
    h.step = share * 512;
    const X *from = x + (uint64_t)min(h.row, m - 1) * ldx;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (h.step * i < k) fetch(from, h.at + h.step * i, k, h.v[i]);
}
// The levels to LDS, the scales to sx; ends with a barrier. `part` holds 8 words.
template <class X>
__device__ __forceinline__ void quantize_to_lds(HeldRow<X> &h, uint32_t m, uint32_t k, uint32_t pitch, int8_t *levels,
                                                float *sx, uint32_t *part) {
    const uint32_t wave = threadIdx.x >> 6, share = waves_of_row(m);
    float y[kHeld][8];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (h.step * i < k) {
            settle(h.at + h.step * i, k, h.v[i], y[i]);
            amax = largest(amax, y[i]);
        }
    amax = wave_max(amax);
    if ((threadIdx.x & 63) == 0) part[wave] = amax;
    __syncthreads();
    for (uint32_t i = 0; i < share; ++i) amax = max(amax, part[wave / share * share + i]);
    const RowScale s = row_scale(amax);
    if (h.row < m) {
        if (h.at == 0) sx[h.row] = s.scale;
        int8_t *out = levels + (uint64_t)h.row * pitch;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const uint32_t c = h.at + h.step * i;
            if (h.step * i < k && c < pitch) put_levels(out, c, pitch, y[i], s);
        }
    }
    __syncthreads();
}

// Copies rows of bytes to a row stride that is a multiple of 16, zeros past the
// row's end, so that the product's tiles can be loaded 16 bytes at a time.
struct RepackParams {
    const int8_t *src;
    int8_t *dst;
    uint64_t lds, ldd;
    uint32_t rows, cols;
};

__device__ __forceinline__ void repack_block(const RepackParams &p, uint64_t block) {
    const uint64_t per_row = p.ldd / 16;
    const uint64_t at = block * 256 + threadIdx.x;
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

static __global__ __launch_bounds__(256) void repack_kernel(RepackParams p) { repack_block(p, block_index()); }

// The layer's rows quantized and its weight copied to aligned rows, in one launch
// (1000 x 777 x 1537 in fp32: 5.2 us; a training step of it 44 us, 46 with two).
template <class T, int TPR, int NV>
__global__ __launch_bounds__(256) void layer_inputs_kernel(QuantizeParams rows, uint64_t n_rows, RepackParams w) {
    __shared__ uint32_t part[4];
    const uint64_t block = block_index();
    if (block < n_rows) quantize_rows_block<T, TPR, NV>(rows, block, part);
    else repack_block(w, block - n_rows);
}

}  // namespace ops
}  // namespace qsgd
