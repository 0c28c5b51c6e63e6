// The product of 8-bit matrices, y = (a b^T) with a scale for each row of a and of
// b, a bias and a rounding to y's type in the epilogue. Formula in
// include/qsgd_ops.h.
//
// Two kernels:
//  - matmul_kernel: tiles of y on the matrix units (v_mfma_i32_16x16x64_i8),
//    bound by their rate for large sizes;
//  - skinny_kernel: few rows of a (single tokens), bound by reading b once.
#pragma once

#include "ops_common.h"

namespace qsgd {
namespace ops {

struct MatmulParams {
    const int8_t *a, *b;
    const float *sa, *sb, *bias;
    void *y;
    int32_t *part;  // [splits, m, n] where the sum is split
    uint64_t lda, ldb, ldy;
    uint32_t m, n, k;
    uint32_t tiles_m, tiles_n;
    uint32_t splits, steps_per_split;  // 64-byte steps of k
};

// Sixteen zero bytes that tile loads past the end of k are pointed at.
static __device__ __align__(16) const uint32_t kZeros[4] = {0, 0, 0, 0};

// The epilogue, one rounding at a time.
__device__ __forceinline__ float finish(float acc, float sa, const float *sb, const float *bias, uint32_t col) {
    float v = acc * sa;
    if (sb) v *= sb[col];
    if (bias) v += bias[col];
    return v;
}

// 16 bytes a lane from global memory straight into LDS: lane i's bytes land at
// `lds` + 16 i. Written as assembly so that the wait for them can be placed by
// hand: the compiler would wait for all of them before the next read of LDS. They
// have no output register; the wait is wait_tiles(). Nothing else in these kernels
// sets m0.
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t offset, const int8_t *base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(lds), "v"(offset), "s"(base) : "memory");
}
__device__ __forceinline__ void load_to_lds(uint32_t lds, const int8_t *from) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :: "s"(lds), "v"(from) : "memory");
}

// Tiles of BM rows of a and BN rows of b. A step is 64 bytes of k. LDS holds a
// ring of S steps, each BM + BN rows of 64 bytes, loaded straight from memory S - 1
// steps ahead. A row's four 16-byte chunks are stored in the order chunk ^ (row /
// 4 % 4), so that the 16 rows that a fragment read takes at one chunk lie in
// different banks.
//
// b is the first operand of the matrix instruction (its rows become the
// accumulator's four consecutive elements) and the rows of b are dealt to LDS so
// that a lane's TN fragments hold 4 TN consecutive columns of y: the epilogue
// writes 16 bytes or more a lane.
template <int WM_, int WN_, int TM_, int TN_, int S_>
struct Tile {
    static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, S = S_;
    static constexpr int BM = WM * TM * 16, BN = WN * TN * 16;
    static constexpr int NW = WM * WN;
    static constexpr int LA = BM / 16 / NW, LB = BN / 16 / NW;  // loads a wave and step
    static constexpr int kStage = (BM + BN) * 64;
    static constexpr int kLds = S * kStage;
    static_assert(LA * 16 * NW == BM && LB * 16 * NW == BN && kLds <= 160 * 1024, "");
};

template <int N>
__device__ __forceinline__ void wait_tiles() {
    // all but the N newest loads have landed, and this wave's reads of LDS are done
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "i"(N) : "memory");
}

template <class C, class OUT>
__global__ __launch_bounds__(C::NW * 64, 1) void matmul_kernel(MatmulParams p) {
    __shared__ __align__(1024) int8_t ring[C::kLds];
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t wm = wave / C::WN, wn = wave % C::WN;

    // Workgroups go round the 8 XCDs in turn; each XCD takes a contiguous run of
    // tiles, in bands of 8 tile rows, so that the tiles an XCD works on together
    // share their rows of a and b in its L2.
    const uint32_t tiles = p.tiles_m * p.tiles_n;
    const uint32_t xcd = blockIdx.x % 8, nth = blockIdx.x / 8;
    const uint32_t id = xcd * (tiles / 8) + min(xcd, tiles % 8) + nth;
    const uint32_t band = id / (8 * p.tiles_n), in_band = id % (8 * p.tiles_n);
    const uint32_t band_rows = min(8u, p.tiles_m - band * 8);
    const uint32_t bm = (band * 8 + in_band % band_rows) * C::BM, bn = in_band / band_rows * C::BN;

    const uint32_t k0 = blockIdx.y * p.steps_per_split;  // first step
    const uint32_t all = (p.k + 63) / 64;
    const uint32_t steps = min(p.steps_per_split, all - k0);
    const uint32_t full = min(steps, p.k / 64 - min(p.k / 64, k0));  // steps wholly inside k

    // This lane's part of the wave's loads. Rows past the end repeat the last one.
    const int8_t *a = p.a + (uint64_t)bm * p.lda + (uint64_t)k0 * 64;
    const int8_t *b = p.b + (uint64_t)bn * p.ldb + (uint64_t)k0 * 64;
    uint32_t oa[C::LA], ob[C::LB];
    const uint32_t chunk = (lane & 3) ^ ((lane >> 4) & 3);
#pragma unroll
    for (int j = 0; j < C::LA; ++j) {
        const uint32_t r = (wave * C::LA + j) * 16 + (lane >> 2);
        oa[j] = min(r, p.m - 1 - bm) * (uint32_t)p.lda + chunk * 16;
    }
#pragma unroll
    for (int j = 0; j < C::LB; ++j) {
        const uint32_t r = (wave * C::LB + j) * 16 + (lane >> 2);
        const uint32_t w = r / (C::TN * 16), f = r / 16 % C::TN, i = r % 16;
        const uint32_t row = w * (C::TN * 16) + i / 4 * (C::TN * 4) + f * 4 + i % 4;
        ob[j] = min(row, p.n - 1 - bn) * (uint32_t)p.ldb + chunk * 16;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t *)ring;

    const auto fill = [&](uint32_t step, uint32_t slot) {
        const uint32_t to = lds0 + slot * C::kStage;
        if (step < full) {
#pragma unroll
            for (int j = 0; j < C::LA; ++j) load_to_lds(to + (wave * C::LA + j) * 1024, oa[j], a + (uint64_t)step * 64);
#pragma unroll
            for (int j = 0; j < C::LB; ++j)
                load_to_lds(to + C::BM * 64 + (wave * C::LB + j) * 1024, ob[j], b + (uint64_t)step * 64);
        } else {
            // the last step, cut by the end of k, and the ring's steps past it: zeros
            const bool in = step < steps && (uint64_t)(k0 + step) * 64 + chunk * 16 < p.k;
#pragma unroll
            for (int j = 0; j < C::LA; ++j)
                load_to_lds(to + (wave * C::LA + j) * 1024, in ? a + (uint64_t)step * 64 + oa[j] : (const int8_t *)kZeros);
#pragma unroll
            for (int j = 0; j < C::LB; ++j)
                load_to_lds(to + C::BM * 64 + (wave * C::LB + j) * 1024,
                            in ? b + (uint64_t)step * 64 + ob[j] : (const int8_t *)kZeros);
        }
    };

    v4i acc[C::TN][C::TM];
#pragma unroll
    for (int i = 0; i < C::TN; ++i)
#pragma unroll
        for (int j = 0; j < C::TM; ++j) acc[i][j] = v4i{0, 0, 0, 0};

    v4i fa[2][C::TM], fb[2][C::TN];
    const uint32_t at = (lane & 15) * 64 + (((lane >> 4) ^ (lane >> 2)) & 3) * 16;
    const auto read = [&](uint32_t slot, v4i (&xa)[C::TM], v4i (&xb)[C::TN]) {
        const int8_t *s = ring + slot * C::kStage + at;
#pragma unroll
        for (int i = 0; i < C::TN; ++i) xb[i] = *(const v4i *)(s + C::BM * 64 + (wn * C::TN + i) * 1024);
#pragma unroll
        for (int j = 0; j < C::TM; ++j) xa[j] = *(const v4i *)(s + (wm * C::TM + j) * 1024);
    };
    const auto multiply = [&](const v4i (&xa)[C::TM], const v4i (&xb)[C::TN]) {
#pragma unroll
        for (int j = 0; j < C::TM; ++j)
#pragma unroll
            for (int i = 0; i < C::TN; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(xb[i], xa[j], acc[i][j], 0, 0, 0);
    };

    constexpr int L = C::LA + C::LB;
#pragma unroll
    for (int s = 0; s < C::S; ++s) fill(s, s);
    wait_tiles<(C::S - 1) * L>();
    read(0, fa[0], fb[0]);
    // Step i: its fragments are in registers. Wait until step i + 1 has landed for
    // every wave and every wave has read step i, refill step i's slot, read step
    // i + 1's fragments under step i's products.
    uint32_t slot = 0;
    const auto advance = [&](uint32_t i, int now) {
        wait_tiles<(C::S - 2) * L>();
        fill(i + C::S, slot);
        slot = slot + 1 == C::S ? 0 : slot + 1;
        read(slot, fa[now ^ 1], fb[now ^ 1]);
        multiply(fa[now], fb[now]);
    };
    uint32_t i = 0;
    for (; i + 2 <= steps; i += 2) {
        advance(i, 0);
        advance(i + 1, 1);
    }
    if (i < steps) multiply(fa[0], fb[0]);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may land after the workgroup's end

    const uint32_t m0 = bm + wm * C::TM * 16 + (lane & 15);
    const uint32_t n0 = bn + wn * C::TN * 16 + (lane >> 4) * (C::TN * 4);
    if (n0 >= p.n) return;
    const uint32_t there = min((uint32_t)(C::TN * 4), p.n - n0);
#pragma unroll
    for (int j = 0; j < C::TM; ++j) {
        const uint32_t m = m0 + j * 16;
        if (m >= p.m) continue;
        if (sizeof(OUT) == 4 && p.part) {
            int32_t *out = p.part + ((uint64_t)blockIdx.y * p.m + m) * p.n + n0;
#pragma unroll
            for (int c = 0; c < C::TN; ++c) {
                if (4 * c + 4 <= (int)there) __builtin_memcpy(out + 4 * c, &acc[c][j], 16);
                else
                    for (int e = 0; e < 4; ++e)
                        if (4 * c + e < (int)there) out[4 * c + e] = acc[c][j][e];
            }
            continue;
        }
        const float sa = p.sa[m];
        OUT *out = (OUT *)p.y + (uint64_t)m * p.ldy + n0;
#pragma unroll
        for (int c = 0; c < C::TN; ++c) {
            if (4 * c + 4 <= (int)there) {
                OUT v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = (OUT)finish((float)acc[c][j][e], sa, p.sb, p.bias, n0 + 4 * c + e);
                __builtin_memcpy(out + 4 * c, v, sizeof(v));
            } else {
                for (int e = 0; e < 4; ++e)
                    if (4 * c + e < (int)there)
                        out[4 * c + e] = (OUT)finish((float)acc[c][j][e], sa, p.sb, p.bias, n0 + 4 * c + e);
            }
        }
    }
}

// Joins the parts of a split sum: exact in 64 bits, then the epilogue.
template <class OUT>
__global__ __launch_bounds__(256) void join_kernel(MatmulParams p) {
    const uint64_t total = (uint64_t)p.m * p.n;
    const uint64_t at = (block_index() * 256 + threadIdx.x) * 4;
    if (at >= total) return;
    int64_t sum[4] = {0, 0, 0, 0};
    const int left = (int)min((uint64_t)4, total - at);
    for (uint32_t s = 0; s < p.splits; ++s) {
        const int32_t *q = p.part + s * total + at;
        if (left == 4) {
            int32_t v[4];
            __builtin_memcpy(v, q, 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += v[e];
        } else {
            for (int e = 0; e < left; ++e) sum[e] += q[e];
        }
    }
    uint32_t row = (uint32_t)(at / p.n), col = (uint32_t)(at % p.n);
    for (int e = 0; e < left; ++e) {
        ((OUT *)p.y)[(uint64_t)row * p.ldy + col] = (OUT)finish((float)sum[e], p.sa[row], p.sb, p.bias, col);
        if (++col == p.n) { col = 0; ++row; }
    }
}

// Few rows of a: a workgroup of 8 waves takes 16 NT rows of b and all of k, its
// waves every eighth 64-byte step. b goes from memory to registers in the matrix
// instruction's own layout (16 bytes of a row a lane), at any alignment; the rows
// of a, at most 16 MT, come from the caches. The waves' sums meet in LDS.
template <int MT, int NT, class OUT>
__global__ __launch_bounds__(512) void skinny_kernel(MatmulParams p) {
    constexpr int kWaves = 8, kUnroll = 4;
    __shared__ int32_t sums[kWaves][MT * NT][256];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t n0 = blockIdx.x * (16 * NT);
    const uint32_t r = lane & 15, chunk = lane >> 4;
    const int8_t *b[NT], *a[MT];
#pragma unroll
    for (int i = 0; i < NT; ++i) b[i] = p.b + (uint64_t)min(n0 + i * 16 + r, p.n - 1) * p.ldb;
#pragma unroll
    for (int j = 0; j < MT; ++j) a[j] = p.a + (uint64_t)min(j * 16 + r, p.m - 1) * p.lda;
    v4i acc[MT][NT];
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[j][i] = v4i{0, 0, 0, 0};
    const auto get = [&](const int8_t *row, uint64_t at) {
        v4i v = {0, 0, 0, 0};
        if (at + 16 <= p.k) {
            __builtin_memcpy(&v, row + at, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (at + e < p.k) v[e / 4] |= (int)((uint32_t)(uint8_t)row[at + e] << (8 * (e % 4)));
        }
        return v;
    };
    const uint32_t steps = (p.k + 63) / 64, full = p.k / 64;
    uint32_t s = wave;
    for (; s + (kUnroll - 1) * kWaves < full; s += kUnroll * kWaves) {
        v4i fb[kUnroll][NT], fa[kUnroll][MT];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t at = (uint64_t)(s + u * kWaves) * 64 + chunk * 16;
#pragma unroll
            for (int i = 0; i < NT; ++i) __builtin_memcpy(&fb[u][i], b[i] + at, 16);
#pragma unroll
            for (int j = 0; j < MT; ++j) __builtin_memcpy(&fa[u][j], a[j] + at, 16);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[u][i], fa[u][j], acc[j][i], 0, 0, 0);
    }
    for (; s < steps; s += kWaves) {
        const uint64_t at = (uint64_t)s * 64 + chunk * 16;
        v4i fb[NT], fa[MT];
#pragma unroll
        for (int i = 0; i < NT; ++i) fb[i] = get(b[i], at);
#pragma unroll
        for (int j = 0; j < MT; ++j) fa[j] = get(a[j], at);
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int i = 0; i < NT; ++i)
                acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[i], fa[j], acc[j][i], 0, 0, 0);
    }
    // lane: rows of y j * 16 + lane % 16, columns i * 16 + lane / 16 * 4 + e
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i)
            *(v4i *)&sums[wave][j * NT + i][lane * 4] = acc[j][i];
    __syncthreads();
    for (uint32_t at = threadIdx.x; at < MT * NT * 256; at += 512) {
        const uint32_t tile = at / 256, j = tile / NT, i = tile % NT, e = at % 256;
        const uint32_t row = j * 16 + e / 4 % 16, col = n0 + i * 16 + e / 64 * 4 + e % 4;
        if (row >= p.m || col >= p.n) continue;
        int32_t sum = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += sums[w][tile][e];
        ((OUT *)p.y)[(uint64_t)row * p.ldy + col] = (OUT)finish((float)sum, p.sa[row], p.sb, p.bias, col);
    }
}

}  // namespace ops
}  // namespace qsgd
