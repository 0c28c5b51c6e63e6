// Distillation from a teacher's top logits: loss of each row, gradient with
// respect to the student's logits. Formulas in include/qsgd_ops.h.
//
// Bound by memory: the logits are read once for the loss, and once more and
// written for the gradient. The softmax's maximum and sum are taken in one pass
// (a thread keeps a running maximum and the sum relative to it). With a teacher
// remainder the running pair covers the logits outside the entries only: taking
// the entries out of a sum over everything would cancel where the student is
// sure of them. They are told apart by a bit for each logit in LDS, read as a
// byte for a thread's eight logits.
//
// In the gradient all logits outside the entries share one factor,
//   dz_j = g / tau e_j (exp(m_r - m) / S - p_r / S_r),   e_j = exp(z_j / tau - m_r),
// with m, S the maximum and sum over all logits and m_r, S_r those outside the
// entries (without a remainder p_r = 0 and m_r = m), so an element costs one
// exponential; the entries are written after it.
#pragma once

#include "ops_common.h"

namespace qsgd {
namespace ops {

constexpr int kMaxEntries = 1024;
constexpr uint32_t kMaxSegment = 1u << 18;  // logits of a workgroup: 32 KB of bits
constexpr int kDT = 512;                    // threads of a workgroup
constexpr int kDW = kDT / 64;

struct DistillParams {
    const void *z, *idx, *t;
    const float *teacher_lse, *grad;
    float *loss, *stats;
    const float *stats_in;
    float2 *part;  // [rows, segments]: maximum and sum of a segment
    void *dz;
    uint64_t ldz, ldi, ldt, lddz;
    uint32_t rows, vocab, k;
    uint32_t segments, segment;  // logits a segment
    uint32_t itype, ttype;
    float inv_tau;
};

// A maximum and a sum of exponentials relative to it. A pair of nothing (or of
// minus infinities) is (-inf, 0); NaN and plus infinity make the sum NaN.
struct Pair {
    float m, s;
};

// Subtractions are relative to this, so that -inf - -inf does not arise.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }

constexpr float kLog2e = 1.44269504088896340736f;
// exp((z - m) / tau), with c = log2(e) / tau
__device__ __forceinline__ float exp_scaled(float z, float base, float c) {
    return __builtin_amdgcn_exp2f((z - base) * c);
}

__device__ __forceinline__ Pair join(Pair a, Pair b, float c) {
    const float m = fmaxf(a.m, b.m), base = base_of(m);
    return {m, a.s * exp_scaled(a.m, base, c) + b.s * exp_scaled(b.m, base, c)};
}

template <class F>
__device__ __forceinline__ float block_reduce(float v, float none, float *lds, F f) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = f(v, __shfl_xor(v, o));
    __syncthreads();  // lds may still be read from the last call
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = none;
    const int waves = blockDim.x >> 6;
    for (int w = 0; w < waves; ++w) v = f(v, lds[w]);
    return v;
}
__device__ __forceinline__ float block_sum(float v, float *lds) {
    return block_reduce(v, 0.0f, lds, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float block_max(float v, float *lds) {
    return block_reduce(v, -INFINITY, lds, [](float a, float b) { return fmaxf(a, b); });
}

__device__ __forceinline__ Pair block_join(Pair v, float c, float *lds) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = join(v, Pair{__shfl_xor(v.m, o), __shfl_xor(v.s, o)}, c);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        lds[threadIdx.x >> 5] = v.m;
        lds[(threadIdx.x >> 5) + 1] = v.s;
    }
    __syncthreads();
    v = {-INFINITY, 0.0f};
    const int waves = blockDim.x >> 6;
    for (int w = 0; w < waves; ++w) v = join(v, Pair{lds[2 * w], lds[2 * w + 1]}, c);
    return v;
}

__device__ __forceinline__ int64_t read_index(const void *p, uint32_t type, uint64_t at) {
    return type == QSGD_I64 ? ((const int64_t *)p)[at] : ((const int32_t *)p)[at];
}
__device__ __forceinline__ float read_logit(const void *p, uint32_t type, uint64_t at) {
    return type == QSGD_F32 ? ((const float *)p)[at]
                            : type == QSGD_F16 ? (float)((const f16 *)p)[at] : (float)((const bf16 *)p)[at];
}

// A row's entries in LDS, and what the teacher says of them.
struct Entries {
    int at[kMaxEntries];    // index in the vocabulary, -1: no entry
    float z[kMaxEntries];   // student's logit
    float p[kMaxEntries];   // teacher's probability
    float red[2 * 16];
};

struct TeacherSums {
    bool some;      // the row has an entry
    float shift;    // log p = t / tau - shift
    float rest;     // p_r
};

// Reads a row's entries (by the whole workgroup; ends with a barrier).
template <class T>
__device__ __forceinline__ TeacherSums read_entries(const DistillParams &p, uint32_t row, Entries &e) {
    const T *z = (const T *)p.z + (uint64_t)row * p.ldz;
    float top = -INFINITY, some = 0.0f;
    for (uint32_t i = threadIdx.x; i < p.k; i += blockDim.x) {
        const int64_t at = read_index(p.idx, p.itype, (uint64_t)row * p.ldi + i);
        const bool there = at >= 0 && at < (int64_t)p.vocab;
        e.at[i] = there ? (int)at : -1;
        e.z[i] = there ? (float)z[at] : -INFINITY;
        const float x = there ? read_logit(p.t, p.ttype, (uint64_t)row * p.ldt + i) * p.inv_tau : -INFINITY;
        e.p[i] = x;
        top = fmaxf(top, x);
        some = there ? 1.0f : some;
    }
    TeacherSums s;
    s.some = block_max(some, e.red) > 0.0f;
    float sum = 0.0f;
    if (p.teacher_lse) {
        s.shift = p.teacher_lse[row];
        for (uint32_t i = threadIdx.x; i < p.k; i += blockDim.x) {
            const float v = e.at[i] >= 0 ? expf(e.p[i] - s.shift) : 0.0f;
            e.p[i] = v;
            sum += v;
        }
        sum = block_sum(sum, e.red);
        s.rest = sum >= 1.0f ? 0.0f : 1.0f - sum;  // NaN stays
    } else {
        top = base_of(block_max(top, e.red));
        for (uint32_t i = threadIdx.x; i < p.k; i += blockDim.x) {
            const float v = e.at[i] >= 0 ? expf(e.p[i] - top) : 0.0f;
            e.p[i] = v;
            sum += v;
        }
        sum = block_sum(sum, e.red);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        for (uint32_t i = threadIdx.x; i < p.k; i += blockDim.x) e.p[i] *= inv;
        s.shift = top + logf(sum);
        s.rest = 0.0f;
    }
    __syncthreads();
    return s;
}

// The bits of the entries inside a segment [lo, lo + n); ends with a barrier.
__device__ __forceinline__ void mark_entries(const Entries &e, uint32_t k, uint32_t lo, uint32_t n, uint32_t *bits) {
    for (uint32_t i = threadIdx.x; i < (n + 31) / 32; i += blockDim.x) bits[i] = 0;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < k; i += blockDim.x) {
        const uint32_t at = (uint32_t)e.at[i] - lo;  // -1 is past every segment
        if (e.at[i] >= 0 && at < n) atomicOr(&bits[at / 32], 1u << (at % 32));
    }
    __syncthreads();
}

// Eight logits (`there` of them; the others are -inf) into a running pair.
__device__ __forceinline__ void take8(Pair &v, const float (&z)[8], float c) {
    float m = v.m;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, z[i]);
    const float base = base_of(m);
    float s = v.s * exp_scaled(v.m, base, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += exp_scaled(z[i], base, c);
    v = {m, s};
}

// The pair of a segment of a row, by one thread's share.
template <class T>
__device__ __forceinline__ Pair scan_segment(const T *z, uint32_t n, const uint32_t *bits, float c) {
    Pair v = {-INFINITY, 0.0f};
    const uint32_t step = blockDim.x * 8;
    for (uint32_t i = threadIdx.x * 8; i < n; i += step) {
        float x[8];
        load_upto8(z + i, (int64_t)n - i, -INFINITY, x);
        if (bits) {
            const uint32_t b = bits[i / 32] >> (i % 32) & 255u;
            if (b) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = b >> j & 1 ? -INFINITY : x[j];
            }
        }
        take8(v, x, c);
    }
    return v;
}

// Loss and statistics of a row from the pair outside the entries (with a
// remainder) or over everything. Every thread returns the statistics.
struct Stats {
    float m, inv, m_rest, inv_rest;
};

__device__ __forceinline__ float inverse(float s) { return s == 0.0f ? 0.0f : 1.0f / s; }

__device__ __forceinline__ Stats finish_row(const DistillParams &p, uint32_t row, const TeacherSums &ts, Pair scanned,
                                            Entries &e) {
    const float c = kLog2e * p.inv_tau;
    Pair all = scanned;
    if (p.teacher_lse) {
        Pair top = {-INFINITY, 0.0f};
        for (uint32_t i = threadIdx.x; i < p.k; i += blockDim.x) top = join(top, Pair{e.z[i], e.at[i] >= 0 ? 1.0f : 0.0f}, c);
        all = join(all, block_join(top, c, e.red), c);
    }
    const float log_sum = logf(all.s), base = base_of(all.m);
    float loss = 0.0f;
    for (uint32_t i = threadIdx.x; i < p.k; i += blockDim.x) {
        const float pi = e.p[i];
        if (e.at[i] < 0 || pi == 0.0f) continue;
        const float log_p = read_logit(p.t, p.ttype, (uint64_t)row * p.ldt + i) * p.inv_tau - ts.shift;
        const float log_q = all.s == 0.0f ? -INFINITY : (e.z[i] - base) * p.inv_tau - log_sum;
        loss += pi * (log_p - log_q);
    }
    loss = block_sum(loss, e.red);
    if (p.teacher_lse && ts.rest != 0.0f && scanned.s != 0.0f)
        loss += ts.rest * (logf(ts.rest) - ((base_of(scanned.m) - base) * p.inv_tau + logf(scanned.s) - log_sum));
    if (threadIdx.x == 0 && p.loss) p.loss[row] = ts.some ? loss : 0.0f;
    return {all.m, inverse(all.s), scanned.m, inverse(scanned.s)};
}

// The gradient of a segment.
template <class T>
__device__ __forceinline__ void write_gradient(const DistillParams &p, uint32_t row, uint32_t lo, uint32_t n,
                                               const TeacherSums &ts, const Stats &st, Entries &e) {
    const float c = kLog2e * p.inv_tau;
    const T *z = (const T *)p.z + (uint64_t)row * p.ldz + lo;
    T *dz = (T *)p.dz + (uint64_t)row * p.lddz + lo;
    const float g = p.grad ? p.grad[row] * p.inv_tau : p.inv_tau;
    const uint32_t step = blockDim.x * 8;
    if (!ts.some || g == 0.0f) {
        const float none[8] = {};
        for (uint32_t i = threadIdx.x * 8; i < n; i += step) {
            if (i + 8 <= n) store8(dz + i, none);
            else
                for (uint32_t j = i; j < n; ++j) dz[j] = (T)0.0f;
        }
        return;
    }
    const float base = base_of(st.m_rest), all = base_of(st.m);
    float factor = st.inv * exp_scaled(base, all, c);
    if (st.m_rest == -INFINITY) factor = st.inv != st.inv ? st.inv : 0.0f;
    factor = g * (factor - ts.rest * st.inv_rest);
    for (uint32_t i = threadIdx.x * 8; i < n; i += step) {
        float x[8];
        load_upto8(z + i, (int64_t)n - i, -INFINITY, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = factor * exp_scaled(x[j], base, c);
        if (i + 8 <= n) store8(dz + i, x);
        else
            for (uint32_t j = i; j < n; ++j) dz[j] = (T)x[j - i];
    }
    // The entries' gradients replace what the loop left there, once it is written.
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < p.k; i += blockDim.x) {
        const uint32_t at = (uint32_t)e.at[i] - lo;
        if (e.at[i] >= 0 && at < n) dz[at] = (T)(g * (exp_scaled(e.z[i], all, c) * st.inv - e.p[i]));
    }
}

// One workgroup a row: loss and statistics, and with GRAD the gradient.
template <class T, bool GRAD>
__global__ __launch_bounds__(kDT) void distill_row_kernel(DistillParams p) {
    __shared__ Entries e;
    __shared__ uint32_t bits[kMaxSegment / 32];
    const uint64_t block = block_index();
    if (block >= p.rows) return;
    const uint32_t row = (uint32_t)block;
    const float c = kLog2e * p.inv_tau;
    const TeacherSums ts = read_entries<T>(p, row, e);
    if (p.teacher_lse) mark_entries(e, p.k, 0, p.vocab, bits);
    const T *z = (const T *)p.z + (uint64_t)row * p.ldz;
    const Pair v = block_join(scan_segment(z, p.vocab, p.teacher_lse ? bits : nullptr, c), c, e.red);
    const Stats st = finish_row(p, row, ts, v, e);
    if (p.stats && threadIdx.x == 0) ((float4 *)p.stats)[row] = make_float4(st.m, st.inv, st.m_rest, st.inv_rest);
    if (GRAD) write_gradient<T>(p, row, 0, p.vocab, ts, st, e);
}

// A row's segment: its pair.
template <class T>
__global__ __launch_bounds__(kDT) void distill_part_kernel(DistillParams p) {
    __shared__ Entries e;
    __shared__ uint32_t bits[kMaxSegment / 32];
    const uint64_t block = block_index();
    if (block >= (uint64_t)p.rows * p.segments) return;
    const uint32_t row = (uint32_t)(block / p.segments), seg = (uint32_t)(block % p.segments);
    const uint32_t lo = seg * p.segment, n = min(p.segment, p.vocab - lo);
    const float c = kLog2e * p.inv_tau;
    if (p.teacher_lse) {
        for (uint32_t i = threadIdx.x; i < p.k; i += blockDim.x) {
            const int64_t at = read_index(p.idx, p.itype, (uint64_t)row * p.ldi + i);
            e.at[i] = at >= 0 && at < (int64_t)p.vocab ? (int)at : -1;
        }
        mark_entries(e, p.k, lo, n, bits);  // a thread reads back its own entries
    }
    const T *z = (const T *)p.z + (uint64_t)row * p.ldz + lo;
    const Pair v = block_join(scan_segment(z, n, p.teacher_lse ? bits : nullptr, c), c, e.red);
    if (threadIdx.x == 0) p.part[block] = make_float2(v.m, v.s);
}

// Joins a row's segments.
template <class T>
__global__ __launch_bounds__(256) void distill_join_kernel(DistillParams p) {
    __shared__ Entries e;
    const uint64_t block = block_index();
    if (block >= p.rows) return;
    const uint32_t row = (uint32_t)block;
    const float c = kLog2e * p.inv_tau;
    const TeacherSums ts = read_entries<T>(p, row, e);
    Pair v = {-INFINITY, 0.0f};
    for (uint32_t i = threadIdx.x; i < p.segments; i += blockDim.x) {
        const float2 q = p.part[(uint64_t)row * p.segments + i];
        v = join(v, Pair{q.x, q.y}, c);
    }
    v = block_join(v, c, e.red);
    const Stats st = finish_row(p, row, ts, v, e);
    if (threadIdx.x == 0) ((float4 *)p.stats)[row] = make_float4(st.m, st.inv, st.m_rest, st.inv_rest);
}

// The gradient of a row's segment from its statistics.
template <class T>
__global__ __launch_bounds__(kDT) void distill_gradient_kernel(DistillParams p) {
    __shared__ Entries e;
    const uint64_t block = block_index();
    if (block >= (uint64_t)p.rows * p.segments) return;
    const uint32_t row = (uint32_t)(block / p.segments), seg = (uint32_t)(block % p.segments);
    const uint32_t lo = seg * p.segment, n = min(p.segment, p.vocab - lo);
    const TeacherSums ts = read_entries<T>(p, row, e);
    const float4 s = ((const float4 *)p.stats_in)[row];
    write_gradient<T>(p, row, lo, n, ts, Stats{s.x, s.y, s.z, s.w}, e);
}

}  // namespace ops
}  // namespace qsgd
