// Drives the operators' host planning and argument checks (no kernel is launched):
// workspace sizes over awkward sizes, and calls that are refused or have nothing to do.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "qsgd_ops.h"

static void need(bool ok, const char *what) {
    if (!ok) {
        std::printf("failed: %s\n", what);
        std::exit(1);
    }
}

int main() {
    const uint64_t sizes[] = {0, 1, 2, 15, 16, 17, 33, 64, 127, 511, 512, 2048, 2049, 4096, 8193, 131072, 1u << 23, (1u << 23) + 1,
                              (1ull << 31) - 1, 1ull << 31, 1ull << 40, ~0ull};
    const int8_t *const p = (const int8_t *)16, *const odd = (const int8_t *)17;
    uint64_t total = 0;
    for (uint64_t m : sizes)
        for (uint64_t n : sizes) {
            total += qsgd_int8_quantize_transposed_workspace(m, n);
            for (int t = 0; t < 5; ++t) total += qsgd_distill_workspace(m, n, (qsgd_dtype)t);
            for (uint64_t k : sizes) {
                total += qsgd_int8_matmul_workspace(p, k, p, k, m, n, k);
                total += qsgd_int8_matmul_workspace(odd, k + 1, p, k + 16, m, n, k);
                total += qsgd_int8_linear_workspace(p, k, m, n, k, 0) + qsgd_int8_linear_workspace(odd, k, m, n, k, 1);
                total += qsgd_int8_linear_backward_workspace(m, n, k);
            }
        }
    need(total > 0, "sizes");
    need(qsgd_int8_matmul_workspace(p, 4096, p, 4096, 8192, 8192, 4096) == 0, "aligned products need no workspace");
    qsgd_teacher te{p, p, QSGD_I32, QSGD_F32, 4, 4, 4, 1.0f, nullptr};
    float *const f = (float *)16;
    need(qsgd_distill_forward(p, QSGD_F32, 0, 10, 10, &te, f, f, nullptr, nullptr) == QSGD_OK, "no rows");
    need(qsgd_distill_forward(p, QSGD_F32, 4, 10, 9, &te, f, f, nullptr, nullptr) == QSGD_ERR_INVALID_ARG, "stride");
    need(qsgd_distill_forward(p, QSGD_F32, 4, 10, 10, nullptr, f, f, nullptr, nullptr) == QSGD_ERR_INVALID_ARG, "no teacher");
    need(qsgd_distill_backward(p, QSGD_F32, 4, 10, 10, &te, f, f, f, 9, nullptr) == QSGD_ERR_INVALID_ARG, "gradient stride");
    te.tau = -1.0f;
    need(qsgd_distill_step(p, QSGD_F32, 4, 10, 10, &te, f, f, f, 10, nullptr, nullptr) == QSGD_ERR_INVALID_ARG, "tau");
    need(qsgd_int8_quantize(p, QSGD_I64, 4, 4, 4, nullptr, (int8_t *)16, 4, f, nullptr) == QSGD_ERR_INVALID_ARG, "type");
    need(qsgd_int8_matmul(p, 8, f, p, 8, f, f, f, QSGD_F32, 8, 8, 8, (1u << 23) + 1, nullptr, nullptr) == QSGD_ERR_INVALID_ARG, "short rows");
    need(qsgd_int8_linear_backward(p, QSGD_F32, 8, p, 8, f, p, 8, f, nullptr, 8, nullptr, 8, 8, 8, 8, nullptr, nullptr) == QSGD_OK,
         "nothing asked");
    std::printf("ok\n");
    return 0;
}
