"""The operators' C ABI on the CPU: exports, workspace sizes and the refusals that
come before anything touches a device."""
import os
import re

import pytest
import torch

import quantized_sgd_amd as q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = q.QSGD_ERR_INVALID_ARG, q.QSGD_ERR_UNSUPPORTED


def test_every_declared_function_is_exported():
    text = open(os.path.join(ROOT, "include", "qsgd_ops.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(qsgd_(?:int8|distill)[a-z0-9_]*)\s*\(", text)))
    assert len(names) >= 8
    for name in names:
        assert hasattr(q.lib(), name), name


def test_int8_argument_checks():
    from quantized_sgd_amd import int8  # noqa: F401 (its C types are set on use)
    from quantized_sgd_amd._ops import bind as function, u64, vp
    import ctypes
    i = ctypes.c_int
    quant = function("qsgd_int8_quantize", i, vp, i, u64, u64, u64, vp, vp, u64, vp, vp)
    assert quant(16, 0, 0, 8, 8, None, 16, 8, 16, None) == 0             # no rows
    assert quant(16, 3, 4, 8, 8, None, 16, 8, 16, None) == INVALID       # an integer type
    assert quant(16, 0, 4, 8, 7, None, 16, 8, 16, None) == INVALID       # overlapping rows of x
    assert quant(16, 0, 4, 8, 8, None, 16, 7, 16, None) == INVALID       # overlapping rows of levels
    assert quant(None, 0, 4, 8, 8, None, 16, 8, 16, None) == INVALID
    assert quant(16, 0, 4, 8, 8, None, 16, 8, None, None) == INVALID
    assert quant(16, 0, 1 << 31, 8, 8, None, 16, 8, 16, None) == INVALID
    size_t = function("qsgd_int8_quantize_transposed_workspace", u64, u64, u64)
    assert size_t(100, 0) == 0 and size_t(0, 100) >= 400 and size_t(4096, 4096) >= 4 * 4096
    quant_t = function("qsgd_int8_quantize_transposed", i, vp, i, u64, u64, u64, vp, vp, u64, vp, vp, vp)
    assert quant_t(16, 0, 8, 0, 8, None, 16, 8, 16, None, None) == 0     # no columns
    assert quant_t(16, 0, 8, 4, 4, None, 16, 8, 16, None, None) == INVALID   # no workspace
    assert quant_t(16, 0, 8, 4, 4, None, 16, 8, 16, 8, None) == INVALID      # misaligned workspace
    assert quant_t(16, 0, 8, 4, 4, None, 16, 7, 16, 16, None) == INVALID
    mm = function("qsgd_int8_matmul", i, vp, u64, vp, vp, u64, vp, vp, vp, i, u64, u64, u64, u64, vp, vp)
    assert mm(16, 8, 16, 16, 8, None, None, 16, 0, 5, 0, 5, 8, None, None) == 0
    assert mm(16, 8, 16, 16, 8, None, None, 16, 0, 5, 4, 5, 9, None, None) == INVALID   # rows shorter than k
    assert mm(16, 8, 16, 16, 8, None, None, 16, 0, 4, 4, 5, 8, None, None) == INVALID   # rows of y shorter than n
    assert mm(16, 8, None, 16, 8, None, None, 16, 0, 5, 4, 5, 8, None, None) == INVALID
    assert mm(16, 8, 16, 16, 8, None, None, 16, 4, 5, 4, 5, 8, None, None) == INVALID   # y of integers
    big = (1 << 23) + 16
    assert mm(16, big, 16, 16, big, None, None, 16, 0, 5, 4, 5, big, None, None) == UNSUPPORTED
    assert mm(16, 33, 16, 16, 33, None, None, 16, 0, 500, 400, 500, 33, None, None) == INVALID  # odd rows, no workspace
    size = function("qsgd_int8_matmul_workspace", u64, vp, u64, vp, u64, u64, u64, u64)
    assert size(16, 4096, 16, 4096, 8192, 8192, 4096) == 0
    assert size(16, 4096, 17, 4096, 8192, 8192, 4096) >= 8192 * 4096       # b is copied to aligned rows
    assert size(16, 65536, 16, 65536, 64, 64, 65536) >= 2 * 64 * 64 * 4    # the sum is split
    lin = function("qsgd_int8_linear", i, vp, i, u64, vp, u64, vp, vp, vp, u64, vp, u64, vp, u64, u64, u64, vp, vp)
    assert lin(16, 0, 8, 16, 8, 16, None, 16, 5, None, 0, None, 0, 5, 8, None, None) == 0
    assert lin(16, 0, 8, 16, 8, 16, None, 16, 5, None, 0, None, 40, 5, 8, None, None) == INVALID  # no workspace
    assert lin(16, 0, 8, 16, 8, 16, None, 16, 5, 16, 16, None, 4, 5, 8, None, None) == INVALID   # xq without sx
    assert lin(16, 0, 8, 16, 8, 16, None, 16, 5, 16, 8, 16, 4, 5, 8, None, None) == INVALID      # rows of xq not padded
    assert lin(16, 0, 8, 16, 8, 16, None, 16, 5, 24, 16, 16, 4, 5, 8, None, None) == INVALID     # xq not aligned
    back = function("qsgd_int8_linear_backward", i, vp, i, u64, vp, u64, vp, vp, u64, vp, vp, u64, vp, u64, u64, u64, u64,
                    vp, vp)
    assert back(16, 0, 5, 16, 8, 16, 16, 8, 16, None, 8, None, 8, 4, 5, 8, 16, None) == 0        # neither is wanted
    assert back(16, 0, 5, 16, 8, 16, 16, 8, 16, 16, 8, 16, 8, 4, 5, 8, None, None) == INVALID    # no workspace
    assert back(16, 0, 4, 16, 8, 16, 16, 8, 16, 16, 8, 16, 8, 4, 5, 8, 16, None) == INVALID
    assert back(16, 0, 5, 16, 8, 16, 16, 8, 16, 16, 7, 16, 8, 4, 5, 8, 16, None) == INVALID


def test_workspaces_of_empty_sizes():
    from quantized_sgd_amd._ops import bind as function, u64, vp
    import ctypes
    back = function("qsgd_int8_linear_backward_workspace", u64, u64, u64, u64)
    linear = function("qsgd_int8_linear_workspace", u64, vp, u64, u64, u64, u64, ctypes.c_int)
    matmul = function("qsgd_int8_matmul_workspace", u64, vp, u64, vp, u64, u64, u64, u64)
    columns = function("qsgd_int8_quantize_transposed_workspace", u64, u64, u64)
    distill = function("qsgd_distill_workspace", u64, u64, u64, ctypes.c_int)
    sizes = (0, 1, 40, 5000)
    for m in sizes:
        for n in sizes:
            assert columns(m, n) >= 0 and distill(m, n, 0) >= 0
            for k in sizes:
                for keep in (0, 1):
                    assert linear(16, max(k, 1), m, n, k, keep) >= 0
                assert back(m, n, k) >= 0 and matmul(16, max(k, 1), 16, max(k, 1), m, n, k) >= 0


def test_bindings_refuse_host_tensors():
    with pytest.raises(ValueError):
        q.int8_quantize(torch.zeros(2, 3))
    with pytest.raises(ValueError):
        q.int8_matmul(torch.zeros(2, 3, dtype=torch.int8), torch.ones(2), torch.zeros(4, 3, dtype=torch.int8))


def test_distill_argument_checks():
    import ctypes

    from quantized_sgd_amd._ops import bind as function, u64, vp
    from quantized_sgd_amd.distill import _Teacher, _teacher_p
    i = ctypes.c_int
    step = function("qsgd_distill_step", i, vp, i, u64, u64, u64, _teacher_p, vp, vp, vp, u64, vp, vp)

    def call(te, dtype=0, rows=300, ldz=100, z=16, loss=16, dz=16, lddz=100, vocab=100):
        return step(z, dtype, rows, vocab, ldz, te, None, loss, dz, lddz, None, None)

    def teacher(idx=16, t=16, itype=3, ttype=0, ldi=5, ldt=5, k=5, tau=1.0):
        return _Teacher(idx, t, itype, ttype, ldi, ldt, k, tau, None)

    assert call(teacher(), rows=0) == 0
    for te in (None, teacher(itype=0), teacher(ttype=3), teacher(ldi=4), teacher(ldt=4), teacher(k=1025, ldi=1025, ldt=1025),
               teacher(tau=0.0), teacher(tau=float("nan")), teacher(tau=float("inf")), teacher(idx=None), teacher(t=None)):
        assert call(te) == INVALID
    te = teacher()
    assert call(te, dtype=4) == INVALID and call(te, ldz=99) == INVALID and call(te, lddz=99) == INVALID
    assert call(te, z=None) == INVALID and call(te, loss=None) == INVALID and call(te, dz=None) == INVALID
    size = function("qsgd_distill_workspace", u64, u64, u64, i)
    assert size(4096, 131072, 0) == 0 and size(0, 131072, 0) == 0 and size(2, 131072, 3) == 0
    assert size(2, 131072, 0) > 0 and size(4096, 300000, 2) > 0          # rows split into segments
    assert call(te, rows=2, vocab=131072, ldz=131072, lddz=131072) == INVALID  # no workspace
    back = function("qsgd_distill_backward", i, vp, i, u64, u64, u64, _teacher_p, vp, vp, vp, u64, vp)
    assert back(16, 0, 3, 100, 100, te, 8, None, 16, 100, None) == INVALID     # misaligned stats
