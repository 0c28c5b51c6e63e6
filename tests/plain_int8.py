"""The 8-bit linear layer's definitions on the CPU, one rounding at a time: the
quantizer in IEEE binary32 steps, sums of products exactly (integers in binary64
below 2^53)."""
import numpy as np
import torch

F32 = np.float32


def to32(x: torch.Tensor) -> np.ndarray:
    return x.detach().cpu().float().numpy()


def quantize_rows(x, fold=None):
    """Levels (int8) and scales of each row of a float32 array."""
    x = np.asarray(x, F32)
    with np.errstate(all="ignore"):
        y = x if fold is None else (x * np.asarray(fold, F32)).astype(F32)
        amax = np.abs(y).max(axis=1) if y.shape[1] else np.zeros(y.shape[0], F32)
        scale = (amax.astype(F32) / F32(127)).astype(F32)
        ok = (scale > 0) & np.isfinite(scale)
        r = np.rint((y / scale[:, None]).astype(F32))
        q = np.where(ok[:, None], np.clip(np.where(np.isnan(r), 0, r), -127, 127), 0)
    return q.astype(np.int8), scale


def quantize_columns(x, fold=None):
    """Levels [C, R] and scales of each column."""
    return quantize_rows(np.ascontiguousarray(np.asarray(x, F32).T), fold)


def product(a, sa, b, sb=None, bias=None):
    """float32 result of the documented sequence of roundings."""
    acc = a.astype(np.float64) @ b.astype(np.float64).T  # integers below 2^53: exact
    with np.errstate(all="ignore"):
        v = (acc.astype(F32) * np.asarray(sa, F32)[:, None]).astype(F32)
        if sb is not None:
            v = (v * np.asarray(sb, F32)).astype(F32)
        if bias is not None:
            v = (v + np.asarray(bias, F32)).astype(F32)
    return v


def cast(v, dtype):
    return torch.from_numpy(np.ascontiguousarray(v)).to(dtype)


def same(got: torch.Tensor, want: torch.Tensor) -> bool:
    """Equal, NaN in the same places."""
    got, want = got.detach().cpu(), want.cpu()
    return got.shape == want.shape and got.dtype == want.dtype and bool(((got == want) | (got.isnan() & want.isnan())).all())
