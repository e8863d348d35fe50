"""Plain 64-bit forms of the operators around the convolution, for the tests.

Tolerances are derived, not tuned.  A result rounded to type T is off by at
most half a step, ``HALF[T]`` relative to its value.  What the kernels compute
in fp32 is off by at most n 2^-24 relative to the sum of the magnitudes that
enter, n the longest chain of dependent fp32 operations: a row statistic is at
most 24 sequential terms, 10 levels of shuffles and a handful of operations a
value, below 2^7 in all, so FP32_ROW = 2^-17; a bf16 result's sigmoid adds
2^-20 relative (hardware exp and reciprocal, 2 ulp each) to that, FP32_ROW_BF16
= 2^-16 covers both.
"""
import torch

HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
ROW = {"bf16": 2.0 ** -16, "fp32": 2.0 ** -17}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def act(u, kind):
    if kind == "silu":
        return u * torch.sigmoid(u)
    if kind == "gelu":
        return 0.5 * u * (1 + torch.tanh(0.7978845608028654 * (u + 0.044715 * u ** 3)))
    return u


def norm(v, kind, w, bias, eps):
    """(norm, normalised rows, rstd, magnitude that bounds the fp32 error)."""
    if kind == "none":
        return v, v, torch.ones_like(v[:, :1]), v.abs()
    mu = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    rstd = ((v - mu).pow(2).mean(1, keepdim=True) + eps).rsqrt()
    n = (v - mu) * rstd
    out = n * w if w is not None else n
    mag = (n.abs() + v.abs().amax(1, keepdim=True) * rstd) * (w.abs() if w is not None else 1)
    if bias is not None:
        out, mag = out + bias, mag + bias.abs()
    return out, n, rstd, mag


def d(t):
    return None if t is None else t.double()


def close(got, want, tol, what):
    """|got - want| <= tol everywhere; NaN where and only where it is wanted."""
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(got.isnan(), want.isnan()), what
    err = (got - want).abs().nan_to_num(0.0, 0.0, 0.0)
    bad = err > tol
    if bad.any():
        i = int((err - tol).flatten().argmax())
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: got "
            f"{got.flatten()[i].item()!r} want {want.flatten()[i].item()!r} tol "
            f"{tol.expand_as(err).flatten()[i].item()!r}")


def guarded(shape, dtype, fill=7.0, pad=64):
    """A tensor inside a larger buffer, and a check that the rest was left alone."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    t = buf[pad:pad + n].view(shape)

    def untouched():
        assert (buf[:pad] == fill).all() and (buf[pad + n:] == fill).all()

    return t, untouched
