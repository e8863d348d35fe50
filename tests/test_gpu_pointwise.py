"""ccv3d_pointwise_forward / ccv3d_pointwise_backward (the 1x1x1 convolution)
against matrix products in 64 bits."""
import itertools

import pytest
import torch

from block_util import DT, HALF, act, close, d, guarded
from causal_conv3d_video_b200 import ccv3d

pytestmark = pytest.mark.gpu


def _acc(k):
    """fp32 accumulation of k products: at most one step of 2^-23 each (the
    tensor cores may truncate where FFMA rounds), and the epilogue's few."""
    return (k + 16) * 2.0 ** -23


def _case(M, K, N, dtype, *, actk="none", bias=True, residual=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(s, device="cuda", generator=g) * std).to(DT[dtype])
    s = dict(M=M, K=K, N=N, dtype=dtype, act=actk, rnd=rnd)
    s["x"], s["w"] = rnd(M, K), rnd(N, K, std=K ** -0.5)
    s["bias"] = rnd(N, std=0.5) if bias else None
    s["residual"] = rnd(M, N) if residual else None
    s["desc"] = ccv3d.make_pointwise_desc(pixels=M, Cin=K, Cout=N, act=actk, dtype=dtype)
    return s


def _ws(s, backward=False):
    n = ccv3d.ccv3d_pointwise_workspace(s["desc"])[1 if backward else 0]
    return guarded((n,), torch.uint8, fill=9) if n else (None, lambda: None)


def _forward(s, pre=False, stream=None, out=None):
    ok_o = lambda: None
    if out is None:
        out, ok_o = guarded((s["M"], s["N"]), DT[s["dtype"]])
    p, ok_p = guarded((s["M"], s["N"]), DT[s["dtype"]]) if pre else (None, lambda: None)
    ws, ok_w = _ws(s)
    ccv3d.ccv3d_pointwise_forward(s["desc"], s["x"], s["w"], s["bias"], s["residual"], out, p, ws,
                                  stream)
    torch.cuda.synchronize()
    for ok in (ok_o, ok_p, ok_w):
        ok()
    return out, p


def _check_forward(s, pre=False):
    out, p = _forward(s, pre)
    half = HALF[s["dtype"]]
    u = d(s["x"]) @ d(s["w"]).t()
    mag = d(s["x"]).abs() @ d(s["w"]).abs().t()
    if s["bias"] is not None:
        u, mag = u + d(s["bias"]), mag + d(s["bias"]).abs()
    e = _acc(s["K"]) * mag
    if pre:
        close(p, u, half * u.abs() + e, "pre")
    want = act(u, s["act"])
    # |act'| <= 1.13, and a bf16 result's sigmoid is off by 2^-20 (block_util)
    e = 1.2 * e + (2.0 ** -18 if s["dtype"] == "bf16" else 2.0 ** -21) * u.abs()
    if s["residual"] is not None:
        e = e + 2.0 ** -23 * (want.abs() + d(s["residual"]).abs())
        want = want + d(s["residual"])
    close(out, want, half * want.abs() + e, "out")


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 4096, 520), (1, 77, 33), (2, 512, 96), (3, 100, 130),
          (5, 1024, 256), (8, 96, 96), (9, 96, 96), (17, 8, 8), (64, 16, 48), (100, 200, 3),
          (127, 24, 40), (128, 64, 64), (129, 65, 17), (200, 96, 192), (256, 192, 96),
          (257, 384, 100), (300, 72, 264), (333, 3, 96), (513, 1000, 72), (640, 128, 1152),
          (1500, 96, 96), (37, 2048, 64), (20, 4096, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_forward_shapes(M, K, N, dtype):
    _check_forward(_case(M, K, N, dtype))
    _check_forward(_case(M, K, N, dtype, actk="silu", residual=True, seed=1), pre=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("actk,bias,residual,pre", list(itertools.product(
    ["none", "silu", "gelu"], [False, True], [False, True], [False, True])))
def test_forward_epilogues(actk, bias, residual, pre, dtype):
    for M, K, N in [(1, 96, 72), (6, 96, 72), (300, 64, 96), (290, 40, 70), (700, 128, 320)]:
        _check_forward(_case(M, K, N, dtype, actk=actk, bias=bias, residual=residual), pre)


def test_forward_many_tiles():
    """More tiles than the GPU has SMs, several per block, odd edges."""
    _check_forward(_case(40_001, 192, 96, "bf16", residual=True), pre=True)
    _check_forward(_case(20_011, 64, 392, "bf16", actk="gelu", residual=True), pre=True)
    _check_forward(_case(30_000, 320, 40, "bf16", residual=True))
    _check_forward(_case(9_000, 1096, 1160, "bf16", actk="silu"))


def test_residual_in_place():
    for dtype, M in itertools.product(["bf16", "fp32"], [1, 7, 1000]):
        s = _case(M, 96, 96, dtype, actk="silu", residual=True)
        want, _ = _forward(s)
        got, _ = _forward(s, out=s["residual"])
        assert torch.equal(want, got) and got.data_ptr() == s["residual"].data_ptr()


@pytest.mark.parametrize("M", [1, 8, 500])
def test_non_finite_stays_in_its_row(M):
    s = _case(M, 96, 72, "bf16", actk="silu", residual=True)
    s["x"][M - 1, 3] = float("nan")
    s["residual"][M // 2, 5] = float("inf")
    out, _ = _forward(s)
    rows = ~out.float().isfinite().all(1)
    want = torch.zeros(M, dtype=torch.bool, device="cuda")
    want[M - 1] = want[M // 2] = True
    assert torch.equal(rows, want)


def _backward(s, want=("x", "w", "bias"), stream=None):
    dt = DT[s["dtype"]]
    pre = s["rnd"](s["M"], s["N"]) if s["act"] != "none" else None
    dout = s["rnd"](s["M"], s["N"])
    got, oks = {"dx": None, "dw": None, "dbias": None}, []
    for k, shape in (("x", (s["M"], s["K"])), ("w", (s["N"], s["K"])), ("bias", (s["N"],))):
        if k in want:
            got["d" + k], ok = guarded(shape, dt)
            oks.append(ok)
    ws, ok = _ws(s, True)
    oks.append(ok)
    ccv3d.ccv3d_pointwise_backward(s["desc"], s["x"], s["w"], pre, dout, got["dx"], got["dw"],
                                   got["dbias"], ws, stream)
    torch.cuda.synchronize()
    for ok in oks:
        ok()
    return pre, dout, {k: v for k, v in got.items() if v is not None}


def _check_backward(s, want=("x", "w", "bias")):
    pre, dout, got = _backward(s, want)
    half = HALF[s["dtype"]]
    dp, e_dp = d(dout), torch.zeros_like(d(dout))
    if pre is not None:
        u = d(pre).requires_grad_()
        slope, = torch.autograd.grad(act(u, s["act"]).sum(), u)
        dp = d(dout) * slope
        # |s|, |u s (1 - s) ...| <= 1.2 and off by a few steps of the sigmoid's error
        e_dp = (2.0 ** -18 if s["dtype"] == "bf16" else 2.0 ** -21) * d(dout).abs() * (
            1 + u.detach().abs())
    e_sum = e_dp
    if pre is not None and s["dtype"] == "bf16":
        e_dp = e_dp + 2.0 ** -8 * dp.abs()   # dP as a bf16 operand
    w, x = d(s["w"]), d(s["x"])
    refs = {
        "dx": (dp @ w, (e_dp + _acc(s["N"]) * dp.abs()) @ w.abs()),
        "dw": (dp.t() @ x, (e_dp + _acc(s["M"]) * dp.abs()).t() @ x.abs()),
        "dbias": (dp.sum(0), (e_sum + _acc(s["M"]) * dp.abs()).sum(0)),
    }
    for k, v in got.items():
        ref, tol = refs[k]
        close(v, ref, half * ref.abs() + tol, k)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_backward_shapes(M, K, N, dtype):
    _check_backward(_case(M, K, N, dtype))
    _check_backward(_case(M, K, N, dtype, actk="gelu", seed=1))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_parts(dtype):
    for actk in ("none", "silu", "gelu"):
        for want in (("x",), ("w",), ("bias",), ("x", "bias"), ("w", "bias")):
            _check_backward(_case(500, 96, 72, dtype, actk=actk), want)


def test_backward_many_tiles():
    _check_backward(_case(40_001, 192, 96, "bf16", actk="silu"))
    _check_backward(_case(9_000, 392, 1160, "bf16", actk="gelu"))
    _check_backward(_case(100_003, 40, 24, "bf16"))


def test_fp32_long_sums_keep_their_accuracy():
    """dw over 60000 pixels in fp32: chains of at most 4096 FMAs.  Rounding errors of
    a chain add up like a random walk whose steps are 2^-24 of the running sum: in
    the 2-norm about 2^-24 sqrt(4096 / 2) / sqrt(3) = 1.6e-6 of a chain's share if
    every step were at its bound, a third of that for steps uniform within it."""
    s = _case(60_000, 40, 72, "fp32")
    _, dout, got = _backward(s)
    for k, want in (("dw", d(dout).t() @ d(s["x"])), ("dbias", d(dout).sum(0))):
        assert (d(got[k]) - want).norm() <= 1.0e-6 * want.norm(), k


@pytest.mark.parametrize("M,K,N,which", [
    (17_571, 200, 300, "dw"), (17_571, 988, 864, "dw"), (90_000, 40, 72, "dw"),
    (300, 4096, 520, "out"), (40_000, 2048, 24, "out"), (300, 77, 4099, "dx"), (520, 1030, 130, "out")])
def test_fp32_chains(M, K, N, which):
    """Sums of many terms in fp32 are taken in chains of 1024.  With terms of random
    signs the running sum after i of n terms is as the root of i, a rounding of it
    2^-24 / sqrt(3) relative, so a chain is 2^-24 sqrt(n / 6) of its sum off in the
    2-norm, 7.8e-7 for 1024; the chains' sums, at most 90 in a row, add 2^-24
    sqrt(90 / 6) = 2.3e-7, the result's rounding 3.4e-8: 8.2e-7 in all."""
    s = _case(M, K, N, "fp32", bias=False)
    if which == "out":
        got, want = _forward(s)[0], d(s["x"]) @ d(s["w"]).t()
    else:
        _, dout, g = _backward(s, ("x",) if which == "dx" else ("w",))
        got = g[which]
        want = d(dout) @ d(s["w"]) if which == "dx" else d(dout).t() @ d(s["x"])
    assert (d(got) - want).norm() <= 8.2e-7 * want.norm()


@pytest.mark.parametrize("terms", [1008, 1024, 1025, 1040, 1041, 2048, 2049, 2064, 3090])
def test_fp32_around_whole_chains(terms):
    """Sums that end at, just before and just after a whole chain, on each tile."""
    for M, N in ((1500, 1400), (700, 70), (9000, 20), (20, 9000)):
        _check_forward(_case(M, terms, N, "fp32", actk="silu", residual=True), pre=True)
    for K, N in ((700, 900), (24, 40)):
        _check_backward(_case(terms, K, N, "fp32"), ("w", "bias"))
    _check_backward(_case(1300, 1400, terms, "fp32"), ("x",))


def test_gradients_against_differences():
    """fp32: central differences of the 64-bit definition along random directions."""
    s = _case(40, 24, 36, "fp32", actk="gelu", bias=True)
    _, pre = _forward(s, pre=True)
    dout = s["rnd"](40, 36)
    outs = [torch.empty_like(t) for t in (s["x"], s["w"], s["bias"])]
    ws, _ = _ws(s, True)
    ccv3d.ccv3d_pointwise_backward(s["desc"], s["x"], s["w"], pre, dout, *outs, ws)
    base = [d(s["x"]), d(s["w"]), d(s["bias"])]
    loss = lambda x, w, b: (act(x @ w.t() + b, "gelu") * d(dout)).sum()
    g = torch.Generator(device="cuda").manual_seed(3)
    for i, grad in enumerate(outs):
        v = torch.randn(base[i].shape, device="cuda", generator=g, dtype=torch.float64)
        e = 1e-5
        up, dn = (loss(*[t + sgn * e * v if j == i else t for j, t in enumerate(base)])
                  for sgn in (1, -1))
        want, terms = (up - dn) / (2 * e), d(grad) * v
        # differences: e^2 and 2^-53 / e of the loss; gradients: the sums' own
        # steps (_acc of 40 terms) of the terms' magnitudes
        assert abs(want - terms.sum()) <= 2.0 ** -15 * terms.abs().sum() + 1e-6 * (1 + want.abs())


def test_same_bits_every_run():
    for M, K, N in [(9_000, 192, 96), (700, 77, 130), (64, 2048, 512)]:
        a = _backward(_case(M, K, N, "bf16", actk="silu"))[2]
        b = _backward(_case(M, K, N, "bf16", actk="silu"))[2]
        assert all(torch.equal(a[k], b[k]) for k in a)
        c, e = (_forward(_case(M, K, N, "bf16", actk="silu"))[0] for _ in range(2))
        assert torch.equal(c, e)


def test_zero_pixels():
    s = _case(0, 16, 24, "bf16")
    _forward(s)
    got = _backward(s)[2]
    assert (got["dw"] == 0).all() and (got["dbias"] == 0).all()


def test_other_stream_and_graph():
    for M in (1, 30, 5000):
        s = _case(M, 192, 96, "bf16", actk="silu", residual=True)
        want, want_pre = _forward(s, pre=True)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got, _ = _forward(s, pre=True)
        assert torch.equal(want, got)
        pre, dout, grads = _backward(s)
        out, p2 = torch.zeros_like(want), torch.zeros_like(want)
        outs = {k: torch.zeros_like(v) for k, v in grads.items()}
        nf, nb = ccv3d.ccv3d_pointwise_workspace(s["desc"])
        wf, wb = ccv3d.alloc_workspace(nf), ccv3d.alloc_workspace(nb)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ccv3d.ccv3d_pointwise_forward(s["desc"], s["x"], s["w"], s["bias"], s["residual"], out,
                                          p2, wf)
            ccv3d.ccv3d_pointwise_backward(s["desc"], s["x"], s["w"], pre, dout, outs["dx"],
                                           outs["dw"], outs["dbias"], wb)
        for _ in range(2):
            for t in (wf, wb):
                if t is not None:
                    t.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(p2, want_pre)
            assert all(torch.equal(outs[k], grads[k]) for k in grads)


def test_far_pixels():
    """Offsets past 2^31 elements: the last rows of a long call, forward and dx."""
    M, K, N = 23_500_001, 96, 96
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, K, device="cuda").bfloat16()
    w = (torch.randn(N, K, device="cuda") * 0.1).bfloat16()
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    desc = ccv3d.make_pointwise_desc(pixels=M, Cin=K, Cout=N)
    nf, nb = ccv3d.ccv3d_pointwise_workspace(desc)
    ccv3d.ccv3d_pointwise_forward(desc, x, w, None, x, out, None, ccv3d.alloc_workspace(nf))
    u, mag = d(x[-3:]) @ d(w).t(), d(x[-3:]).abs() @ d(w).abs().t()
    want = u + d(x[-3:])
    close(out[-3:], want, HALF["bf16"] * want.abs() + 2 * _acc(K) * (mag + d(x[-3:]).abs()), "out")
    assert int((out[:-3] != 0).sum()) == 0
    ccv3d.ccv3d_pointwise_backward(desc, None, w, None, x, out, None, None,
                                   ccv3d.alloc_workspace(nb))
    want, mag = d(x[-3:]) @ d(w), d(x[-3:]).abs() @ d(w).abs()
    close(out[-3:], want, HALF["bf16"] * want.abs() + _acc(N) * mag, "dx")
    assert int((out[:-3] != 0).sum()) == 0
    assert ccv3d.ccv3d_block_get_status() == ccv3d.CCV3D_OK


@pytest.fixture(autouse=True)
def status_is_clean():
    """No call of a test left an error (a wait that ran out; in the checked build
    an address outside its buffer) in the library's status word."""
    yield
    assert ccv3d.ccv3d_block_get_status() == ccv3d.CCV3D_OK
